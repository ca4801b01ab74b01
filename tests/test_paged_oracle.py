"""Pins of oracle/paged.py, on the CPU."""
import numpy as np
import pytest

import oracle.paged as paged
import oracle.ref as ref
from paged_util import holders, numpy_cache


@pytest.mark.parametrize("lens,page,n,causal", [((1, 37, 64), 16, 1, True), ((9, 40, 5), 8, 4, True),
                                                ((64, 3, 17), 32, 3, False)])
def test_decode_is_dense_attention_over_the_row(lens, page, n, causal):
    rng = np.random.default_rng(1)
    H, Hkv, d, dv = 6, 2, 8, 16
    c = numpy_cache(rng, 3, Hkv, page, d, dv, lens)
    q = rng.standard_normal((3, H, n, d))
    q_len = [min(n, L) for L in lens]
    O, lse, _, _ = paged.decode(q, c["k_pages"], c["v_pages"], c["table"], lens, q_len, causal)
    for b, L in enumerate(lens):
        K = paged.read_back(c["k_pages"], c["table"][b], L).astype(np.float64)
        V = paged.read_back(c["v_pages"], c["table"][b], L).astype(np.float64)
        for h in range(H):
            hk = h // (H // Hkv)
            for i in range(q_len[b]):
                see = L - (q_len[b] - 1 - i) if causal else L
                o, l = ref.head_forward(q[b, h, i:i + 1], K[hk, :see], V[hk, :see], False, d ** -0.5)
                assert np.allclose(O[b, h, i], o[0], rtol=1e-12, atol=1e-14)
                assert np.allclose(lse[b, h, i], l[0], rtol=1e-12)
        assert np.isnan(O[b, :, q_len[b]:]).all()


def test_decode_of_the_last_rows_is_causal_attention():
    """With the whole sequence as queries, decode is oracle.ref's causal attention."""
    rng = np.random.default_rng(2)
    n, d = 21, 8
    c = numpy_cache(rng, 1, 1, 8, d, d, (n,))
    q = rng.standard_normal((1, 1, n, d))
    O, lse, _, _ = paged.decode(q, c["k_pages"], c["v_pages"], c["table"], (n,))
    K = paged.read_back(c["k_pages"], c["table"][0], n).astype(np.float64)[0]
    V = paged.read_back(c["v_pages"], c["table"][0], n).astype(np.float64)[0]
    o, l = ref.head_forward(q[0, 0], K, V, True, d ** -0.5)
    assert np.allclose(O[0, 0], o, rtol=1e-12, atol=1e-14) and np.allclose(lse[0, 0], l, rtol=1e-12)


def test_decode_without_keys():
    rng = np.random.default_rng(3)
    c = numpy_cache(rng, 2, 1, 8, 8, 8, (0, 2))
    q = rng.standard_normal((2, 1, 4, 8))
    O, lse, _, _ = paged.decode(q, c["k_pages"], c["v_pages"], c["table"], (0, 2))
    assert (O[0] == 0).all() and np.isneginf(lse[0]).all()
    assert (O[1, 0, :2] == 0).all() and np.isneginf(lse[1, 0, :2]).all() and np.isfinite(lse[1, 0, 2:]).all()


class Model:
    """Every sequence as the list of its token values."""

    def __init__(self, cache, B):
        self.page = cache["k_pages"].shape[2]
        self.seqs = [self.values(cache, b) for b in range(B)]

    def values(self, c, b):
        return [tuple(x) for x in paged.read_back(c["k_pages"], c["table"][b], int(c["lens"][b]))[0]]

    def check(self, c, extra):
        P = c["ref"].shape[0]
        for b, want in enumerate(self.seqs):
            assert int(c["lens"][b]) == len(want)
            assert self.values(c, b) == want
        assert (holders(c["table"], c["lens"], self.page, P) + extra == c["ref"]).all()
        for b in range(len(self.seqs)):          # a partly filled last page has one holder
            L = int(c["lens"][b])
            if L % self.page:
                assert c["ref"][c["table"][b, L // self.page]] == 1


@pytest.mark.parametrize("seed", range(6))
def test_a_run_of_cache_calls_against_lists_of_tokens(seed):
    rng = np.random.default_rng(seed)
    B, Hkv, page = 5, 2, 8
    c = numpy_cache(rng, B, Hkv, page, 8, 8, rng.integers(0, 40, size=B), spare=30, M=12)
    m = Model(c, B)
    extra = np.zeros_like(c["ref"])
    keys = ("k_pages", "v_pages", "table", "lens", "ref")
    refused = 0
    for step in range(60):
        kind = rng.integers(0, 3)
        if kind == 0:
            n = int(rng.integers(1, 20))
            k = rng.standard_normal((B, Hkv, n, 8)).astype(np.float32)
            v = rng.standard_normal((B, Hkv, n, 8)).astype(np.float32)
            new = rng.integers(0, n + 1, size=B)
            out = paged.append(k, v, *(c[x] for x in keys), new_len=new)
            if out[-1][0] == paged.INFO_OK:
                for b in range(B):
                    m.seqs[b] += [tuple(x) for x in k[b, 0, :new[b]]]
            else:
                refused += 1
            c = dict(zip(keys, out[:5]))
        elif kind == 1:
            src = rng.integers(-1, B, size=B)
            stay = rng.random(B) < 0.4
            src[stay] = np.arange(B)[stay]
            keep = rng.integers(0, 100, size=B)
            out = paged.fork(*(c[x] for x in keys), src, keep)
            if out[-1][0] == paged.INFO_OK:
                m.seqs = [list(m.seqs[s][:keep[b]]) if s >= 0 else [] for b, s in enumerate(src)]
            c = dict(zip(keys, out[:5]))
        else:
            kp, vp, table, refs, remap, info = paged.compact(*(c[x] for x in keys))
            live = int((refs > 0).sum())
            assert (refs[:live] > 0).all() and (refs[live:] == 0).all()
            assert info[1] == len(refs) - live
            moved = np.zeros_like(extra)
            for p, to in enumerate(remap):
                if to >= 0:
                    moved[to] = extra[p]
            extra = moved
            c = dict(k_pages=kp, v_pages=vp, table=table, lens=c["lens"], ref=refs)
        assert out[-1][1] == (out[4] <= 0).sum() if kind < 2 else True
        m.check(c, extra)
        if rng.random() < 0.1:                    # a reference of the caller's own to some full page
            full = [p for b in range(B) for p in c["table"][b, :int(c["lens"][b]) // page]]
            if full:
                p = full[int(rng.integers(len(full)))]
                extra[p] += 1
                c["ref"] = c["ref"].copy()
                c["ref"][p] += 1
    assert refused < 60


def test_refusals_change_nothing():
    rng = np.random.default_rng(9)
    c = numpy_cache(rng, 2, 1, 8, 8, 8, (12, 8), spare=1, M=3)
    k = rng.standard_normal((2, 1, 12, 8)).astype(np.float32)
    args = [c[x] for x in ("k_pages", "v_pages", "table", "lens", "ref")]
    for new, status in (((12, 0), 0), ((12, 1), 1), ((13, 0), 0), ((12, 12), 1)):
        out = paged.append(k, k, *args, new_len=new)
        assert out[-1][0] == status, new
        if status:
            assert all((a == b).all() for a, b in zip(args, out[:5]))
    out = paged.append(np.repeat(k, 2, 2), np.repeat(k, 2, 2), *args, new_len=(13, 0))
    assert out[-1][0] == paged.INFO_TABLE_FULL
    shared = c["ref"].copy()
    shared[c["table"][0, 1]] = 2
    assert paged.append(k, k, *args[:4], shared, new_len=(1, 0))[-1][0] == paged.INFO_SHARED_TAIL
    assert paged.append(k, k, *args[:4], shared, new_len=(0, 1))[-1][0] == paged.INFO_OK
    # two copies of the partly filled page of 0 do not fit beside it in one free page
    out = paged.fork(*args, src=(0, 0))
    assert out[-1][0] == paged.INFO_OK and out[-1][2] == 1
    c3 = numpy_cache(rng, 3, 1, 8, 8, 8, (12, 8, 8), spare=0, M=3)
    args = [c3[x] for x in ("k_pages", "v_pages", "table", "lens", "ref")]
    full = c3["ref"].copy()
    full[c3["table"][1, 0]] = full[c3["table"][2, 0]] = 2      # kept by the caller: not freed
    out = paged.fork(*args[:4], full, src=(0, 0, 0))
    assert out[-1] == (paged.INFO_NO_PAGES, 0, 0)
    assert all((a == b).all() for a, b in zip(args[:4], out[:4])) and (out[4] == full).all()
