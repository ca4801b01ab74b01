"""The paged cache's append, fork and compact on the GPU against the oracle:
every table entry, length, count, status word and pool element, exactly."""
import numpy as np
import pytest
import torch

import oracle.paged as paged
from paged_util import DT, numpy_cache, on_gpu

pytestmark = pytest.mark.gpu

lib = pytest.importorskip("scaled_dot_product_saving_b200")

BOOKS = ("table", "lens", "ref")
POOLS = ("k_pages", "v_pages")


def ints(x):
    return None if x is None else torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def same(dev, want):
    for name, w in want.items():
        g = dev[name]
        g = g.double().cpu().numpy() if name in POOLS else g.cpu().numpy()
        assert g.shape == np.asarray(w).shape, name
        assert (g == w).all(), f"{name} differs in {np.argwhere(g != w)[:5].tolist()}"


def outs(dev, in_place, names=BOOKS):
    if in_place:
        return {f"{n}_out": dev[n] for n in names}
    return {f"{n}_out": torch.full_like(dev[n], -77) for n in names}


def append(dev, host, k, v, new_len=None, in_place=False, **kw):
    """One call on the device and the oracle, compared; returns the status."""
    before = {n: dev[n].clone() for n in BOOKS}
    t, l, r, info = lib.attn_cache_append(k, v, dev["k_pages"], dev["v_pages"], *(dev[n] for n in BOOKS),
                                          new_len=ints(new_len), **outs(dev, in_place), **kw)
    torch.cuda.synchronize()
    out = paged.append(k.double().cpu().numpy(), v.double().cpu().numpy(), host["k_pages"], host["v_pages"],
                       host["table"], host["lens"], host["ref"], new_len)
    if not in_place:
        for n in BOOKS:
            assert torch.equal(dev[n], before[n]), n
    dev.update(table=t, lens=l, ref=r)
    host.update(zip(POOLS + BOOKS, out[:5]))
    same(dev, {n: host[n] for n in POOLS + BOOKS})
    assert tuple(info.tolist()) == out[5]
    return out[5]


def fork(dev, host, src, keep=None, in_place=False, **kw):
    t, l, r, info = lib.attn_cache_fork(dev["k_pages"], dev["v_pages"], *(dev[n] for n in BOOKS), ints(src),
                                        keep=ints(keep), **outs(dev, in_place), **kw)
    torch.cuda.synchronize()
    out = paged.fork(host["k_pages"], host["v_pages"], host["table"], host["lens"], host["ref"], src, keep)
    dev.update(table=t, lens=l, ref=r)
    host.update(zip(POOLS + BOOKS, out[:5]))
    same(dev, {n: host[n] for n in POOLS + BOOKS})
    assert tuple(info.tolist()) == out[5]
    return out[5]


def compact(dev, host, in_place=False, **kw):
    t, r, remap, info = lib.attn_cache_compact(dev["k_pages"], dev["v_pages"], *(dev[n] for n in BOOKS),
                                               **outs(dev, in_place, ("table", "ref")), **kw)
    torch.cuda.synchronize()
    out = paged.compact(host["k_pages"], host["v_pages"], host["table"], host["lens"], host["ref"])
    dev.update(table=t, ref=r, remap=remap)
    host.update(zip(POOLS + ("table", "ref"), out[:4]))
    same(dev, {n: host[n] for n in POOLS + ("table", "ref")})
    assert (remap.cpu().numpy() == out[4]).all()
    assert tuple(info.tolist()) == out[5]
    return out[5]


def rows(rng, B, Hkv, n, w, dt):
    return torch.tensor(rng.standard_normal((B, Hkv, n, w)), device="cuda").to(DT[dt])


both = pytest.mark.parametrize("in_place", [False, True], ids=["out", "in_place"])


@both
@pytest.mark.parametrize("lens,n,Hkv,d,dv,page,dt,new_len", [
    ((0,), 1, 1, 64, 64, 16, "bf16", None),                       # a new cache's first token
    ((0, 5, 16, 31, 32), 1, 2, 128, 128, 16, "bf16", None),       # page borders
    ((0, 5, 16, 31, 33), 50, 2, 64, 64, 16, "bf16", (50, 0, 1, 17, 33)),
    ((7, 300), 130, 3, 40, 72, 64, "bf16", (130, 2)),
    ((9, 1), 20, 2, 36, 4, 8, "f32", (20, -3)),                   # below zero: none
    ((9, 1), 20, 2, 128, 128, 256, "f32", (99, 20)),              # past n: n
    ((3, 4, 5), 2, 1, 8, 8, 8, "bf16", (0, 0, 0)),
])
def test_append(lens, n, Hkv, d, dv, page, dt, new_len, in_place):
    rng = np.random.default_rng(n + d)
    M = max(-(-(L + n) // page) for L in lens) + 1
    dev, host = on_gpu(numpy_cache(rng, len(lens), Hkv, page, d, dv, lens, spare=2 * len(lens) + sum(lens) + 60, M=M), dt)
    k, v = rows(rng, len(lens), Hkv, n, d, dt), rows(rng, len(lens), Hkv, n, dv, dt)
    assert append(dev, host, k, v, new_len, in_place)[0] == 0
    assert append(dev, host, k, v, [0] * len(lens), in_place)[0] == 0


@both
def test_append_refusals_change_nothing(in_place):
    rng = np.random.default_rng(3)
    c = numpy_cache(rng, 3, 2, 8, 64, 64, (12, 8, 0), spare=2, M=4)
    dev, host = on_gpu(c, "bf16")
    k, v = rows(rng, 3, 2, 32, 64, "bf16"), rows(rng, 3, 2, 32, 64, "bf16")
    assert append(dev, host, k, v, (4, 8, 9), in_place)[0] == 1          # one page short
    assert append(dev, host, k, v, (21, 0, 0), in_place)[0] == 2         # longer than the row
    assert append(dev, host, k, v, (21, 32, 32), in_place)[0] == 2       # and not enough pages
    p = host["table"][0, 1]
    dev["ref"][p] += 1
    host["ref"] = host["ref"].copy()
    host["ref"][p] += 1
    assert append(dev, host, k, v, (1, 1, 0), in_place)[0] == 3          # a last page that others refer to
    assert append(dev, host, k, v, (0, 1, 1), in_place)[0] == 0          # not touched: no matter
    host["table"] = host["table"].copy()
    for bad in (-1, host["ref"].shape[0], 2 ** 31 - 1, -2 ** 31):
        dev["table"][0, 1] = bad
        host["table"][0, 1] = bad
        assert append(dev, host, k, v, (1, 0, 0), in_place)[0] == 3


@both
@pytest.mark.parametrize("lens,src,keep,page", [
    ((0,), (0,), None, 16),
    ((20,), (-1,), None, 16),                                    # freed
    ((20, 0, 32), (0, 0, 0), None, 16),                          # one forked over others
    ((20, 33, 32), (1, 2, 0), None, 16),                         # all change at once
    ((20, 33, 47), (0, 1, 2), (5, 32, 46), 16),                  # roll-back: in a page, to its border, by one
    ((20, 33, 47), (2, 2, 2), (16, 40, 47), 16),                 # prefixes: full, cut, whole
    ((20, 33, 47), (2, 2, -7), (40, 40, 1), 16),                 # the same cut page, its owner gone
    ((20, 33, 47), (2, 2, -7), (33, 40, 1), 16),                 # ... in different places
    ((20, 33, 47), (99, 1, 1), (-4, 0, 1000), 16),               # out of range, none kept, more than there is
    ((100, 9, 8, 256, 257), (4, 3, 3, 4, 3), (256, 256, 255, 257, 1), 256),
    ((100, 9, 8, 64), (3, 0, 1, 2), None, 8),                    # a cycle
])
def test_fork(lens, src, keep, page, in_place):
    rng = np.random.default_rng(len(lens) + page)
    dev, host = on_gpu(numpy_cache(rng, len(lens), 2, page, 64, 40, lens, spare=6), "bf16")
    assert fork(dev, host, src, keep, in_place)[0] == 0
    assert fork(dev, host, [-1] * len(lens), None, in_place)[:2] == (0, host["ref"].shape[0])


@both
def test_fork_refused_and_references_of_the_caller(in_place):
    rng = np.random.default_rng(4)
    dev, host = on_gpu(numpy_cache(rng, 3, 2, 8, 64, 64, (12, 8, 8), spare=0, M=3), "f32")
    kept = [host["table"][1, 0], host["table"][2, 0]]
    dev["ref"][ints(kept).long()] += 1
    host["ref"] = host["ref"].copy()
    host["ref"][kept] += 1
    assert fork(dev, host, (0, 0, 0), None, in_place) == (1, 0, 0)
    assert fork(dev, host, (0, -1, -1), None, in_place) == (0, 0, 0)     # kept pages stay referred to
    assert fork(dev, host, (-1, -1, -1), None, in_place) == (0, 2, 0)
    assert sorted(np.flatnonzero(host["ref"])) == sorted(kept)


@both
@pytest.mark.parametrize("lens,src,page,dt", [
    ((20, 33, 47), (0, 1, 2), 16, "bf16"),
    ((20, 33, 47), (-1, 1, 2), 16, "f32"),
    ((200, 3, 470, 90), (-1, 3, -1, 3), 8, "bf16"),
    ((0, 0), (0, 1), 8, "bf16"),                                  # nothing live
    ((300, 300), (0, 1), 128, "f32"),
])
def test_compact(lens, src, page, dt, in_place):
    rng = np.random.default_rng(len(lens) * page)
    dev, host = on_gpu(numpy_cache(rng, len(lens), 2, page, 64, 24, lens, spare=13), dt)
    assert fork(dev, host, src, None, in_place)[0] == 0
    compact(dev, host, in_place)
    assert compact(dev, host, in_place)[2] == 0                   # nothing left to move


def test_compact_of_a_full_pool():
    rng = np.random.default_rng(6)
    dev, host = on_gpu(numpy_cache(rng, 2, 1, 8, 64, 64, (64, 80), spare=0), "bf16")
    assert compact(dev, host) == (0, 0, 0)


@both
def test_bad_page_numbers_are_carried_along(in_place):
    rng = np.random.default_rng(7)
    c = numpy_cache(rng, 3, 1, 8, 64, 64, (20, 20, 20), spare=5)
    P = c["ref"].shape[0]
    c["table"][1, :3] = [P, -1, 2 ** 31 - 1]
    c["lens"][2] = -9
    dev, host = on_gpu(c, "bf16")
    fork(dev, host, (1, 1, 0), (20, 9, 15), in_place)
    compact(dev, host, in_place)


@pytest.mark.parametrize("seed,page,dt,B", [(0, 16, "bf16", 6), (1, 8, "f32", 6), (2, 32, "bf16", 40)])
def test_a_run_of_calls(seed, page, dt, B):
    """Cache calls in random order, in place and not, with attn_decode over
    the result (values are whole numbers: uniform weights at scale 0)."""
    rng = np.random.default_rng(seed)
    Hkv, H, d = 2, 4, 64
    c = numpy_cache(rng, B, Hkv, page, d, d, rng.integers(0, 5 * page, size=B), spare=12 * B, M=16, unit=True)
    dev, host = on_gpu(c, dt)
    ws = torch.full((lib.attn_cache_workspace_size(B, 16, c["ref"].shape[0]),), 255, dtype=torch.uint8, device="cuda")
    done = 0
    for step in range(25):
        in_place = bool(rng.random() < 0.5)
        kind = rng.integers(0, 4)
        if kind <= 1:
            n = int(rng.integers(1, 2 * page)) if kind else 1
            k = torch.tensor(rng.integers(-9, 10, size=(B, Hkv, n, d)), device="cuda").to(DT[dt])
            status = append(dev, host, k, k + 1, rng.integers(0, n + 1, size=B), in_place, workspace=ws)[0]
        elif kind == 2:
            src = np.where(rng.random(B) < 0.5, np.arange(B), rng.integers(-1, B, size=B))
            status = fork(dev, host, src, rng.integers(0, 8 * page, size=B), in_place, workspace=ws)[0]
        else:
            status = compact(dev, host, in_place, workspace=ws)[0]
        done += status == 0
        q = torch.tensor(rng.standard_normal((B, H, 1, d)), device="cuda").to(DT[dt])
        o, _ = lib.attn_decode(q, dev["k_pages"], dev["v_pages"], dev["table"], dev["lens"], scale=0.0)
        torch.cuda.synchronize()
        for b in range(B):
            L = int(host["lens"][b])
            V = paged.read_back(host["v_pages"], host["table"][b], L)
            want = V.mean(1) if L else np.zeros((Hkv, d))
            got = o[b, :, 0].double().cpu().numpy().reshape(Hkv, H // Hkv, d)
            # whole numbers: the sum is exact, one division and one rounding
            assert np.allclose(got, want[:, None], rtol=2.0 ** -8 * 1.01 if dt == "bf16" else 2.0 ** -22, atol=1e-30)
    assert done >= 10


def test_many_sequences_and_pages():
    """More sequences than a block has threads, and a pool of many pages."""
    rng = np.random.default_rng(8)
    B = 2500
    lens = rng.integers(0, 30, size=B)
    dev, host = on_gpu(numpy_cache(rng, B, 1, 8, 8, 8, lens, spare=9000, M=6), "bf16")
    k = rows(rng, B, 1, 12, 8, "bf16")
    assert append(dev, host, k, k, rng.integers(0, 13, size=B))[0] == 0
    src = np.where(rng.random(B) < 0.5, np.arange(B), rng.integers(-1, B, size=B))
    assert fork(dev, host, src, rng.integers(0, 40, size=B), True)[0] == 0
    compact(dev, host, True)


def test_captured_step():
    """append and decode of a token captured once and replayed: the cache grows
    over page borders with no word from the host; then a captured roll-back."""
    rng = np.random.default_rng(9)
    B, Hkv, H, d, page = 3, 2, 8, 64, 8
    dev, host = on_gpu(numpy_cache(rng, B, Hkv, page, d, d, (0, 7, 30), spare=20, M=8), "bf16")
    k, v = rows(rng, B, Hkv, 1, d, "bf16"), rows(rng, B, Hkv, 1, d, "bf16")
    q = rows(rng, B, H, 1, d, "bf16")
    ws = torch.empty(lib.attn_cache_workspace_size(B, 8, host["ref"].shape[0]), dtype=torch.uint8, device="cuda")
    info = torch.zeros(3, dtype=torch.int32, device="cuda")
    books = {f"{n}_out": dev[n] for n in BOOKS}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.attn_cache_append(k, v, dev["k_pages"], dev["v_pages"], *(dev[n] for n in BOOKS), info=info,
                              workspace=ws, **books)
        o, lse = lib.attn_decode(q, dev["k_pages"], dev["v_pages"], dev["table"], dev["lens"])
    for _ in range(12):
        k.copy_(rows(rng, B, Hkv, 1, d, "bf16"))
        v.copy_(rows(rng, B, Hkv, 1, d, "bf16"))
        g.replay()
        torch.cuda.synchronize()
        out = paged.append(k.double().cpu().numpy(), v.double().cpu().numpy(), *(host[n] for n in POOLS + BOOKS))
        host.update(zip(POOLS + BOOKS, out[:5]))
        same(dev, {n: host[n] for n in POOLS + BOOKS})
        assert tuple(info.tolist()) == out[5] and out[5][0] == 0
        eager = lib.attn_decode(q, dev["k_pages"], dev["v_pages"], dev["table"], dev["lens"])
        assert torch.equal(o, eager[0]) and torch.equal(lse, eager[1])
    src, keep = ints((0, 1, 2)), ints((3, 16, 41))
    g2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g2):
        lib.attn_cache_fork(dev["k_pages"], dev["v_pages"], *(dev[n] for n in BOOKS), src, keep=keep, info=info,
                            workspace=ws, **books)
    g2.replay()
    g2.replay()                                                   # a second time: nothing more to do
    torch.cuda.synchronize()
    out = paged.fork(*(host[n] for n in POOLS + BOOKS), (0, 1, 2), (3, 16, 41))
    same(dev, dict(zip(POOLS + BOOKS, out[:5])))


def test_prompt_then_tokens_is_causal_attention():
    """attn_fwd over a prompt, its keys appended, then token after token through
    attn_decode: the rows of attn_fwd over the whole sequence."""
    B, H, d, n, m = 2, 4, 64, 50, 70
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(B, H, m, d, generator=g).to(torch.bfloat16).cuda() for _ in range(3))
    whole, whole_lse = lib.attn_fwd(q, k, v, causal=True)
    P, page, M = 12, 16, 5
    kp = torch.full((P, H, page, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vp = torch.full_like(kp, float("nan"))
    table = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    ref = torch.zeros(P, dtype=torch.int32, device="cuda")
    part = lambda x, a, b: x[:, :, a:b].contiguous()
    table, lens, ref, info = lib.attn_cache_append(part(k, 0, n), part(v, 0, n), kp, vp, table, lens, ref)
    at = n
    for step in (1, 1, 3, 8, 7):
        table, lens, ref, info = lib.attn_cache_append(part(k, at, at + step), part(v, at, at + step), kp, vp,
                                                       table, lens, ref)
        o, lse = lib.attn_decode(part(q, at, at + step), kp, vp, table, lens)
        torch.cuda.synchronize()
        assert info[0].item() == 0
        # both round the weights (2^-8 of sum P|v| <= max|v|) and the result (2^-8) to bf16
        top = v.float().abs().max().item()
        assert (o.float() - whole[:, :, at:at + step].float()).abs().max().item() <= 4 * 2.0 ** -8 * top
        assert (lse - whole_lse[:, :, at:at + step]).abs().max().item() <= 1e-3
        at += step
    assert at == m and lib.attn_get_device_error() == 0


def test_on_another_stream():
    rng = np.random.default_rng(10)
    dev, host = on_gpu(numpy_cache(rng, 4, 2, 16, 64, 64, (5, 20, 40, 0), spare=12), "bf16")
    s = torch.cuda.Stream()
    k = rows(rng, 4, 2, 3, 64, "bf16")
    torch.cuda.synchronize()
    assert append(dev, host, k, k, (3, 2, 1, 0), stream=s)[0] == 0
    assert fork(dev, host, (1, 1, 3, 2), stream=s)[0] == 0
    compact(dev, host, stream=s)


def test_refusals():
    rng = np.random.default_rng(11)
    dev, _ = on_gpu(numpy_cache(rng, 2, 2, 16, 64, 64, (20, 30)), "bf16")
    pools, books = (dev["k_pages"], dev["v_pages"]), tuple(dev[n] for n in BOOKS)
    k = rows(rng, 2, 2, 1, 64, "bf16")
    for bad in (k[:1], k.float(), k[..., :32].contiguous(), k.cpu()):
        with pytest.raises((ValueError, TypeError)):
            lib.attn_cache_append(bad, k, *pools, *books)
    for bad in (None, dev["ref"][:3], dev["ref"].long(), dev["ref"].cpu()):
        with pytest.raises(ValueError):
            lib.attn_cache_append(k, k, *pools, dev["table"], dev["lens"], bad)
        with pytest.raises(ValueError):
            lib.attn_cache_compact(*pools, dev["table"], dev["lens"], bad)
    for bad in (None, ints((0,)), torch.zeros(2, device="cuda")):
        with pytest.raises(ValueError):
            lib.attn_cache_fork(*pools, *books, bad)
    with pytest.raises(ValueError):
        lib.attn_cache_append(k, k, dev["k_pages"], dev["v_pages"][:, :, :8].contiguous(), *books)
    with pytest.raises(lib.AttnError) as e:
        lib.attn_cache_fork(*pools, *books, ints((0, 1)), table_out=dev["table"], lens_out=ints((0, 1)),
                            workspace=dev["k_pages"])
    assert e.value.code == 9
    with pytest.raises(lib.AttnError) as e:
        lib.attn_cache_append(k, k, *(p[:, :, :4].contiguous() for p in pools), *books)
    assert e.value.code == 4


@both
def test_a_pool_of_very_many_pages(in_place):
    """More pages than the books hold in registers, most of them the caller's."""
    rng = np.random.default_rng(12)
    P, B = 300001, 3
    c = numpy_cache(rng, B, 1, 8, 8, 8, (9, 800, 0), spare=P - 102, M=600, unit=True)
    assert c["ref"].shape[0] == P
    c["ref"][rng.random(P) < 0.99] |= 1
    dev, host = on_gpu(c, "bf16")
    k, v = rows(rng, B, 1, 3000, 8, "bf16"), rows(rng, B, 1, 3000, 8, "bf16")
    out = append(dev, host, k, v, (3000, 17, 2900), in_place)
    assert out[0] == 0 and out[2] > 700
    assert fork(dev, host, (2, 1, 1), (2000, 500, 813), in_place)[0] == 0
    assert compact(dev, host, in_place)[2] > 1000


def test_captured_round():
    """A step of a search captured whole, in place: new tokens, attention, new
    parents, then the pool closed up; replayed while the cache grows."""
    rng = np.random.default_rng(13)
    B, Hkv, d, page, M = 4, 2, 64, 8, 6
    dev, host = on_gpu(numpy_cache(rng, B, Hkv, page, d, d, (3, 9, 0, 16), spare=20, M=M), "bf16")
    P = host["ref"].shape[0]
    k, q = rows(rng, B, Hkv, 3, d, "bf16"), rows(rng, B, 4, 3, d, "bf16")
    src, new_len = ints((1, 1, 0, 3)), ints((3, 0, 1, 2))
    books = {f"{n}_out": dev[n] for n in BOOKS}
    ws = torch.empty(lib.attn_cache_workspace_size(B, M, P), dtype=torch.uint8, device="cuda")
    infos = torch.full((3, 3), -1, dtype=torch.int32, device="cuda")
    args = (dev["k_pages"], dev["v_pages"], *(dev[n] for n in BOOKS))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.attn_cache_append(k, k, *args, new_len=new_len, info=infos[0], workspace=ws, **books)
        o, lse = lib.attn_decode(q, *args[:4], q_len=new_len)
        lib.attn_cache_fork(*args, src, info=infos[1], workspace=ws, **books)
        lib.attn_cache_compact(*args, info=infos[2], workspace=ws, table_out=dev["table"], ref_out=dev["ref"])
    for turn in range(6):
        parents = rng.integers(-1, B, size=B) if turn else np.arange(B)
        grow = rng.integers(0, 4, size=B)
        src.copy_(ints(parents))
        new_len.copy_(ints(grow))
        k.copy_(rows(rng, B, Hkv, 3, d, "bf16"))
        g.replay()
        torch.cuda.synchronize()
        kk = k.double().cpu().numpy()
        want = []
        out = paged.append(kk, kk, *(host[n] for n in POOLS + BOOKS), grow)
        want.append(out[5])
        out = paged.fork(*out[:5], parents)
        want.append(out[5])
        lens = out[3]
        out = paged.compact(*out[:5])
        want.append(out[5])
        host.update(zip(POOLS + ("table", "ref"), out[:4]), lens=lens)
        same(dev, {n: host[n] for n in POOLS + BOOKS})
        assert infos.tolist() == [list(x) for x in want]
    assert lib.attn_get_device_error() == 0


@both
def test_which_refusal_is_told(in_place):
    """3 goes before 2 and 2 before 1; a partly filled last page is looked at in every
    sequence with new tokens, whether or not they fit its row."""
    rng = np.random.default_rng(14)
    dev, host = on_gpu(numpy_cache(rng, 3, 2, 8, 64, 64, (12, 8, 5), spare=1, M=2), "bf16")
    k, v = rows(rng, 3, 2, 9, 64, "bf16"), rows(rng, 3, 2, 9, 64, "bf16")
    host["ref"] = host["ref"].copy()

    def share(b, j, by):
        p = int(host["table"][b, j])
        dev["ref"][p] += by
        host["ref"][p] += by

    assert append(dev, host, k, v, (1, 0, 8), in_place)[0] == 0
    dev, host = on_gpu(numpy_cache(rng, 3, 2, 8, 64, 64, (12, 8, 5), spare=1, M=2), "bf16")
    host["ref"] = host["ref"].copy()
    assert append(dev, host, k, v, (4, 8, 8), in_place)[0] == 1          # one page for two
    assert append(dev, host, k, v, (5, 8, 8), in_place)[0] == 2          # ... and a full row
    share(0, 1, 1)
    assert append(dev, host, k, v, (1, 8, 8), in_place)[0] == 3          # no pages, and a shared last page
    assert append(dev, host, k, v, (1, 9, 8), in_place)[0] == 3          # a full row elsewhere
    assert append(dev, host, k, v, (5, 0, 0), in_place)[0] == 3          # the full row is the shared one's
    assert append(dev, host, k, v, (5, 9, 8), in_place)[0] == 3          # all of them
    assert append(dev, host, k, v, (0, 9, 1), in_place)[0] == 2          # shared, but not added to
    share(0, 1, -1)
    share(2, 0, 1)
    assert append(dev, host, k, v, (5, 0, 9), in_place)[0] == 3
    share(2, 0, -1)
    assert append(dev, host, k, v, (4, 0, 8), in_place)[0] == 0
