"""attn_decode on the GPU against the float64 oracle, on the rounded inputs.

Bounds, per element, from the arithmetic (u = 2^-24; A = sum_j P_j |v_j|,
X = max_j scale * sum_c |q_c k_jc|, both from the oracle; L keys):
  a score is a sum of d products scaled once and taken through exp2: its error
  is at most (d + 4) u X, plus 4 u for the exponential itself, and enters the
  weights and their sum once each; the two sums over the keys add L u each:
    fp32  |dO|   <= A u (2 ((d + 4) X + 4) + 2 L + 16),
          |dLSE| <= u ((d + 4) X + 4 + L + 16 + 2 |LSE|)
  in bf16 the weights may be rounded to bf16 before the second product (half a
  step, 2^-8 of each) and the result is rounded once more:
    bf16  |dO|   <= 2^-8 (1 + 2^-8) A + 2^-8 |O| + the fp32 terms
"""
import math

import numpy as np
import pytest
import torch

import oracle.paged as paged
from paged_util import DT, numpy_cache, on_gpu

pytestmark = pytest.mark.gpu

lib = pytest.importorskip("scaled_dot_product_saving_b200")

U = 2.0 ** -24


def run(dev, q, causal=True, q_len=None, scale=None, **kw):
    ql = None if q_len is None else torch.tensor(q_len, dtype=torch.int32, device="cuda")
    o, lse = lib.attn_decode(q, dev["k_pages"], dev["v_pages"], dev["table"], dev["lens"], causal=causal,
                             scale=scale, q_len=ql, **kw)
    torch.cuda.synchronize()
    assert lib.attn_get_device_error() == 0
    return o, lse


def compare(o, lse, dt, host, q, causal=True, q_len=None, scale=None):
    table, lens = host["table"], host["lens"]
    O, LSE, A, X = paged.decode(q.double().cpu().numpy(), host["k_pages"], host["v_pages"], table, lens,
                                q_len, causal, scale)
    d, L = q.shape[-1], max(1, int(np.max(lens)))
    live = ~np.isnan(LSE)
    empty = np.isneginf(LSE)
    got, gl = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert (got[empty] == 0).all() and np.isneginf(gl[empty]).all()
    some = live & ~empty
    x = X[..., None]
    tol = A * U * (2 * ((d + 4) * x + 4) + 2 * L + 16)
    if dt == "bf16":
        tol = tol + 2.0 ** -8 * ((1 + 2.0 ** -8) * A + np.abs(O)) * (1 + 2.0 ** -8)
    err = np.abs(got - O)
    assert (err <= tol)[some].all(), f"O: worst error / bound {np.nanmax((err / tol)[some])}"
    tl = U * ((d + 4) * X + 4 + L + 16 + 2 * np.abs(np.where(empty, 0, LSE)))
    el = np.abs(np.where(empty, 0, gl) - np.where(empty, 0, LSE))
    assert (el <= tl)[some].all(), f"LSE: worst error / bound {np.nanmax((el / tl)[some])}"
    return live


CASES = [
    # lens, H, Hkv, n, d, dv, page, causal, dtype
    ((1,), 1, 1, 1, 64, 64, 16, True, "bf16"),                       # one token
    ((0, 1, 2, 63, 64, 65), 8, 2, 1, 128, 128, 16, True, "bf16"),    # an empty sequence; tile borders
    ((700, 129, 1000), 32, 8, 1, 128, 128, 16, True, "bf16"),
    ((513, 77), 16, 16, 1, 64, 64, 32, True, "bf16"),                # heads not shared
    ((300, 5, 64), 16, 1, 1, 128, 128, 64, True, "bf16"),            # one key head for all
    ((95, 640), 48, 2, 1, 128, 128, 128, True, "bf16"),              # 24 rows per key head
    ((260, 1), 6, 2, 5, 64, 64, 256, True, "bf16"),                  # a draft; fewer keys than queries
    ((33, 150), 8, 2, 9, 128, 128, 8, True, "bf16"),                 # 36 rows, the smallest page
    ((200, 64), 4, 4, 4, 128, 128, 16, False, "bf16"),               # not causal
    ((150, 90), 6, 3, 2, 40, 72, 16, True, "bf16"),                  # odd widths
    ((150, 90), 6, 3, 1, 8, 128, 8, True, "bf16"),
    ((150, 90), 2, 1, 3, 96, 16, 32, True, "bf16"),
    ((150, 0, 70), 72, 1, 1, 128, 128, 16, True, "bf16"),            # more rows than one item takes
    ((150, 3, 70), 30, 2, 5, 64, 128, 16, True, "bf16"),             # 75 rows, the last item nearly empty
    ((150, 3, 70), 26, 2, 4, 128, 64, 32, True, "bf16"),
    ((700, 64, 1, 0, 130), 40, 1, 1, 128, 128, 16, True, "bf16"),    # one to eleven key tiles; none
    ((400, 65), 16, 1, 8, 64, 64, 64, True, "bf16"),                 # 128 rows
    ((400, 65), 17, 1, 8, 128, 64, 8, False, "bf16"),                # 136: a second item of 8
    ((129, 300), 36, 1, 1, 72, 40, 256, True, "bf16"),               # odd widths
    ((1,), 2, 1, 1, 64, 64, 16, True, "f32"),
    ((0, 1, 63, 64, 65, 129), 8, 2, 1, 128, 128, 16, True, "f32"),
    ((700, 129), 20, 4, 1, 64, 64, 16, True, "f32"),
    ((333, 40), 7, 1, 5, 36, 100, 8, True, "f32"),                   # 35 rows, odd widths
    ((95, 300), 24, 2, 3, 128, 128, 64, False, "f32"),
    ((50, 260), 3, 3, 1, 4, 4, 256, True, "f32"),
]


# A long table row alone decides how a call is split: short rows and few items
# are taken by teams of CTAs, one launch; else the split goes over all CTAs.
SPLITS = pytest.mark.parametrize("room", [None, 5000], ids=["short_rows", "long_rows"])


def width(lens, page, room):
    return None if room is None else -(-max(room, *lens) // page) + 2


@SPLITS
@pytest.mark.parametrize("lens,H,Hkv,n,d,dv,page,causal,dt", CASES)
def test_decode(lens, H, Hkv, n, d, dv, page, causal, dt, room):
    rng = np.random.default_rng(len(lens) * 1000 + d + n)
    dev, host = on_gpu(numpy_cache(rng, len(lens), Hkv, page, d, dv, lens, M=width(lens, page, room)), dt)
    q = torch.tensor(rng.standard_normal((len(lens), H, n, d)), device="cuda").to(DT[dt])
    o, lse = run(dev, q, causal)
    compare(o, lse, dt, host, q, causal)


@pytest.mark.parametrize("dt,H", [("bf16", 8), ("bf16", 48), ("bf16", 100), ("f32", 8), ("f32", 16), ("f32", 40)])
def test_split_and_joined(dt, H):
    """Lengths far apart: the long sequence is cut over many CTAs."""
    rng = np.random.default_rng(5)
    lens = (9000, 3, 130, 0, 2500)
    dev, host = on_gpu(numpy_cache(rng, 5, 2, 16, 64, 64, lens), dt)
    q = torch.tensor(rng.standard_normal((5, H, 1, 64)), device="cuda").to(DT[dt])
    o, lse = run(dev, q)
    compare(o, lse, dt, host, q)
    again = run(dev, q)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@SPLITS
@pytest.mark.parametrize("dt,H", [("bf16", 4), ("bf16", 40), ("f32", 4)])
def test_large_scores(dt, H, room):
    """Scores of several hundred, of both signs of the scale, and a zero scale."""
    rng = np.random.default_rng(6)
    dev, host = on_gpu(numpy_cache(rng, 2, 2, 16, 64, 64, (400, 90), M=width((400,), 16, room)), dt)
    q = torch.tensor(20 * rng.standard_normal((2, H, 2, 64)), device="cuda").to(DT[dt])
    for scale in (1.0, -1.0, 0.0):
        o, lse = run(dev, q, scale=scale)
        compare(o, lse, dt, host, q, scale=scale)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 4, 15])
@SPLITS
def test_ragged_queries_leave_other_rows(dt, n, room):
    rng = np.random.default_rng(7)
    lens, q_len = (70, 0, 200, 129, 3), (n, n, 0, max(1, n - 1), n)
    dev, host = on_gpu(numpy_cache(rng, 5, 2, 8, 64, 64, lens, M=width(lens, 8, room)), dt)
    q = torch.tensor(rng.standard_normal((5, 6, n, 64)), device="cuda").to(DT[dt])
    out = torch.full((5, 6, n, 64), 7.0, dtype=DT[dt], device="cuda")
    lse = torch.full((5, 6, n), 7.0, device="cuda")
    o, l = run(dev, q, q_len=q_len, out=out, lse=lse)
    assert o.data_ptr() == out.data_ptr() and l.data_ptr() == lse.data_ptr()
    live = compare(o, l, dt, host, q, q_len=q_len)
    rest = torch.tensor(~live, device="cuda")
    assert (o[rest] == 7).all() and (l[rest] == 7).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("page", [8, 64])
@pytest.mark.parametrize("H", [4, 24])
@SPLITS
def test_unused_rows_have_no_influence(dt, page, H, room):
    """NaN and infinities in every row that no token owns, free pages included,
    and table entries past the last page that lead nowhere."""
    rng = np.random.default_rng(8)
    lens = (1, 65, 131, 0)
    c = numpy_cache(rng, 4, 2, page, 64, 64, lens, M=width(lens, page, room))
    q = torch.tensor(rng.standard_normal((4, H, 3, 64)), device="cuda").to(DT[dt])
    dev, host = on_gpu(c, dt)
    want = run(dev, q)
    compare(*want, dt, host, q)
    used = np.zeros(c["k_pages"].shape[:1] + (page,), dtype=bool)
    for b, L in enumerate(lens):
        t = np.arange(L)
        used[c["table"][b, t // page], t % page] = True
        c["table"][b, -(-L // page):] = rng.integers(-2 ** 31, 2 ** 31 - 1, size=c["table"].shape[1] + L // -page)
    for pool, bad in (("k_pages", np.nan), ("v_pages", np.inf)):
        c[pool].transpose(0, 2, 1, 3)[~used] = bad
    c["v_pages"].transpose(0, 2, 1, 3)[~used] = np.where(rng.random(c["v_pages"].transpose(0, 2, 1, 3)[~used].shape) < 0.5,
                                                         np.nan, -np.inf)
    dev, _ = on_gpu(c, dt)
    got = run(dev, q)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("H", [2, 12, 20])
@SPLITS
def test_later_tokens_of_a_draft_have_no_influence(dt, H, room):
    """An infinite or NaN key or value of a draft's last tokens reaches the
    queries that see it and no other."""
    rng = np.random.default_rng(9)
    lens, n = (64, 70, 8), 5
    c = numpy_cache(rng, 3, 1, 16, 64, 64, lens, M=width(lens, 16, room))
    q = torch.tensor(rng.standard_normal((3, H, n, 64)), device="cuda").to(DT[dt])
    dev, host = on_gpu(c, dt)
    want = run(dev, q)
    compare(*want, dt, host, q)
    for pool, bad in (("v_pages", np.nan), ("v_pages", np.inf), ("k_pages", np.nan)):
        dirty = {k: v.copy() for k, v in c.items()}
        for b, L in enumerate(lens):
            t = L - 2                                       # seen by the last two queries
            dirty[pool][c["table"][b, t // 16], 0, t % 16, 7] = bad
        o, lse = run(on_gpu(dirty, dt)[0], q)
        assert torch.equal(lse[..., :3], want[1][..., :3])
        # the weights meet the finite values by another route: same sums to rounding
        assert (o[..., :3, :].float() - want[0][..., :3, :].float()).abs().max() <= 2.0 ** -7 * want[0].float().abs().max()
        reached = o[..., 3:, 7] if pool == "v_pages" else lse[..., 3:]
        assert not torch.isfinite(reached).any()
        if pool == "v_pages":
            rest = [x for x in range(64) if x != 7]
            assert torch.isfinite(o[..., rest]).all() and torch.equal(lse, want[1])


@pytest.mark.parametrize("dt,H", [("bf16", 4), ("bf16", 44), ("f32", 4)])
def test_bad_page_numbers_and_lengths(dt, H):
    """Page numbers outside the pool mask their tokens; lengths are clamped."""
    rng = np.random.default_rng(10)
    c = numpy_cache(rng, 3, 2, 16, 64, 64, (100, 100, 100), M=7)
    P = c["ref"].shape[0]
    c["table"][0, :7] = [c["table"][0, 0], -1, P, 2 ** 31 - 1, -2 ** 31, c["table"][0, 5], c["table"][0, 6]]
    c["table"][1, :7] = -1                                 # nothing left: an empty row
    c["lens"] = np.array([100, 100, -5], dtype=np.int32)
    dev, host = on_gpu(c, dt)
    q = torch.tensor(rng.standard_normal((3, H, 2, 64)), device="cuda").to(DT[dt])
    compare(*run(dev, q), dt, host, q)
    c["lens"] = np.array([2 ** 31 - 1, 5, 1000], dtype=np.int32)     # the row holds 112
    c["table"][2, 6] = 0
    dev, host = on_gpu(c, dt)
    compare(*run(dev, q), dt, host, dict(q=q)["q"])


def test_pages_past_32_bits():
    """A pool of more than 2^32 bytes per half, pages at both ends of it."""
    P, Hkv, page, d = 20000, 8, 128, 128                    # 2.6e9 elements per pool
    k = torch.empty(P, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    g = torch.Generator(device="cuda").manual_seed(1)
    picks = [P - 1, 0, P - 2, P // 2, 16384, 16383]
    for p in picks:
        k[p] = torch.randn(Hkv, page, d, device="cuda", generator=g).to(k.dtype)
        v[p] = torch.randn(Hkv, page, d, device="cuda", generator=g).to(k.dtype)
    q = torch.randn(2, 16, 1, d, device="cuda", generator=g).to(k.dtype)
    lens = torch.tensor([300, 290], dtype=torch.int32, device="cuda")
    o, lse = lib.attn_decode(q, k, v, torch.tensor([picks[:3], picks[3:]], dtype=torch.int32, device="cuda"), lens)
    ks, vs = k[picks].clone(), v[picks].clone()
    small = torch.tensor([[0, 1, 2], [3, 4, 5]], dtype=torch.int32, device="cuda")
    o2, lse2 = lib.attn_decode(q, ks, vs, small, lens)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    host = dict(k_pages=ks.double().cpu().numpy(), v_pages=vs.double().cpu().numpy(),
                table=small.cpu().numpy(), lens=lens.cpu().numpy())
    compare(o, lse, "bf16", host, q)


def test_many_sequences():
    """More sequences than threads of a block, most of them short or idle."""
    rng = np.random.default_rng(11)
    B = 700
    lens = rng.integers(0, 20, size=B)
    lens[[3, 500]] = (900, 1500)
    q_len = rng.integers(0, 2, size=B)
    dev, host = on_gpu(numpy_cache(rng, B, 1, 8, 64, 64, lens), "bf16")
    q = torch.tensor(rng.standard_normal((B, 2, 1, 64)), device="cuda").to(torch.bfloat16)
    out = torch.zeros(B, 2, 1, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = run(dev, q, q_len=q_len, out=out)
    compare(o, lse, "bf16", host, q, q_len=q_len)
    assert (run(dev, q, q_len=np.zeros(B, dtype=np.int32), out=out.clone().fill_(3))[0] == 3).all()


@SPLITS
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_captured_streams_and_workspaces(dt, room):
    """A captured call replayed on new inputs in place; calls at once on two
    streams with workspaces of their own; a workspace of any contents."""
    rng = np.random.default_rng(12)
    lens = (700, 20)
    dev, host = on_gpu(numpy_cache(rng, 2, 2, 16, 64, 64, lens, M=width(lens, 16, room)), dt)
    qs = [torch.tensor(rng.standard_normal((2, 4, 1, 64)), device="cuda").to(DT[dt]) for _ in range(2)]
    want = [run(dev, q) for q in qs]
    need = lib.attn_decode_workspace_size(2, 4, 2, 1, 64, 64, DT[dt])
    ws = [torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [lib.attn_decode(q, dev["k_pages"], dev["v_pages"], dev["table"], dev["lens"], workspace=w, stream=s)
           for q, w, s in zip(qs, ws, streams) for _ in range(3)]
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i // 3][0]) and torch.equal(l, want[i // 3][1])
    q = qs[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, l = lib.attn_decode(q, dev["k_pages"], dev["v_pages"], dev["table"], dev["lens"])
    for i in (1, 0):
        q.copy_(qs[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])


def test_paths():
    """attn_set_path holds for attn_decode: the CUDA-core path for both types,
    the tensor-core path for bf16 alone."""
    rng = np.random.default_rng(14)
    for dt in ("bf16", "f32"):
        dev, host = on_gpu(numpy_cache(rng, 2, 2, 16, 64, 64, (200, 30)), dt)
        q = torch.tensor(rng.standard_normal((2, 8, 2, 64)), device="cuda").to(DT[dt])
        try:
            lib.attn_set_path(lib.ATTN_PATH_SIMT)
            compare(*run(dev, q), dt, host, q)
            lib.attn_set_path(lib.ATTN_PATH_TENSOR)
            if dt == "bf16":
                compare(*run(dev, q), dt, host, q)
            else:
                with pytest.raises(lib.AttnError) as e:
                    run(dev, q)
                assert e.value.code == 4
        finally:
            lib.attn_set_path(lib.ATTN_PATH_AUTO)


def test_refusals():
    rng = np.random.default_rng(13)
    dev, _ = on_gpu(numpy_cache(rng, 2, 2, 16, 64, 64, (20, 30)), "bf16")
    q = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    args = (dev["k_pages"], dev["v_pages"], dev["table"], dev["lens"])
    for bad in (q[:1], q.float(), q[..., :32].contiguous(), q.cpu(), q.transpose(1, 2)):
        with pytest.raises((ValueError, TypeError, lib.AttnError)):
            lib.attn_decode(bad, *args)
    with pytest.raises(TypeError):
        lib.attn_decode(q.half(), dev["k_pages"].half(), dev["v_pages"].half(), *args[2:])
    with pytest.raises(ValueError):
        lib.attn_decode(q, *args[:2], dev["table"].long(), dev["lens"])
    with pytest.raises(ValueError):
        lib.attn_decode(q, *args[:3], dev["lens"][:1])
    with pytest.raises(ValueError):
        lib.attn_decode(q, *args, q_len=torch.ones(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        lib.attn_decode(q, *args, out=torch.empty(2, 4, 1, 32, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(lib.AttnError) as e:
        lib.attn_decode(torch.zeros(2, 5, 1, 64, dtype=torch.bfloat16, device="cuda"), *args)
    assert e.value.code == 2
    with pytest.raises(lib.AttnError) as e:
        lib.attn_decode(q, *args, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.code == 6
    with pytest.raises(lib.AttnError) as e:
        lib.attn_decode(q, *args, out=q)
    assert e.value.code == 9


@SPLITS
@pytest.mark.parametrize("dt,H", [("bf16", 6), ("bf16", 40), ("f32", 6)])
def test_a_query_of_nan_stays_its_own(dt, H, room):
    rng = np.random.default_rng(15)
    lens = (130, 20)
    dev, _ = on_gpu(numpy_cache(rng, 2, 2, 16, 64, 64, lens, M=width(lens, 16, room)), dt)
    q = torch.tensor(rng.standard_normal((2, H, 2, 64)), device="cuda").to(DT[dt])
    want = run(dev, q)
    q[0, 1, 1, 5] = float("nan")
    o, lse = run(dev, q)
    other = torch.ones(2, H, 2, dtype=torch.bool, device="cuda")
    other[0, 1, 1] = False
    assert torch.isnan(o[0, 1, 1]).all() and torch.isnan(lse[0, 1, 1])
    assert torch.equal(o[other], want[0][other]) and torch.equal(lse[other], want[1][other])


def test_launches_and_trace():
    """What a call launches, as the library counts and traces it."""
    rng = np.random.default_rng(16)
    for dt, room, H, names in (("bf16", None, 4, ["decode_tensor"]), ("bf16", 5000, 4, ["decode_tensor", "decode_join"]),
                               ("bf16", None, 80, ["decode_wide", "decode_join"]),
                               ("f32", None, 4, ["decode_f32", "decode_join"])):
        dev, host = on_gpu(numpy_cache(rng, 2, 2, 16, 64, 64, (90, 30), M=width((90,), 16, room)), dt)
        q = torch.tensor(rng.standard_normal((2, H, 1, 64)), device="cuda").to(DT[dt])
        lib.attn_trace_begin(8)
        try:
            o, lse = run(dev, q)
        finally:
            trace = lib.attn_trace_end()
        assert [name for name, _ in trace] == names
        assert lib.attn_last_launch_count() == len(names)
        compare(o, lse, dt, host, q)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_after_a_timeout_until_it_is_read(dt):
    """While the error word is set a call returns and changes nothing outside its
    outputs; once it has been read, calls work again."""
    rng = np.random.default_rng(17)
    for room, H in ((None, 4), (5000, 4), (None, 80)):
        dev, host = on_gpu(numpy_cache(rng, 2, 2, 16, 64, 64, (90, 30), M=width((90,), 16, room)), dt)
        q = torch.tensor(rng.standard_normal((2, H, 1, 64)), device="cuda").to(DT[dt])
        lib.attn_probe_timeout(1000)
        lib.attn_decode(q, dev["k_pages"], dev["v_pages"], dev["table"], dev["lens"])
        assert lib.attn_get_device_error() == lib.ATTN_ERR_DEVICE_TIMEOUT
        o, lse = run(dev, q)
        compare(o, lse, dt, host, q)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_shared_pages(dt):
    """Sequences over the same pages, and one whose row repeats a page."""
    rng = np.random.default_rng(18)
    c = numpy_cache(rng, 3, 2, 16, 64, 64, (64, 64, 64))
    c["table"][1, :3] = c["table"][0, :3]
    c["table"][2, :4] = c["table"][2, 0]
    dev, host = on_gpu(c, dt)
    q = torch.tensor(rng.standard_normal((3, 4, 1, 64)), device="cuda").to(DT[dt])
    compare(*run(dev, q), dt, host, q)


def test_long_drafts():
    """As many queries as a short prompt has: many items of query rows."""
    rng = np.random.default_rng(19)
    lens, n = (150, 100), 100
    dev, host = on_gpu(numpy_cache(rng, 2, 2, 16, 64, 64, lens), "bf16")
    q = torch.tensor(rng.standard_normal((2, 4, n, 64)), device="cuda").to(torch.bfloat16)
    compare(*run(dev, q), "bf16", host, q)


@pytest.mark.parametrize("dt,H", [("bf16", 40), ("bf16", 150), ("f32", 20)])
def test_many_rows_captured_and_at_once(dt, H):
    """Many query rows per key head: a call replayed on new queries, and calls at
    once on two streams, give what calls by themselves give."""
    rng = np.random.default_rng(20)
    lens = (1500, 70, 333)
    dev, host = on_gpu(numpy_cache(rng, 3, 2, 16, 64, 64, lens), dt)
    qs = [torch.tensor(rng.standard_normal((3, 2 * H, 1, 64)), device="cuda").to(DT[dt]) for _ in range(2)]
    want = [run(dev, q) for q in qs]
    compare(*want[0], dt, host, qs[0])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [lib.attn_decode(q, dev["k_pages"], dev["v_pages"], dev["table"], dev["lens"], stream=s)
           for _ in range(3) for q, s in zip(qs, streams)]
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(l, want[i % 2][1])
    q = qs[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, l = lib.attn_decode(q, dev["k_pages"], dev["v_pages"], dev["table"], dev["lens"])
    for i in (1, 0):
        q.copy_(qs[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])
    assert lib.attn_get_device_error() == 0


@pytest.mark.parametrize("H,d,dv,page", [(4, 128, 128, 16), (16, 128, 128, 64), (64, 128, 64, 8), (12, 72, 40, 16),
                                         (40, 128, 128, 32), (8, 64, 64, 16), (8, 48, 128, 16)])
def test_many_short_sequences(H, d, dv, page):
    """Several pieces in a row to every CTA, most of a single tile, some of none."""
    rng = np.random.default_rng(21)
    B, n = 400, 2
    lens = rng.integers(0, 150, size=B)
    lens[[0, 7, 250]] = (700, 0, 640)
    q_len = rng.integers(0, n + 1, size=B)
    dev, host = on_gpu(numpy_cache(rng, B, 4, page, d, dv, lens), "bf16")
    q = torch.tensor(rng.standard_normal((B, H, n, d)), device="cuda").to(torch.bfloat16)
    out = torch.full((B, H, n, dv), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, H, n), 7.0, device="cuda")
    run(dev, q, q_len=q_len, out=out, lse=lse)
    compare(out, lse, "bf16", host, q, q_len=q_len)
    idle = torch.tensor(np.arange(n)[None, :] >= q_len[:, None], device="cuda")
    assert (out.transpose(1, 2)[idle] == 7).all() and (lse.transpose(1, 2)[idle] == 7).all()
    again = run(dev, q, q_len=q_len, out=out.clone(), lse=lse.clone())
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@SPLITS
def test_a_query_of_nan_among_wide_heads(room):
    """d = 128: a query row that is not a number leaves the others as they are."""
    rng = np.random.default_rng(22)
    lens = (300, 64)
    dev, host = on_gpu(numpy_cache(rng, 2, 2, 16, 128, 128, lens, M=width(lens, 16, room)), "bf16")
    q = torch.tensor(rng.standard_normal((2, 12, 1, 128)), device="cuda").to(torch.bfloat16)
    want = run(dev, q)
    q[0, 2], q[1, 11] = float("nan"), float("inf")
    o, lse = run(dev, q)
    hit = torch.zeros(2, 12, 1, dtype=torch.bool, device="cuda")
    hit[0, 2] = hit[1, 11] = True
    assert torch.isnan(o[hit]).all() and torch.isnan(lse[hit]).all()
    for got, ref, mask in ((o, want[0], ~hit), (lse, want[1], ~hit)):
        assert torch.equal(got[mask], ref[mask])


KERNELS = pytest.mark.parametrize("dt,H,path", [("bf16", 4, "AUTO"), ("bf16", 24, "AUTO"), ("bf16", 40, "AUTO"),
                                                ("bf16", 12, "SIMT"), ("f32", 4, "AUTO"), ("f32", 8, "AUTO"),
                                                ("f32", 16, "AUTO")])


@SPLITS
@KERNELS
@pytest.mark.parametrize("d", [64, 128])
def test_infinite_scores(dt, H, path, d, room):
    """A score of +inf: LSE = +inf and O = softmax = NaN, for its query alone; with
    a score that is not a number beside it, both NaN. A score of -inf weighs nothing."""
    rng = np.random.default_rng(24)
    lens = (1300, 75)
    c = numpy_cache(rng, 2, 1, 16, d, d, lens, M=width(lens, 16, room))
    q = rng.standard_normal((2, H, 1, d))
    q[..., 7] = np.where(np.arange(H) % 3 == 1, 1.0, -1.0)[None, :, None]
    q = torch.tensor(q, device="cuda").to(DT[dt])
    up = torch.tensor(np.broadcast_to(np.arange(H)[None, :, None] % 3 == 1, (2, H, 1)).copy(), device="cuda")
    try:
        lib.attn_set_path(getattr(lib, f"ATTN_PATH_{path}"))
        for t in ((0, 0), (65, 64), (700, 70), (1299, 74)):
            runs = {}
            for bad in (1e4, np.inf):
                dirty = {k: v.copy() for k, v in c.items()}
                for b in range(2):
                    dirty["k_pages"][c["table"][b, t[b] // 16], 0, t[b] % 16, 7] = bad
                dev, _ = on_gpu(dirty, dt)
                runs[bad] = run(dev, q)
            o, lse = runs[np.inf]
            assert torch.isposinf(lse[up]).all() and torch.isnan(o[up]).all()
            # The others: the same weights, perhaps from another running maximum.
            # In bf16 the weights and the result are rounded once in each call (2^-8 of
            # sum P |v| <= max |v|); in fp32 errors are some (L + d) 2^-24 of it, below 2^-12.
            top = float(dev["v_pages"].float().abs().max())
            far = (o[~up].float() - runs[1e4][0][~up].float()).abs().max()
            assert far <= (4 * 2.0 ** -8 if dt == "bf16" else 2.0 ** -12) * top
            assert (lse[~up] - runs[1e4][1][~up]).abs().max() <= 2.0 ** -12 * 16
            # one more token with a score of NaN
            for b in range(2):
                dirty["k_pages"][c["table"][b, 2], 0, 3, 9] = np.nan
            o, lse = run(on_gpu(dirty, dt)[0], q)
            assert torch.isnan(lse).all() and torch.isnan(o).all()
    finally:
        lib.attn_set_path(lib.ATTN_PATH_AUTO)


@SPLITS
@KERNELS
def test_scores_of_minus_infinity_alone(dt, H, path, room):
    """Every score -inf: as if there were no key."""
    rng = np.random.default_rng(26)
    lens = (70, 1)
    c = numpy_cache(rng, 2, 1, 16, 64, 64, lens, M=width(lens, 16, room))
    c["k_pages"][..., 7] = -np.inf
    q = rng.standard_normal((2, H, 1, 64))
    q[..., 7] = 1.0
    q = torch.tensor(q, device="cuda").to(DT[dt])
    try:
        lib.attn_set_path(getattr(lib, f"ATTN_PATH_{path}"))
        o, lse = run(on_gpu(c, dt)[0], q)
        assert (o == 0).all() and torch.isneginf(lse).all()
    finally:
        lib.attn_set_path(lib.ATTN_PATH_AUTO)


@SPLITS
@KERNELS
@pytest.mark.parametrize("n", [1, 4])
def test_values_not_finite_of_a_vanishing_weight(dt, H, path, n, room):
    """A weight that underflows to zero is not a mask: an infinite or NaN value of a
    token reaches every query that sees it, wherever in a tile the token lies,
    and no other."""
    rng = np.random.default_rng(25)
    lens, heads = (1300, 75), max(1, H // n)
    c = numpy_cache(rng, 2, 1, 16, 64, 64, lens, M=width(lens, 16, room))
    q = rng.standard_normal((2, heads, n, 64))
    q[..., 7] = 8.0
    q = torch.tensor(q, device="cuda").to(DT[dt])
    try:
        lib.attn_set_path(getattr(lib, f"ATTN_PATH_{path}"))
        for back in (2, 1200, 20):
            for bad in (np.inf, np.nan):
                dirty = {k: v.copy() for k, v in c.items()}
                see = np.zeros((2, heads, n), dtype=bool)
                for b, L in enumerate(lens):
                    t = max(L - back, 0)
                    dirty["k_pages"][c["table"][b, t // 16], 0, t % 16, 7] = -2000.0     # score about -2000
                    dirty["v_pages"][c["table"][b, t // 16], 0, t % 16, 5] = bad
                    see[b] = t < L - (n - 1 - np.arange(n))
                o, lse = run(on_gpu(dirty, dt)[0], q)
                see = torch.tensor(see, device="cuda")
                assert torch.isfinite(lse).all()
                assert not torch.isfinite(o[..., 5][see]).any()
                assert torch.isfinite(o[..., 5][~see]).all()
                assert torch.isfinite(o[..., [x for x in range(64) if x != 5]]).all()
    finally:
        lib.attn_set_path(lib.ATTN_PATH_AUTO)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("room,H", [(None, 4), (5000, 4), (None, 48), (None, 80)])
def test_after_a_timeout_nothing_is_written(dt, room, H):
    """While the error word is set the call leaves its outputs as they were,
    whichever kernel takes it: a team, the split, two row groups, many rows."""
    rng = np.random.default_rng(23)
    dev, host = on_gpu(numpy_cache(rng, 2, 2, 16, 64, 64, (90, 30), M=width((90,), 16, room)), dt)
    q = torch.tensor(rng.standard_normal((2, H, 1, 64)), device="cuda").to(DT[dt])
    out = torch.full((2, H, 1, 64), 7.0, dtype=DT[dt], device="cuda")
    lse = torch.full((2, H, 1), 7.0, device="cuda")
    lib.attn_probe_timeout(1000)
    lib.attn_decode(q, dev["k_pages"], dev["v_pages"], dev["table"], dev["lens"], out=out, lse=lse)
    assert lib.attn_get_device_error() == lib.ATTN_ERR_DEVICE_TIMEOUT
    assert (out == 7).all() and (lse == 7).all()
    compare(*run(dev, q, out=out, lse=lse), dt, host, q)


@SPLITS
@KERNELS
def test_values_not_finite_where_every_score_is_minus_infinity(dt, H, path, room):
    """Zero weights alone: zero times an infinite value is not zero."""
    rng = np.random.default_rng(27)
    lens = (70, 700, 1)
    c = numpy_cache(rng, 3, 1, 16, 64, 64, lens, M=width(lens, 16, room))
    c["k_pages"][..., 7] = -np.inf
    for b, L in enumerate(lens):
        c["v_pages"][c["table"][b, (L - 1) // 32], 0, 0, 5] = np.inf
    q = rng.standard_normal((3, H, 1, 64))
    q[..., 7] = 1.0
    q = torch.tensor(q, device="cuda").to(DT[dt])
    try:
        lib.attn_set_path(getattr(lib, f"ATTN_PATH_{path}"))
        o, lse = run(on_gpu(c, dt)[0], q)
        assert torch.isnan(o[..., 5]).all() and torch.isneginf(lse).all()
        assert (o[..., [x for x in range(64) if x != 5]] == 0).all()
    finally:
        lib.attn_set_path(lib.ATTN_PATH_AUTO)
