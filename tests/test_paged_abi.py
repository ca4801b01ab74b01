"""The paged cache's entry points on the CPU: argument checks before any CUDA
work, workspace sizes, and the binding's refusals."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    import scaled_dot_product_saving_b200 as m
    return m


# Fake device addresses, far apart; checks must answer before any is used.
def addr(i, off=0):
    return ctypes.c_void_p((i + 1) * (1 << 36) + off)


NUL = ctypes.c_void_p(0)
BIG = 1 << 34
OK_ON_CPU = 7             # every check passed: the launch fails without a device


def call(fn, ptrs, sizes, tail, change):
    """fn(*pointers, workspace bytes, *sizes, *tail) with named changes."""
    p = {name: addr(i) for i, name in enumerate(ptrs)}
    s = dict(sizes)
    t = dict(tail)
    wsb = change.pop("wsb", BIG)
    for key, value in change.items():
        (p if key in p else s if key in s else t)[key] = value
    return fn(*p.values(), wsb, *s.values(), *t.values())


def decode(L, **change):
    return call(L.lib.attn_decode, ("q", "kp", "vp", "table", "lens", "q_len", "o", "lse", "ws"),
                dict(B=2, H=8, Hkv=2, n=1, d=64, dv=64, P=32, page=16, M=8, dtype=1, causal=1),
                dict(scale=0.125, stream=NUL), change)


def append(L, **change):
    return call(L.lib.attn_cache_append,
                ("k", "v", "kp", "vp", "table", "lens", "ref", "new_len", "table_out", "lens_out",
                 "ref_out", "info", "ws"),
                dict(B=2, Hkv=2, n=3, d=64, dv=64, P=32, page=16, M=8, dtype=1), dict(stream=NUL), change)


def fork(L, **change):
    return call(L.lib.attn_cache_fork,
                ("kp", "vp", "table", "lens", "ref", "src", "keep", "table_out", "lens_out", "ref_out",
                 "info", "ws"),
                dict(B=2, Hkv=2, d=64, dv=64, P=32, page=16, M=8, dtype=1), dict(stream=NUL), change)


def compact(L, **change):
    return call(L.lib.attn_cache_compact,
                ("kp", "vp", "table", "lens", "ref", "table_out", "ref_out", "remap", "info", "ws"),
                dict(B=2, Hkv=2, d=64, dv=64, P=32, page=16, M=8, dtype=1), dict(stream=NUL), change)


ALL = [decode, append, fork, compact]
nocuda = pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses must not be launched on")


@nocuda
@pytest.mark.parametrize("f", ALL)
def test_valid_calls_reach_the_launch(L, f):
    assert f(L) == OK_ON_CPU
    assert f(L, dtype=0) == OK_ON_CPU
    assert f(L, page=8) == OK_ON_CPU and f(L, page=256) == OK_ON_CPU
    assert f(L, d=8, dv=128) == OK_ON_CPU
    assert f(L, dtype=0, d=4, dv=12) == OK_ON_CPU


@pytest.mark.parametrize("f", ALL)
def test_sizes(L, f):
    for name in ("B", "Hkv", "d", "dv", "P", "page", "M"):
        assert f(L, **{name: 0}) == 2, name
        assert f(L, **{name: -1}) == 2, name
    assert f(L, page=4) == 4 and f(L, page=512) == 4 and f(L, page=24) == 4
    assert f(L, d=136) == 4 and f(L, dv=136) == 4
    assert f(L, d=60) == 2 and f(L, dv=4) == 2             # rows of whole 16 bytes
    assert f(L, dtype=0, d=62) == 2
    assert f(L, dtype=2) == 3
    assert f(L, P=1 << 30) == 2                            # P * Hkv
    assert f(L, B=1 << 16, M=1 << 15) == 2                 # B * M
    assert f(L, M=1 << 27) == 2                            # M * page


@pytest.mark.parametrize("f", ALL)
def test_limits_leave_room_for_a_tile(L, f):
    """Tokens, pages and query rows are numbered in 32 bits, and so is what lies
    a tile past the last of them."""
    assert f(L, Hkv=1, H=8, P=(1 << 30) + 1) == 2 if f is decode else f(L, Hkv=1, P=(1 << 30) + 1) == 2
    for page in (8, 16, 256):
        assert f(L, B=1, page=page, M=(1 << 30) // page + 1) == 2
        assert f(L, B=1, page=page, M=(1 << 31) // page - 1) == 2
        if not torch.cuda.is_available():
            assert f(L, B=1, page=page, M=(1 << 30) // page) == OK_ON_CPU
    if f is decode:
        assert f(L, B=1, H=1, Hkv=1, n=(1 << 30) + 1) == 2
        assert f(L, B=(1 << 30) + 1, H=1, Hkv=1, M=1) == 2


@pytest.mark.parametrize("f", ALL)
def test_workspace(L, f):
    need = (L.attn_decode_workspace_size(2, 8, 2, 1, 64, 64, 1) if f is decode
            else L.attn_cache_workspace_size(2, 8, 32))
    assert need > 0
    assert f(L, wsb=need - 1) == 6
    assert f(L, ws=NUL) == 6
    assert f(L, ws=addr(40, 8)) == 5


@pytest.mark.parametrize("f,names,optional", [
    (decode, ("q", "kp", "vp", "table", "lens", "o", "lse"), ("q_len",)),
    (append, ("k", "v", "kp", "vp", "table", "lens", "ref", "table_out", "lens_out", "ref_out", "info"),
     ("new_len",)),
    (fork, ("kp", "vp", "table", "lens", "ref", "src", "table_out", "lens_out", "ref_out", "info"),
     ("keep",)),
    (compact, ("kp", "vp", "table", "lens", "ref", "table_out", "ref_out", "remap", "info"), ()),
])
def test_pointers(L, f, names, optional):
    ints = {"table", "lens", "ref", "table_out", "lens_out", "ref_out", "info", "src", "remap"}
    for name in names:
        assert f(L, **{name: NUL}) == 1, name
        assert f(L, **{name: addr(40, 2 if name in ints else 8)}) == 5, name
    for name in optional:
        assert f(L, **{name: addr(40, 2)}) == 5
        if not torch.cuda.is_available():
            assert f(L, **{name: NUL}) == OK_ON_CPU


def test_decode_sizes(L):
    assert decode(L, H=7) == 2                              # H % Hkv
    assert decode(L, H=0) == 2 and decode(L, n=0) == 2
    assert decode(L, scale=float("nan")) == 2 and decode(L, scale=float("inf")) == 2
    assert decode(L, B=1 << 15, H=1 << 10, n=1 << 6) == 2   # B * H * n
    assert append(L, n=0) == 2
    assert append(L, B=1 << 15, Hkv=1 << 10, n=1 << 6, M=1) == 2


@nocuda
def test_in_place_and_overlaps(L):
    """Outputs may be their inputs, and nothing else."""
    t, l, r = addr(20), addr(21), addr(22)
    assert append(L, table=t, table_out=t, lens=l, lens_out=l, ref=r, ref_out=r) == OK_ON_CPU
    assert fork(L, table=t, table_out=t, lens=l, lens_out=l, ref=r, ref_out=r) == OK_ON_CPU
    assert compact(L, table=t, table_out=t, ref=r, ref_out=r) == OK_ON_CPU
    assert append(L, table=t, table_out=addr(20, 16)) == 9   # shifted by some entries
    assert append(L, lens=l, ref_out=l) == 9                 # another array's input
    assert append(L, k=t, kp=t) == 9
    assert append(L, kp=t, vp=t) == 9
    assert fork(L, lens_out=l, src=l) == 9
    assert fork(L, table_out=t, ref_out=t) == 9
    assert compact(L, remap=r, ref=r) == 9
    assert compact(L, lens=l, ref_out=l) == 9
    assert decode(L, q=t, o=t) == 9
    assert decode(L, ws=t, kp=t) == 9
    assert decode(L, kp=t, vp=t) == OK_ON_CPU                # both only read


def test_workspace_sizes(L):
    r = lambda x: -(-x // 256) * 256
    def cache(B, M, P):
        return (r(512) + 2 * r(4 * B) + 2 * r(4 * P) + r(4 * B * M) + r(16 * max(B, P)))
    for args in ((1, 1, 1), (64, 1024, 20000), (300, 7, 5)):
        assert L.attn_cache_workspace_size(*args) == cache(*args)
    assert L.attn_cache_workspace_size(0, 1, 1) == 0 and L.attn_cache_workspace_size(1 << 16, 1 << 15, 1) == 0
    assert L.attn_decode_workspace_size(1, 7, 2, 1, 64, 64, 1) == 0
    assert L.attn_decode_workspace_size(1, 8, 2, 1, 64, 200, 1) == 0
    # bounded: pieces per CTA, whatever the batch and the lengths
    assert (L.attn_decode_workspace_size(512, 64, 8, 4, 128, 128, 1)
            == L.attn_decode_workspace_size(1, 64, 8, 4, 128, 128, 1) < 16 << 20)


def test_workspace_of_many_rows(L):
    """More than 32 rows per key head go through items of 128."""
    few, many = (L.attn_decode_workspace_size(4, H, 1, 1, 64, 128, 1) for H in (32, 33))
    assert few < many == L.attn_decode_workspace_size(4, 5000, 1, 1, 64, 128, 1) < 40 << 20
    assert decode(L, H=66, wsb=L.attn_decode_workspace_size(2, 66, 2, 1, 64, 64, 1) - 1) == 6


def test_binding_refuses_before_the_library(L):
    kp = torch.zeros(4, 2, 8, 64)
    with pytest.raises(ValueError, match="CUDA"):
        L.attn_decode(torch.zeros(1, 2, 1, 64), kp, kp, torch.zeros(1, 2, dtype=torch.int32),
                      torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        L.attn_cache_compact(kp, kp, torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                             torch.zeros(4, dtype=torch.int32))


def test_status_string_of_overlap(L):
    assert "overlap" in L.attn_status_string(9)


def test_workspace_has_room_for_every_cta(L):
    """Two pieces of an item for each of the CTAs that the GPU holds at once: on
    each of 148 SMs three of 16 rows at d = dv = 64 and two of 32, two of 16 rows and
    one of 32 at larger widths; a row is dv outputs, a maximum and a sum."""
    sms, ask = 148, L.attn_decode_workspace_size
    for rows, d, dv, ctas, tile in ((8, 64, 64, 3, 16), (24, 64, 64, 2, 32), (32, 48, 40, 2, 32), (16, 128, 128, 2, 16),
                                    (17, 128, 128, 1, 32), (33, 128, 128, 1, 128)):
        assert ask(4, rows, 1, 1, d, dv, 1) >= 2 * sms * ctas * tile * (dv + 2) * 4 + sms * ctas * 16, (rows, d, dv)


def test_workspace_size_is_zero_for_what_every_call_refuses(L):
    big = 1 << 30
    assert L.attn_cache_workspace_size(1, 1, big + 1) == 0 < L.attn_cache_workspace_size(1, 1, big)
    assert L.attn_cache_workspace_size(1, (big >> 3) + 1, 1) == 0 < L.attn_cache_workspace_size(1, big >> 3, 1)
    for d, dv, dtype in ((60, 64, 1), (64, 4, 1), (62, 64, 0), (64, 2, 0), (136, 64, 1)):
        assert L.attn_decode_workspace_size(1, 8, 2, 1, d, dv, dtype) == 0, (d, dv, dtype)
    assert L.attn_decode_workspace_size(1, 1, 1, big + 1, 64, 64, 1) == 0


def test_limits_of_single_calls(L):
    """At a limit a call goes on to the launch, past it it is refused."""
    def at(f, status, **change):
        if status != OK_ON_CPU or not torch.cuda.is_available():
            assert f(L, wsb=1 << 45, **change) == status, change

    def far(**sizes):                                     # pools and rows that do not meet
        names = ("k", "v", "kp", "vp", "table", "lens", "ref", "new_len", "table_out", "lens_out", "ref_out",
                 "info", "ws", "src", "keep")
        return {**sizes, **{x: ctypes.c_void_p((i + 1) << 48) for i, x in enumerate(names)}}

    app = lambda **s: {k: v for k, v in far(**s).items() if k not in ("src", "keep")}
    frk = lambda **s: {k: v for k, v in far(**s).items() if k not in ("k", "v", "new_len")}
    at(append, OK_ON_CPU, **app(B=1, Hkv=1, n=(1 << 30) - 1, d=8, dv=8))
    at(append, 2, **app(B=1, Hkv=1, n=1 << 30, d=8, dv=8))
    at(append, 2, **app(B=1 << 10, Hkv=1 << 10, n=1 << 10, d=8, dv=8))
    at(fork, OK_ON_CPU, **frk(B=1 << 29, M=1))
    at(fork, 2, **frk(B=(1 << 29) + 1, M=1))


def test_scale_whose_factor_in_base_two_is_not_finite(L):
    """Scores are taken in base 2: a scale that overflows there would make a score of
    zero one that is not a number."""
    for scale in (2.4e38, 3.4e38, -3e38):
        assert decode(L, scale=scale) == 2
    if not torch.cuda.is_available():
        assert decode(L, scale=2.3e38) == OK_ON_CPU and decode(L, scale=-2.3e38) == OK_ON_CPU
