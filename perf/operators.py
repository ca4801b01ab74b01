"""What is measured of the paged key-value cache and the attention that reads it.

Four operators of the library, each in plain torch and as a user calls it:

  attn_decode         attention of one new token (or the few tokens of a draft)
                      of every sequence over its pages, with grouped heads
  attn_cache_append   pages for new tokens, and their K and V rows written
  attn_cache_fork     sequence b becomes the first keep[b] tokens of src[b]:
                      beam reordering, forks, shared prefixes, roll-back, freeing
  attn_cache_compact  the live pages moved to the front of the pool

A cache is a pair of pools [P, Hkv, page, width] (K and V), a page table
[B, M], the lengths [B] and a reference count per page [P]; a page is free
when its count is zero. Integers are int32. The table, lengths and counts
that a call gives back are other arrays than those it reads, so a pass can be
repeated; the pools are changed in place, the same way in every pass.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # One user of a served model, a short chat: latency is all that counts.
        dict(name="decode_one_user", op="decode", B=1, H=32, Hkv=8, d=128, dv=128, page=16, n=1,
             lo=1000, hi=1000, ragged=False, causal=True, dtype="bf16"),
        # A served batch of ordinary size: chats of very different lengths.
        dict(name="decode_batch", op="decode", B=64, H=32, Hkv=8, d=128, dv=128, page=16, n=1,
             lo=128, hi=16384, ragged=False, causal=True, dtype="bf16"),
        # A few very long contexts (documents): the cache's length is the only parallelism.
        dict(name="decode_long", op="decode", B=4, H=32, Hkv=8, d=128, dv=128, page=64, n=1,
             lo=65536, hi=262144, ragged=False, causal=True, dtype="bf16"),
        # Checking drafts of up to five tokens, heads not shared, odd lengths.
        dict(name="decode_draft", op="decode", B=24, H=16, Hkv=16, d=64, dv=64, page=32, n=5,
             lo=101, hi=4093, ragged=True, causal=True, dtype="bf16"),
        # The library's fp32 type, as used to check a bf16 server against.
        dict(name="decode_f32", op="decode", B=8, H=16, Hkv=4, d=64, dv=64, page=16, n=1,
             lo=64, hi=8192, ragged=False, causal=True, dtype="f32"),
        # The step that goes before each decode: one token for every sequence.
        dict(name="append_token", op="append", B=128, Hkv=8, d=128, dv=128, page=16, n=1,
             lo=128, hi=4096, ragged=False, spare=0.25, dtype="bf16"),
        # Prompts of a batch written into the cache at once, padded to the longest.
        dict(name="append_prompts", op="append", B=8, Hkv=8, d=128, dv=128, page=64, n=4096,
             lo=1, hi=2000, ragged=True, spare=0.25, dtype="bf16"),
        # A chunk of odd size in small pages, unequal widths, fp32.
        dict(name="append_chunk_f32", op="append", B=3, Hkv=5, d=72, dv=40, page=8, n=257,
             lo=30, hi=900, ragged=True, spare=0.5, dtype="f32"),
        # Beam search: groups of four beams pick their parents anew after every token.
        dict(name="fork_beams", op="fork", B=16, Hkv=8, d=128, dv=128, page=16, lo=1800, hi=2200,
             kind="beams", spare=0.5, dtype="bf16"),
        # A large batch between two steps: some end, some restart from another's prefix, some roll back.
        dict(name="fork_mixed", op="fork", B=256, Hkv=8, d=128, dv=128, page=16, lo=64, hi=4096,
             kind="mixed", spare=0.25, dtype="bf16"),
        # A small pool after a few sequences ended.
        dict(name="compact_small", op="compact", B=8, Hkv=4, d=64, dv=64, page=16, lo=100, hi=700,
             spare=0.5, dtype="bf16"),
        # A pool of more than a gigabyte, two fifths of it freed here and there.
        dict(name="compact_large", op="compact", B=96, Hkv=8, d=128, dv=128, page=16, lo=500, hi=4096,
             spare=0.67, dtype="bf16"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "append", "fork", "compact"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    step = 8 if dtype == "bf16" else 4
    wide = rng.random() < 0.6
    d = rng.choice([64, 128]) if wide else step * rng.randint(1, 128 // step)
    dv = d if wide or rng.random() < 0.5 else step * rng.randint(1, 128 // step)
    page = rng.choice([8, 16, 16, 32, 64, 128, 256])
    Hkv = _log_uniform(rng, 1, 16)
    case = dict(op=op, Hkv=Hkv, d=d, dv=dv, page=page, dtype=dtype)
    row = Hkv * (d + dv) * BYTES[dtype]
    if op == "decode":
        B = _log_uniform(rng, 1, 160)
        group = rng.choice([1, 2, 3, 4, 4, 5, 6, 7, 8, 8, 16])
        n = rng.choice([1, 1, 1, 2, 3, 5, 8])
        # at most a gigabyte of keys and values, and a bounded number of products
        top = min(1.0e9 / (B * row), 3.0e11 / (2.0 * Hkv * group * n * (d + dv) * B), 262144)
        hi = max(n + 1, _log_uniform(rng, 32, max(64, int(top))))
        lo = max(n, _log_uniform(rng, max(1, hi // 64), hi))
        case.update(B=B, H=Hkv * group, n=n, lo=lo, hi=hi, ragged=n > 1 and rng.random() < 0.5,
                    causal=rng.random() < 0.9)
    else:
        B = _log_uniform(rng, 1, 256)
        top = max(64, int(min(8192, 0.7e9 / (B * row))))
        hi = _log_uniform(rng, 32, top)
        lo = _log_uniform(rng, max(1, hi // 32), hi)
        case.update(B=B, lo=lo, hi=hi, spare=round(rng.uniform(0.1, 0.8), 2))
        if op == "append":
            n = 1 if rng.random() < 0.4 else _log_uniform(rng, 1, top)
            case.update(n=n, ragged=n > 1 and rng.random() < 0.7)
        elif op == "fork":
            case.update(kind=rng.choice(["beams", "mixed"]))
    return case


def _lengths(case, B, lo, hi):
    """B lengths spread evenly over [lo, hi] on a logarithmic scale; a case has
    the same lengths whatever the seed, which only shuffles them."""
    return np.array([int(round(lo * (hi / lo) ** ((i + 0.5) / B))) for i in range(B)], dtype=np.int64)


def _news(case):
    """New tokens (or queries) of each sequence: n, or spread over [0, n]."""
    B, n = case["B"], case["n"]
    if not case["ragged"]:
        return np.full(B, n, dtype=np.int64)
    return np.array([int(round((i + 0.5) / B * n)) for i in range(B)], dtype=np.int64)


def _row_bytes(case):
    return case["Hkv"] * (case["d"] + case["dv"]) * BYTES[case["dtype"]]


def _plan(case, rng):
    """Host side of a cache: lengths, table, reference counts. Pages are handed
    out in random order, as in a pool that has been in use for a while."""
    B, page = case["B"], case["page"]
    lens = _lengths(case, B, case["lo"], case["hi"])
    rng.shuffle(lens)
    new = _news(case) if "n" in case else np.zeros(B, dtype=np.int64)
    rng.shuffle(new)
    if case["op"] == "decode":
        lens = np.maximum(lens, case["n"])    # the new tokens are in the cache already
    # sizes that do not depend on which sequence got which length
    most = int(new.max()) if case["op"] == "append" else 0
    M = -(-(int(lens.max()) + most) // page) + 1
    held = -(-lens // page)
    if case["op"] == "decode":
        P = int(held.sum())
    else:
        P = int(held.sum() * (1.0 + case["spare"])) + int((-(-new // page)).sum()) + 2 * B
    order = rng.permutation(P)
    table = np.full((B, M), -1, dtype=np.int64)
    ref = np.zeros(P, dtype=np.int64)
    at = 0
    for b in range(B):
        c = int(held[b])
        table[b, :c] = order[at:at + c]
        ref[order[at:at + c]] = 1
        at += c
    return lens, new, table, ref


def _fork_plan(case, lens, rng):
    """src and keep of a fork."""
    B = case["B"]
    b = np.arange(B)
    keep = np.full(B, 1 << 30, dtype=np.int64)
    if case["kind"] == "beams":
        group = b // 4 * 4
        src = group + rng.integers(0, np.minimum(4, B - group))
        return src, keep
    src = b.copy()
    kind = rng.permutation(B) % 8
    src[kind == 0] = -1                                            # ended: freed
    restart = kind == 1                                            # starts on another's prefix
    src[restart] = rng.integers(0, B, size=int(restart.sum()))
    keep[restart] = lens[src[restart]] * rng.integers(1, 9, size=int(restart.sum())) // 8
    back = kind == 2                                               # rolls back up to eight tokens
    keep[back] = np.maximum(lens[back] - rng.integers(1, 9, size=int(back.sum())), 0)
    return src, keep


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    lens, new, table, ref = _plan(case, rng)
    B, Hkv, page, d, dv = (case[k] for k in ("B", "Hkv", "page", "d", "dv"))
    P = ref.shape[0]

    def ints(a):
        return torch.tensor(a, dtype=torch.int32, device="cuda")

    def normal(*shape):
        return torch.randn(*shape, dtype=dt, device="cuda", generator=gen)

    s = dict(case=case, table=ints(table), lens=ints(lens), ref=ints(ref),
             k_pages=normal(P, Hkv, page, d), v_pages=normal(P, Hkv, page, dv))
    if case["op"] == "decode":
        s["q"] = normal(B, case["H"], case["n"], d)
        s["scale"] = 1.0 / math.sqrt(d)
        s["q_len"] = ints(new) if case["ragged"] else None
        s["out"] = torch.zeros(B, case["H"], case["n"], dv, dtype=dt, device="cuda")
        s["lse"] = torch.zeros(B, case["H"], case["n"], dtype=torch.float32, device="cuda")
    if case["op"] == "append":
        s["k"] = normal(B, Hkv, case["n"], d)
        s["v"] = normal(B, Hkv, case["n"], dv)
        s["new_len"] = ints(new) if case["ragged"] else None
    if case["op"] == "fork":
        src, keep = _fork_plan(case, lens, rng)
        s["src"], s["keep"] = ints(src), ints(keep)
    if case["op"] != "decode":
        s["table_out"], s["lens_out"] = torch.empty_like(s["table"]), torch.empty_like(s["lens"])
        s["ref_out"], s["remap"] = torch.empty_like(s["ref"]), torch.empty_like(s["ref"])
        s["info"] = torch.empty(3, dtype=torch.int32, device="cuda")
    if own:
        import scaled_dot_product_saving_b200 as lib
        if case["op"] == "decode":
            need = lib.attn_decode_workspace_size(B, case["H"], Hkv, case["n"], d, dv, dt)
        else:
            need = lib.attn_cache_workspace_size(B, table.shape[1], P)
        s["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    return s


# --------------------------------------------------------------- plain forms
def _plain_decode(s):
    """One sequence at a time: its pages gathered, all scores in fp32, those
    past the last visible key set to -inf, softmax, products."""
    case, q, table = s["case"], s["q"], s["table"]
    B, H, n, d = q.shape
    P, Hkv, page, _ = s["k_pages"].shape
    M = table.shape[1]
    out, lse = s["out"], s["lse"]
    j = torch.arange(M * page, device=q.device)
    i = torch.arange(n, device=q.device)
    for b in range(B):
        pages = table[b].long().clamp(0, P - 1)
        k = s["k_pages"][pages].transpose(0, 1).reshape(Hkv, M * page, d).float()
        v = s["v_pages"][pages].transpose(0, 1).reshape(Hkv, M * page, -1).float()
        count = n if s["q_len"] is None else s["q_len"][b]
        seen = s["lens"][b] - (count - 1 - i) if case["causal"] else s["lens"][b].expand(n)
        mask = (j[None, :] < seen[:, None]) & (table[b].repeat_interleave(page) >= 0)[None, :]
        qb = q[b].float().reshape(Hkv, H // Hkv, n, d)
        x = torch.einsum("hgid,hjd->hgij", qb, k) * s["scale"]
        x = torch.where(mask, x, torch.full_like(x, -math.inf))
        top = x.amax(-1, keepdim=True)
        top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
        e = torch.exp(x - top)
        z = e.sum(-1, keepdim=True)
        o = torch.einsum("hgij,hjd->hgid", e, v) / torch.where(z > 0, z, torch.ones_like(z))
        row = (top + torch.log(z)).reshape(H, n)
        live = (i < count)[None, :].expand(H, n)
        out[b] = torch.where(live[..., None], o.reshape(H, n, -1).to(out.dtype), out[b])
        lse[b] = torch.where(live, row, lse[b])
    return out, lse


def _lowest_free(free):
    """The free pages in order, then -1s."""
    P = free.shape[0]
    rank = torch.cumsum(free.long(), 0) - 1
    where = torch.where(free, rank, torch.full_like(rank, P))
    pages = torch.full((P + 1,), -1, dtype=torch.int64, device=free.device)
    pages[where] = torch.where(free, torch.arange(P, device=free.device), pages[:P])
    pages[P] = -1
    return pages


def _plain_append(s):
    table, lens, ref = s["table"].long(), s["lens"].long(), s["ref"].long()
    B, M = table.shape
    P, Hkv, page, _ = s["k_pages"].shape
    n = s["k"].shape[2]
    new = torch.full_like(lens, n) if s["new_len"] is None else s["new_len"].long().clamp(0, n)
    after = lens + new
    had, has = (lens + page - 1) // page, (after + page - 1) // page
    need = has - had
    first = torch.cumsum(need, 0) - need
    free = ref == 0
    pages = _lowest_free(free)
    slot = torch.arange(M, device=table.device)[None, :]
    fresh = (slot >= had[:, None]) & (slot < has[:, None])
    pick = pages[(first[:, None] + slot - had[:, None]).clamp(0, P)]
    shared = (new > 0) & (lens % page > 0) & (ref[table.gather(1, (lens // page).clamp(max=M - 1)[:, None])[:, 0]] != 1)
    status = torch.where(need.sum() > free.sum(), 1, 0)
    status = torch.where((after > M * page).any(), 2, status)
    status = torch.where(shared.any(), 3, status)
    ok = status == 0
    table = torch.where(fresh & ok, pick, table)
    taken = torch.zeros(P + 1, dtype=torch.int64, device=table.device)
    taken[torch.where(fresh, pick, torch.full_like(pick, P))] = 1
    ref = torch.where(ok, ref + taken[:P], ref)
    # every new row to its place: page table[b, t // page], row t % page
    b, i = torch.nonzero((torch.arange(n, device=table.device)[None, :] < new[:, None]) & ok, as_tuple=True)
    t = lens[b] + i
    at = table[b, t // page]
    s["k_pages"][at, :, t % page] = s["k"][b, :, i]
    s["v_pages"][at, :, t % page] = s["v"][b, :, i]
    taken_count = torch.where(ok, need.sum(), 0)
    info = torch.stack([status, (ref == 0).sum(), taken_count]).int()
    return (table.int(), torch.where(ok, after, lens).int(), ref.int(), info, s["k_pages"], s["v_pages"])


def _plain_fork(s):
    table, lens, ref = s["table"].long(), s["lens"].long(), s["ref"].long()
    src, keep = s["src"].long(), s["keep"].long()
    B, M = table.shape
    P, Hkv, page, _ = s["k_pages"].shape
    dev = table.device
    valid = (src >= 0) & (src < B)
    frm = src.clamp(0, B - 1)
    after = torch.where(valid, torch.minimum(keep.clamp(min=0), lens[frm]), torch.zeros_like(lens))
    had, full, has = (lens + page - 1) // page, after // page, (after + page - 1) // page
    rows = table[frm]
    slot = torch.arange(M, device=dev)[None, :]
    dump = torch.full_like(table, P)
    ones = torch.ones(B * M, dtype=torch.int64, device=dev)

    def uses(pages, mask):
        c = torch.zeros(P + 1, dtype=torch.int64, device=dev)
        return c.index_add_(0, torch.where(mask, pages, dump).reshape(-1), ones)[:P]

    base = ref - uses(table, slot < had[:, None]) + uses(rows, slot < full[:, None])
    # a partly filled last page stays with one sequence if nobody holds it in full
    tail = has > full
    tp = torch.where(tail, rows.gather(1, full.clamp(max=M - 1)[:, None])[:, 0], torch.full_like(full, P))
    me = torch.arange(B, device=dev)
    key = torch.where(src == me, me, me + B)
    base_d = torch.cat([base, base.new_ones(1)])
    lowest = torch.full((P + 1,), 2 * B, dtype=torch.int64, device=dev)
    lowest = lowest.scatter_reduce(0, torch.where(base_d[tp] == 0, tp, torch.full_like(tp, P)), key, "amin")
    copy = tail & ((base_d[tp] > 0) | (lowest[tp] != key))
    free = (base <= 0) & (lowest[:P] == 2 * B)
    pages = _lowest_free(free)
    pick = pages[(torch.cumsum(copy.long(), 0) - 1).clamp(0, P)]
    ok = copy.sum() <= free.sum()
    last = torch.where(copy, pick, tp)
    made = torch.where(slot < full[:, None], rows,
                       torch.where((slot == full[:, None]) & tail[:, None], last[:, None],
                                   torch.where(slot < had[:, None], torch.full_like(table, -1), table)))
    count = base.clamp(min=0) + uses(last[:, None].expand(B, M), (slot == 0) & tail[:, None])
    sel = torch.nonzero(copy & ok)[:, 0]
    put = (torch.arange(page, device=dev)[None, :] < (after[sel] % page)[:, None])[:, None, :, None]
    for pool in (s["k_pages"], s["v_pages"]):
        pool[pick[sel]] = torch.where(put, pool[tp[sel]], pool[pick[sel]])
    ref = torch.where(ok, count, ref)
    info = torch.stack([torch.where(ok, 0, 1), (ref == 0).sum(), torch.where(ok, copy.sum(), 0)]).int()
    return (torch.where(ok, made, table).int(), torch.where(ok, after, lens).int(), ref.int(), info,
            s["k_pages"], s["v_pages"])


def _plain_compact(s):
    table, lens, ref = s["table"].long(), s["lens"].long(), s["ref"].long()
    B, M = table.shape
    P, Hkv, page, _ = s["k_pages"].shape
    me = torch.arange(P, device=table.device)
    live = ref > 0
    L = live.sum()
    holes, high = torch.nonzero(~live & (me < L))[:, 0], torch.nonzero(live & (me >= L))[:, 0]
    remap = torch.where(live, me, torch.full_like(me, -1))
    remap[high] = holes
    s["k_pages"][holes] = s["k_pages"][high]
    s["v_pages"][holes] = s["v_pages"][high]
    ref = ref.clone()
    ref[holes] = ref[high]
    ref[high] = 0
    held = torch.arange(M, device=table.device)[None, :] < ((lens + page - 1) // page)[:, None]
    table = torch.where(held, remap[table.clamp(0, P - 1)], table)
    info = torch.stack([torch.zeros_like(L), P - L, torch.tensor(holes.numel(), device=table.device)]).int()
    return table.int(), ref.int(), remap.int(), info, s["k_pages"], s["v_pages"]


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"decode": _plain_decode, "append": _plain_append, "fork": _plain_fork,
                "compact": _plain_compact}[op](s)
    import scaled_dot_product_saving_b200 as lib
    pools = (s["k_pages"], s["v_pages"])
    outs = {k: s[k] for k in ("table_out", "ref_out", "info", "workspace") if k in s}
    if op == "decode":
        return lib.attn_decode(s["q"], *pools, s["table"], s["lens"], causal=s["case"]["causal"],
                               scale=s["scale"], q_len=s["q_len"], out=s["out"], lse=s["lse"],
                               workspace=s["workspace"])
    if op == "append":
        return lib.attn_cache_append(s["k"], s["v"], *pools, s["table"], s["lens"], s["ref"],
                                     new_len=s["new_len"], lens_out=s["lens_out"], **outs) + pools
    if op == "fork":
        return lib.attn_cache_fork(*pools, s["table"], s["lens"], s["ref"], s["src"], keep=s["keep"],
                                   lens_out=s["lens_out"], **outs) + pools
    return lib.attn_cache_compact(*pools, s["table"], s["lens"], s["ref"], remap=s["remap"],
                                  **outs) + pools


# ---------------------------------------------------------------- the cost
def work(case):
    """Bytes: what is read and written at least once. Decode reads the keys and
    values of every held token; append moves the new rows; fork and compact
    read the counts and write them, read and write the table entries that
    change, and move the rows of the partly filled pages or the moved pages."""
    B, page, es = case["B"], case["page"], BYTES[case["dtype"]]
    lens = _lengths(case, B, case["lo"], case["hi"])
    row = _row_bytes(case)
    if case["op"] == "decode":
        new = _news(case)
        tokens = float(np.maximum(lens, case["n"]).sum())
        H, d, dv = case["H"], case["d"], case["dv"]
        rows = float(new.sum()) * H
        per = rows / B
        return {"bytes": tokens * row + rows * ((d + dv) * es + 4) + 4.0 * tokens / page,
                "flops": 2.0 * per * (d + dv) * tokens}
    held = float((-(-lens // page)).sum())
    pages = held * (1.0 + case["spare"]) + 2.0 * B
    if case["op"] == "append":
        new = float(_news(case).sum())
        return {"bytes": 2.0 * new * row + 4.0 * pages, "flops": 0.0}
    if case["op"] == "fork":
        moved = B * (0.5 if case["kind"] == "beams" else 0.15)     # partly filled pages copied, about
        share = 0.7 if case["kind"] == "beams" else 0.25           # table rows that change, about
        return {"bytes": 2.0 * moved * row * page / 2 + 8.0 * pages + 8.0 * held * share, "flops": 0.0}
    high = held * (1.0 - held / pages)                             # live pages above the live count, about
    return {"bytes": 2.0 * high * row * page + 8.0 * pages + 8.0 * held, "flops": 0.0}


# -------------------------------------------------------------- 64-bit answers
def _host(t):
    return t.cpu().numpy().astype(np.int64)


def _exact_decode(s):
    """Key by key from the definition: softmax weights in 64 bits over the
    tokens a query may see, gathered token by token through the table."""
    case = s["case"]
    B, H, n, d = s["q"].shape
    P, Hkv, page, dv = s["v_pages"].shape
    table, lens = _host(s["table"]), _host(s["lens"])
    count = [n] * B if s["q_len"] is None else _host(s["q_len"]).tolist()
    out = torch.zeros(B, H, n, dv, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, H, n, dtype=torch.float64, device="cuda")
    kf, vf = s["k_pages"].view(P * Hkv * page, d), s["v_pages"].view(P * Hkv * page, dv)
    for b in range(B):
        token = np.arange(int(lens[b]))
        place = table[b, token // page] * (Hkv * page) + token % page
        for h in range(Hkv):
            at = torch.tensor(place + h * page, device="cuda")
            keys, values = kf[at].double(), vf[at].double()
            for i in range(int(count[b])):
                see = int(lens[b]) - (int(count[b]) - 1 - i if case["causal"] else 0)
                heads = slice(h * (H // Hkv), (h + 1) * (H // Hkv))
                if see <= 0:
                    lse[b, heads, i] = -math.inf
                    continue
                x = (s["q"][b, heads, i].double() @ keys[:see].T) * float(s["scale"])
                lse[b, heads, i] = torch.logsumexp(x, -1)
                out[b, heads, i] = torch.softmax(x, -1) @ values[:see]
    return out, lse


def _exact_append(s):
    """A token at a time, as a user's host code would keep the books."""
    table, lens, ref = _host(s["table"]), _host(s["lens"]), _host(s["ref"])
    B, M = table.shape
    page, n = s["k_pages"].shape[2], s["k"].shape[2]
    new = [n] * B if s["new_len"] is None else _host(s["new_len"]).tolist()
    free = [p for p in range(len(ref)) if ref[p] == 0]
    used, frm, to = 0, [], []
    for b in range(B):
        for i in range(int(new[b])):
            t = int(lens[b])
            if t % page == 0:
                table[b, t // page] = free[used]
                ref[free[used]] = 1
                used += 1
            frm.append((b, i))
            to.append((int(table[b, t // page]), t % page))
            lens[b] = t + 1
    k, v = s["k_pages"], s["v_pages"]
    if frm:
        fb, fi = (torch.tensor(c, device="cuda") for c in zip(*frm))
        tp, tr = (torch.tensor(c, device="cuda") for c in zip(*to))
        k[tp, :, tr] = s["k"][fb, :, fi]
        v[tp, :, tr] = s["v"][fb, :, fi]
    return table, lens, ref, np.array([0, len(free) - used, used]), k, v


def _exact_fork(s):
    """The holders of every page listed, then each rule applied as it is said."""
    table, lens, ref = _host(s["table"]), _host(s["lens"]), _host(s["ref"])
    src, keep = _host(s["src"]), _host(s["keep"])
    B = len(lens)
    P, page = len(ref), s["k_pages"].shape[2]
    after = [min(max(int(keep[b]), 0), int(lens[src[b]])) if 0 <= src[b] < B else 0 for b in range(B)]
    count = ref.copy()
    for b in range(B):
        for p in table[b, :-(-int(lens[b]) // page)]:
            count[p] -= 1
    made = table.copy()
    takers = {}
    for b in range(B):
        whole = after[b] // page
        made[b, :-(-int(lens[b]) // page)] = -1
        for j in range(whole):
            made[b, j] = table[src[b], j]
            count[made[b, j]] += 1
        if after[b] % page:
            takers.setdefault(int(table[src[b], whole]), []).append(b)
    copies = []
    keeper = {}
    for p, who in takers.items():
        stay = None
        if count[p] == 0:
            at_home = [b for b in who if src[b] == b]
            stay = (at_home or who)[0]
            keeper[p] = stay
        for b in who:
            if b == stay:
                made[b, after[b] // page] = p
            else:
                copies.append((b, p))
    for p in keeper:
        count[p] = 1
    free = [p for p in range(P) if count[p] == 0]
    k, v = s["k_pages"], s["v_pages"]
    for rank, (b, p) in enumerate(sorted(copies)):
        to = free[rank]                      # free afterwards: never one that is copied from
        made[b, after[b] // page] = to
        count[to] = 1
        for pool in (k, v):
            pool[to, :, :after[b] % page] = pool[p, :, :after[b] % page]
    return (made, np.array(after), count, np.array([0, len(free) - len(copies), len(copies)]), k, v)


def _exact_compact(s):
    """One page at a time: the next live page past the front goes to the next hole."""
    table, lens, ref = _host(s["table"]), _host(s["lens"]), _host(s["ref"])
    P, page = len(ref), s["k_pages"].shape[2]
    total = int((ref > 0).sum())
    remap = np.array([p if ref[p] > 0 else -1 for p in range(P)])
    high = [p for p in range(total, P) if ref[p] > 0]
    at = 0
    for hole in range(total):
        if ref[hole] == 0:
            p = high[at]
            at += 1
            remap[p] = hole
            ref[hole], ref[p] = ref[p], 0
            for pool in (s["k_pages"], s["v_pages"]):
                pool[hole] = pool[p]
    for b in range(len(lens)):
        for j in range(-(-int(lens[b]) // page)):
            table[b, j] = remap[table[b, j]]
    return table, ref, remap, np.array([0, P - total, at]), s["k_pages"], s["v_pages"]


def exact(case, seed):
    s = prepare(case, seed)
    answer = {"decode": _exact_decode, "append": _exact_append, "fork": _exact_fork,
              "compact": _exact_compact}[case["op"]](s)
    return tuple(torch.as_tensor(a) if isinstance(a, np.ndarray) else a for a in answer)
