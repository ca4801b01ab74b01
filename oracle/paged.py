"""Plain float64 oracle of the paged key-value cache and of the attention of
the newest tokens over it.

TEST INFRASTRUCTURE ONLY, like oracle/ref.py: tests alone import it, and it
shares no code with the kernels. Each function is the definition, token by
token and page by page, in the order in which it is said:

  decode    S_ij = scale * q_i . k_j over the tokens j of the sequence, found
            through the table; query i of the c newest tokens sees the tokens
            up to itself (if causal); softmax; O = P V; LSE. A query that sees
            nothing has O = 0 and LSE = -inf.
  append    a token at a time; the lowest free page at every page border.
  fork      the holders of every page counted; full pages shared; a partly
            filled last page has one holder, the others get copies.
  compact   the next live page past the front goes to the next hole.

Pinned by tests/test_paged_oracle.py: decode against oracle.ref's dense
attention on the same keys laid out in a row; the cache functions against a
model that keeps every sequence as a list of tokens, over random runs of calls.
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["decode", "append", "fork", "compact", "read_back", "INFO_OK", "INFO_NO_PAGES",
           "INFO_TABLE_FULL", "INFO_SHARED_TAIL"]

INFO_OK, INFO_NO_PAGES, INFO_TABLE_FULL, INFO_SHARED_TAIL = 0, 1, 2, 3


def _pages(length: int, page: int) -> int:
    return -(-length // page)


def decode(q, k_pages, v_pages, table, lens, q_len=None, causal=True, scale=None):
    """(O, LSE, A, X): A = sum_j P_ij |v_j| and X = max_j scale * sum_c |q_ic k_jc|
    are what error bounds need. Rows past q_len are NaN."""
    B, H, n, d = q.shape
    P, Hkv, page, dv = v_pages.shape
    M = table.shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    O = np.full((B, H, n, dv), np.nan)
    A = np.full((B, H, n, dv), np.nan)
    lse = np.full((B, H, n), np.nan)
    X = np.full((B, H, n), np.nan)
    for b in range(B):
        length = min(max(int(lens[b]), 0), M * page)
        c = n if q_len is None else min(max(int(q_len[b]), 0), n)
        t = np.arange(length)
        pages = table[b, t // page] if length else np.zeros(0, dtype=np.int64)
        there = (pages >= 0) & (pages < P)
        for h in range(H):
            hk = h // (H // Hkv)
            K = k_pages[pages[there], hk, t[there] % page]
            V = v_pages[pages[there], hk, t[there] % page]
            for i in range(c):
                see = length - (c - 1 - i) if causal else length
                seen = t[there] < see
                if not seen.any():
                    O[b, h, i], A[b, h, i], lse[b, h, i], X[b, h, i] = 0.0, 0.0, -np.inf, 0.0
                    continue
                s = (K[seen] @ q[b, h, i]) * scale
                top = s.max()
                e = np.exp(s - top)
                O[b, h, i] = (e @ V[seen]) / e.sum()
                A[b, h, i] = (e @ np.abs(V[seen])) / e.sum()
                lse[b, h, i] = top + math.log(e.sum())
                X[b, h, i] = (np.abs(K[seen]) @ np.abs(q[b, h, i])).max() * abs(scale)
    return O, lse, A, X


def append(k, v, k_pages, v_pages, table, lens, ref, new_len=None):
    """(k_pages, v_pages, table, lens, ref, info) after the call."""
    B, Hkv, n, _ = k.shape
    P, _, page, _ = k_pages.shape
    M = table.shape[1]
    new = [n if new_len is None else min(max(int(new_len[b]), 0), n) for b in range(B)]
    old = [min(max(int(x), 0), M * page) for x in lens]
    free = [p for p in range(P) if ref[p] <= 0]
    status = INFO_OK
    need = sum(_pages(old[b] + new[b], page) - _pages(old[b], page) for b in range(B))
    if need > len(free):
        status = INFO_NO_PAGES
    if any(old[b] + new[b] > M * page for b in range(B)):
        status = INFO_TABLE_FULL
    for b in range(B):
        if new[b] > 0 and old[b] % page:
            p = table[b, old[b] // page]
            if not 0 <= p < P or ref[p] != 1:
                status = INFO_SHARED_TAIL
    k_pages, v_pages, table, lens, ref = (x.copy() for x in (k_pages, v_pages, table, lens, ref))
    if status != INFO_OK:
        return k_pages, v_pages, table, lens, ref, (status, len(free), 0)
    for b in range(B):
        for i in range(new[b]):
            t = old[b] + i
            if t % page == 0:
                p = free.pop(0)
                table[b, t // page] = p
                ref[p] = 1
            p = table[b, t // page]
            k_pages[p, :, t % page] = k[b, :, i]
            v_pages[p, :, t % page] = v[b, :, i]
        lens[b] = old[b] + new[b]
    return k_pages, v_pages, table, lens, ref, (status, len(free), need)


def fork(k_pages, v_pages, table, lens, ref, src, keep=None):
    """(k_pages, v_pages, table, lens, ref, info) after the call."""
    P, _, page, _ = k_pages.shape
    B, M = table.shape
    old = [min(max(int(x), 0), M * page) for x in lens]
    L = []
    for b in range(B):
        s = int(src[b])
        if not 0 <= s < B:
            L.append(0)
        else:
            L.append(old[s] if keep is None else min(max(int(keep[b]), 0), old[s]))
    held = [int(x) for x in ref]
    made = table.copy()
    for b in range(B):
        for p in table[b, :_pages(old[b], page)]:
            if 0 <= p < P:
                held[p] -= 1
        made[b, :_pages(old[b], page)] = -1
    continues = {}
    for b in range(B):
        full = L[b] // page
        for j in range(full):
            p = table[src[b], j]
            made[b, j] = p
            if 0 <= p < P:
                held[p] += 1
        if L[b] % page:
            p = int(table[src[b], full])
            made[b, full] = p
            if 0 <= p < P:
                continues.setdefault(p, []).append(b)
    copies = []
    kept = set()
    for p, who in continues.items():
        stays = None
        if held[p] <= 0:
            own = [b for b in who if src[b] == b]
            stays = own[0] if own else who[0]
            kept.add(p)
        copies += [(b, p) for b in who if b != stays]
    free = [p for p in range(P) if held[p] <= 0 and p not in kept]
    if len(copies) > len(free):
        now = sum(1 for x in ref if x <= 0)
        return (k_pages.copy(), v_pages.copy(), table.copy(), lens.copy(), ref.copy(),
                (INFO_NO_PAGES, now, 0))
    ref = np.array([max(x, 0) for x in held], dtype=ref.dtype)
    for p in kept:
        ref[p] += 1
    k_new, v_new = k_pages.copy(), v_pages.copy()
    for b, p in sorted(copies):
        to = free.pop(0)
        rows = L[b] % page
        made[b, L[b] // page] = to
        ref[to] = 1
        k_new[to, :, :rows] = k_pages[p, :, :rows]
        v_new[to, :, :rows] = v_pages[p, :, :rows]
    return (k_new, v_new, made, np.array(L, dtype=lens.dtype), ref, (INFO_OK, len(free), len(copies)))


def compact(k_pages, v_pages, table, lens, ref):
    """(k_pages, v_pages, table, ref, remap, info) after the call."""
    P, _, page, _ = k_pages.shape
    B, M = table.shape
    live = [p for p in range(P) if ref[p] > 0]
    remap = np.full(P, -1, dtype=table.dtype)
    for p in live:
        remap[p] = p
    holes = [p for p in range(len(live)) if ref[p] <= 0]
    high = [p for p in live if p >= len(live)]
    k_pages, v_pages, ref, made = k_pages.copy(), v_pages.copy(), ref.copy(), table.copy()
    for hole, p in zip(holes, high):
        remap[p] = hole
        k_pages[hole], v_pages[hole] = k_pages[p], v_pages[p]
        ref[hole], ref[p] = ref[p], 0
    for b in range(B):
        for j in range(_pages(min(max(int(lens[b]), 0), M * page), page)):
            if 0 <= table[b, j] < P:
                made[b, j] = remap[table[b, j]]
    return k_pages, v_pages, made, ref, remap, (INFO_OK, P - len(live), len(holes))


def read_back(pages, table, length):
    """Rows [Hkv, length, width] of one sequence, through its table row."""
    page = pages.shape[2]
    t = np.arange(length)
    return pages[table[t // page], :, t % page].swapaxes(0, 1) if length else pages[:0, :, 0].swapaxes(0, 1)
