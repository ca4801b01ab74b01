// cache.cuh -- the books of a paged key-value cache (append, fork, compact)
// and the kernels that move its rows.
//
// A page is free when its reference count is zero (or, which no call makes,
// less). Pages are handed out
// lowest number first, so every result is a function of the inputs alone. The
// three book-keeping kernels run as one cluster of kBookCtas CTAs: their
// phases depend on one another through counts over all pages, and a cluster's
// hardware barrier separates them without a launch per phase. They work from
// device memory only, never through the host, and leave the list of rows to
// move in the workspace for the copy kernel launched after them.
//
// A table, length array or count array may be written in place (output ==
// input): every value that a phase overwrites has been read before the
// barrier in front of it, or is read and written by the same thread.
#pragma once

#include <cstdint>

#include "paged.cuh"

namespace attn {
namespace paged {

constexpr int kBookCtas = 1;
constexpr int kBookThreads = 1024;
constexpr int kBookWarps = kBookThreads / 32;
constexpr int kNone = 0x7fffffff;

// info[0]; the header documents the values.
enum : int { kInfoOk = 0, kInfoNoPages = 1, kInfoTableFull = 2, kInfoSharedTail = 3 };

struct Move {            // rows [0, rows) of every head of page src, to page dst
    int src, dst, rows, pad;
};

// Words of the control block at the start of the workspace.
enum : int { kCtlNeed = 0, kCtlFlags = 1, kCtlMoves = 2, kCtlSums = 32, kCtlFreed = 64, kCtlWords = 128 };

struct Books {
    Geometry g;
    const int* table;
    const int* lens;
    const int* ref;
    int* table_out;
    int* lens_out;
    int* ref_out;
    int* info;           // status, free pages, pages taken / copied / moved
    // workspace
    int* control;        // [kCtlWords]
    int* first;          // [B + 1]
    int* after;          // [B]
    int* start;          // [B]  append: old length; fork: last page of the source, if partly filled
    int* base;           // [P]
    int* key;            // [P]
    int* stage;          // [B, M]
    Move* moves;         // [max(B, P)]
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// All threads of the cluster meet, and see each other's earlier writes.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The pages of this warp: a contiguous range, ranges in the order of
// (CTA, warp), so that ranks follow page numbers.
__device__ __forceinline__ void page_range(int P, int* lo, int* hi) {
    const long long w = (long long)cluster_rank() * kBookWarps + (threadIdx.x >> 5);
    constexpr long long n = kBookCtas * kBookWarps;
    *lo = int(P * w / n);
    *hi = int(P * (w + 1) / n);
}

// How many pages of the warp's range satisfy the predicate.
template <typename F>
__device__ __forceinline__ int count_pages(int lo, int hi, F&& pred) {
    int c = 0;
#pragma unroll 4
    for (int p = lo + int(threadIdx.x & 31); p < hi; p += 32) c += pred(p) ? 1 : 0;
    return __reduce_add_sync(0xffffffffu, c);
}

// Rank of the warp's first hit among the hits of all CTAs: begin() before a
// cluster_sync, end() after it.
struct Ranker {
    int warp_before;
    __device__ void begin(int hits, int* scratch, int* sums) {
        int total;
        const int before = block_exclusive((threadIdx.x & 31) == 0 ? hits : 0, scratch, &total);
        warp_before = __shfl_sync(0xffffffffu, before, 0);
        if (threadIdx.x == 0) sums[cluster_rank()] = total;
    }
    __device__ int end(const int* sums, int* total) const {
        int before = 0, all = 0;
        for (int c = 0; c < kBookCtas; ++c) {
            const int s = sums[c];
            if (c < int(cluster_rank())) before += s;
            all += s;
        }
        *total = all;
        return before + warp_before;
    }
};

// This thread's contiguous share of the sequences, over one CTA.
__device__ __forceinline__ void thread_share(int B, int* b0, int* b1) {
    const int chunk = (B + kBookThreads - 1) / kBookThreads;
    *b0 = int(min((long long)B, (long long)threadIdx.x * chunk));
    *b1 = min(B, *b0 + chunk);
}

// ------------------------------------------------------------------- append
__global__ void __launch_bounds__(kBookThreads, 1) append_books(Books k, const int* new_len, int n) {
    __shared__ int scratch[33];
    const Geometry& g = k.g;
    const int tid = threadIdx.x, lane = tid & 31;
    const int rank = int(cluster_rank());
    const int gwarp = rank * kBookWarps + (tid >> 5);
    const int page_mask = (1 << g.page_log2) - 1, room = g.M << g.page_log2;

    // Free pages, and (first CTA) the pages that each sequence needs.
    int lo, hi;
    page_range(g.P, &lo, &hi);
    Ranker ranker;
    ranker.begin(count_pages(lo, hi, [&](int p) { return k.ref[p] <= 0; }), scratch, k.control + kCtlSums);
    if (rank == 0) {
        int b0, b1;
        thread_share(g.B, &b0, &b1);
        int need = 0, full = 0, shared = 0;
        for (int b = b0; b < b1; ++b) {
            const int len = clamp_len(k.lens[b], g);
            const int add = new_len ? min(max(new_len[b], 0), n) : n;
            if (add > room - len) {
                full = 1;
                continue;
            }
            if (add > 0 && (len & page_mask) != 0) {
                // The page that goes on being filled must be this sequence's alone.
                const int p = k.table[size_t(b) * g.M + (len >> g.page_log2)];
                if (!page_ok(p, g.P) || k.ref[p] != 1) shared = 1;
            }
            need += pages_of(len + add, g.page_log2) - pages_of(len, g.page_log2);
        }
        int total;
        int before = block_exclusive(need, scratch, &total);
        for (int b = b0; b < b1; ++b) {
            const int len = clamp_len(k.lens[b], g);
            int add = new_len ? min(max(new_len[b], 0), n) : n;
            if (add > room - len) add = 0;          // the call is refused as a whole below
            k.first[b] = before;
            k.start[b] = len;
            k.after[b] = len + add;
            before += pages_of(len + add, g.page_log2) - pages_of(len, g.page_log2);
        }
        full = __syncthreads_or(full);
        shared = __syncthreads_or(shared);
        if (tid == 0) {
            k.first[g.B] = total;
            k.control[kCtlNeed] = total;
            k.control[kCtlFlags] = shared ? kInfoSharedTail : full ? kInfoTableFull : kInfoOk;
        }
    }
    cluster_sync();

    int total_free;
    int at = ranker.end(k.control + kCtlSums, &total_free);
    const int need = k.control[kCtlNeed];
    int status = k.control[kCtlFlags];
    if (status == kInfoOk && need > total_free) status = kInfoNoPages;
    const bool ok = status == kInfoOk;
    if (rank == 0 && tid == 0) {
        k.info[0] = status;
        k.info[1] = total_free - (ok ? need : 0);
        k.info[2] = ok ? need : 0;
        k.control[kCtlMoves] = ok;                  // the copy kernel writes nothing otherwise
    }
    // The free page of rank q goes to the sequence b with first[b] <= q < first[b + 1].
    const bool same_ref = k.ref_out == k.ref;
    for (int p0 = lo; p0 < hi; p0 += 32) {
        if (same_ref && (!ok || at >= need)) break;
        const int p = p0 + lane;
        const int r = p < hi ? k.ref[p] : 1;
        const unsigned hits = __ballot_sync(0xffffffffu, r <= 0);
        const int q = at + __popc(hits & ((1u << lane) - 1u));
        at += __popc(hits);
        if (ok && r <= 0 && q < need) {
            int b0 = 0, b1 = g.B;                   // last b with first[b] <= q
            while (b1 - b0 > 1) {
                const int mid = (b0 + b1) >> 1;
                if (k.first[mid] <= q) b0 = mid;
                else b1 = mid;
            }
            const int slot = pages_of(k.start[b0], g.page_log2) + (q - k.first[b0]);
            k.table_out[size_t(b0) * g.M + slot] = p;
            k.ref_out[p] = 1;
        } else if (!same_ref && p < hi) {
            k.ref_out[p] = r;
        }
    }
    if (k.table_out != k.table) {
        for (int b = gwarp; b < g.B; b += kBookCtas * kBookWarps) {
            const int from = ok ? pages_of(k.start[b], g.page_log2) : 0;
            const int to = ok ? pages_of(k.after[b], g.page_log2) : 0;
            const size_t row = size_t(b) * g.M;
            for (int j = lane; j < g.M; j += 32)
                if (j < from || j >= to) k.table_out[row + j] = k.table[row + j];
        }
    }
    if (ok || k.lens_out != k.lens)
        for (int b = rank * kBookThreads + tid; b < g.B; b += kBookCtas * kBookThreads)
            k.lens_out[b] = ok ? k.after[b] : k.lens[b];
}

// New rows K [B, Hkv, n, wk], V [B, Hkv, n, wv] into their pages; widths in
// 16-byte units. One thread per 16 bytes.
constexpr int kCopyThreads = 256;

__global__ void __launch_bounds__(kCopyThreads)
append_rows(Geometry g, const uint4* __restrict__ K, const uint4* __restrict__ V, uint4* __restrict__ Kp,
            uint4* __restrict__ Vp, const int* __restrict__ table, const int* control, const int* start,
            const int* after, int n, int wk, int wv) {
    if (!control[kCtlMoves]) return;
    const int w = wk + wv, page = 1 << g.page_log2;
    const unsigned long long total = (unsigned long long)g.B * g.Hkv * n * w;
    for (unsigned long long x = (unsigned long long)blockIdx.x * kCopyThreads + threadIdx.x; x < total;
         x += (unsigned long long)gridDim.x * kCopyThreads) {
        const unsigned long long row = x / w;
        const int c = int(x - row * w);
        const unsigned long long bh = row / n;
        const int i = int(row - bh * n), b = int(bh / g.Hkv), h = int(bh - (unsigned long long)b * g.Hkv);
        const int t = start[b] + i;
        if (t >= after[b]) continue;
        const int p = table[size_t(b) * g.M + (t >> g.page_log2)];
        if (!page_ok(p, g.P)) continue;
        const size_t dst = (size_t(p) * g.Hkv + h) * page + (t & (page - 1));
        if (c < wk) Kp[dst * wk + c] = K[row * wk + c];
        else Vp[dst * wv + c - wk] = V[row * wv + c - wk];
    }
}

// --------------------------------------------------------------------- fork
// Sequence b becomes the first L_b tokens of sequence src[b]: full pages are
// shared, and a partly filled last page belongs to one sequence alone.
//   base(p) = ref(p) - (uses in the old rows) + (full uses in the new rows)
// counts who holds p besides its takers as a last page. With base(p) = 0 one
// taker keeps p (the one it belonged to, else the lowest); every other taker
// gets a copy in a fresh page.
__global__ void __launch_bounds__(kBookThreads, 1) fork_books(Books k, const int* src, const int* keep) {
    __shared__ int scratch[33];
    const Geometry& g = k.g;
    const int tid = threadIdx.x, lane = tid & 31;
    const int rank = int(cluster_rank());
    const int gwarp = rank * kBookWarps + (tid >> 5);
    const int gthread = rank * kBookThreads + tid;
    constexpr int kWarps = kBookCtas * kBookWarps, kThreads = kBookCtas * kBookThreads;
    const int page_mask = (1 << g.page_log2) - 1;
    int lo, hi;
    page_range(g.P, &lo, &hi);

    for (int p = gthread; p < g.P; p += kThreads) {
        k.base[p] = k.ref[p];
        k.key[p] = kNone;
    }
    cluster_sync();

    // Uses given up and taken. Pages that a sequence keeps in its own row cancel.
    for (int b = gwarp; b < g.B; b += kWarps) {
        const int len = clamp_len(k.lens[b], g), s = src[b];
        const bool valid = s >= 0 && s < g.B;
        int L = valid ? clamp_len(k.lens[s], g) : 0;
        if (valid && keep) L = min(max(keep[b], 0), L);
        const int had = pages_of(len, g.page_log2), full = L >> g.page_log2;
        const int* mine = k.table + size_t(b) * g.M;
        const int* from = k.table + size_t(valid ? s : b) * g.M;
        for (int j = (s == b ? full : 0) + lane; j < had; j += 32) {
            const int p = mine[j];
            if (page_ok(p, g.P)) atomicSub(k.base + p, 1);
        }
        if (s != b) {
            for (int j = lane; j < full; j += 32) {
                const int p = from[j];
                if (page_ok(p, g.P)) atomicAdd(k.base + p, 1);
                k.stage[size_t(b) * g.M + j] = p;
            }
        }
        if (lane == 0) {
            k.start[b] = (L & page_mask) != 0 ? from[full] : -1;
            k.after[b] = L;
        }
    }
    cluster_sync();

    auto order_of = [&](int b) { return src[b] == b ? b : b + g.B; };
    auto tail_of = [&](int b) {                        // a last page that can be followed, or -1
        const int p = k.start[b];
        return (k.after[b] & page_mask) != 0 && page_ok(p, g.P) ? p : -1;
    };
    for (int b = gthread; b < g.B; b += kThreads) {
        const int p = tail_of(b);
        if (p >= 0 && k.base[p] <= 0) atomicMin(k.key + p, order_of(b));
    }
    cluster_sync();

    // Who copies (in the order of sequences), and which pages are free.
    auto copies = [&](int b) {
        const int p = tail_of(b);
        return p >= 0 && (k.base[p] > 0 || k.key[p] != order_of(b));
    };
    Ranker ranker;
    ranker.begin(count_pages(lo, hi, [&](int p) { return k.base[p] <= 0 && k.key[p] == kNone; }), scratch,
                 k.control + kCtlSums);
    if (rank == 0) {
        int b0, b1;
        thread_share(g.B, &b0, &b1);
        int mine = 0, total;
        for (int b = b0; b < b1; ++b) mine += copies(b) ? 1 : 0;
        int at = block_exclusive(mine, scratch, &total);
        for (int b = b0; b < b1; ++b) {
            const bool c = copies(b);
            k.first[b] = c ? at : -1;
            if (c) {
                k.moves[at].src = k.start[b];
                k.moves[at].rows = k.after[b] & page_mask;
                ++at;
            }
        }
        if (tid == 0) k.control[kCtlNeed] = total;
    }
    cluster_sync();

    int total_free;
    int at = ranker.end(k.control + kCtlSums, &total_free);
    const int need = k.control[kCtlNeed];
    const bool ok = need <= total_free;
    const bool same_ref = k.ref_out == k.ref;
    int free_before = 0;                               // free pages of the counts as they came
    for (int p0 = lo; p0 < hi; p0 += 32) {
        const int p = p0 + lane;
        const int base = p < hi ? k.base[p] : 1, key = p < hi ? k.key[p] : kNone;
        const bool free_page = base <= 0 && key == kNone;
        const unsigned hits = __ballot_sync(0xffffffffu, free_page);
        const int q = at + __popc(hits & ((1u << lane) - 1u));
        at += __popc(hits);
        if (p >= hi) continue;
        if (ok) {
            const bool taken = free_page && q < need;
            if (taken) k.moves[q].dst = p;
            k.ref_out[p] = taken ? 1 : max(base, 0) + (key != kNone ? 1 : 0);
        } else {
            const int r = k.ref[p];
            free_before += r <= 0 ? 1 : 0;
            if (!same_ref) k.ref_out[p] = r;
        }
    }
    if (!ok) {
        int total;
        (void)block_exclusive(free_before, scratch, &total);
        if (tid == 0) k.control[kCtlFreed + rank] = total;
    }
    cluster_sync();
    if (rank == 0 && tid == 0) {
        int free_now = total_free - need;
        if (!ok) {
            free_now = 0;
            for (int c = 0; c < kBookCtas; ++c) free_now += k.control[kCtlFreed + c];
        }
        k.info[0] = ok ? kInfoOk : kInfoNoPages;
        k.info[1] = free_now;
        k.info[2] = ok ? need : 0;
        k.control[kCtlMoves] = ok ? need : 0;
    }

    const bool same_table = k.table_out == k.table;
    for (int b = gwarp; b < g.B; b += kWarps) {
        const size_t row = size_t(b) * g.M;
        const int old_len = k.lens[b];
        __syncwarp();
        if (!ok) {
            if (!same_table)
                for (int j = lane; j < g.M; j += 32) k.table_out[row + j] = k.table[row + j];
            if (lane == 0) k.lens_out[b] = old_len;
            continue;
        }
        const int had = pages_of(clamp_len(old_len, g), g.page_log2);
        const int L = k.after[b], full = L >> g.page_log2, has = pages_of(L, g.page_log2);
        const bool home = src[b] == b;
        const int c = k.first[b];
        const int last = c >= 0 ? k.moves[c].dst : k.start[b];
        // In place, a sequence's own row only changes from its last page on.
        const int end = same_table ? max(had, has) : g.M;
        for (int j = (same_table && home ? full : 0) + lane; j < end; j += 32) {
            int p;
            if (j < full) p = home ? k.table[row + j] : k.stage[row + j];
            else if (j < has) p = last;
            else p = j < had ? -1 : k.table[row + j];
            k.table_out[row + j] = p;
        }
        if (lane == 0) k.lens_out[b] = L;
    }
}

// ------------------------------------------------------------------ compact
// L live pages. The k-th live page at or past L moves to the k-th free page
// before L: the fewest moves, no page both read and written.
__global__ void __launch_bounds__(kBookThreads, 1) compact_books(Books k, int* remap) {
    __shared__ int scratch[33];
    const Geometry& g = k.g;
    const int tid = threadIdx.x, lane = tid & 31;
    const int rank = int(cluster_rank());
    const int gwarp = rank * kBookWarps + (tid >> 5);
    const int gthread = rank * kBookThreads + tid;
    constexpr int kThreads = kBookCtas * kBookThreads;
    int lo, hi;
    page_range(g.P, &lo, &hi);
    int* holes = k.base;
    int* high = k.key;

    Ranker ranker;
    ranker.begin(count_pages(lo, hi, [&](int p) { return k.ref[p] > 0; }), scratch, k.control + kCtlSums);
    cluster_sync();
    int live;
    int at = ranker.end(k.control + kCtlSums, &live);
    for (int p0 = lo; p0 < hi; p0 += 32) {
        const int p = p0 + lane;
        const bool is_live = p < hi && k.ref[p] > 0;
        const unsigned hits = __ballot_sync(0xffffffffu, is_live);
        const int q = at + __popc(hits & ((1u << lane) - 1u));   // live pages before p
        at += __popc(hits);
        if (p >= hi) continue;
        if (p < live && !is_live) holes[p - q] = p;               // p - q free pages before p
        if (p >= live && is_live) high[live - 1 - q] = p;         // numbered from the last one down
        // The free pages before L are as many as the live pages from L on.
        if (p == live) k.control[kCtlNeed] = p - q;
        if (!is_live) remap[p] = -1;
        else if (p < live) remap[p] = p;
    }
    if (gthread == 0 && live == g.P) k.control[kCtlNeed] = 0;
    cluster_sync();
    const int m = k.control[kCtlNeed];
    // A moved page's count goes to its hole. Counts of holes and of moved pages
    // are written by the second loop alone; the others stay.
    if (k.ref_out != k.ref) {
        for (int p = gthread; p < g.P; p += kThreads) {
            const int r = k.ref[p];
            if (r > 0 ? p < live : p >= live) k.ref_out[p] = r;
        }
    }
    for (int q = gthread; q < m; q += kThreads) {
        const int from = high[m - 1 - q], to = holes[q];
        remap[from] = to;
        k.ref_out[to] = k.ref[from];
        k.ref_out[from] = 0;
        k.moves[q] = Move{from, to, 1 << g.page_log2, 0};
    }
    if (gthread == 0) {
        k.info[0] = kInfoOk;
        k.info[1] = g.P - live;
        k.info[2] = m;
        k.control[kCtlMoves] = m;
    }
    cluster_sync();
    const bool same_table = k.table_out == k.table;
    for (int b = gwarp; b < g.B; b += kBookCtas * kBookWarps) {
        const int had = pages_of(clamp_len(k.lens[b], g), g.page_log2);
        const size_t row = size_t(b) * g.M;
        for (int j = lane; j < (same_table ? had : g.M); j += 32) {
            const int p = k.table[row + j];
            k.table_out[row + j] = j < had && page_ok(p, g.P) ? remap[p] : p;
        }
    }
}

// Rows [0, rows) of every head of the listed pages, K then V; widths in
// 16-byte units. One block per (move, head) at a time.
__global__ void __launch_bounds__(kCopyThreads)
move_rows(Geometry g, uint4* Kp, uint4* Vp, const int* control, const Move* moves, int wk, int wv) {
    const unsigned long long items = (unsigned long long)control[kCtlMoves] * g.Hkv;
    for (unsigned long long x = blockIdx.x; x < items; x += gridDim.x) {
        const unsigned long long q = x / g.Hkv;
        const int h = int(x - q * g.Hkv);
        const Move mv = moves[q];
        const size_t from = (size_t(mv.src) * g.Hkv + h) << g.page_log2;
        const size_t to = (size_t(mv.dst) * g.Hkv + h) << g.page_log2;
        for (int c = threadIdx.x; c < mv.rows * wk; c += kCopyThreads) Kp[to * wk + c] = Kp[from * wk + c];
        for (int c = threadIdx.x; c < mv.rows * wv; c += kCopyThreads) Vp[to * wv + c] = Vp[from * wv + c];
    }
}

}  // namespace paged
}  // namespace attn
