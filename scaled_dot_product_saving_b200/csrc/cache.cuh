// cache.cuh -- the books of a paged key-value cache (append, fork, compact)
// and the kernels that move its rows.
//
// A page is free when its reference count is zero (or, which no call makes,
// less). Pages are handed out lowest number first, so every result is a
// function of the inputs alone. The three book-keeping kernels run as one
// cluster of kBookCtas CTAs: their phases depend on one another through counts
// over all pages, and a cluster's hardware barrier separates them without a
// launch per phase. They work from device memory only, never through the
// host, and leave the list of rows to move in the workspace.
//
// What bounds the books is latency: a phase is two or three dependent reads of
// L2 and a barrier, about 2 us, whatever the sizes up to some ten thousand
// pages. So a phase reads what it can at once, sums that can go together go
// through one scan, and what a thread knows of its sequence stays in registers.
// One B200, whole calls: append of a token to 128 sequences 10 us (25 with a single
// CTA's books), fork of 16 beams 15, of 256 sequences over 20,000 pages 20, compact
// of 250 pages 8.5. Where there is much to copy, HBM bounds the call: 17,400 pages
// of 64 KB, 516 MB read and written, 97 us (5.8 TB/s for the copy), prompts of 134 MB
// 30 us.
//
// A table, length array or count array may be written in place (output ==
// input): every value that a phase overwrites has been read before the
// barrier in front of it, or is read and written by the same thread.
#pragma once

#include <cstdint>

#include "paged.cuh"
#include "sm100.cuh"

namespace attn {
namespace paged {

constexpr int kBookCtas = 8;
constexpr int kBookThreads = 1024;
constexpr int kBookWarps = kBookThreads / 32;
constexpr int kAllWarps = kBookCtas * kBookWarps, kAllThreads = kBookCtas * kBookThreads;
constexpr int kNone = 0x7fffffff;

// info[0]; the header documents the values.
enum : int { kInfoOk = 0, kInfoNoPages = 1, kInfoTableFull = 2, kInfoSharedTail = 3 };

struct Move {            // rows [0, rows) of every head of page src, to page dst
    int src, dst, rows, entry;   // fork: the table entry that gets dst
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
    int* after;          // [B]  new length
    int* start;          // [B]  append: old length; fork: last page of the source, if partly filled
    int* base;           // [P]  fork: references besides last pages; compact: holes
    int* key;            // [P]  append: table entry of each page taken; fork: who keeps it; compact: pages to move
    int* stage;          // [B, M]
    Move* moves;         // [max(B, P)]
};

// The pages of this warp: a contiguous range, ranges in the order of
// (CTA, warp), so that ranks follow page numbers.
__device__ __forceinline__ void page_range(int P, int* lo, int* hi) {
    const long long w = (long long)cluster_rank() * kBookWarps + (threadIdx.x >> 5);
    *lo = int(P * w / kAllWarps);
    *hi = int(P * (w + 1) / kAllWarps);
}

// Two sums through one scan: pages (high word) counted per warp, and a count
// per thread (low word). Both totals are below 2^31.
__device__ __forceinline__ long long both(int pages, int count) {
    return ((threadIdx.x & 31) == 0 ? (long long)pages << 32 : 0ll) + count;
}

// The totals of all CTAs' pages, read after a cluster_sync: those of earlier
// CTAs, and all.
__device__ __forceinline__ int pages_before(const int* sums, int* total) {
    int before = 0, all = 0;
#pragma unroll
    for (int c = 0; c < kBookCtas; ++c) {
        const int s = __ldcg(sums + c);
        if (c < int(cluster_rank())) before += s;
        all += s;
    }
    *total = all;
    return before;
}

// This thread's contiguous share of the sequences, over one CTA.
__device__ __forceinline__ void thread_share(int B, int* b0, int* b1) {
    const int chunk = (B + kBookThreads - 1) / kBookThreads;
    *b0 = int(min((long long)B, (long long)threadIdx.x * chunk));
    *b1 = min(B, *b0 + chunk);
}

// f(b, j0) for blocks of 128 entries [j0, j0 + 128) of every table row, a warp
// each, over the cluster: four entries a lane keep loads in flight.
constexpr int kRowBlock = 128;
template <typename F>
__device__ __forceinline__ void table_blocks(const Geometry& g, F&& f) {
    const int blocks = (g.M + kRowBlock - 1) / kRowBlock;
    const long long items = (long long)g.B * blocks;
    for (long long x = (long long)cluster_rank() * kBookWarps + (threadIdx.x >> 5); x < items; x += kAllWarps) {
        const int b = int(x / blocks);
        f(b, int(x - (long long)b * blocks) * kRowBlock);
    }
}

// -------------------------------------------------------------- copying rows
// A warp takes a span at a time: up to kSpan 16-byte units (four a lane in
// flight) of consecutive rows of K, or of V. Spans are whole rows, so that where
// a lane's units lie in a row is the same in every span, and the loops divide by
// multiplication. Copies of up to kHereSpans spans are made by the cluster that
// keeps the books; larger ones by a kernel of their own over the whole GPU, which
// starts while the books are still being written and reads what it needs of
// them from L2, after its wait.
constexpr int kCopyThreads = 256, kUnits = 4, kSpan = 32 * kUnits;
constexpr unsigned kHereSpans = 512;

// n / d for 0 <= n < 2^31.
struct Divisor {
    unsigned d, mul, shift;
    static Divisor of(unsigned d) {
        unsigned l = 0;
        while (l < 31 && (1u << l) < d) ++l;
        return Divisor{d, unsigned(((1ull << 32) * ((1ull << l) - d)) / d + 1), l};
    }
    __device__ __forceinline__ unsigned divide(unsigned n) const { return (__umulhi(n, mul) + n) >> shift; }
};

// What is copied. Widths in 16-byte units. A part is a run of rows that spans do
// not cross: one head of a page to move; of new rows one head of a sequence, or,
// when that is less than four spans (few tokens a sequence), all of them.
struct Rows {
    const uint4* K;      // append: the new rows [B, Hkv, n, w]
    const uint4* V;
    uint4* Kp;
    uint4* Vp;
    const int* new_len;  // append: may be null
    int n;
    int wk, wv, k_rows, v_rows;              // widths, rows of a span
    unsigned k_spans;                        // of a part's K; the rest are of its V
    Divisor spans, by_n, by_heads;           // spans of a part
    bool flat;                               // append: one part
    bool here;                               // by the books' own cluster

    static Rows of(void* Kp, void* Vp, int wk, int wv, long long rows, int heads, int n, bool flat) {
        Rows r{};
        r.Kp = static_cast<uint4*>(Kp);
        r.Vp = static_cast<uint4*>(Vp);
        r.n = n;
        r.wk = wk;
        r.wv = wv;
        r.k_rows = kSpan / wk;
        r.v_rows = kSpan / wv;
        r.k_spans = unsigned((rows + r.k_rows - 1) / r.k_rows);
        r.spans = Divisor::of(r.k_spans + unsigned((rows + r.v_rows - 1) / r.v_rows));
        r.by_n = Divisor::of(n);
        r.by_heads = Divisor::of(heads);
        r.flat = flat;
        return r;
    }
    static Rows of_new(void* Kp, void* Vp, int wk, int wv, int B, int heads, int n) {
        const bool flat = n < 4 * (kSpan / wk);
        return of(Kp, Vp, wk, wv, flat ? 1ll * B * heads * n : n, heads, n, flat);
    }
};

// Rows of sequence b that are not padding.
__device__ __forceinline__ int new_rows(const Rows& r, int b) {
    return r.new_len ? min(max(__ldg(r.new_len + b), 0), r.n) : r.n;
}

// Span x of the new rows, all of them one part, to their pages. `wait` is called
// once the rows are on their way, if `early`, and says whether to go on.
template <typename F>
__device__ __forceinline__ bool append_span_flat(const Books& k, const Rows& r, unsigned x, bool early, F&& wait) {
    const Geometry& g = k.g;
    const int lane = threadIdx.x & 31, page = 1 << g.page_log2;
    const bool is_v = x >= r.k_spans;
    const unsigned w = is_v ? r.wv : r.wk, span_rows = is_v ? r.v_rows : r.k_rows;
    const unsigned row0 = (is_v ? x - r.k_spans : x) * span_rows;      // of all new rows
    const unsigned rows = min(span_rows, unsigned(g.B) * g.Hkv * r.n - row0);
    const uint4* from = (is_v ? r.V : r.K) + size_t(row0) * w + lane;
    uint4* pool = is_v ? r.Vp : r.Kp;
    uint4 v[kUnits];
    unsigned c[kUnits];
    int b[kUnits], h[kUnits], i[kUnits], t[kUnits];
#pragma unroll
    for (int e = 0; e < kUnits; ++e) {
        const unsigned u = lane + 32 * e, row = u / w;
        c[e] = u - row * w;
        b[e] = -1;
        if (row >= rows) continue;
        const unsigned bh = r.by_n.divide(row0 + row);
        i[e] = int(row0 + row - bh * r.n);
        b[e] = int(r.by_heads.divide(bh));
        h[e] = int(bh - b[e] * r.by_heads.d);
        v[e] = __ldcs(from + 32 * e);
    }
    if (early && !wait()) return false;
#pragma unroll
    for (int e = 0; e < kUnits; ++e) {
        if (b[e] < 0) continue;
        t[e] = __ldcg(k.start + b[e]) + i[e];
        if (t[e] >= __ldcg(k.after + b[e])) b[e] = -1;
        else i[e] = __ldcg(k.table_out + size_t(b[e]) * g.M + (t[e] >> g.page_log2));
    }
#pragma unroll
    for (int e = 0; e < kUnits; ++e)
        if (b[e] >= 0 && page_ok(i[e], g.P))
            pool[((size_t(i[e]) * g.Hkv + h[e]) * page + (t[e] & (page - 1))) * w + c[e]] = v[e];
    return true;
}

// Where a lane's units lie in a span of rows of w units.
struct Lanes {
    int row[kUnits], col[kUnits];
    __device__ __forceinline__ Lanes(int w, int rows) {
#pragma unroll
        for (int e = 0; e < kUnits; ++e) {
            const int u = (threadIdx.x & 31) + 32 * e;
            row[e] = u / w;
            col[e] = u - row[e] * w;
            if (row[e] >= rows) row[e] = 0x3fffffff;       // past the span
        }
    }
};

// Span x of the new rows, a part for each head of a sequence. Padding is told by
// the call's own numbers, so that it is passed over, and the first rows are on
// their way, before the books are there; `ready` waits for them and says whether
// to go on.
template <typename F>
__device__ __forceinline__ bool append_span(const Books& k, const Rows& r, unsigned x, const Lanes& in_k,
                                            const Lanes& in_v, F&& ready) {
    const Geometry& g = k.g;
    const int page = 1 << g.page_log2;
    const unsigned bh = r.spans.divide(x), b = r.by_heads.divide(bh), h = bh - b * r.by_heads.d;
    unsigned span = x - bh * r.spans.d;
    const bool is_v = span >= r.k_spans;
    if (is_v) span -= r.k_spans;
    const int w = is_v ? r.wv : r.wk, i0 = int(span) * (is_v ? r.v_rows : r.k_rows);
    const int left = new_rows(r, b) - i0;
    if (left <= 0) return true;
    const uint4* from = (is_v ? r.V : r.K) + (size_t(bh) * r.n + i0) * w + (threadIdx.x & 31);
    uint4* pool = (is_v ? r.Vp : r.Kp);
    uint4 v[kUnits];
    int p[kUnits];
#pragma unroll
    for (int e = 0; e < kUnits; ++e)
        if ((is_v ? in_v.row[e] : in_k.row[e]) < left) v[e] = __ldcs(from + 32 * e);
    if (!ready()) return false;
    const int t0 = __ldcg(k.start + b) + i0;
    const int* row = k.table_out + size_t(b) * g.M;
#pragma unroll
    for (int e = 0; e < kUnits; ++e) {
        const int i = is_v ? in_v.row[e] : in_k.row[e];
        if (i < left) p[e] = __ldcg(row + ((t0 + i) >> g.page_log2));
    }
#pragma unroll
    for (int e = 0; e < kUnits; ++e) {
        const int i = is_v ? in_v.row[e] : in_k.row[e], c = is_v ? in_v.col[e] : in_k.col[e];
        if (i < left && page_ok(p[e], g.P))
            pool[((size_t(p[e]) * g.Hkv + h) * page + ((t0 + i) & (page - 1))) * w + c] = v[e];
    }
    return true;
}

// Span x of the moves: rows [0, rows) of every head of the listed pages.
__device__ __forceinline__ void move_span(const Books& k, const Rows& r, unsigned long long x) {
    const Geometry& g = k.g;
    const int lane = threadIdx.x & 31;
    const unsigned qh = (x >> 31) == 0 ? r.spans.divide(unsigned(x)) : unsigned(x / r.spans.d);
    const unsigned q = r.by_heads.divide(qh), h = qh - q * r.by_heads.d;
    unsigned span = unsigned(x - (unsigned long long)qh * r.spans.d);
    const bool is_v = span >= r.k_spans;
    if (is_v) span -= r.k_spans;
    const int w = is_v ? r.wv : r.wk, rows = is_v ? r.v_rows : r.k_rows;
    const int4 m = __ldcg(reinterpret_cast<const int4*>(k.moves) + q);
    const int units = min(rows, m.z - int(span) * rows) * w, u0 = int(span) * rows * w + lane;
    uint4* pool = is_v ? r.Vp : r.Kp;
    const uint4* from = pool + ((size_t(m.x) * g.Hkv + h) << g.page_log2) * w + u0;
    uint4* to = pool + ((size_t(m.y) * g.Hkv + h) << g.page_log2) * w + u0;
    uint4 v[kUnits];
#pragma unroll
    for (int e = 0; e < kUnits; ++e)
        if (lane + 32 * e < units) v[e] = __ldcs(from + 32 * e);
#pragma unroll
    for (int e = 0; e < kUnits; ++e)
        if (lane + 32 * e < units) __stcs(to + 32 * e, v[e]);
}

__global__ void __launch_bounds__(kCopyThreads) append_rows(Books k, Rows r) {
    const unsigned stride = gridDim.x * (kCopyThreads / 32), first = blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5);
    auto wait = [&] {
        grid_dependency_wait();
        return __ldcg(k.control + kCtlMoves) != 0;
    };
    if (r.flat) {
        // The first rows are on the way before the books are read.
        for (unsigned x = first; x < r.spans.d; x += stride)
            if (!append_span_flat(k, r, x, x == first, wait)) return;
    } else {
        const Lanes in_k(r.wk, r.k_rows), in_v(r.wv, r.v_rows);
        const unsigned items = r.spans.d * unsigned(k.g.B) * unsigned(k.g.Hkv);
        bool waited = false;
        auto ready = [&] {
            if (waited) return true;
            waited = true;
            return wait();
        };
        for (unsigned x = first; x < items; x += stride)
            if (!append_span(k, r, x, in_k, in_v, ready)) return;
        // The grid ends after the books even if there is nothing but padding.
        if (blockIdx.x == 0) (void)ready();
    }
}

__global__ void __launch_bounds__(kCopyThreads) move_rows(Books k, Rows r) {
    grid_dependency_wait();
    const unsigned long long items = (unsigned long long)__ldcg(k.control + kCtlMoves) * k.g.Hkv * r.spans.d;
    const unsigned stride = gridDim.x * (kCopyThreads / 32);
    for (unsigned long long x = blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); x < items; x += stride)
        move_span(k, r, x);
}

// The moves by the books' cluster, after its last writes.
__device__ __forceinline__ void move_here(const Books& k, const Rows& r) {
    cluster_sync();
    const unsigned items = unsigned(__ldcg(k.control + kCtlMoves)) * k.g.Hkv * r.spans.d;
    for (unsigned x = cluster_rank() * kBookWarps + (threadIdx.x >> 5); x < items; x += kAllWarps) move_span(k, r, x);
}

// ------------------------------------------------------------------- append
__global__ void __launch_bounds__(kBookThreads, 1) append_books(Books k, Rows r) {
    grid_launch_dependents();                       // the copy kernel may set up meanwhile
    __shared__ long long scratch[33];
    __shared__ int full_s, shared_s;
    const Geometry& g = k.g;
    const int tid = threadIdx.x, lane = tid & 31;
    const int rank = int(cluster_rank());
    const int page_mask = (1 << g.page_log2) - 1, room = g.M << g.page_log2;
    const bool same_ref = k.ref_out == k.ref, same_table = k.table_out == k.table;
    if (tid == 0) full_s = shared_s = 0;

    // (First CTA) the pages that each sequence needs.
    int b0 = 0, b1 = 0, need = 0, full = 0, shared = 0, len = 0, add = 0;
    if (rank == 0) {
        thread_share(g.B, &b0, &b1);
        for (int b = b0; b < b1; ++b) {
            len = clamp_len(k.lens[b], g);
            add = new_rows(r, b);
            if (add > 0 && (len & page_mask) != 0) {
                // The page that goes on being filled must be this sequence's alone.
                const int p = k.table[size_t(b) * g.M + (len >> g.page_log2)];
                if (!page_ok(p, g.P) || k.ref[p] != 1) shared = 1;
            }
            if (add > room - len) {
                full = 1;
                add = 0;                            // the call is refused as a whole below
            }
            need += pages_of(len + add, g.page_log2) - pages_of(len, g.page_log2);
        }
    }
    // Free pages; the counts are copied on the way. Lane i holds which pages of
    // the warp's i-th block of 32 are free, for its first 1,024 pages.
    int lo, hi, count = 0;
    unsigned held = 0;
    page_range(g.P, &lo, &hi);
#pragma unroll 4
    for (int p0 = lo, i = 0; p0 < hi; p0 += 32, ++i) {
        const int p = p0 + lane;
        const int r = p < hi ? k.ref[p] : 1;
        if (!same_ref && p < hi) k.ref_out[p] = r;
        const unsigned hits = __ballot_sync(0xffffffffu, r <= 0);
        if (lane == i) held = hits;
        count += __popc(hits);
    }
    if (!same_table) {
        table_blocks(g, [&](int b, int j0) {
#pragma unroll
            for (int j = j0 + lane; j < j0 + kRowBlock; j += 32)
                if (j < g.M) k.table_out[size_t(b) * g.M + j] = k.table[size_t(b) * g.M + j];
        });
    }
    __syncthreads();                                // full_s, shared_s are zero
    if (full) full_s = 1;
    if (shared) shared_s = 1;
    long long totals;
    const long long before = block_exclusive(both(count, need), scratch, &totals);
    if (tid == 0) k.control[kCtlSums + rank] = int(totals >> 32);
    if (rank == 0) {
        // Page q of the call goes to table entry key[q]; sequences in order.
        int q0 = int(before & 0x7fffffff);
        for (int b = b0; __any_sync(0xffffffffu, b < b1); ++b) {
            if (b < b1 && b1 - b0 > 1) {            // else it is in registers still
                len = clamp_len(k.lens[b], g);
                add = new_rows(r, b);
                if (add > room - len) add = 0;
            }
            int mine = 0, at = 0;
            if (b < b1) {
                k.start[b] = len;
                k.after[b] = len + add;
                at = pages_of(len, g.page_log2);
                mine = pages_of(len + add, g.page_log2) - at;
            }
            for (unsigned some = __ballot_sync(0xffffffffu, mine > 0); some; some &= some - 1) {
                const int l = __ffs(some) - 1;
                const int c = __shfl_sync(0xffffffffu, mine, l), q = __shfl_sync(0xffffffffu, q0, l);
                const int e = __shfl_sync(0xffffffffu, b * g.M + at, l);
                for (int x = lane; x < min(c, g.P - q); x += 32) k.key[q + x] = e + x;
            }
            q0 += mine;
        }
        if (tid == 0) {
            k.control[kCtlNeed] = int(totals & 0x7fffffff);
            k.control[kCtlFlags] = shared_s ? kInfoSharedTail : full_s ? kInfoTableFull : kInfoOk;
        }
    }
    cluster_sync();

    int total_free;
    int at = pages_before(k.control + kCtlSums, &total_free) + int(__shfl_sync(0xffffffffu, before, 0) >> 32);
    need = __ldcg(k.control + kCtlNeed);
    int status = __ldcg(k.control + kCtlFlags);
    if (status == kInfoOk && need > total_free) status = kInfoNoPages;
    const bool ok = status == kInfoOk;
    if (rank == 0 && tid == 0) {
        k.info[0] = status;
        k.info[1] = total_free - (ok ? need : 0);
        k.info[2] = ok ? need : 0;
        k.control[kCtlMoves] = ok;                  // the copy kernel writes nothing otherwise
    }
    if (ok) {
        for (int p0 = lo, i = 0; p0 < hi && at < need; p0 += 32, ++i) {
            const int p = p0 + lane;
            const unsigned hits = i < 32 ? __shfl_sync(0xffffffffu, held, i)
                                         : __ballot_sync(0xffffffffu, p < hi && k.ref[p] <= 0);
            const int q = at + __popc(hits & ((1u << lane) - 1u));
            at += __popc(hits);
            if ((hits >> lane & 1) && q < need) {
                k.table_out[__ldcg(k.key + q)] = p;
                k.ref_out[p] = 1;
            }
        }
    }
    if (rank == 0) {
        for (int b = b0; b < b1; ++b) {
            if (b1 - b0 > 1) add = k.after[b] - (len = k.start[b]);
            if (ok) k.lens_out[b] = len + add;
            else if (k.lens_out != k.lens) k.lens_out[b] = k.lens[b];
        }
    }
    if (r.here && ok) {
        cluster_sync();
        for (unsigned x = rank * kBookWarps + (tid >> 5); x < r.spans.d; x += kAllWarps)
            append_span_flat(k, r, x, false, [] { return true; });
    }
}

// --------------------------------------------------------------------- fork
// Sequence b becomes the first L_b tokens of sequence src[b]: full pages are
// shared, and a partly filled last page belongs to one sequence alone.
//   base(p) = ref(p) - (uses in the old rows) + (full uses in the new rows)
// counts who holds p besides its takers as a last page. With base(p) = 0 one
// taker keeps p (the one it belonged to, else the lowest: the least of `key`);
// every other taker gets a copy in a fresh page.
__global__ void __launch_bounds__(kBookThreads, 1) fork_books(Books k, const int* src, const int* keep, Rows r) {
    grid_launch_dependents();                       // the copy kernel may set up meanwhile
    __shared__ long long scratch[33];
    const Geometry& g = k.g;
    const int tid = threadIdx.x, lane = tid & 31;
    const int rank = int(cluster_rank());
    const int page_mask = (1 << g.page_log2) - 1;
    const bool same_ref = k.ref_out == k.ref, same_table = k.table_out == k.table;

    // (First CTA) the last pages; a thread keeps its first sequence in registers.
    int b0 = 0, b1 = 0;
    if (rank == 0) {
        thread_share(g.B, &b0, &b1);
    } else {
#pragma unroll 4
        for (int p = (rank - 1) * kBookThreads + tid; p < g.P; p += kAllThreads - kBookThreads) {
            k.base[p] = k.ref[p];
            k.key[p] = kNone;
        }
    }
    int my_src = -1, my_L = 0, tail = -1;
    for (int b = b0; b < b1; ++b) {
        my_src = src[b];
        const bool valid = my_src >= 0 && my_src < g.B;
        my_L = valid ? clamp_len(k.lens[my_src], g) : 0;
        if (valid && keep) my_L = min(max(keep[b], 0), my_L);
        tail = (my_L & page_mask) != 0 ? k.table[size_t(my_src) * g.M + (my_L >> g.page_log2)] : -1;
        k.start[b] = tail;
        k.after[b] = my_L;
    }
    const bool one = b1 - b0 <= 1;
    cluster_sync();

    // Uses given up and taken; pages that a sequence keeps in its own row
    // cancel. Rows that come from elsewhere are staged: they may be overwritten.
    table_blocks(g, [&](int b, int j0) {
        const int had = pages_of(clamp_len(k.lens[b], g), g.page_log2), full = __ldcg(k.after + b) >> g.page_log2;
        const int s = src[b];
        const bool home = s == b;
        if (j0 >= max(had, full)) return;
        const int* own = k.table + size_t(b) * g.M;
        const int* from = k.table + size_t(full > 0 ? s : b) * g.M;
#pragma unroll
        for (int j = j0 + lane; j < j0 + kRowBlock; j += 32) {
            if (j < had && !(home && j < full)) {
                const int p = own[j];
                if (page_ok(p, g.P)) atomicSub(k.base + p, 1);
            }
            if (j < full && !home) {
                const int p = from[j];
                if (page_ok(p, g.P)) atomicAdd(k.base + p, 1);
                k.stage[size_t(b) * g.M + j] = p;
            }
        }
    });
    // A last page that can be followed, or -1; its takers in order.
    auto tail_of = [&](int b) {
        const int p = one ? tail : k.start[b];
        return ((one ? my_L : k.after[b]) & page_mask) != 0 && page_ok(p, g.P) ? p : -1;
    };
    auto order_of = [&](int b) { return (one ? my_src : src[b]) == b ? b : b + g.B; };
    for (int b = b0; b < b1; ++b) {
        const int p = tail_of(b);
        if (p >= 0) atomicMin(k.key + p, order_of(b));
    }
    cluster_sync();

    // Who copies (in the order of sequences), and which pages are free: lane i
    // holds those of the warp's i-th block of 32, for its first 1,024 pages.
    auto copies = [&](int b) {
        const int p = tail_of(b);
        return p >= 0 && (__ldcg(k.base + p) > 0 || __ldcg(k.key + p) != order_of(b));
    };
    int ncopy = 0;
    for (int b = b0; b < b1; ++b) ncopy += copies(b) ? 1 : 0;
    int lo, hi, count = 0;
    unsigned held = 0;
    page_range(g.P, &lo, &hi);
    auto is_free = [&](int p) { return p < hi && __ldcg(k.base + p) <= 0 && __ldcg(k.key + p) == kNone; };
#pragma unroll 4
    for (int p0 = lo, i = 0; p0 < hi; p0 += 32, ++i) {
        const unsigned hits = __ballot_sync(0xffffffffu, is_free(p0 + lane));
        if (lane == i) held = hits;
        count += __popc(hits);
    }
    long long totals;
    const long long before = block_exclusive(both(count, ncopy), scratch, &totals);
    if (tid == 0) k.control[kCtlSums + rank] = int(totals >> 32);
    if (rank == 0) {
        int q = int(before & 0x7fffffff);
        for (int b = b0; b < b1; ++b) {
            const int L = one ? my_L : k.after[b];
            if ((L & page_mask) == 0) continue;
            const bool c = one ? ncopy != 0 : copies(b);
            const int entry = b * g.M + (L >> g.page_log2);
            k.stage[entry] = c;                                  // staged entries end before it
            if (c) k.moves[q++] = Move{one ? tail : k.start[b], -1, L & page_mask, entry};
        }
        if (tid == 0) k.control[kCtlNeed] = int(totals & 0x7fffffff);
    }
    cluster_sync();

    int total_free;
    int at = pages_before(k.control + kCtlSums, &total_free) + int(__shfl_sync(0xffffffffu, before, 0) >> 32);
    const int need = __ldcg(k.control + kCtlNeed);
    if (need > total_free) {
        // Nothing changes; the free pages are those of the counts as they came.
        int was_free = 0;
        for (int p = lo + lane; p < hi; p += 32) {
            const int r = k.ref[p];
            was_free += r <= 0 ? 1 : 0;
            if (!same_ref) k.ref_out[p] = r;
        }
        if (!same_table) {
            table_blocks(g, [&](int b, int j0) {
                for (int j = j0 + lane; j < min(g.M, j0 + kRowBlock); j += 32)
                    k.table_out[size_t(b) * g.M + j] = k.table[size_t(b) * g.M + j];
            });
        }
        if (k.lens_out != k.lens)
            for (int b = b0; b < b1; ++b) k.lens_out[b] = k.lens[b];
        long long sum;
        (void)block_exclusive((long long)was_free, scratch, &sum);
        if (tid == 0) k.control[kCtlFreed + rank] = int(sum);
        cluster_sync();
        if (rank == 0 && tid == 0) {
            int now = 0;
            for (int c = 0; c < kBookCtas; ++c) now += __ldcg(k.control + kCtlFreed + c);
            k.info[0] = kInfoNoPages;
            k.info[1] = now;
            k.info[2] = 0;
            k.control[kCtlMoves] = 0;
        }
        return;
    }
    if (rank == 0 && tid == 0) {
        k.info[0] = kInfoOk;
        k.info[1] = total_free - need;
        k.info[2] = need;
        k.control[kCtlMoves] = need;
    }
#pragma unroll 4
    for (int p0 = lo, i = 0; p0 < hi; p0 += 32, ++i) {
        const int p = p0 + lane;
        const unsigned hits = i < 32 ? __shfl_sync(0xffffffffu, held, i) : __ballot_sync(0xffffffffu, is_free(p));
        const int q = at + __popc(hits & ((1u << lane) - 1u));
        at += __popc(hits);
        if (p >= hi) continue;
        if (hits >> lane & 1) {
            if (q < need) {
                k.moves[q].dst = p;
                k.table_out[__ldcg(&k.moves[q].entry)] = p;
            }
            k.ref_out[p] = q < need ? 1 : 0;
        } else {
            const int held_by = __ldcg(k.base + p);
            k.ref_out[p] = held_by > 0 ? held_by : 1;            // a last page that stays, if nobody else
        }
    }
    // The rows. In place, a sequence's own row only changes from its last page on.
    table_blocks(g, [&](int b, int j0) {
        const int L = __ldcg(k.after + b), had = pages_of(clamp_len(k.lens[b], g), g.page_log2);
        const int full = L >> g.page_log2, has = pages_of(L, g.page_log2);
        const bool home = src[b] == b;
        const int last = __ldcg(k.start + b);
        const bool copied = has > full && __ldcg(k.stage + size_t(b) * g.M + full);
        const int from = same_table && home ? full : 0, end = same_table ? max(had, has) : g.M;
        if (j0 + kRowBlock <= from || j0 >= end) return;
        const size_t row = size_t(b) * g.M;
#pragma unroll
        for (int j = j0 + lane; j < j0 + kRowBlock; j += 32) {
            if (j < from || j >= end || (copied && j == full)) continue;   // written with its page
            int p;
            if (j < full) p = home ? k.table[row + j] : __ldcg(k.stage + row + j);
            else if (j < has) p = last;
            else p = j < had ? -1 : k.table[row + j];
            k.table_out[row + j] = p;
        }
    });
    if (k.lens_out == k.lens) cluster_sync();                    // every row has read its old length
    for (int b = b0; b < b1; ++b) k.lens_out[b] = one ? my_L : k.after[b];
    if (r.here) move_here(k, r);
}

// ------------------------------------------------------------------ compact
// L live pages. The k-th live page at or past L moves to the k-th free page
// before L: the fewest moves, no page both read and written.
__global__ void __launch_bounds__(kBookThreads, 1) compact_books(Books k, int* remap, Rows r) {
    grid_launch_dependents();                       // the copy kernel may set up meanwhile
    __shared__ long long scratch[33];
    const Geometry& g = k.g;
    const int tid = threadIdx.x, lane = tid & 31;
    const int rank = int(cluster_rank());
    const int gthread = rank * kBookThreads + tid;
    int lo, hi;
    page_range(g.P, &lo, &hi);
    int* holes = k.base;
    int* high = k.key;

    int count = 0;
    unsigned held = 0;                              // live pages, as in append_books
#pragma unroll 4
    for (int p0 = lo, i = 0; p0 < hi; p0 += 32, ++i) {
        const unsigned hits = __ballot_sync(0xffffffffu, p0 + lane < hi && k.ref[p0 + lane] > 0);
        if (lane == i) held = hits;
        count += __popc(hits);
    }
    long long totals;
    const long long before = block_exclusive(both(count, 0), scratch, &totals);
    if (tid == 0) k.control[kCtlSums + rank] = int(totals >> 32);
    cluster_sync();
    int live;
    int at = pages_before(k.control + kCtlSums, &live) + int(__shfl_sync(0xffffffffu, before, 0) >> 32);
    for (int p0 = lo, i = 0; p0 < hi; p0 += 32, ++i) {
        const int p = p0 + lane;
        const unsigned hits = i < 32 ? __shfl_sync(0xffffffffu, held, i)
                                     : __ballot_sync(0xffffffffu, p < hi && k.ref[p] > 0);
        const bool is_live = hits >> lane & 1;
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
    const int m = __ldcg(k.control + kCtlNeed);
    // A moved page's count goes to its hole. Counts of holes and of moved pages
    // are written by the second loop alone; the others stay.
    if (k.ref_out != k.ref) {
#pragma unroll 4
        for (int p = gthread; p < g.P; p += kAllThreads) {
            const int r = k.ref[p];
            if (r > 0 ? p < live : p >= live) k.ref_out[p] = r;
        }
    }
    for (int q = gthread; q < m; q += kAllThreads) {
        const int from = __ldcg(high + (m - 1 - q)), to = __ldcg(holes + q);
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
    table_blocks(g, [&](int b, int j0) {
        const int had = pages_of(clamp_len(k.lens[b], g), g.page_log2);
        const int end = same_table ? had : g.M;
        const size_t row = size_t(b) * g.M;
        int p[kRowBlock / 32];
#pragma unroll
        for (int e = 0; e < kRowBlock / 32; ++e) {
            const int j = j0 + lane + 32 * e;
            p[e] = j < end ? k.table[row + j] : -1;
        }
#pragma unroll
        for (int e = 0; e < kRowBlock / 32; ++e) {
            const int j = j0 + lane + 32 * e;
            if (j < had && page_ok(p[e], g.P)) p[e] = __ldcg(remap + p[e]);
        }
#pragma unroll
        for (int e = 0; e < kRowBlock / 32; ++e) {
            const int j = j0 + lane + 32 * e;
            if (j < end) k.table_out[row + j] = p[e];
        }
    });
    if (r.here) move_here(k, r);
}

}  // namespace paged
}  // namespace attn
