// paged.cuh -- what the kernels of the paged key-value cache share: its
// geometry, block-wide scans, and the split of a decode call over CTAs.
//
// A cache is two pools of pages (K [P, Hkv, page, d], V [P, Hkv, page, dv]), a
// table of page numbers [B, M], the lengths [B] and one reference count per
// page [P]. Token t of sequence b lies in page table[b][t / page], row
// t % page. Page numbers and lengths live in device memory, so no kernel
// trusts them: lengths are clamped to [0, M * page], and a page number outside
// [0, P) is never followed.
#pragma once

#include <cstdint>

namespace attn {
namespace paged {

constexpr int kMinPageLog2 = 3, kMaxPageLog2 = 8;    // 8 .. 256 tokens

struct Geometry {
    int B, M, P, Hkv;
    int page_log2;
};

__device__ __forceinline__ int clamp_len(int len, const Geometry& g) {
    return min(max(len, 0), g.M << g.page_log2);
}
__device__ __forceinline__ int pages_of(int len, int page_log2) {
    return int((unsigned(len) + (1u << page_log2) - 1u) >> page_log2);
}
__device__ __forceinline__ bool page_ok(int p, int P) { return unsigned(p) < unsigned(P); }

// Exclusive scan of one value per thread over the block; `total` gets the sum.
// `scratch` holds one value per warp and one more; the call ends with every
// thread past a barrier, so scratch can be reused at once.
template <typename T>
__device__ __forceinline__ T block_exclusive(T v, T* scratch, T* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = int(blockDim.x + 31) >> 5;
    T inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
    }
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        T w = lane < warps ? scratch[lane] : T(0);
        T winc = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const T up = __shfl_up_sync(0xffffffffu, winc, o);
            if (lane >= o) winc += up;
        }
        if (lane < warps) scratch[lane] = winc - w;
        if (lane == 31) scratch[32] = winc;
    }
    __syncthreads();
    const T r = scratch[warp] + inc - v;
    *total = scratch[32];
    __syncthreads();
    return r;
}

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

// ------------------------------------------------- the split of a decode call
// A call's work is counted in units. An item (sequence, key head, tile of query
// rows) costs one per key tile (kTileKeys keys) and kItemUnits for its start
// and end. A sequence with queries and no keys has one (empty) tile per item,
// so that its rows are written. Units are numbered sequence by sequence, item
// by item, and every CTA takes the same number of consecutive ones, however
// the lengths are spread, which the host does not know. (64 sequences of 128 to
// 16384 tokens: 173 us with kItemUnits = 0, 148 with 1, 145 with 2; 24 drafts of
// 100 to 4000 tokens: 39, 30 and 28.) An item cut by a CTA
// border is joined afterwards from its pieces.
constexpr int kTileKeys = 64;
constexpr int kItemUnits = 2;

struct DecodeArgs {
    Geometry g;
    const int* table;
    const int* lens;
    const int* q_len;       // may be null: n queries everywhere
    int H, n, d, dv;
    int rows;               // query rows per key head: (H / Hkv) * n
    int tile_rows;          // query rows per item
    int row_tiles;          // items per key head
    int causal;
    float scale;
};

struct Piece {
    int b, item;            // item: key head * row_tiles + row tile
    int len, nq;            // keys and queries of the sequence
    int t0, t1, tiles;      // key tiles [t0, t1) of `tiles`
    long long end;          // number of the unit after the item's last
};

__device__ __forceinline__ int queries_of(const DecodeArgs& a, int b) {
    return a.q_len ? min(max(__ldg(a.q_len + b), 0), a.n) : a.n;
}
__device__ __forceinline__ int tiles_of(int len) { return max(1, (len + kTileKeys - 1) / kTileKeys); }

// x / y for x >= 0, y > 0: mostly both fit 32 bits, where it is much cheaper.
__device__ __forceinline__ long long divide(long long x, long long y) {
    if (((x | y) >> 32) == 0) return (unsigned)x / (unsigned)y;
    return x / y;
}

// The sequence in [b0, b1) that holds unit pos, *x being the units before b0 and
// then those before it. The last one if none does, which only lengths that change
// during the call can bring about: they must not lead past the arrays.
template <typename Units>
__device__ __forceinline__ int sequence_of(Units&& units, int b0, int b1, long long pos, long long* x) {
    int b = b0;
    for (; b < b1 - 1; ++b) {
        const long long u = units(b);
        if (pos < *x + u) break;
        *x += u;
    }
    return b;
}

// A CTA's share, walked by one warp (all lanes hold the same walker). With
// total = q * ctas + r, the first r CTAs take q + 1 units and the others q.
struct Walker {
    int b, ctas;            // ctas: those that have work
    long long off;          // units of sequence b already passed
    long long left;         // units left to this CTA
    long long pos;          // number of the next unit
    long long q, r;

    static __device__ __forceinline__ long long units_of(const DecodeArgs& a, int b) {
        if (queries_of(a, b) <= 0) return 0;
        return (long long)(a.g.Hkv * a.row_tiles) * (tiles_of(clamp_len(__ldg(a.lens + b), a.g)) + kItemUnits);
    }

    __device__ void start(const DecodeArgs& a) {
        const int lane = threadIdx.x & 31, chunk = (a.g.B + 31) / 32;
        const int b0 = int(min((long long)a.g.B, (long long)lane * chunk)), b1 = min(a.g.B, b0 + chunk);
        long long sum = 0;
#pragma unroll 4
        for (int k = b0; k < b1; ++k) sum += units_of(a, k);
        long long inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long up = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += up;
        }
        const long long total = __shfl_sync(0xffffffffu, inc, 31), before = inc - sum;
        ctas = int(min((long long)gridDim.x, max(1ll, total)));
        q = divide(total, ctas);
        r = total - q * ctas;
        const long long c = blockIdx.x;
        left = c < ctas ? q + (c < r ? 1 : 0) : 0;
        pos = q * c + min(c, r);
        // The lane whose sequences hold unit pos looks for the sequence.
        const bool mine = left > 0 && pos >= before && pos < inc;
        int found = 0;
        long long x = before;
        if (mine) found = sequence_of([&](int k) { return units_of(a, k); }, b0, b1, pos, &x);
        const unsigned who = __ballot_sync(0xffffffffu, mine);
        const int from = who ? __ffs(who) - 1 : 0;
        b = __shfl_sync(0xffffffffu, found, from);
        off = pos - __shfl_sync(0xffffffffu, x, from);
    }

    __device__ bool next(const DecodeArgs& a, Piece* p) {
        const int items = a.g.Hkv * a.row_tiles;
        while (left > 0) {
            for (;; ++b, off = 0) {
                // (Past the last sequence only if the lengths change meanwhile.)
                if (b >= a.g.B) return false;
                p->nq = queries_of(a, b);
                if (p->nq <= 0) continue;
                p->len = clamp_len(__ldg(a.lens + b), a.g);
                p->tiles = tiles_of(p->len);
                if (off < (long long)items * (p->tiles + kItemUnits)) break;
            }
            const int cost = p->tiles + kItemUnits;
            p->b = b;
            p->item = int(divide(off, cost));
            const int at = int(off - (long long)p->item * cost);
            const int used = int(min((long long)(cost - at), left));
            p->t0 = max(0, at - kItemUnits);
            p->t1 = max(0, at + used - kItemUnits);
            p->end = pos - at + cost;
            off += used;
            pos += used;
            left -= used;
            if (p->t0 < p->t1) return true;
        }
        return false;
    }

    // The CTA that takes unit x.
    __device__ int owner(long long x) const {
        const long long longer = r * (q + 1);
        return int(x < longer ? divide(x, q + 1) : r + divide(x - longer, q));
    }
};

// A small call (few items, short rows of the table) is split otherwise: a team,
// one cluster of kTeam CTAs, takes an item and joins it through its own shared
// memory, in one launch.
constexpr int kTeam = 8;

struct Member {
    Piece p;
    bool left;
    __device__ void start(const DecodeArgs& a) {
        const int items = a.g.Hkv * a.row_tiles, rank = int(cluster_rank());
        const int item = blockIdx.x / kTeam;
        p.b = item / items;
        p.item = item - p.b * items;
        p.nq = queries_of(a, p.b);
        p.len = clamp_len(__ldg(a.lens + p.b), a.g);
        p.tiles = tiles_of(p.len);
        p.t0 = int((long long)p.tiles * rank / kTeam);
        p.t1 = int((long long)p.tiles * (rank + 1) / kTeam);
        left = p.nq > 0 && p.t0 < p.t1;
    }
    __device__ bool next(const DecodeArgs&, Piece* to) {
        if (!left) return false;
        *to = p;
        left = false;
        return true;
    }
    __device__ int owner(long long) const { return 0; }
};

// Pieces of cut items go through the workspace: CTA c writes its piece that
// starts its item to slot 2c + 1, one that continues an earlier CTA's item to
// slot 2c (it has at most one of each). head[c] describes the item that starts
// in CTA c and goes on in later ones. Between the first and the last CTA of an
// item every CTA holds a piece of it.
struct Head {
    int b;                  // -1: none
    int item;
    int last;               // last CTA that holds a piece of it
    int nq;
};
// How many pieces the item has that starts in CTA first of ctas. (None past the
// slots, should lengths have changed during the call. Bounded here, once an item
// and row: in owner() it cost fp32 with 8 rows at d = 128 2 %.)
__device__ __forceinline__ int pieces_of(const Head& h, int first, int ctas) {
    return max(0, min(h.last, ctas - 1) - first + 1);
}
struct Parts {
    float* o;               // [2G][tile_rows][dv], not divided by l
    float* ml;              // [2G][tile_rows][2]: maximum (base 2) and sum
    Head* head;             // [G]
};

}  // namespace paged
}  // namespace attn
