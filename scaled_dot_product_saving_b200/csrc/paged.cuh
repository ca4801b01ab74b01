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

// ------------------------------------------------- the split of a decode call
// A call's work is counted in units: one key tile (kTileKeys keys) of one item
// (sequence, key head, tile of query rows). A sequence with queries and no
// keys counts one unit per item, so that its rows are written. Units are
// numbered sequence by sequence, item by item, tile by tile, and CTA c of G
// takes [total * c / G, total * (c + 1) / G): every CTA gets the same number
// of tiles however the lengths are spread, which the host does not know. An
// item cut by a CTA border is joined afterwards from its pieces.
constexpr int kTileKeys = 64;
constexpr int kMinUnits = 1;

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

// The CTA's share: walks its pieces in order. Every thread of the block holds
// the same walker.
struct Walker {
    int b;
    long long off;          // units of sequence b already passed
    long long left;         // units left to this CTA
    long long pos, total;   // number of the next unit, and of all units
    int ctas;               // CTAs that have work: each gets kMinUnits at least

    static __device__ __forceinline__ long long units_of(const DecodeArgs& a, int b) {
        if (queries_of(a, b) <= 0) return 0;
        return (long long)(a.g.Hkv * a.row_tiles) * tiles_of(clamp_len(__ldg(a.lens + b), a.g));
    }

    // Collective over the block. scratch: 33 values; found: 2 values.
    __device__ void start(const DecodeArgs& a, long long* scratch, long long* found) {
        const int chunk = (a.g.B + int(blockDim.x) - 1) / int(blockDim.x);
        const int b0 = int(min((long long)a.g.B, (long long)threadIdx.x * chunk));
        const int b1 = min(a.g.B, b0 + chunk);
        long long sum = 0;
        for (int k = b0; k < b1; ++k) sum += units_of(a, k);
        const long long before = block_exclusive(sum, scratch, &total);
        ctas = int(min((long long)gridDim.x, max(1ll, total / kMinUnits)));
        const long long c = min((int)blockIdx.x, ctas);
        pos = total * c / ctas;
        left = total * min(c + 1, (long long)ctas) / ctas - pos;
        if (left > 0 && pos >= before && pos < before + sum) {
            long long x = before;
            int k = b0;
            for (;; ++k) {
                const long long u = units_of(a, k);
                if (pos < x + u) break;
                x += u;
            }
            found[0] = k;
            found[1] = pos - x;
        }
        __syncthreads();
        if (left > 0) {
            b = int(found[0]);
            off = found[1];
        }
    }

    __device__ bool next(const DecodeArgs& a, Piece* p) {
        if (left <= 0) return false;
        const int items = a.g.Hkv * a.row_tiles;
        for (;; ++b, off = 0) {
            p->nq = queries_of(a, b);
            if (p->nq <= 0) continue;
            p->len = clamp_len(__ldg(a.lens + b), a.g);
            p->tiles = tiles_of(p->len);
            if (off < (long long)items * p->tiles) break;
        }
        p->b = b;
        p->item = int(off / p->tiles);
        p->t0 = int(off - (long long)p->item * p->tiles);
        p->t1 = int(min((long long)p->tiles, p->t0 + left));
        p->end = pos - p->t0 + p->tiles;
        const int used = p->t1 - p->t0;
        off += used;
        pos += used;
        left -= used;
        return true;
    }

    // The CTA that takes unit x: the largest c with total * c / ctas <= x.
    __device__ int owner(long long x) const { return int(((x + 1) * ctas - 1) / total); }
};

// Pieces of cut items go through the workspace: CTA c writes its piece that
// starts its item to slot 2c + 1, one that continues an earlier CTA's item to
// slot 2c (it has at most one of each). head[c] describes the item that starts
// in CTA c and goes on in later ones.
struct Head {
    int b;                  // -1: none
    int item;
    int last;               // last CTA that holds a piece of it
    int nq;
};
struct Parts {
    float* o;               // [2G][tile_rows][dv], not divided by l
    float* ml;              // [2G][tile_rows][2]: maximum (base 2) and sum
    Head* head;             // [G]
};

}  // namespace paged
}  // namespace attn
