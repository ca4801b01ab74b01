// decode.cuh -- attention of the newest tokens of every sequence over its
// paged keys and values: what the kernels share, the joining of split items, and
// the kernel for bf16 that ATTN_PATH_SIMT asks for (the others are decode_tc.cuh,
// decode_wide.cuh and decode_f32.cuh).
//
//   S_rj = scale * q_r . k_j  over the keys j that row r may see,
//   O_r = sum_j softmax(S_r)_j v_j,  LSE_r = ln sum_j exp(S_rj)
//
// A row that sees no key gets O = 0 and LSE = -inf. Query rows of one key head
// (its group of query heads, times the new tokens) are taken together, so that
// every key and value is read once for all of them. One pass over the keys
// with a running maximum and sum per row (base 2, fp32).
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "paged.cuh"
#include "simt.cuh"
#include "sm100.cuh"

namespace attn {
namespace paged {

constexpr int kRows = 16;             // query rows per item on the CUDA cores
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxWidth = 128;
// Where a running maximum stops (the largest finite number): a score of +inf then
// weighs 2^inf = inf, not 2^(inf - inf), so that LSE is +inf and O = inf / inf is NaN,
// as the logarithm of the sum and the softmax have it. A score of NaN makes both NaN.
constexpr float kTopScore = 3.402823466e38f;

// Last key (exclusive) that query i of nq sees in a sequence of len tokens,
// the queries being its last nq tokens.
__device__ __forceinline__ int visible(const DecodeArgs& a, int len, int nq, int i) {
    return a.causal ? len - (nq - 1 - i) : len;
}

// Rows of an item are numbered r = g * n + i (query head hk * G + g, query i),
// which are consecutive rows of Q, O and LSE.
__device__ __forceinline__ size_t row_base(const DecodeArgs& a, int b, int hk) {
    return (size_t(b) * a.H + size_t(hk) * (a.H / a.g.Hkv)) * a.n;
}

constexpr int kSimtThreads = 128;

__host__ __device__ constexpr int simt_smem_bytes(int d, int dv) {
    return (kRows * d + kTileKeys * (d + 1) + kTileKeys * dv + kRows * kTileKeys + 3 * kRows) * 4;
}

__global__ void __launch_bounds__(kSimtThreads)
decode_simt(DecodeArgs a, const __nv_bfloat16* __restrict__ Q, const __nv_bfloat16* __restrict__ Kp,
            const __nv_bfloat16* __restrict__ Vp, __nv_bfloat16* __restrict__ O, float* __restrict__ LSE,
            Parts parts) {
    extern __shared__ float sm[];
    __shared__ int pages[kTileKeys];
    const int d = a.d, dv = a.dv, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float* Qs = sm;                              // [16][d]
    float* Ks = Qs + kRows * d;                  // [64][d + 1]
    float* Vs = Ks + kTileKeys * (d + 1);        // [64][dv]
    float* Ps = Vs + kTileKeys * dv;             // [16][64]
    float* Ms = Ps + kRows * kTileKeys;          // [16] maximum
    float* Ls = Ms + kRows;                      // [16] sum
    float* Cs = Ls + kRows;                      // [16] factor of the old sums

    // Every warp walks the CTA's pieces.
    Walker w;
    w.start(a);
    if (tid == 0) parts.head[blockIdx.x].b = -1;
    grid_launch_dependents();
    const float scale_log2 = a.scale * 1.4426950408889634f;
    const int page = 1 << a.g.page_log2;

    Piece p;
    while (w.next(a, &p)) {
        const int hk = p.item / a.row_tiles, r0 = (p.item % a.row_tiles) * kRows;
        const int rows = min(kRows, a.rows - r0);
        const size_t base = row_base(a, p.b, hk) + r0;
        __syncthreads();
        for (int x = tid; x < rows * d; x += kSimtThreads) Qs[x] = simt::to_f(Q[base * d + x]);
        if (tid < kRows) {
            Ms[tid] = -INFINITY;
            Ls[tid] = 0.f;
        }
        float acc[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) acc[r] = 0.f;

        for (int t = p.t0; t < p.t1; ++t) {
            const int k0 = t * kTileKeys;
            __syncthreads();
            if (tid < kTileKeys) {
                const int j = k0 + tid;
                int pg = -1;
                if (j < p.len) {
                    pg = a.table[size_t(p.b) * a.g.M + (j >> a.g.page_log2)];
                    if (!page_ok(pg, a.g.P)) pg = -1;
                }
                pages[tid] = pg;
            }
            __syncthreads();
            // Rows of absent tokens are zeros: their weight is zero, and zero
            // times what an unused row may hold need not be.
            for (int j = warp; j < kTileKeys; j += kSimtThreads / 32) {
                const int pg = pages[j];
                const size_t row = (size_t(max(pg, 0)) * a.g.Hkv + hk) * page + ((k0 + j) & (page - 1));
                for (int c = lane; c < d; c += 32) Ks[j * (d + 1) + c] = pg >= 0 ? simt::to_f(Kp[row * d + c]) : 0.f;
                for (int c = lane; c < dv; c += 32) Vs[j * dv + c] = pg >= 0 ? simt::to_f(Vp[row * dv + c]) : 0.f;
            }
            __syncthreads();
            {
                const int j = tid & 63;
                const bool there = pages[j] >= 0;
                for (int r = tid >> 6; r < rows; r += 2) {
                    float s = 0.f;
                    for (int c = 0; c < d; ++c) s = fmaf(Qs[r * d + c], Ks[j * (d + 1) + c], s);
                    const bool see = there && k0 + j < visible(a, p.len, p.nq, (r0 + r) % a.n);
                    Ps[r * kTileKeys + j] = see ? s * scale_log2 : -INFINITY;
                }
            }
            __syncthreads();
            for (int r = warp; r < rows; r += kSimtThreads / 32) {
                const float s0 = Ps[r * kTileKeys + lane], s1 = Ps[r * kTileKeys + 32 + lane];
                const float old = Ms[r];
                const float m = fminf(fmaxf(old, simt::warp_max(fmaxf(s0, s1))), kTopScore);
                const float ms = m == -INFINITY ? 0.f : m;     // a row without keys so far
                const float e0 = exp2f(s0 - ms), e1 = exp2f(s1 - ms), c = exp2f(old - ms);
                const float sum = simt::warp_sum(e0 + e1);
                Ps[r * kTileKeys + lane] = e0;
                Ps[r * kTileKeys + 32 + lane] = e1;
                __syncwarp();
                if (lane == 0) {
                    Ms[r] = m;
                    Ls[r] = Ls[r] * c + sum;
                    Cs[r] = c;
                }
            }
            __syncthreads();
            if (tid < dv) {
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    if (r < rows) {
                        float s = acc[r] * Cs[r];
                        // A token that this row does not see may hold anything.
                        const int end = min(kTileKeys, visible(a, p.len, p.nq, (r0 + r) % a.n) - k0);
                        for (int j = 0; j < end; ++j) s = fmaf(Ps[r * kTileKeys + j], Vs[j * dv + tid], s);
                        acc[r] = s;
                    }
                }
            }
        }
        __syncthreads();
        const bool whole = p.t0 == 0 && p.t1 == p.tiles;
        const size_t slot = 2 * size_t(blockIdx.x) + (p.t0 == 0 ? 1 : 0);
        if (whole) {
            if (tid < dv) {
#pragma unroll
                for (int r = 0; r < kRows; ++r)
                    if (r < rows && (r0 + r) % a.n < p.nq)
                        O[(base + r) * dv + tid] = simt::from_f<__nv_bfloat16>(Ls[r] > 0.f ? acc[r] / Ls[r] : acc[r]);
            }
            if (tid < rows && (r0 + tid) % a.n < p.nq)
                LSE[base + tid] = (Ms[tid] + log2f(Ls[tid])) * kLn2;
        } else {
            if (tid < dv) {
#pragma unroll
                for (int r = 0; r < kRows; ++r)
                    if (r < rows) parts.o[(slot * kRows + r) * dv + tid] = acc[r];
            }
            if (tid < rows) {
                parts.ml[(slot * kRows + tid) * 2] = Ms[tid];
                parts.ml[(slot * kRows + tid) * 2 + 1] = Ls[tid];
            }
            if (tid == 0 && p.t0 == 0) {
                Head h;
                h.b = p.b;
                h.item = p.item;
                h.nq = p.nq;
                h.last = w.owner(p.end - 1);
                parts.head[blockIdx.x] = h;
            }
        }
    }
}

// The item that starts in CTA blockIdx.x and goes on, a row on `split` warps:
// O = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s over its pieces, in an order
// that only depends on their number, so that a repeated call gives the same
// bits. What bounds it is latency: up to 32 maxima and sums are read at once,
// and eight pieces' rows.
constexpr int kJoinThreads = 128;

template <typename T>
__global__ void __launch_bounds__(kJoinThreads)
decode_join(DecodeArgs a, T* __restrict__ O, float* __restrict__ LSE, Parts parts, int split) {
    __shared__ float4 sums[kJoinThreads];
    grid_dependency_wait();
    const int4 hw = __ldcg(reinterpret_cast<const int4*>(parts.head) + blockIdx.x);
    const Head h{hw.x, hw.y, hw.z, hw.w};
    if (h.b < 0) return;                                    // the whole block
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hk = h.item / a.row_tiles, r0 = (h.item % a.row_tiles) * a.tile_rows;
    const int r = (blockIdx.y * (kJoinThreads / 32) + warp) / split, part = warp % split;
    const bool live = r < min(a.tile_rows, a.rows - r0) && (r0 + r) % a.n < h.nq;
    const int first = blockIdx.x, pieces = pieces_of(h, first, gridDim.x);
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live) {
        auto row_of = [&](int c) {
            return (2 * size_t(first + c) + (c == 0 ? 1 : 0)) * a.tile_rows + r;
        };
        const float2* ml = reinterpret_cast<const float2*>(parts.ml);
        // Pieces c + e * split of the 32 from c0 on.
        float4 o[8];
        auto outputs = [&](int c0, int c, int end) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (c + e * split < end && 4 * lane < a.dv)
                    o[e] = __ldcg(reinterpret_cast<const float4*>(parts.o + row_of(c0 + c + e * split) * a.dv + 4 * lane));
            }
        };
        // The first 32 maxima and sums and the first eight outputs in one go.
        const float2 none = make_float2(-INFINITY, 0.f), x0 = lane < pieces ? __ldcg(ml + row_of(lane)) : none;
        outputs(0, part, min(32, pieces));
        m = x0.x;
        for (int c = lane + 32; c < pieces; c += 32) m = fmaxf(m, __ldcg(&ml[row_of(c)].x));
        m = simt::warp_max(m);
        const float ms = m == -INFINITY ? 0.f : m;
        for (int c0 = 0; c0 < pieces; c0 += 32) {
            const float2 x = c0 == 0 ? x0 : c0 + lane < pieces ? __ldcg(ml + row_of(c0 + lane)) : none;
            const float w = exp2f(x.x - ms);
            l = fmaf(x.y, w, l);
            const int end = min(32, pieces - c0);
            for (int c = part; c < end; c += 8 * split) {
                if (c0 + c != part) outputs(c0, c, end);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float f = __shfl_sync(0xffffffffu, w, (c + e * split) & 31);
                    if (c + e * split >= end) continue;
                    acc.x = fmaf(o[e].x, f, acc.x);
                    acc.y = fmaf(o[e].y, f, acc.y);
                    acc.z = fmaf(o[e].z, f, acc.z);
                    acc.w = fmaf(o[e].w, f, acc.w);
                }
            }
        }
        l = simt::warp_sum(l);
    }
    if (split > 1) {
        sums[threadIdx.x] = acc;
        __syncthreads();
        if (part != 0) return;
        for (int x = 1; x < split; ++x) {
            const float4 o = sums[threadIdx.x + 32 * x];
            acc.x += o.x;
            acc.y += o.y;
            acc.z += o.z;
            acc.w += o.w;
        }
    }
    if (!live) return;
    const size_t row = row_base(a, h.b, hk) + r0 + r;
    const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;           // NaN stays
    if (4 * lane < a.dv) {
        T* o = O + row * a.dv + 4 * lane;
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float4*>(o) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        } else {
            *reinterpret_cast<uint2*>(o) =
                make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        }
    }
    if (lane == 0) LSE[row] = (m + log2f(l)) * kLn2;
}

}  // namespace paged
}  // namespace attn
