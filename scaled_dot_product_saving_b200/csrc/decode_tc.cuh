// decode_tc.cuh -- attention of the newest tokens over paged bf16 keys and
// values on the tensor cores.
//
// The mathematics is decode.cuh's. What bounds it is memory: every key and
// value is read once from HBM (512 bytes a token and key head at d = 128) and
// meets the few query rows of its key head, 16 to 64 here. So the design is a
// stream: one warp copies tiles of 64 keys with the TMA, page by page, through
// a ring of stages, as far ahead as shared memory lets it and across the
// borders of pieces; the other warps only consume.
//
// Each of four key warps takes 16 keys of every tile and keeps its own running
// maximum, sum and output for 16 query rows, so that no warp waits for another
// inside a piece; the four are joined when the piece ends. A warp's scores
// leave mma.m16n8k16 in the layout in which their exponentials enter the second
// product, and its share of K and V comes from the TMA's 128-byte-swizzled rows
// through ldmatrix without bank conflicts. Query rows past 16 go to further
// groups of four warps that read the same tiles.
//
// mma.sync and not tcgen05: 16 query rows are an eighth of a tcgen05 tile, its
// accumulator would pass through TMEM twice per 64 keys for the softmax, and
// the four key warps would have to meet at every tile. At 16 rows the tensor
// work of a tile is a few hundred cycles of an SM that gets 22 bytes a cycle
// from HBM (a 32 KB tile every 1,450 cycles).
#pragma once

#include "decode_ring.cuh"

namespace attn {
namespace paged {

constexpr int kKeyWarps = 4;                       // warps that share a tile's keys

template <int DK, int DV, int R>                   // padded widths, groups of 16 query rows
struct DecodeCfg {
    static constexpr int kPanelCols = 64, kKPanels = DK / 64, kVPanels = DV / 64;
    static constexpr int kKBytes = kKPanels * kPanelBytes;
    static constexpr int kStageBytes = kKBytes + kVPanels * kPanelBytes;
    static constexpr int kThreads = (kKeyWarps * R + 1) * 32;
    // Two CTAs an SM for 16 rows (96 KB of stages each), one for more.
    static constexpr int kCtasPerSm = R == 1 ? 2 : 1;
    static constexpr int kStages = (R == 1 ? 96 : 160) * 1024 / kStageBytes;
    static constexpr int kJoinBytes = R * 16 * DV * 4;
    // With four groups a thread has 96 registers: query fragments are read from
    // shared memory at every use instead of being held.
    static constexpr bool kQShared = R == 4;
    static constexpr int kQPitch = DK * 2 + 16;
    static constexpr int kOffQ = kStages * kStageBytes + kJoinBytes;
    static constexpr int kSmemBytes = kOffQ + (kQShared ? R * 16 * kQPitch : 0);
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void group_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Either half of a pair of bf16 infinite or NaN.
__device__ __forceinline__ bool not_finite(uint32_t w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

template <int DK, int DV, int R>
__global__ void __launch_bounds__(DecodeCfg<DK, DV, R>::kThreads, DecodeCfg<DK, DV, R>::kCtasPerSm)
decode_tc(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, DecodeArgs a,
          const __nv_bfloat16* __restrict__ Q, __nv_bfloat16* __restrict__ O, float* __restrict__ LSE,
          Parts parts, unsigned long long budget_ns) {
    using C = DecodeCfg<DK, DV, R>;
    constexpr int kTileRows = 16 * R, kStages = C::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ long long scratch[33], found[2];
    __shared__ Ring<kStages> ring;
    __shared__ float stat_m[R][kKeyWarps][16], stat_l[R][kKeyWarps][16];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    Walker w;
    if (!set_up(a, parts, ring, smem, kKeyWarps * R, scratch, found, &w)) return;

    if (warp == kKeyWarps * R) {
        produce<C>(&tmK, &tmV, a, w, ring, smem, budget_ns);
        return;
    }

    // ---------------------------------------------------------- key warps
    const int kg = warp % kKeyWarps, mt = warp / kKeyWarps;
    const int g = lane >> 2, t4 = lane & 3;
    const float scale_log2 = a.scale * 1.4426950408889634f;
    float4* joined = reinterpret_cast<float4*>(smem + kStages * C::kStageBytes) + mt * (16 * DV / 4);
    // ldmatrix rows of this lane: K by (key half, 8-dim half) = (bit 4, bit 3)
    // of the lane, V by (8-dim half, key half).
    const uint32_t sm = smem_addr(smem);
    const uint32_t k_row = (kg * 16 + ((lane >> 4) << 3) + (lane & 7)) * 128;
    const uint32_t k_x = (((lane >> 3) & 1) ^ (lane & 7)) << 4;
    const uint32_t v_row = C::kKBytes + (kg * 16 + (((lane >> 3) & 1) << 3) + (lane & 7)) * 128;
    const uint32_t v_x = ((lane >> 4) ^ (lane & 7)) << 4;

    int n = 0;
    Piece p;
    while (w.next(a, &p)) {
        const int hk = p.item / a.row_tiles, r0 = (p.item % a.row_tiles) * kTileRows + mt * 16;
        const size_t base = row_base(a, p.b, hk);
        const bool rows_here = r0 < a.rows;               // else only the barriers
        // Query rows as A fragments: rows g and g + 8, widths past d as zeros.
        uint32_t qf[C::kQShared ? 1 : DK / 16][4];
        const uint32_t q_at = sm + C::kOffQ + (mt * 16 + (lane & 15)) * C::kQPitch + (lane >> 4) * 16;
        if constexpr (C::kQShared) {
            group_sync(1 + mt, kKeyWarps * 32);           // the last piece's are read
            for (int x = kg * 32 + lane; x < 16 * (DK / 2); x += kKeyWarps * 32) {
                const int r = x / (DK / 2), c = x % (DK / 2) * 2;
                *reinterpret_cast<uint32_t*>(smem + C::kOffQ + (mt * 16 + r) * C::kQPitch + c * 2) =
                    r0 + r < a.rows && c < a.d ? *reinterpret_cast<const uint32_t*>(Q + (base + r0 + r) * a.d + c)
                                               : 0u;
            }
            group_sync(1 + mt, kKeyWarps * 32);
        } else {
#pragma unroll
            for (int ks = 0; ks < DK / 16; ++ks) {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int r = r0 + g + (x & 1) * 8, c = ks * 16 + 2 * t4 + (x >> 1) * 8;
                    qf[ks][x] = r < a.rows && c < a.d
                                    ? *reinterpret_cast<const uint32_t*>(Q + (base + r) * a.d + c)
                                    : 0u;
                }
            }
        }
        // Keys that rows g and g + 8 see, and that every row sees.
        const int see0 = visible(a, p.len, p.nq, (r0 + g) % a.n);
        const int see1 = visible(a, p.len, p.nq, (r0 + g + 8) % a.n);
        const int see_all = a.causal ? p.len - (p.nq - 1) : p.len;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
        float acc[DV / 8][4];
#pragma unroll
        for (int x = 0; x < DV / 8; ++x) acc[x][0] = acc[x][1] = acc[x][2] = acc[x][3] = 0.f;

        for (int t = p.t0; t < p.t1; ++t, ++n) {
            const int s = n % kStages;
            ring_wait(ring, &ring.full[s], (n / kStages) & 1, budget_ns);
            const uint32_t st = sm + s * C::kStageBytes;
            const int k0 = t * kTileKeys + kg * 16;       // this warp's keys
            const uint32_t there = uint32_t(ring.present[s] >> (kg * 16)) & 0xffffu;
            if (rows_here && there != 0) {
                float sc[2][4] = {};
#pragma unroll
                for (int ks = 0; ks < DK / 16; ++ks) {
                    uint32_t b[4];
                    ldsm4(st + (ks / 4) * kPanelBytes + k_row + (k_x ^ ((ks & 3) << 5)), b);
                    uint32_t(&q)[4] = qf[C::kQShared ? 0 : ks];
                    if constexpr (C::kQShared) ldsm4(q_at + ks * 32, q);
                    mma16816(sc[0], q, b[0], b[1]);
                    mma16816(sc[1], q, b[2], b[3]);
                }
                // sc[h][0..1]: row g, keys 8 h + 2 t4 + {0, 1}; sc[h][2..3]: row g + 8.
                const bool whole = there == 0xffffu && k0 + 16 <= see_all;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) sc[h][x] *= scale_log2;
                }
                if (!whole) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int j = 8 * h + 2 * t4 + (x & 1);
                            if (!(there >> j & 1) || k0 + j >= (x < 2 ? see0 : see1)) sc[h][x] = -INFINITY;
                        }
                    }
                }
                float x0 = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
                float x1 = fmaxf(fmaxf(sc[0][2], sc[0][3]), fmaxf(sc[1][2], sc[1][3]));
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
                // The reference value moves, and the sums are rescaled, only when
                // a maximum has grown by more than 8 (base 2): weights stay below
                // 2^8 and are summed in fp32.
                if (__any_sync(0xffffffffu, x0 > m0 + 8.f || x1 > m1 + 8.f)) {
                    const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
                    const float f0 = n0 == -INFINITY ? 1.f : ex2(m0 - n0), f1 = n1 == -INFINITY ? 1.f : ex2(m1 - n1);
                    m0 = n0;
                    m1 = n1;
                    l0 *= f0;
                    l1 *= f1;
#pragma unroll
                    for (int x = 0; x < DV / 8; ++x) {
                        acc[x][0] *= f0;
                        acc[x][1] *= f0;
                        acc[x][2] *= f1;
                        acc[x][3] *= f1;
                    }
                }
                const float z0 = m0 == -INFINITY ? 0.f : m0, z1 = m1 == -INFINITY ? 0.f : m1;
                uint32_t pf[4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float e0 = ex2(sc[h][0] - z0), e1 = ex2(sc[h][1] - z0);
                    const float e2 = ex2(sc[h][2] - z1), e3 = ex2(sc[h][3] - z1);
                    l0 += e0 + e1;
                    l1 += e2 + e3;
                    // Weights in bf16 for the second product (half a step, 2^-8 of
                    // each); their sum is of the unrounded ones.
                    pf[2 * h] = pack_bf16x2(e0, e1);
                    pf[2 * h + 1] = pack_bf16x2(e2, e3);
                }
                if (whole) {
#pragma unroll
                    for (int c = 0; c < DV / 16; ++c) {
                        uint32_t b[4];
                        ldsm4_t(st + (c / 4) * kPanelBytes + v_row + (v_x ^ ((c & 3) << 5)), b);
                        mma16816(acc[2 * c], pf, b[0], b[1]);
                        mma16816(acc[2 * c + 1], pf, b[2], b[3]);
                    }
                } else {
                    // Rows of V that no token owns may hold anything: zero times
                    // them is made zero. A token that only some rows see may hold
                    // infinities or NaN; those are left to the loop below.
                    const uint32_t lo = (there >> (2 * t4) & 1 ? 0xffffu : 0u) |
                                        (there >> (2 * t4 + 1) & 1 ? 0xffff0000u : 0u);
                    const uint32_t hi = (there >> (2 * t4 + 8) & 1 ? 0xffffu : 0u) |
                                        (there >> (2 * t4 + 9) & 1 ? 0xffff0000u : 0u);
                    bool odd = false;
#pragma unroll
                    for (int c = 0; c < DV / 16; ++c) {
                        uint32_t b[4];
                        ldsm4_t(st + (c / 4) * kPanelBytes + v_row + (v_x ^ ((c & 3) << 5)), b);
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            b[x] &= x & 1 ? hi : lo;
                            if (not_finite(b[x])) {
                                odd = true;
                                if ((b[x] & 0x7f80u) == 0x7f80u) b[x] &= 0xffff0000u;
                                if ((b[x] & 0x7f800000u) == 0x7f800000u) b[x] &= 0xffffu;
                            }
                        }
                        mma16816(acc[2 * c], pf, b[0], b[1]);
                        mma16816(acc[2 * c + 1], pf, b[2], b[3]);
                    }
                    if (__any_sync(0xffffffffu, odd)) {
                        // Value by value: infinities and NaN times the weights of
                        // the rows that see them.
                        for (int j = 0; j < 16; ++j) {
                            if (!(there >> j & 1)) continue;
                            const int from = (lane & ~3) | ((j & 7) >> 1);
                            const uint32_t w0 = __shfl_sync(0xffffffffu, pf[j >> 3 ? 2 : 0], from);
                            const uint32_t w1 = __shfl_sync(0xffffffffu, pf[j >> 3 ? 3 : 1], from);
                            const float p0 = __uint_as_float(j & 1 ? w0 & 0xffff0000u : w0 << 16);
                            const float p1 = __uint_as_float(j & 1 ? w1 & 0xffff0000u : w1 << 16);
                            const int key = kg * 16 + j;
#pragma unroll
                            for (int c = 0; c < DV / 8; ++c) {
                                const uint8_t* at = smem + s * C::kStageBytes + C::kKBytes + (c / 8) * kPanelBytes +
                                                    key * 128 + (((c & 7) ^ (key & 7)) << 4) + t4 * 4;
                                const uint32_t v = *reinterpret_cast<const uint32_t*>(at);
#pragma unroll
                                for (int x = 0; x < 2; ++x) {
                                    const float y = __uint_as_float(x ? v & 0xffff0000u : v << 16);
                                    if (isfinite(y)) continue;
                                    if (p0 != 0.f) acc[c][x] += p0 * y;
                                    if (p1 != 0.f) acc[c][2 + x] += p1 * y;
                                }
                            }
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ring.empty[s]);
        }

        // ------------------------------------------- the four warps joined
        // Their maxima and sums meet in shared memory; each scales its output
        // to the common maximum, and they are added in the order of the warps.
        l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
        if (t4 == 0) {
            stat_m[mt][kg][g] = m0;
            stat_m[mt][kg][g + 8] = m1;
            stat_l[mt][kg][g] = l0;
            stat_l[mt][kg][g + 8] = l1;
        }
        group_sync(R == 1 ? 1 : 1 + mt, kKeyWarps * 32);
        float M0 = -INFINITY, M1 = -INFINITY, L0 = 0.f, L1 = 0.f;
#pragma unroll
        for (int x = 0; x < kKeyWarps; ++x) {
            M0 = fmaxf(M0, stat_m[mt][x][g]);
            M1 = fmaxf(M1, stat_m[mt][x][g + 8]);
        }
        const float Z0 = M0 == -INFINITY ? 0.f : M0, Z1 = M1 == -INFINITY ? 0.f : M1;
#pragma unroll
        for (int x = 0; x < kKeyWarps; ++x) {
            L0 = fmaf(stat_l[mt][x][g], ex2(stat_m[mt][x][g] - Z0), L0);
            L1 = fmaf(stat_l[mt][x][g + 8], ex2(stat_m[mt][x][g + 8] - Z1), L1);
        }
        const float f0 = ex2(m0 - Z0), f1 = ex2(m1 - Z1);
#pragma unroll
        for (int x = 0; x < DV / 8; ++x) {
            acc[x][0] *= f0;
            acc[x][1] *= f0;
            acc[x][2] *= f1;
            acc[x][3] *= f1;
        }
#pragma unroll 1
        for (int turn = kKeyWarps - 1; turn >= 0; --turn) {
            if (kg == turn) {
#pragma unroll
                for (int x = 0; x < DV / 8; ++x) {
                    if (turn < kKeyWarps - 1) {
                        const float4 o = joined[x * 32 + lane];
                        acc[x][0] += o.x;
                        acc[x][1] += o.y;
                        acc[x][2] += o.z;
                        acc[x][3] += o.w;
                    }
                    if (turn > 0) joined[x * 32 + lane] = make_float4(acc[x][0], acc[x][1], acc[x][2], acc[x][3]);
                }
            }
            if (turn > 0) group_sync(R == 1 ? 1 : 1 + mt, kKeyWarps * 32);
        }
        if (kg != 0) continue;

        const bool all = p.t0 == 0 && p.t1 == p.tiles;
        const size_t slot = 2 * size_t(blockIdx.x) + (p.t0 == 0 ? 1 : 0);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = r0 + g + 8 * half;
            if (r >= a.rows) continue;
            const float L = half ? L1 : L0, M = half ? M1 : M0;
            if (all) {
                if (r % a.n >= p.nq) continue;
                const float inv = L > 0.f ? 1.f / L : L == 0.f ? 0.f : L;     // NaN stays
                __nv_bfloat16* o = O + (base + r) * a.dv;
#pragma unroll
                for (int x = 0; x < DV / 8; ++x) {
                    const int c = 8 * x + 2 * t4;
                    if (c < a.dv)
                        *reinterpret_cast<uint32_t*>(o + c) =
                            pack_bf16x2(acc[x][2 * half] * inv, acc[x][2 * half + 1] * inv);
                }
                if (t4 == 0) LSE[base + r] = (M + log2f(L)) * kLn2;
            } else {
                const int rt = mt * 16 + g + 8 * half;                        // row of the slot
                float* o = parts.o + (slot * kTileRows + rt) * a.dv;
#pragma unroll
                for (int x = 0; x < DV / 8; ++x) {
                    const int c = 8 * x + 2 * t4;
                    if (c < a.dv) *reinterpret_cast<float2*>(o + c) = make_float2(acc[x][2 * half], acc[x][2 * half + 1]);
                }
                if (t4 == 0) {
                    parts.ml[(slot * kTileRows + rt) * 2] = M;
                    parts.ml[(slot * kTileRows + rt) * 2 + 1] = L;
                }
            }
        }
        if (!all && p.t0 == 0 && mt == 0 && lane == 0) {
            Head h;
            h.b = p.b;
            h.item = p.item;
            h.nq = p.nq;
            h.last = w.owner(p.end - 1);
            parts.head[blockIdx.x] = h;
        }
    }
}

}  // namespace paged
}  // namespace attn
