// decode_f32.cuh -- attention of the newest tokens over paged fp32 keys and
// values, on the CUDA cores in fp32 arithmetic.
//
// The mathematics is decode.cuh's; the stream of tiles is decode_ring.cuh's.
// Memory bounds it here too (1 KB a token and key head at d = 128) as long as
// the arithmetic of a key, 2 (d + dv) fused multiply-adds per query row, keeps
// up with 22 bytes a cycle and SM; for that neither operand of the products may
// come from shared memory more than once:
//  - scores: half a warp per key, 16 lanes over its width, query values of all
//    rows in registers. The partial sums of 8 keys times 4 rows are reduced
//    across the 16 lanes by halving: at each step a lane passes on half of its
//    sums and adds the other half, so that 15 shuffles reduce 16 sums and leave
//    one score per lane;
//  - values: a lane owns 4 columns of the output for all rows, reads each value
//    once, and the weights of a key come as one broadcast per 4 rows.
// One B200, 32768 tokens, d = 128: 4 rows 167 us (6.4 TB/s), 8 rows 208, 16 rows 361,
// where the issue and latency of the arithmetic bound it.
#pragma once

#include "decode_ring.cuh"

namespace attn {
namespace paged {

// DK, DV: padded widths; RB: query rows of a warp (4 or 8); R: groups of RB rows.
template <int DK, int DV, int RB, int R>
struct DecodeF32Cfg {
    static constexpr int kPanelCols = 32, kKPanels = DK / 32, kVPanels = DV / 32, kQPitch = 0, kQBytes = 0, kOffQ = 0;
    static constexpr int kKBytes = kKPanels * kPanelBytes;
    static constexpr int kStageBytes = kKBytes + kVPanels * kPanelBytes;
    // Two CTAs an SM where their stages fit: with 16 consumers instead of 8 the
    // stream is busy (4 x 32768 tokens of 16 heads, d = 64: 165 us, 6.5 TB/s,
    // against 237). At wider rows 16 consumers in one CTA, half of them on every
    // other tile, gained nothing (197 us against 191).
    static constexpr int kCtasPerSm = RB == 4 && DK == 64 && DV == 64 ? 2 : 1;
    static constexpr int kStages = 192 / kCtasPerSm * 1024 / kStageBytes;
    static constexpr int kWarps = 8;                       // consumers: 8 / R key warps per group
    static constexpr int kKeyWarps = kWarps / R, kWarpKeys = kTileKeys / kKeyWarps;
    static constexpr int kProducers = kCtasPerSm == 1 ? 2 : 1;
    static constexpr int kThreads = (kWarps + kProducers) * 32;
    static constexpr int kTileRows = RB * R;
    // The warps' outputs, when a piece ends, lie in the stage of its last tile.
    static_assert(kWarps * RB * DV * 4 <= kStageBytes, "outputs larger than a stage");
    static constexpr int kOffW = kStages * kStageBytes;
    static constexpr int kSmemBytes = kOffW + kWarps * 8 * RB * 4;
};

template <int DK, int DV, int RB, int R>
__global__ void __launch_bounds__(DecodeF32Cfg<DK, DV, RB, R>::kThreads, DecodeF32Cfg<DK, DV, RB, R>::kCtasPerSm)
decode_f32(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, DecodeArgs a,
           const float* __restrict__ Q, float* __restrict__ O, float* __restrict__ LSE, Parts parts,
           unsigned long long budget_ns) {
    using C = DecodeF32Cfg<DK, DV, RB, R>;
    constexpr int kStages = C::kStages, kQ = DK / 64, kSets = RB / 4;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ Ring<kStages, 1> ring;                      // all groups meet, since they share the stage
    __shared__ float stat_m[C::kWarps][RB], stat_l[C::kWarps][RB];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    Walker w;
    if (warp >= C::kWarps) w.start(a);                     // while the barriers are set up
    if (!set_up<false>(parts, ring, smem, C::kWarps, C::kProducers)) return;
    if (warp >= C::kWarps) {
        auto begin = [&](const Stage& p) { return prefetch_rows(Q, p.row, p.rows, a.d); };
        if (C::kProducers == 1) produce<C, Loads::kBoth>(&tmK, &tmV, a, nullptr, w, ring, smem, budget_ns, begin);
        else if (warp == C::kWarps) produce<C, Loads::kKeys>(&tmK, &tmV, a, nullptr, w, ring, smem, budget_ns, begin);
        else produce<C, Loads::kValues>(&tmK, &tmV, a, nullptr, w, ring, smem, budget_ns, begin);
        return;
    }

    const int kg = warp % C::kKeyWarps, group = warp / C::kKeyWarps;
    const int s16 = lane & 15, kp = lane >> 4;             // slice of the width, key of a pair
    const int my_row = s16 & 3, my_key = 2 * (s16 >> 2) + kp;   // of the score this lane ends with
    const float scale_log2 = a.scale * 1.4426950408889634f;
    float* weights = reinterpret_cast<float*>(smem + C::kOffW) + warp * 8 * RB;   // [key][row]
    constexpr int kVKeys = 128 / DV;                       // keys that a warp's 32 chunks of V cover
    const int v_chunk = lane % (DV / 4), v_key = lane / (DV / 4);

    At at{};
    uint32_t joints = 0;                                   // parity of the next meeting
    int tile0 = 0, see_all = 0;
    float4 q[RB][kQ];
    int see[kSets];
    float m[kSets], l[kSets];
    float4 acc[RB];
#pragma unroll
    for (int x = 0; x < kSets; ++x) m[x] = l[x] = 0.f, see[x] = 0;

    // The warps joined, when a piece ends: maxima and sums meet in shared
    // memory; each scales its output to the common maximum and leaves it in the
    // stage, and each sums and writes some rows of its group.
    auto finish = [&](float4* scratch) -> bool {
#pragma unroll
        for (int x = 0; x < kSets; ++x) {
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) l[x] += __shfl_xor_sync(0xffffffffu, l[x], o);
            if (lane < 4) {
                stat_m[warp][4 * x + lane] = m[x];
                stat_l[warp][4 * x + lane] = l[x];
            }
        }
        if constexpr (kVKeys == 2) {                       // the two keys' halves of the output
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                acc[r].x += __shfl_xor_sync(0xffffffffu, acc[r].x, 16);
                acc[r].y += __shfl_xor_sync(0xffffffffu, acc[r].y, 16);
                acc[r].z += __shfl_xor_sync(0xffffffffu, acc[r].z, 16);
                acc[r].w += __shfl_xor_sync(0xffffffffu, acc[r].w, 16);
            }
        }
        constexpr int kGroup = C::kKeyWarps, kChunks = DV / 4;
        const int w0 = group * kGroup;
        warp_arrive(&ring.joint[0][0]);
        if (!ring_wait(ring, &ring.joint[0][0], joints, budget_ns)) return false;
        // Common maximum and sum of row `lane` (the first RB lanes), and what
        // this warp's outputs are scaled with.
        float M = -INFINITY, L = 0.f, f = 0.f;
        if (lane < RB) {
#pragma unroll
            for (int x = 0; x < kGroup; ++x) M = fmaxf(M, stat_m[w0 + x][lane]);
            const float z = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int x = 0; x < kGroup; ++x) L = fmaf(stat_l[w0 + x][lane], exp2f(stat_m[w0 + x][lane] - z), L);
            f = exp2f(stat_m[warp][lane] - z);
        }
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            const float fr = __shfl_sync(0xffffffffu, f, r);
            if (lane < kChunks)
                scratch[(warp * RB + r) * kChunks + lane] =
                    make_float4(acc[r].x * fr, acc[r].y * fr, acc[r].z * fr, acc[r].w * fr);
        }
        warp_arrive(&ring.joint[0][1]);
        if (!ring_wait(ring, &ring.joint[0][1], joints, budget_ns)) return false;
        joints ^= 1;
        const bool all = (at.flags & (kStarts | kEnds)) == (kStarts | kEnds);
        const size_t slot = (2 * size_t(blockIdx.x) + (at.flags & kStarts ? 1 : 0)) * C::kTileRows;
        if (!all && warp == 0 && lane == 0) note_head(parts, at);
        for (int r = kg; r < RB; r += kGroup) {
            const int row = group * RB + r;
            const float Mr = __shfl_sync(0xffffffffu, M, r), Lr = __shfl_sync(0xffffffffu, L, r);
            if (row >= at.rows || (all && query_of(a, at, row) >= at.nq)) continue;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            if (lane < kChunks) {
#pragma unroll
                for (int x = 0; x < kGroup; ++x) {
                    const float4 y = scratch[((w0 + x) * RB + r) * kChunks + lane];
                    o.x += y.x;
                    o.y += y.y;
                    o.z += y.z;
                    o.w += y.w;
                }
            }
            const size_t to = (all ? size_t(at.row) : slot) + row;
            if (all) {
                const float inv = Lr > 0.f ? 1.f / Lr : Lr == 0.f ? 0.f : Lr;            // NaN stays
                if (4 * lane < a.dv)
                    *reinterpret_cast<float4*>(O + to * a.dv + 4 * lane) =
                        make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
                if (lane == 0) LSE[to] = (Mr + log2f(Lr)) * kLn2;
            } else {
                if (4 * lane < a.dv) *reinterpret_cast<float4*>(parts.o + to * a.dv + 4 * lane) = o;
                if (lane == 0) *reinterpret_cast<float2*>(parts.ml + to * 2) = make_float2(Mr, Lr);
            }
        }
        return true;
    };

    uint32_t parity = 0;
    for (int s = 0;; s = s + 1 == kStages ? 0 : s + 1, parity ^= s == 0) {
        if (!ring_wait(ring, &ring.full[s], parity, budget_ns)) return;
        const int flags = ring.stage[s].flags;
        if (flags & kStop) return;
        if (flags & kFirst) {
            at = piece_at(ring, s);
            const int len = ring.stage[s].len, r0 = group * RB;
            // Query columns 4 (s16 + 16 x) of every row.
#pragma unroll
            for (int r = 0; r < RB; ++r) {
#pragma unroll
                for (int x = 0; x < kQ; ++x) {
                    const int c = 4 * (s16 + 16 * x);
                    q[r][x] = r0 + r < at.rows && c < a.d
                                  ? *reinterpret_cast<const float4*>(Q + (size_t(at.row) + r0 + r) * a.d + c)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
                }
            }
            see_all = a.causal ? len - (at.nq - 1) : len;
            tile0 = ring.stage[s].t0 * kTileKeys;
#pragma unroll
            for (int x = 0; x < kSets; ++x) {
                see[x] = visible(a, len, at.nq, query_of(a, at, r0 + 4 * x + my_row));
                m[x] = -INFINITY;
                l[x] = 0.f;
            }
#pragma unroll
            for (int r = 0; r < RB; ++r) acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        {
            const bool rows_here = group * RB < at.rows;
            const uint8_t* st = smem + s * C::kStageBytes;
#pragma unroll 1
            for (int k8 = kg * C::kWarpKeys; rows_here && k8 < (kg + 1) * C::kWarpKeys; k8 += 8) {
                const uint32_t there = uint32_t(ring.stage[s].present >> k8) & 0xffu;
                if (there == 0) continue;
                // Scores of keys k8 + 2 pair + kp, partial over this lane's columns.
                float part[kSets][16];
#pragma unroll
                for (int pair = 0; pair < 4; ++pair) {
                    const int key = k8 + 2 * pair + kp;
                    float4 k[kQ];
#pragma unroll
                    for (int x = 0; x < kQ; ++x)
                        k[x] = *reinterpret_cast<const float4*>(st + ((s16 >> 3) + 2 * x) * kPanelBytes + key * 128 +
                                                                (((s16 & 7) ^ (key & 7)) << 4));
#pragma unroll
                    for (int r = 0; r < RB; ++r) {
                        float sum = 0.f;
#pragma unroll
                        for (int x = 0; x < kQ; ++x) {
                            sum = fmaf(q[r][x].x, k[x].x, sum);
                            sum = fmaf(q[r][x].y, k[x].y, sum);
                            sum = fmaf(q[r][x].z, k[x].z, sum);
                            sum = fmaf(q[r][x].w, k[x].w, sum);
                        }
                        part[r >> 2][pair * 4 + (r & 3)] = sum;
                    }
                }
                float sc[kSets];
#pragma unroll
                for (int x = 0; x < kSets; ++x) {
#pragma unroll
                    for (int o = 8; o >= 1; o >>= 1) {
                        const bool up = s16 & o;
#pragma unroll
                        for (int e = 0; e < o; ++e) {
                            const float pass = up ? part[x][e] : part[x][e + o];
                            const float stay = up ? part[x][e + o] : part[x][e];
                            part[x][e] = stay + __shfl_xor_sync(0xffffffffu, pass, o);
                        }
                    }
                    sc[x] = part[x][0] * scale_log2;       // row 4 x + my_row, key k8 + my_key
                }
                const int k0 = tile0 + k8;
                const bool whole = there == 0xffu && k0 + 8 <= see_all;
                if (!whole) {
#pragma unroll
                    for (int x = 0; x < kSets; ++x)
                        if (!(there >> my_key & 1) || k0 + my_key >= see[x]) sc[x] = -INFINITY;
                }
                // Running maximum over the keys of a row (lanes that differ in bits
                // 2, 3 and 4); the reference moves when it has grown by more than 8.
                float top[kSets];
                bool grown = false;
#pragma unroll
                for (int x = 0; x < kSets; ++x) {
                    top[x] = sc[x];
#pragma unroll
                    for (int o = 4; o <= 16; o <<= 1) top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], o));
                    grown |= top[x] > m[x] + 8.f;
                }
                if (__any_sync(0xffffffffu, grown)) {
                    float f[kSets];
#pragma unroll
                    for (int x = 0; x < kSets; ++x) {
                        const float next = fminf(fmaxf(m[x], top[x]), kTopScore);
                        f[x] = next == -INFINITY ? 1.f : exp2f(m[x] - next);
                        m[x] = next;
                        l[x] *= f[x];
                    }
#pragma unroll
                    for (int r = 0; r < RB; ++r) {
                        const float fr = __shfl_sync(0xffffffffu, f[r >> 2], r & 3);
                        acc[r].x *= fr;
                        acc[r].y *= fr;
                        acc[r].z *= fr;
                        acc[r].w *= fr;
                    }
                }
#pragma unroll
                for (int x = 0; x < kSets; ++x) {
                    const float e = exp2f(sc[x] - (m[x] == -INFINITY ? 0.f : m[x]));
                    l[x] += e;
                    weights[my_key * RB + 4 * x + my_row] = e;
                }
                if (!whole) {
#pragma unroll
                    for (int x = 0; x < kSets; ++x)
                        if (!(there >> my_key & 1) || k0 + my_key >= see[x]) weights[my_key * RB + 4 * x + my_row] = -0.f;
                }
                __syncwarp();
#pragma unroll
                for (int j0 = 0; j0 < 8; j0 += kVKeys) {
                    const int j = j0 + v_key, key = k8 + j;
                    const float4 v = *reinterpret_cast<const float4*>(
                        st + C::kKBytes + (v_chunk >> 3) * kPanelBytes + key * 128 + (((v_chunk & 7) ^ (key & 7)) << 4));
                    if (!whole && !(there >> j & 1)) continue;     // a row that no token owns may hold anything
#pragma unroll
                    for (int x = 0; x < kSets; ++x) {
                        const float4 e4 = *reinterpret_cast<const float4*>(weights + j * RB + 4 * x);
                        const float e[4] = {e4.x, e4.y, e4.z, e4.w};
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            // ... and a token that only some rows see: the others have
                            // -0 (a weight that vanished is +0, and infinity times it NaN)
                            if (!whole && __float_as_uint(e[r]) == 0x80000000u) continue;
                            float4& o = acc[4 * x + r];
                            o.x = fmaf(e[r], v.x, o.x);
                            o.y = fmaf(e[r], v.y, o.y);
                            o.z = fmaf(e[r], v.z, o.z);
                            o.w = fmaf(e[r], v.w, o.w);
                        }
                    }
                }
                __syncwarp();                              // weights are read before the next 8 keys'
            }
        }
        tile0 += kTileKeys;
        if (flags & kLast) {
            // Every warp has read the stage once they have met.
            if (!finish(reinterpret_cast<float4*>(smem + s * C::kStageBytes))) return;
            fence_proxy_async_smem();                      // before the TMA writes there again
        }
        warp_arrive(&ring.empty[s]);
    }
}

}  // namespace paged
}  // namespace attn
