// decode_tc.cuh -- attention of the newest tokens over paged bf16 keys and
// values on the tensor cores.
//
// The mathematics is decode.cuh's. What bounds it is memory: every key and
// value is read once from HBM (512 bytes a token and key head at d = 128) and
// meets the few query rows of its key head, up to 32 here. So the design is a
// stream: one warp copies tiles of 64 keys with the TMA, page by page, through
// a ring of stages, as far ahead as shared memory lets it and across the
// borders of pieces; the other warps only consume.
//
// Each of four key warps takes 16 keys of every tile and keeps its own running
// maximum, sum and output for 16 query rows, so that no warp waits for another
// inside a piece. A warp's scores leave mma.m16n8k16 in the layout in which their
// exponentials enter the second product, and its share of K and V comes from the
// TMA's 128-byte-swizzled rows through ldmatrix without bank conflicts. Query rows
// past 16 go to a second group of four warps that read the same tiles.
//
// At the end of a piece the four are joined. Where there is room for it (d = 128, up
// to 16 rows) they do not wait for that either: each leaves what it has in the place
// of its own keys in the last tile's stage, and a warp of its own joins and writes
// the rows while they go on; the query rows come with a piece's first tile. Else
// they meet twice, and each writes a quarter of the columns. (Meeting costs 3,000
// cycles a piece, leaving 500; query rows from global memory 800 to 1,900. 200
// sequences of 30 to 400 tokens, d = 128: 32 key heads 137 us with meetings, 111
// without; 8 key heads 45.5 and 37.2; 64 sequences of 128 to 16384: 143.4, 144.5.)
//
// mma.sync and not tcgen05, up to 32 rows: 16 query rows are an eighth of a
// tcgen05 tile, its accumulator would pass through TMEM twice per 64 keys for the
// softmax, and the four key warps would have to meet at every tile. At 16 rows
// the tensor work of a tile is a few hundred cycles of an SM that gets 22 bytes a
// cycle from HBM (a 32 KB tile every 1,450 cycles). At 32 the instruction itself
// becomes the limit: a tile takes 64 of them a sub-partition, at about 16 cycles.
//
// One B200: 4 x 65536 tokens of 8 key heads, d = 128, 4 rows: 6.5 TB/s in pages
// of 16, 6.0 in pages of 8; 4 x 65536 to 262144 in pages of 64: 6.7 TB/s (the
// measured copy runs at 6.54). 64 sequences of 128 to 16384: 6.1 TB/s. The rest
// of a small call is latency: 1.7 us until the first copy is issued, 0.8 for it to
// arrive, about 1 us a tile and 1 us to join.
#pragma once

#include <type_traits>

#include "decode_ring.cuh"

namespace attn {
namespace paged {

constexpr int kKeyWarps = 4;                       // warps that share a tile's keys

// DK, DV: padded widths; R: groups of 16 query rows; kTeamed: a team an item.
template <int DK, int DV, int R, bool kTeamed>
struct DecodeCfg {
    static constexpr int kTileRows = 16 * R;
    static constexpr int kPanelCols = 64, kKPanels = DK / 64, kVPanels = DV / 64;
    static constexpr int kKBytes = kKPanels * kPanelBytes;
    static constexpr int kStageBytes = kKBytes + kVPanels * kPanelBytes;
    static constexpr int kProducers = R == 2 ? 2 : 1;
    static constexpr bool kNarrow = DK == 64 && DV == 64;
    // A warp of its own joins the key warps' outputs, [16][DV] each, left in the
    // place of a warp's 16 keys (2 KB of each panel) in the stage of the piece's last
    // tile. Not where they do not fit there (dv > d); not with two groups, for which
    // one warp is too slow (200 x 64 tokens, 20 rows, d = 128: 49.5 us against 41.0),
    // nor at d = dv = 64, where three CTAs of six warps leave a thread 96 registers (24
    // drafts: 22.4 against 21.6): there the key warps meet.
    static constexpr int kWarpRows = 2048 / (DV * 4);                             // rows in 2 KB
    static constexpr bool kJoiner = R == 1 && !kNarrow && kWarpRows * (kKPanels + kVPanels) >= 16;
    static constexpr int kThreads = (kKeyWarps * R + kProducers + (kJoiner ? 1 : 0)) * 32;
    // CTAs an SM: for 16 rows two of 113 KB, or at d = dv = 64, where a tile is
    // half the bytes and costs a warp 0.7 of the time, three of 72 KB (24 sequences
    // x 16 heads of about 1,100 tokens: 25.7 us with two, 21.6 with three, 22.6 with
    // four); for 32 rows one, or two at d = dv = 64 (8 sequences of 16500 tokens, 8
    // key heads, 24 rows: 86.0 us with one, 60.0 with two; 64 of 100 to 3000: 53.4
    // and 44.2).
    static constexpr int kCtasPerSm = 3 - R + (kNarrow ? 1 : 0);
    static constexpr int kStages = R == 2 ? 128 * 1024 / kCtasPerSm / kStageBytes : kNarrow ? 4 : 3;
    // Where the key warps meet: all their outputs, in the stage of the piece's last
    // tile, if they fit, or beside the stages.
    static constexpr int kScratchBytes = kKeyWarps * 16 * DV * 4;
    static constexpr bool kInStage = R == 1 && kScratchBytes <= kStageBytes;
    static constexpr int kOffOut = kStages * kStageBytes;
    // Query rows of a piece that begins in a stage (where there is room), each turned
    // by 16 bytes more than the one before, so that ldmatrix meets no bank twice.
    static constexpr int kOffQ = kOffOut + (kInStage || kJoiner ? 0 : R * kScratchBytes);
    static constexpr int kQPitch = !kNarrow && (kJoiner || R == 2) ? DK * 2 : 0, kQBytes = 16 * R * kQPitch;
    // A team's CTA leaves its output here for the others, [16][DV]: its only piece
    // has read its query rows.
    static constexpr int kOffTeam = kOffQ;
    static constexpr int kTeamBytes = kTeamed ? 16 * DV * 4 : 0;
    static constexpr int kSmemBytes = kOffQ + (kStages * kQBytes > kTeamBytes ? kStages * kQBytes : kTeamBytes);
    static_assert(!kTeamed || R == 1, "a team has one group of rows");
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
// Either half of a pair of bf16 infinite or NaN.
__device__ __forceinline__ bool not_finite(uint32_t w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// Row r of the output that key warp kg leaves for the joining warp when a piece
// ends with the tile in stage s; blocks of 8 columns lie at block ^ (r % 8).
template <typename C>
__device__ __forceinline__ uint8_t* out_row(uint8_t* smem, int s, int kg, int r) {
    return smem + s * C::kStageBytes + (r / C::kWarpRows) * kPanelBytes + kg * 2048 +
           (r % C::kWarpRows) * (2048 / C::kWarpRows);
}

// An address of this CTA's shared memory in another CTA of the cluster.
__device__ __forceinline__ uint32_t of_member(uint32_t addr, int rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float2 ld_member(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ int ld_member_int(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

template <int DK, int DV, int R, bool kTeamed>
__global__ void __launch_bounds__(DecodeCfg<DK, DV, R, kTeamed>::kThreads, DecodeCfg<DK, DV, R, kTeamed>::kCtasPerSm)
decode_tc(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, DecodeArgs a,
          const __nv_bfloat16* __restrict__ Q, __nv_bfloat16* __restrict__ O, float* __restrict__ LSE,
          Parts parts, unsigned long long budget_ns) {
    using C = DecodeCfg<DK, DV, R, kTeamed>;
    constexpr int kTileRows = C::kTileRows, kStages = C::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr int kKeys = kKeyWarps * R;                  // key warps; then the producers, then the joining warp
    __shared__ Ring<kStages, R> ring;
    // Maxima and sums of the key warps; with a joining warp by the stage of a piece's
    // last tile, and the warps' arrivals there.
    constexpr int kSlots = C::kJoiner ? kStages : R;
    __shared__ float2 stat[kSlots][kKeyWarps][16];
    __shared__ uint64_t left[kSlots];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    __shared__ float2 team_ml[kTeamed ? 16 : 1];          // maximum and sum of each row, for the team; a sum
                                                          // below zero: the CTA had no tile

    std::conditional_t<kTeamed, Member, Walker> w;
    if (kTeamed || (warp >= kKeys && warp < kKeys + C::kProducers)) w.start(a);   // while the barriers are set up
    if (threadIdx.x == 0)
        for (int x = 0; x < kSlots; ++x) mbar_init(&left[x], kKeys);
    if (kTeamed && threadIdx.x < 16) team_ml[threadIdx.x] = make_float2(-INFINITY, -1.f);   // until it has a tile's
    const bool going = set_up<kTeamed>(parts, ring, smem, kKeys + (C::kJoiner ? 1 : 0), C::kProducers);   // fences the barriers' initialisation
    if (!kTeamed && !going) return;

    auto consume = [&] {
    // ---------------------------------------------------------- key warps
    const int kg = warp % kKeyWarps, mt = warp / kKeyWarps;
    const int g = lane >> 2, t4 = lane & 3;
    const float scale_log2 = a.scale * 1.4426950408889634f;
    // ldmatrix rows of this lane: K by (key half, 8-dim half) = (bit 4, bit 3)
    // of the lane, V by (8-dim half, key half).
    const uint32_t sm = smem_addr(smem);
    const uint32_t k_row = (kg * 16 + ((lane >> 4) << 3) + (lane & 7)) * 128;
    const uint32_t k_x = (((lane >> 3) & 1) ^ (lane & 7)) << 4;
    const uint32_t v_row = C::kKBytes + (kg * 16 + (((lane >> 3) & 1) << 3) + (lane & 7)) * 128;
    const uint32_t v_x = ((lane >> 4) ^ (lane & 7)) << 4;

    At at{};
    uint32_t joints = 0;                                  // parity of the group's next meeting
    uint32_t qf[DK / 16][4];
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float acc[DV / 8][4];
    int see0 = 0, see1 = 0, see_all = 0, k0 = 0;

    auto sums = [&](int slot) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
        if (t4 == 0) {
            stat[slot][kg][g] = make_float2(m0, l0);
            stat[slot][kg][g + 8] = make_float2(m1, l1);
        }
    };

    // What this warp has of a piece, where the joining warp finds it.
    auto leave = [&](int s) {
        sums(s);
        __syncwarp();                                     // the warp has read its keys and values
        uint8_t* ra = out_row<C>(smem, s, kg, g) + t4 * 8;
        uint8_t* rb = out_row<C>(smem, s, kg, g + 8) + t4 * 8;
        if (g < at.rows) {
#pragma unroll
            for (int x = 0; x < DV / 8; ++x) *reinterpret_cast<float2*>(ra + ((x ^ g) << 5)) = make_float2(acc[x][0], acc[x][1]);
        }
        if (g + 8 < at.rows) {
#pragma unroll
            for (int x = 0; x < DV / 8; ++x) *reinterpret_cast<float2*>(rb + ((x ^ g) << 5)) = make_float2(acc[x][2], acc[x][3]);
        }
        warp_arrive(&left[s]);
    };

    // The four warps of the group joined, when a piece ends: their maxima and
    // sums meet in shared memory; each scales its output to the common maximum
    // and leaves it there, and each sums and writes a quarter of the columns.
    auto finish = [&](uint8_t* scratch) -> bool {
        sums(mt);
        warp_arrive(&ring.joint[mt][0]);
        if (!ring_wait(ring, &ring.joint[mt][0], joints, budget_ns)) return false;
        float M0 = -INFINITY, M1 = -INFINITY, L0 = 0.f, L1 = 0.f;
#pragma unroll
        for (int x = 0; x < kKeyWarps; ++x) {
            M0 = fmaxf(M0, stat[mt][x][g].x);
            M1 = fmaxf(M1, stat[mt][x][g + 8].x);
        }
        const float Z0 = M0 == -INFINITY ? 0.f : M0, Z1 = M1 == -INFINITY ? 0.f : M1;
        const float f0 = ex2(m0 - Z0), f1 = ex2(m1 - Z1);
        float4* out = reinterpret_cast<float4*>(scratch) + lane;
#pragma unroll
        for (int x = 0; x < DV / 8; ++x)
            out[(kg * (DV / 8) + x) * 32] = make_float4(acc[x][0] * f0, acc[x][1] * f0, acc[x][2] * f1, acc[x][3] * f1);
#pragma unroll
        for (int x = 0; x < kKeyWarps; ++x) {
            const float2 u0 = stat[mt][x][g], u1 = stat[mt][x][g + 8];
            L0 = fmaf(u0.y, ex2(u0.x - Z0), L0);
            L1 = fmaf(u1.y, ex2(u1.x - Z1), L1);
        }
        warp_arrive(&ring.joint[mt][1]);
        const bool all = !kTeamed && (at.flags & (kStarts | kEnds)) == (kStarts | kEnds);
        const int ra = mt * 16 + g, rb = ra + 8;
        const bool put0 = ra < at.rows && (!all || query_of(a, at, ra) < at.nq);
        const bool put1 = rb < at.rows && (!all || query_of(a, at, rb) < at.nq);
        const float inv0 = all ? (L0 > 0.f ? 1.f / L0 : L0 == 0.f ? 0.f : L0) : 1.f;         // NaN stays
        const float inv1 = all ? (L1 > 0.f ? 1.f / L1 : L1 == 0.f ? 0.f : L1) : 1.f;
        const size_t slot = (2 * size_t(blockIdx.x) + (at.flags & kStarts ? 1 : 0)) * kTileRows;
        const size_t to0 = (all ? size_t(at.row) : slot) + ra, to1 = to0 + 8;
        float* team_o = reinterpret_cast<float*>(smem + C::kOffTeam);
        if (kg == 0 && t4 == 0) {
            if constexpr (kTeamed) {
                team_ml[ra] = make_float2(M0, L0);
                team_ml[rb] = make_float2(M1, L1);
            } else if (all) {
                if (put0) LSE[to0] = (M0 + log2f(L0)) * kLn2;
                if (put1) LSE[to1] = (M1 + log2f(L1)) * kLn2;
            } else {
                if (put0) *reinterpret_cast<float2*>(parts.ml + to0 * 2) = make_float2(M0, L0);
                if (put1) *reinterpret_cast<float2*>(parts.ml + to1 * 2) = make_float2(M1, L1);
                if (mt == 0 && lane == 0) note_head(parts, at);
            }
        }
        if (!ring_wait(ring, &ring.joint[mt][1], joints, budget_ns)) return false;
        joints ^= 1;
        constexpr int kCols = DV / 8 / kKeyWarps;         // blocks of 8 columns a warp
#pragma unroll
        for (int x = 0; x < kCols; ++x) {
            const int c8 = kg * kCols + x, c = 8 * c8 + 2 * t4;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kKeyWarps; ++k) {
                const float4 o = out[(k * (DV / 8) + c8) * 32];
                y.x += o.x;
                y.y += o.y;
                y.z += o.z;
                y.w += o.w;
            }
            if constexpr (kTeamed) {
                *reinterpret_cast<float2*>(team_o + ra * DV + c) = make_float2(y.x, y.y);
                *reinterpret_cast<float2*>(team_o + rb * DV + c) = make_float2(y.z, y.w);
                continue;
            }
            if (c >= a.dv) continue;
            if (all) {
                if (put0) *reinterpret_cast<uint32_t*>(O + to0 * a.dv + c) = pack_bf16x2(y.x * inv0, y.y * inv0);
                if (put1) *reinterpret_cast<uint32_t*>(O + to1 * a.dv + c) = pack_bf16x2(y.z * inv1, y.w * inv1);
            } else {
                if (put0) *reinterpret_cast<float2*>(parts.o + to0 * a.dv + c) = make_float2(y.x, y.y);
                if (put1) *reinterpret_cast<float2*>(parts.o + to1 * a.dv + c) = make_float2(y.z, y.w);
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
            const int len = ring.stage[s].len, r = mt * 16 + g;
            // Query rows g and g + 8 as A fragments, widths past d as zeros.
            if constexpr (C::kQPitch > 0) {
                const int row = mt * 16 + (lane & 15);
                const uint32_t q = sm + C::kOffQ + s * C::kQBytes + row * C::kQPitch;
#pragma unroll
                for (int ks = 0; ks < DK / 16; ++ks) {
                    ldsm4(q + (((row + 2 * ks + (lane >> 4)) << 4) & (C::kQPitch - 1)), qf[ks]);
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if (r + (x & 1) * 8 >= at.rows || 2 * t4 + ks * 16 + (x >> 1) * 8 >= a.d) qf[ks][x] = 0u;
                }
            } else {
                const __nv_bfloat16* q = Q + (size_t(at.row) + r) * a.d + 2 * t4;
#pragma unroll
                for (int ks = 0; ks < DK / 16; ++ks) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int c = ks * 16 + (x >> 1) * 8;
                        qf[ks][x] = r + (x & 1) * 8 < at.rows && c < a.d
                                        ? *reinterpret_cast<const uint32_t*>(q + (x & 1) * 8 * a.d + c)
                                        : 0u;
                    }
                }
            }
            // Keys that rows g and g + 8 see, and that every row sees.
            see0 = visible(a, len, at.nq, query_of(a, at, r));
            see1 = visible(a, len, at.nq, query_of(a, at, r + 8));
            see_all = a.causal ? len - (at.nq - 1) : len;
            k0 = ring.stage[s].t0 * kTileKeys + kg * 16;
            m0 = m1 = -INFINITY;
            l0 = l1 = 0.f;
#pragma unroll
            for (int x = 0; x < DV / 8; ++x) acc[x][0] = acc[x][1] = acc[x][2] = acc[x][3] = 0.f;
        }
        {
            const bool rows_here = mt * 16 < at.rows;     // else only the barriers
            const uint32_t st = sm + s * C::kStageBytes;
            const uint32_t there = uint32_t(ring.stage[s].present >> (kg * 16)) & 0xffffu;
            if (rows_here && there != 0) {
                float sc[2][4] = {};
#pragma unroll
                for (int ks = 0; ks < DK / 16; ++ks) {
                    uint32_t b[4];
                    ldsm4(st + (ks / 4) * kPanelBytes + k_row + (k_x ^ ((ks & 3) << 5)), b);
                    mma16816(sc[0], qf[ks], b[0], b[1]);
                    mma16816(sc[1], qf[ks], b[2], b[3]);
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
                    const float n0 = fminf(fmaxf(m0, x0), kTopScore), n1 = fminf(fmaxf(m1, x1), kTopScore);
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
                        // the rows that see them, a weight of zero included.
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
                                    if (k0 + j < see0) acc[c][x] += p0 * y;
                                    if (k0 + j < see1) acc[c][2 + x] += p1 * y;
                                }
                            }
                        }
                    }
                }
            }
        }
        k0 += kTileKeys;
        if (flags & kLast) {
            if constexpr (C::kJoiner) {
                leave(s);
            } else {
                // Every warp of the group has read the stage once they have met.
                uint8_t* scratch = smem + (C::kInStage ? s * C::kStageBytes : C::kOffOut + mt * C::kScratchBytes);
                if (!finish(scratch)) return;
                if (C::kInStage) fence_proxy_async_smem();    // before the TMA writes there again
            }
        }
        warp_arrive(&ring.empty[s]);
    }
    };

    // The joining warp follows the stream and takes what the key warps left of each
    // piece: O = sum_w 2^(m_w - m) o_w, with its maximum and sum, or divided by the sum
    // if the piece is its whole item. A row is 4 columns a lane.
    auto join = [&] {
    At at{};
    uint32_t parity = 0, turn = 0;                        // turn: parity of left, a bit a stage
    constexpr int kLanes = DV / 4, kRowsAtOnce = 32 / kLanes;
    const int col = lane % kLanes, sub = lane / kLanes;
    for (int s = 0;; s = s + 1 == kStages ? 0 : s + 1, parity ^= s == 0) {
        if (!ring_wait(ring, &ring.full[s], parity, budget_ns)) return;
        const int flags = ring.stage[s].flags;
        if (flags & kStop) return;
        if (flags & kFirst) at = piece_at(ring, s);
        if (!(flags & kLast)) {
            warp_arrive(&ring.empty[s]);
            continue;
        }
        if (!ring_wait(ring, &left[s], (turn >> s) & 1, budget_ns)) return;
        turn ^= 1u << s;
        const bool all = !kTeamed && (at.flags & (kStarts | kEnds)) == (kStarts | kEnds);
        const size_t first = all ? size_t(at.row) : (2 * size_t(blockIdx.x) + (at.flags & kStarts ? 1 : 0)) * kTileRows;
        if (!kTeamed && !all && lane == 0) note_head(parts, at);
        const int mine = lane & 15;                     // statistics: a row a lane
        float2 x[kKeyWarps];
        float M = -INFINITY, L = 0.f, f[kKeyWarps];
#pragma unroll
        for (int k = 0; k < kKeyWarps; ++k) {
            x[k] = stat[s][k][mine];
            M = fmaxf(M, x[k].x);
        }
        const float Z = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int k = 0; k < kKeyWarps; ++k) {
            f[k] = ex2(x[k].x - Z);
            L = fmaf(x[k].y, f[k], L);
        }
        const float inv = all ? (L > 0.f ? 1.f / L : L == 0.f ? 0.f : L) : 1.f;          // NaN stays
        const bool put = mine < at.rows && (!all || query_of(a, at, mine) < at.nq);
        const unsigned puts = __ballot_sync(0xffffffffu, put);
        if (lane < 16 && put) {
            if constexpr (kTeamed) team_ml[mine] = make_float2(M, L);
            else if (all) LSE[first + mine] = (M + log2f(L)) * kLn2;
            else *reinterpret_cast<float2*>(parts.ml + (first + mine) * 2) = make_float2(M, L);
        }
        // Four rows at once: what bounds this warp is the latency of its reads.
        constexpr int kBatch = 4 / kRowsAtOnce;
        for (int r0 = 0; r0 < at.rows; r0 += 4) {
            float4 o[kBatch][kKeyWarps];
#pragma unroll
            for (int y0 = 0; y0 < kBatch; ++y0) {
                const int r = r0 + y0 * kRowsAtOnce + sub;
#pragma unroll
                for (int k = 0; k < kKeyWarps; ++k)
                    o[y0][k] = *reinterpret_cast<const float4*>(out_row<C>(smem, s, k, r) +
                                                               (((col >> 1) ^ (r & 7)) << 5) + (col & 1) * 16);
            }
#pragma unroll
            for (int y0 = 0; y0 < kBatch; ++y0) {
                const int r = r0 + y0 * kRowsAtOnce + sub;
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < kKeyWarps; ++k) {
                    const float fk = __shfl_sync(0xffffffffu, f[k], r);
                    y.x = fmaf(o[y0][k].x, fk, y.x);
                    y.y = fmaf(o[y0][k].y, fk, y.y);
                    y.z = fmaf(o[y0][k].z, fk, y.z);
                    y.w = fmaf(o[y0][k].w, fk, y.w);
                }
                const float i = __shfl_sync(0xffffffffu, inv, r);
                const size_t to = (first + r) * a.dv + 4 * col;
                if (!(puts >> r & 1)) {
                } else if (kTeamed) {
                    *reinterpret_cast<float4*>(smem + C::kOffTeam + (r * DV + 4 * col) * 4) = y;
                } else if (4 * col < a.dv) {
                    if (all)
                        *reinterpret_cast<uint2*>(O + to) =
                            make_uint2(pack_bf16x2(y.x * i, y.y * i), pack_bf16x2(y.z * i, y.w * i));
                    else
                        *reinterpret_cast<float4*>(parts.o + to) = y;
                }
            }
        }
        fence_proxy_async_smem();                       // before the TMA writes there again
        warp_arrive(&ring.empty[s]);
    }
    };

    if (!going) {
    } else if (warp < kKeys) {
        consume();
    } else if (C::kJoiner && warp == kKeys + C::kProducers) {
        if constexpr (C::kJoiner) join();
    } else {
        auto begin = [&](const Stage& p) { return C::kQPitch > 0 || prefetch_rows(Q, p.row, p.rows, a.d); };
        if (C::kProducers == 1) produce<C, Loads::kBoth>(&tmK, &tmV, a, Q, w, ring, smem, budget_ns, begin);
        else if (warp == kKeys) produce<C, Loads::kKeys>(&tmK, &tmV, a, Q, w, ring, smem, budget_ns, begin);
        else produce<C, Loads::kValues>(&tmK, &tmV, a, Q, w, ring, smem, budget_ns, begin);
    }
    if constexpr (kTeamed) {
        // The team joined: every CTA takes an eighth of the columns of all rows
        // from all of them. No CTA leaves before its memory has been read, on
        // whatever way it got here.
        __syncwarp();
        cluster_sync();
        const int rank = int(cluster_rank()), kCols = DV / kTeam / 2;                 // pairs of columns
        const int r = threadIdx.x / kCols, c = (rank * kCols + threadIdx.x % kCols) * 2;
        const int rows = a.rows - (w.p.item % a.row_tiles) * 16;
        if (w.p.nq > 0 && r < min(16, rows)) {
            const int first = (w.p.item % a.row_tiles) * 16;
            const size_t row = row_base(a, w.p.b, w.p.item / a.row_tiles) + first + r;
            const uint32_t ml = smem_addr(&team_ml[r]), o = smem_addr(smem + C::kOffTeam) + (r * DV + c) * 4;
            float2 x[kTeam], y[kTeam];
            int gone = 0;                                 // a member gave up: nothing is written
#pragma unroll
            for (int k = 0; k < kTeam; ++k) {
                x[k] = ld_member(of_member(ml, k));
                y[k] = ld_member(of_member(o, k));
                gone |= ld_member_int(of_member(smem_addr(&ring.abort), k));
            }
            float M = -INFINITY, L = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll
            for (int k = 0; k < kTeam; ++k) M = fmaxf(M, x[k].x);
            const float Z = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int k = 0; k < kTeam; ++k) {
                if (x[k].y < 0.f) continue;               // no tile there: its output is not written
                const float f = ex2(x[k].x - Z);
                L = fmaf(x[k].y, f, L);
                y0 = fmaf(y[k].x, f, y0);
                y1 = fmaf(y[k].y, f, y1);
            }
            const float inv = L > 0.f ? 1.f / L : L == 0.f ? 0.f : L;                // NaN stays
            if (gone == 0 && (first + r) % a.n < w.p.nq) {
                if (c < a.dv) *reinterpret_cast<uint32_t*>(O + row * a.dv + c) = pack_bf16x2(y0 * inv, y1 * inv);
                if (c == 0) LSE[row] = (M + log2f(L)) * kLn2;
            }
        }
        __syncwarp();
        cluster_sync();
    }
}

}  // namespace paged
}  // namespace attn
