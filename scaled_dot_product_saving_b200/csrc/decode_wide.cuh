// decode_wide.cuh -- attention over paged bf16 keys and values for many query
// rows per key head (drafts, many heads on one key head): up to 128 rows an
// item, on tcgen05.
//
// The mathematics is decode.cuh's; the stream of tiles is decode_ring.cuh's.
// mma.sync takes 16 cycles an instruction and SM sub-partition here, so that
// decode_tc.cuh's 32 rows already cost what a tile takes to arrive; one tcgen05
// instruction takes 128 rows at that price, and memory bounds the call again.
//
// The item's rows are the 128 lanes of tensor memory. The key tiles of a piece
// go in turn to two streams, each with its scores, its running maximum and sum
// (a row a thread) and its output in tensor memory, so that the softmax of one
// tile runs under the products of the other; the two are joined when the piece
// ends. One warp issues: S of tile i, then O += P V of tile i - 1.
#pragma once

#include "decode_ring.cuh"

namespace attn {
namespace paged {

constexpr int kWideRows = 128;

template <int DK, int DV>
struct DecodeWideCfg {
    static constexpr int kPanelCols = 64, kKPanels = DK / 64, kVPanels = DV / 64;
    static constexpr int kKBytes = kKPanels * kPanelBytes;
    static constexpr int kStageBytes = kKBytes + kVPanels * kPanelBytes;
    static constexpr int kQPanelBytes = kWideRows * 128, kQBytes = kKPanels * kQPanelBytes;
    // Two buffers for the query rows, the rest of 224 KB for the ring (which
    // leaves 3 KB for what is declared in the kernel).
    static constexpr int kFit = (224 * 1024 - 2 * kQBytes) / kStageBytes, kStages = kFit < 8 ? kFit : 8;
    static constexpr int kOffQ = kStages * kStageBytes, kSmemBytes = kOffQ + 2 * kQBytes;
    static constexpr int kThreads = 10 * 32;               // two softmax warpgroups, producer, MMA issuer
    static constexpr uint32_t kColS = 0, kColO = 2 * kTileKeys;      // S_x at 64 x, O_x at 128 + DV x
};

// What the issuing warp tells a stream with each tile.
enum : int { kMsgFirst = 1, kMsgNone = 2, kMsgFinal = 4, kMsgStop = 8 };
struct Message {
    unsigned long long present;
    int flags;       // kMsgFirst: a piece begins; kMsgNone: it has no tile for this stream;
                     // kMsgFinal: the stream's last of the piece; kMsgStop: the end
    int stage, k0;   // where the tile lies, its first key
    uint32_t parity; // of the stage's arrival
    int par;         // parity of the piece: which description
};

struct WideBars {
    uint64_t q_full[2], q_free[2];
    uint64_t s_full[2];              // the tile's scores and its message: the MMAs, and the issuing warp
    uint64_t msg_free[2];            // the stream's warps have read the message
    uint64_t p_full[2], o_done[2];   // weights written; the piece's last product into O_x
    uint64_t met, o_free, drain;     // both warpgroups' statistics; O read out
    uint32_t tmem;
};

template <int DK, int DV>
__global__ void __launch_bounds__(DecodeWideCfg<DK, DV>::kThreads, 1)
decode_wide(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, DecodeArgs a,
            const __nv_bfloat16* __restrict__ Q, __nv_bfloat16* __restrict__ O, float* __restrict__ LSE, Parts parts,
            unsigned long long budget_ns, const __grid_constant__ CUtensorMap tmQ,
            const __nv_bfloat16* __restrict__ Kp, const __nv_bfloat16* __restrict__ Vp) {
    using C = DecodeWideCfg<DK, DV>;
    constexpr int kStages = C::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ Ring<kStages, 1> ring;
    __shared__ WideBars bars;
    __shared__ Message msg[2];
    __shared__ Stage piece[2];                             // descriptions, by parity of the piece
    __shared__ float2 stat[2][kWideRows];                  // by stream and row: maximum, sum
    __shared__ int odd[4];                                 // by piece: values that are not finite were set aside
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    Walker w;
    if (warp == 8) w.start(a);
    if (threadIdx.x == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(&bars.q_full[x], 1);
            mbar_init(&bars.q_free[x], 1);
            mbar_init(&bars.s_full[x], 2);
            mbar_init(&bars.msg_free[x], 4);
            mbar_init(&bars.p_full[x], 4);
            mbar_init(&bars.o_done[x], 1);
        }
        for (int x = 0; x < 4; ++x) odd[x] = 0;
        mbar_init(&bars.met, 8);
        mbar_init(&bars.o_free, 8);
        mbar_init(&bars.drain, 1);
    }
    if (!set_up<false>(parts, ring, smem, 1)) return;      // fences the barriers' initialisation
    if (warp == 9) {
        tmem_alloc(&bars.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem;

    if (warp == 8) {
        // -------------------------------------------------------- producer
        if (lane == 0) prefetch_tensor_map(&tmQ);
        int pieces = 0;
        produce<C>(&tmK, &tmV, a, w, ring, smem, budget_ns, [&](int row, int) {
            const int x = pieces & 1;
            if (pieces >= 2 && !ring_wait(ring, &bars.q_free[x], ((pieces >> 1) - 1) & 1, budget_ns)) return false;
            if (lane == 0) {
                mbar_arrive_expect_tx(&bars.q_full[x], C::kQBytes);
                for (int y = 0; y < C::kKPanels; ++y)
                    tma_load_3d(smem + C::kOffQ + x * C::kQBytes + y * C::kQPanelBytes, &tmQ, &bars.q_full[x], 64 * y,
                                row, 0);
            }
            __syncwarp();
            ++pieces;
            return true;
        });
        for (int p = max(0, pieces - 2); p < pieces; ++p)
            (void)mbar_wait_timed(&bars.q_full[p & 1], (p >> 1) & 1, budget_ns);
    } else if (warp == 9) {
        // ------------------------------------------------------ MMA issuer
        const uint32_t leader = elect_leader();
        constexpr uint32_t idS = idesc_bf16_f32(kWideRows, kTileKeys, 0, 0);
        constexpr uint32_t idO = idesc_bf16_f32(kWideRows, DV, 0, 1);
        int pieces = 0, tile = 0, tiles = 0, k0 = 0;       // of the piece: tile index, count, first key
        int sent[2] = {0, 0}, used[2] = {0, 0};            // messages, weights taken
        bool pend = false;
        int pend_x = 0, pend_s = 0, pend_tile = 0, pend_tiles = 0, pend_piece = 0;
        auto tell = [&](int x, const Message& m, bool with_mma) -> bool {
            if (sent[x] > 0 && !ring_wait(ring, &bars.msg_free[x], (sent[x] - 1) & 1, budget_ns)) return false;
            ++sent[x];
            if (lane == 0) {
                msg[x] = m;
                mbar_arrive(&bars.s_full[x]);
                if (!with_mma) mbar_arrive(&bars.s_full[x]);
            }
            __syncwarp();
            return true;
        };
        auto flush = [&]() -> bool {
            if (!pend) return true;
            pend = false;
            const int x = pend_x;
            if (!ring_wait(ring, &bars.p_full[x], used[x] & 1, budget_ns)) return false;
            ++used[x];
            // The first product of a piece overwrites O: the piece before is read.
            if (pend_tile < 2 && pend_piece > 1 &&
                !ring_wait(ring, &bars.o_free, (pend_piece - 2) & 1, budget_ns))
                return false;
            tc_fence_after();
            const uint32_t sV = smem_addr(smem + pend_s * C::kStageBytes + C::kKBytes);
#pragma unroll
            for (int kk = 0; kk < kTileKeys / 16; ++kk)
                mma_ts_w(tmem + C::kColO + DV * x, tmem + C::kColS + kTileKeys * x + kk * 8,
                         sdesc_at(sV, kk * 2048, kPanelBytes, 1024), idO, pend_tile >= 2 || kk > 0, leader);
            mma_commit_w(&ring.empty[pend_s], leader);
            if (pend_tile + 2 >= pend_tiles) mma_commit_w(&bars.o_done[x], leader);
            return true;
        };
        uint32_t parity = 0;
        for (int s = 0;; s = s + 1 == kStages ? 0 : s + 1, parity ^= s == 0) {
            if (!ring_wait(ring, &ring.full[s], parity, budget_ns)) break;
            const int flags = ring.stage[s].flags;
            if (flags & kStop) {
                if (!flush()) break;
                const Message stop{0ull, kMsgStop, 0, 0, 0u, 0};
                if (tell(0, stop, false)) (void)tell(1, stop, false);
                break;
            }
            if (flags & kFirst) {
                ++pieces;
                tile = 0;
                tiles = ring.stage[s].tiles;
                k0 = ring.stage[s].t0 * kTileKeys;
                // Two pieces back the description has been read: a product of the
                // last one waited for that piece's output.
                if (pieces > 2 && !flush()) break;
                if (lane == 0) piece[pieces & 1] = ring.stage[s];
                if (!ring_wait(ring, &bars.q_full[(pieces - 1) & 1], ((pieces - 1) >> 1) & 1, budget_ns)) break;
            }
            const int x = tile & 1;
            if (pend && pend_x == x && !flush()) break;    // its weights lie where these scores go
            Message m{ring.stage[s].present, tile < 2 ? kMsgFirst : 0, s, k0, parity, pieces & 1};
            if (tile + 2 >= tiles) m.flags |= kMsgFinal;
            tc_fence_after();
            const uint32_t sQ = smem_addr(smem + C::kOffQ + ((pieces - 1) & 1) * C::kQBytes);
            const uint32_t sK = smem_addr(smem + s * C::kStageBytes);
#pragma unroll
            for (int kk = 0; kk < DK / 16; ++kk)
                mma_ss_w(tmem + C::kColS + kTileKeys * x,
                         sdesc_at(sQ, (kk >> 2) * C::kQPanelBytes + (kk & 3) * 32, 16, 1024),
                         sdesc_at(sK, (kk >> 2) * kPanelBytes + (kk & 3) * 32, 16, 1024), idS, kk > 0, leader);
            mma_commit_w(&bars.s_full[x], leader);
            if (!tell(x, m, true)) break;
            if (tile == tiles - 1) mma_commit_w(&bars.q_free[(pieces - 1) & 1], leader);
            if (tiles == 1) {
                m.flags = kMsgFirst | kMsgNone | kMsgFinal;
                if (!tell(1, m, false)) break;
            }
            if (!flush()) break;
            pend = true;
            pend_x = x;
            pend_s = s;
            pend_tile = tile;
            pend_tiles = tiles;
            pend_piece = pieces;
            ++tile;
            k0 += kTileKeys;
        }
        // All MMAs issued here complete before tensor memory is given back.
        mma_commit_w(&bars.drain, leader);
        (void)mbar_wait_timed(&bars.drain, 0, budget_ns);
    } else {
        // ------------------------------------------------ softmax, a row a thread
        const int x = warp >> 2, r = threadIdx.x & 127;
        const uint32_t tl = tmem + (uint32_t((warp & 3) * 32) << 16);
        const uint32_t tS = tl + C::kColS + kTileKeys * x, tO = tl + C::kColO;
        const float scale_log2 = a.scale * 1.4426950408889634f;
        At at{};
        int see = 0, see_all = 0, len = 0, first_key = 0, tiles = 0, pieces = 0, got = 0;
        int done[2] = {0, 0};                              // pieces with tiles, per stream
        float m_run = -INFINITY, l_run = 0.f;
        bool fresh = true;                                 // no product of this piece in O_x yet
        for (;;) {
            if (!ring_wait(ring, &bars.s_full[x], got & 1, budget_ns)) break;
            ++got;
            tc_fence_after();
            const Message m = msg[x];
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.msg_free[x]);
            if (m.flags & kMsgStop) break;
            if (m.flags & kMsgFirst) {
                const Stage& st = piece[m.par];
                at = At{st.row, st.rows, st.i0, st.nq, st.flags, st.b, st.item, st.last};
                len = st.len;
                first_key = st.t0 * kTileKeys;
                tiles = st.tiles;
                see = visible(a, len, at.nq, query_of(a, at, r));
                see_all = a.causal ? len - (at.nq - 1) : len;
                m_run = -INFINITY;
                l_run = 0.f;
                fresh = true;
                ++pieces;
            }
            if (!(m.flags & kMsgNone)) {
                const bool whole = m.present == ~0ull && m.k0 + kTileKeys <= see_all;
                if (!whole) {
                    // V as the products may read it: rows that no token owns are
                    // zeros; so are values that are not finite in rows that only
                    // some queries see, which are added at the end.
                    if (!ring_wait(ring, &ring.full[m.stage], m.parity, budget_ns)) break;   // done: sees the copies
                    uint8_t* v = smem + m.stage * C::kStageBytes + C::kKBytes;
                    for (int u = r; u < kTileKeys * (DV / 8); u += 128) {
                        const int j = u / (DV / 8), c = u % (DV / 8);
                        uint4* p = reinterpret_cast<uint4*>(v + (c / 8) * kPanelBytes + j * 128 + (((c & 7) ^ (j & 7)) << 4));
                        if (!(m.present >> j & 1)) {
                            *p = make_uint4(0u, 0u, 0u, 0u);
                        } else if (m.k0 + j >= see_all) {
                            uint32_t y[4];
                            *reinterpret_cast<uint4*>(y) = *p;
                            bool bad = false;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if ((y[e] & 0x7f80u) == 0x7f80u) y[e] &= 0xffff0000u, bad = true;
                                if ((y[e] & 0x7f800000u) == 0x7f800000u) y[e] &= 0xffffu, bad = true;
                            }
                            if (bad) {
                                *p = *reinterpret_cast<const uint4*>(y);
                                odd[pieces & 3] = 1;
                            }
                        }
                    }
                    fence_proxy_async_smem();
                }
                if ((warp & 3) * 32 < at.rows) {           // else no row of this warp is one
                    uint32_t s0[32], s1[32];
                    tmem_ld32(tS, s0);
                    tmem_ld32(tS + 32, s1);
                    tmem_ld_wait(s0);
                    tmem_ld_wait(s1);
                    float top = -INFINITY;
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        float y0 = __uint_as_float(s0[e]) * scale_log2, y1 = __uint_as_float(s1[e]) * scale_log2;
                        if (!whole) {
                            if (!(m.present >> e & 1) || m.k0 + e >= see) y0 = -INFINITY;
                            if (!(m.present >> (e + 32) & 1) || m.k0 + e + 32 >= see) y1 = -INFINITY;
                        }
                        s0[e] = __float_as_uint(y0);
                        s1[e] = __float_as_uint(y1);
                        top = fmax3(top, y0, y1);
                    }
                    // The reference value moves, and O is rescaled, only when the
                    // maximum has grown by more than 8 (base 2).
                    const bool want = top > m_run + 8.f;
                    const bool rescale = __any_sync(0xffffffffu, want && !fresh);
                    float alpha = 1.f;
                    if (want) {
                        alpha = ex2(m_run - top);
                        m_run = top;
                        l_run *= alpha;
                    }
                    if (rescale) {
                        // S of this tile was issued after the stream's last product.
#pragma unroll
                        for (int c = 0; c < DV / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld32(tO + DV * x + 32 * c, o);
                            tmem_ld_wait(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tmem_st32(tO + DV * x + 32 * c, o);
                        }
                    }
                    const float z = m_run == -INFINITY ? 0.f : m_run;
                    float sum0 = 0.f, sum1 = 0.f;
                    uint32_t pk[16];
                    // Weights in bf16 for the second product (half a step, 2^-8 of
                    // each), over the scores; their sum is of the unrounded ones.
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float p0 = ex2(__uint_as_float(s0[2 * e]) - z), p1 = ex2(__uint_as_float(s0[2 * e + 1]) - z);
                        sum0 += p0;
                        sum1 += p1;
                        pk[e] = pack_bf16x2(p0, p1);
                    }
                    tmem_st16(tS, pk);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float p0 = ex2(__uint_as_float(s1[2 * e]) - z), p1 = ex2(__uint_as_float(s1[2 * e + 1]) - z);
                        sum0 += p0;
                        sum1 += p1;
                        pk[e] = pack_bf16x2(p0, p1);
                    }
                    tmem_st16(tS + 16, pk);
                    l_run += sum0 + sum1;
                    tmem_st_wait();
                }
                tc_fence_before();
                warp_arrive(&bars.p_full[x]);
                fresh = false;
            }
            if (!(m.flags & kMsgFinal)) continue;

            // ------------------------------------- the two streams joined
            const int ph = (pieces - 1) & 1;
            // The statistics of the piece before have been read.
            if (pieces > 1 && !ring_wait(ring, &bars.o_free, ph ^ 1, budget_ns)) break;
            stat[x][r] = make_float2(m_run, l_run);
            // Cleared for the next piece but one: read for the last time two pieces
            // ago, and not written before both have met for this one.
            if (threadIdx.x == 0) odd[(pieces + 2) & 3] = 0;
            warp_arrive(&bars.met);
            if (!ring_wait(ring, &bars.met, ph, budget_ns)) break;
            const float2 u0 = stat[0][r], u1 = stat[1][r];
            const bool two = tiles > 1;
            if (!ring_wait(ring, &bars.o_done[0], done[0] & 1, budget_ns)) break;
            ++done[0];
            if (two) {
                if (!ring_wait(ring, &bars.o_done[1], done[1] & 1, budget_ns)) break;
                ++done[1];
            }
            tc_fence_after();
            const float M = fmaxf(u0.x, u1.x), Z = M == -INFINITY ? 0.f : M;
            const float f0 = ex2(u0.x - Z), f1 = ex2(u1.x - Z), L = fmaf(u0.y, f0, u1.y * f1);
            const bool all = (at.flags & (kStarts | kEnds)) == (kStarts | kEnds);
            const bool put = r < at.rows && (!all || query_of(a, at, r) < at.nq);
            const float inv = all ? (L > 0.f ? 1.f / L : L == 0.f ? 0.f : L) : 1.f;          // NaN stays
            const size_t slot = (2 * size_t(blockIdx.x) + (at.flags & kStarts ? 1 : 0)) * kWideRows;
            const size_t to = (all ? size_t(at.row) : slot) + r;
            const bool extra = odd[pieces & 3] != 0 && put;
            if ((warp & 3) * 32 < at.rows) {
                // Each warpgroup takes half of the columns.
#pragma unroll 1
                for (int c0 = x * (DV / 2); c0 < (x + 1) * (DV / 2); c0 += 32) {
                    uint32_t o0[32], o1[32];
                    tmem_ld32(tO + c0, o0);
                    if (two) tmem_ld32(tO + DV + c0, o1);
                    tmem_ld_wait(o0);
                    float y[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) y[e] = __uint_as_float(o0[e]) * f0;
                    if (two) {
                        tmem_ld_wait(o1);
#pragma unroll
                        for (int e = 0; e < 32; ++e) y[e] = fmaf(__uint_as_float(o1[e]), f1, y[e]);
                    }
                    if (extra) {
                        // Infinities and NaN of the newest tokens, times the weights
                        // of the rows that see them, from the cache itself.
                        const int hk = at.item / a.row_tiles, page = 1 << a.g.page_log2;
                        const int end = min(min(len, first_key + tiles * kTileKeys), see);
                        for (int j = max(see_all, first_key); j < end; ++j) {
                            const int p = a.table[size_t(at.b) * a.g.M + (j >> a.g.page_log2)];
                            if (!page_ok(p, a.g.P)) continue;
                            const size_t row = (size_t(p) * a.g.Hkv + hk) * page + (j & (page - 1));
                            float dot = 0.f;
                            for (int c = 0; c < a.d; ++c)
                                dot = fmaf(__bfloat162float(Q[(size_t(at.row) + r) * a.d + c]),
                                           __bfloat162float(Kp[row * a.d + c]), dot);
                            const float wgt = ex2(dot * scale_log2 - Z);
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                const float v = c0 + e < a.dv ? __bfloat162float(Vp[row * a.dv + c0 + e]) : 0.f;
                                if (!isfinite(v) && wgt != 0.f) y[e] += wgt * v;
                            }
                        }
                    }
                    if (!put) continue;
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        if (c0 + e >= a.dv) continue;
                        if (all) {
                            uint4 o;
                            o.x = pack_bf16x2(y[e] * inv, y[e + 1] * inv);
                            o.y = pack_bf16x2(y[e + 2] * inv, y[e + 3] * inv);
                            o.z = pack_bf16x2(y[e + 4] * inv, y[e + 5] * inv);
                            o.w = pack_bf16x2(y[e + 6] * inv, y[e + 7] * inv);
                            *reinterpret_cast<uint4*>(O + to * a.dv + c0 + e) = o;
                        } else {
                            float4* o = reinterpret_cast<float4*>(parts.o + to * a.dv + c0 + e);
                            o[0] = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
                            o[1] = make_float4(y[e + 4], y[e + 5], y[e + 6], y[e + 7]);
                        }
                    }
                }
            }
            tc_fence_before();
            if (x == 0 && put) {
                if (all) LSE[to] = (M + log2f(L)) * kLn2;
                else *reinterpret_cast<float2*>(parts.ml + to * 2) = make_float2(M, L);
            }
            if (threadIdx.x == 0) note_head(parts, at);
            warp_arrive(&bars.o_free);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace paged
}  // namespace attn
