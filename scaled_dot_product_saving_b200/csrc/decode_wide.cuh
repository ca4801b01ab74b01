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
// go in turn to two streams, each with its running maximum and sum (a row a
// thread) and its output in tensor memory, so that the softmax of one tile runs
// beside that of the other; the two are joined when the piece ends. One warp
// issues the first products, into four buffers in turn, so that a stream finds
// its next scores ready when it has left its weights; another issues the second
// ones. (What bounded the kernel with one issuing warp was that warp: two waits,
// twelve MMAs and a message to the stream, 1,900 cycles a tile.)
//
// One B200, 8 sequences of 32768 tokens, 8 key heads, d = 128: 64 rows 186 to
// 220 us, 128 rows 205 to 250 (5.8 and 5.2 TB/s at best; runs differ). 8 of 16384 to
// 32768 tokens, 16 key heads, d = 64, 48 rows: 200 to 246 us (3.9 TB/s at best): a tile
// has half the bytes, and the softmax of one CTA an SM does not keep up.
#pragma once

#include "decode_ring.cuh"

namespace attn {
namespace paged {

constexpr int kWideRows = 128;

template <int DK, int DV>
struct DecodeWideCfg {
    static constexpr int kCtasPerSm = 1, kTileRows = kWideRows;
    static constexpr int kPanelCols = 64, kKPanels = DK / 64, kVPanels = DV / 64, kQPitch = 0;
    static constexpr int kKBytes = kKPanels * kPanelBytes;
    static constexpr int kStageBytes = kKBytes + kVPanels * kPanelBytes;
    static constexpr int kQPanelBytes = kWideRows * 128, kQBytes = kKPanels * kQPanelBytes;
    // Two buffers for the query rows, the rest of 224 KB for the ring (which
    // leaves 3 KB for what is declared in the kernel).
    static constexpr int kFit = (224 * 1024 - 2 * kQBytes) / kStageBytes, kStages = kFit < 7 ? kFit : 7;
    static constexpr int kOffQ = kStages * kStageBytes, kSmemBytes = kOffQ + 2 * kQBytes;
    static constexpr int kThreads = 12 * 32;               // two softmax warpgroups, two MMA issuers, two producers
    static constexpr uint32_t kColS = 0, kColO = 4 * kTileKeys;      // S at 64 (tile % 4), O_x at 256 + DV x
};

// Tiles are numbered through all pieces of the CTA: tile g lies in stage
// g % kStages and has its scores in buffer g % 4. A barrier of a buffer moves on
// once per four tiles, after everyone has seen it: tile g + 4 follows the product
// of tile g, which follows its weights, which follow its scores.
struct WideBars {
    uint64_t q_full[2], q_free[2];       // by parity of the piece
    uint64_t told[4];                    // descriptions, of pieces in turn
    uint64_t s_full[4], p_full[4], pv_done[4];   // by buffer: scores there; weights there; product complete
    uint64_t o_done[2];                  // the piece's last product into O_x complete
    uint64_t met, o_free;                // both warpgroups' statistics written; O read out
    uint64_t drain[2];
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
    __shared__ Stage piece[4];                             // descriptions, of pieces in turn; tiles = 0: the end
    __shared__ float2 stat[2][kWideRows];                  // by stream and row: maximum, sum
    __shared__ int odd[4];                                 // by piece: values that are not finite were set aside
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    Walker w;
    if (warp == 8 || warp == 11) w.start(a);
    if (threadIdx.x == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(&bars.q_full[x], 1);
            mbar_init(&bars.q_free[x], 1);
            mbar_init(&bars.o_done[x], 1);
            mbar_init(&bars.drain[x], 1);
        }
        for (int x = 0; x < 4; ++x) {
            mbar_init(&bars.told[x], 1);
            mbar_init(&bars.s_full[x], 1);
            mbar_init(&bars.p_full[x], 4);
            mbar_init(&bars.pv_done[x], 1);
            odd[x] = 0;
        }
        mbar_init(&bars.met, 8);
        mbar_init(&bars.o_free, 8);
    }
    if (!set_up<false>(parts, ring, smem, 1, 2)) return;      // fences the barriers' initialisation
    if (warp == 9) {
        tmem_alloc(&bars.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem;

    if (warp == 8) {
        // ------------------------------------- producer of Q and K, which leads
        if (lane == 0) prefetch_tensor_map(&tmQ);
        int pieces = 0;
        // Piece p's description takes the place of piece p - 4's. Its query rows
        // wait for the last product of piece p - 2, whose first one followed the
        // output of piece p - 3: everyone is past that piece.
        auto tell = [&](const Stage& d) {
            if (lane == 0) {
                piece[pieces & 3] = d;
                mbar_arrive(&bars.told[pieces & 3]);
            }
            __syncwarp();
        };
        auto q_free = [&] {
            return pieces < 2 || ring_wait(ring, &bars.q_free[pieces & 1], ((pieces >> 1) - 1) & 1, budget_ns);
        };
        produce<C, Loads::kKeys>(&tmK, &tmV, a, nullptr, w, ring, smem, budget_ns, [&](const Stage& d) {
            if (!q_free()) return false;
            if (lane == 0) {
                const int x = pieces & 1;
                mbar_arrive_expect_tx(&bars.q_full[x], C::kQBytes);
                for (int y = 0; y < C::kKPanels; ++y)
                    tma_load_3d(smem + C::kOffQ + x * C::kQBytes + y * C::kQPanelBytes, &tmQ, &bars.q_full[x], 64 * y,
                                d.row, 0);
            }
            tell(d);
            ++pieces;
            return true;
        });
        if (q_free()) {
            Stage end{};
            end.tiles = 0;
            tell(end);
        }
        for (int p = max(0, pieces - 2); p < pieces; ++p)
            (void)mbar_wait_timed(&bars.q_full[p & 1], (p >> 1) & 1, budget_ns);
    } else if (warp == 11) {
        produce<C, Loads::kValues>(&tmK, &tmV, a, nullptr, w, ring, smem, budget_ns, [](const Stage&) { return true; });
    } else if (warp == 9) {
        // ------------------------------------------------ issuer of S = Q K^T
        const uint32_t leader = elect_leader();
        constexpr uint32_t idS = idesc_bf16_f32(kWideRows, kTileKeys, 0, 0);
        int g = 0, s = 0;
        uint32_t parity = 0;
        bool ok = true;
        for (int p = 0; ok; ++p) {
            ok = ring_wait(ring, &bars.told[p & 3], (p >> 2) & 1, budget_ns);
            const int tiles = ok ? piece[p & 3].tiles : 0;
            if (tiles == 0) break;
            ok = ring_wait(ring, &bars.q_full[p & 1], (p >> 1) & 1, budget_ns);
            const uint32_t sQ = smem_addr(smem + C::kOffQ + (p & 1) * C::kQBytes);
            for (int i = 0; ok && i < tiles; ++i, ++g) {
                const int b = g & 3;
                ok = ring_wait(ring, &ring.full[s], parity, budget_ns) &&
                     (g < 4 || ring_wait(ring, &bars.pv_done[b], ((g >> 2) - 1) & 1, budget_ns));
                if (!ok) break;
                tc_fence_after();
                const uint32_t sK = smem_addr(smem + s * C::kStageBytes);
#pragma unroll
                for (int kk = 0; kk < DK / 16; ++kk)
                    mma_ss_w(tmem + C::kColS + kTileKeys * b,
                             sdesc_at(sQ, (kk >> 2) * C::kQPanelBytes + (kk & 3) * 32, 16, 1024),
                             sdesc_at(sK, (kk >> 2) * kPanelBytes + (kk & 3) * 32, 16, 1024), idS, kk > 0, leader);
                mma_commit_w(&bars.s_full[b], leader);
                if (++s == kStages) {
                    s = 0;
                    parity ^= 1;
                }
            }
        }
        // All MMAs issued here complete before tensor memory is given back.
        mma_commit_w(&bars.drain[0], leader);
        (void)mbar_wait_timed(&bars.drain[0], 0, budget_ns);
    } else if (warp == 10) {
        // ------------------------------------------------ issuer of O += P V
        const uint32_t leader = elect_leader();
        constexpr uint32_t idO = idesc_bf16_f32(kWideRows, DV, 0, 1);
        int g = 0, s = 0;
        uint32_t parity = 0;
        bool ok = true;
        for (int p = 0; ok; ++p) {
            ok = ring_wait(ring, &bars.told[p & 3], (p >> 2) & 1, budget_ns);
            const int tiles = ok ? piece[p & 3].tiles : 0;
            if (tiles == 0) break;
            // The first product overwrites O: the piece before is read.
            if (p > 0) ok = ring_wait(ring, &bars.o_free, (p - 1) & 1, budget_ns);
            for (int i = 0; ok && i < tiles; ++i, ++g) {
                const int b = g & 3, x = i & 1;
                ok = ring_wait(ring, &bars.p_full[b], (g >> 2) & 1, budget_ns) &&
                     ring_wait(ring, &ring.full[s], parity, budget_ns);    // done: sees the copies
                if (!ok) break;
                tc_fence_after();
                const uint32_t sV = smem_addr(smem + s * C::kStageBytes + C::kKBytes);
#pragma unroll
                for (int kk = 0; kk < kTileKeys / 16; ++kk)
                    mma_ts_w(tmem + C::kColO + DV * x, tmem + C::kColS + kTileKeys * b + kk * 8,
                             sdesc_at(sV, kk * 2048, kPanelBytes, 1024), idO, i >= 2 || kk > 0, leader);
                mma_commit_w(&bars.pv_done[b], leader);
                mma_commit_w(&ring.empty[s], leader);
                if (i + 2 >= tiles) mma_commit_w(&bars.o_done[x], leader);
                if (i + 1 == tiles) mma_commit_w(&bars.q_free[p & 1], leader);
                if (++s == kStages) {
                    s = 0;
                    parity ^= 1;
                }
            }
        }
        mma_commit_w(&bars.drain[1], leader);
        (void)mbar_wait_timed(&bars.drain[1], 0, budget_ns);
    } else {
        // ------------------------------------------------ softmax, a row a thread
        const int x = warp >> 2, r = threadIdx.x & 127;
        const uint32_t tl = tmem + (uint32_t((warp & 3) * 32) << 16);
        const uint32_t tO = tl + C::kColO;
        const float scale_log2 = a.scale * 1.4426950408889634f;
        int done[2] = {0, 0};                              // pieces with tiles, per stream
        int g0 = 0;                                        // tiles of the pieces before
        bool ok = true;
        for (int p = 0; ok; ++p) {
            ok = ring_wait(ring, &bars.told[p & 3], (p >> 2) & 1, budget_ns);
            const Stage& st = piece[p & 3];
            const int tiles = ok ? st.tiles : 0;
            if (tiles == 0) break;
            const At at{st.row, st.rows, st.i0, st.nq, st.flags, st.b, st.item, st.last};
            const int len = st.len, first_key = st.t0 * kTileKeys;
            const int see = visible(a, len, at.nq, query_of(a, at, r));
            const int see_all = a.causal ? len - (at.nq - 1) : len;
            float m_run = -INFINITY, l_run = 0.f;
            for (int i = x; ok && i < tiles; i += 2) {
                const int g = g0 + i, b = g & 3, s = g % kStages, k0 = first_key + i * kTileKeys;
                // The second wait is over as soon as it begins: it is for what was
                // written beside the tile, and for V where it is mended below.
                ok = ring_wait(ring, &bars.s_full[b], (g >> 2) & 1, budget_ns) &&
                     ring_wait(ring, &ring.full[s], (g / kStages) & 1, budget_ns);
                if (!ok) break;
                tc_fence_after();
                const unsigned long long present = ring.stage[s].present;
                const bool whole = present == ~0ull && k0 + kTileKeys <= see_all;
                if (!whole) {
                    // V as the products may read it: rows that no token owns are
                    // zeros; so are values that are not finite in rows that only
                    // some queries see, which are added at the end.
                    uint8_t* v = smem + s * C::kStageBytes + C::kKBytes;
                    for (int u = r; u < kTileKeys * (DV / 8); u += 128) {
                        const int j = u / (DV / 8), c = u % (DV / 8);
                        uint4* y4 = reinterpret_cast<uint4*>(v + (c / 8) * kPanelBytes + j * 128 + (((c & 7) ^ (j & 7)) << 4));
                        if (!(present >> j & 1)) {
                            *y4 = make_uint4(0u, 0u, 0u, 0u);
                        } else if (k0 + j >= see_all) {
                            uint32_t y[4];
                            *reinterpret_cast<uint4*>(y) = *y4;
                            bool bad = false;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if ((y[e] & 0x7f80u) == 0x7f80u) y[e] &= 0xffff0000u, bad = true;
                                if ((y[e] & 0x7f800000u) == 0x7f800000u) y[e] &= 0xffffu, bad = true;
                            }
                            if (bad) {
                                *y4 = *reinterpret_cast<const uint4*>(y);
                                odd[p & 3] = 1;
                            }
                        }
                    }
                    fence_proxy_async_smem();
                }
                if ((warp & 3) * 32 < at.rows) {           // else no row of this warp is one
                    const uint32_t tS = tl + C::kColS + kTileKeys * b;
                    uint32_t s0[32], s1[32];
                    tmem_ld32(tS, s0);
                    tmem_ld32(tS + 32, s1);
                    tmem_ld_wait(s0);
                    tmem_ld_wait(s1);
                    uint32_t lo = ~0u, hi = ~0u;             // keys that exist and that this row sees
                    if (!whole) {
                        const int left = see - k0;
                        const unsigned long long seen =
                            present & (left >= kTileKeys ? ~0ull : left > 0 ? (1ull << left) - 1ull : 0ull);
                        lo = uint32_t(seen);
                        hi = uint32_t(seen >> 32);
                        // Scaled scores of the others are -inf below, whatever they hold.
                        const uint32_t worst = __float_as_uint(scale_log2 < 0.f ? INFINITY : -INFINITY);
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            if (!(lo >> e & 1)) s0[e] = worst;
                            if (!(hi >> e & 1)) s1[e] = worst;
                        }
                    }
                    // Weights against the reference value as it is, in bf16 for the
                    // second product (half a step, 2^-8 of each); their sum is of the
                    // unrounded ones, and the extreme raw score is found on the way.
                    const f32x2 sl2 = make_f32x2(scale_log2, scale_log2);
                    const bool falling = scale_log2 < 0.f;
                    uint32_t pk[32];
                    float sum = 0.f, far = falling ? INFINITY : -INFINITY;
                    auto weigh = [&](const uint32_t(&sc)[32], uint32_t seen, uint32_t* to, f32x2 nz2, f32x2& acc, auto masked) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float a0 = __uint_as_float(sc[2 * e]), a1 = __uint_as_float(sc[2 * e + 1]);
                            const float2 y = split_f32x2(fma_x2(make_f32x2(a0, a1), sl2, nz2));
                            float q0 = ex2(y.x), q1 = ex2(y.y);
                            if constexpr (decltype(masked)::value) {
                                if (!(seen >> (2 * e) & 1)) q0 = 0.f;
                                if (!(seen >> (2 * e + 1) & 1)) q1 = 0.f;
                            }
                            far = falling ? fmin3(far, a0, a1) : fmax3(far, a0, a1);
                            acc = add_x2(acc, make_f32x2(q0, q1));
                            to[e] = pack_bf16x2(q0, q1);
                        }
                    };
                    auto weigh_all = [&](float z) {
                        const f32x2 nz2 = make_f32x2(-z, -z);
                        f32x2 u = make_f32x2(0.f, 0.f), v = u;
                        if (whole) {
                            weigh(s0, lo, pk, nz2, u, std::false_type{});
                            weigh(s1, hi, pk + 16, nz2, v, std::false_type{});
                        } else {
                            weigh(s0, lo, pk, nz2, u, std::true_type{});
                            weigh(s1, hi, pk + 16, nz2, v, std::true_type{});
                        }
                        const float2 w = split_f32x2(add_x2(u, v));
                        sum = w.x + w.y;
                    };
                    weigh_all(m_run == -INFINITY ? 0.f : m_run);
                    const float top = (lo | hi) != 0 ? far * scale_log2 : -INFINITY;
                    // The reference value moves, and O is rescaled, only when the
                    // maximum has grown by more than 8 (base 2): on a piece's first tile
                    // and rarely after it. The weights are then taken again.
                    const bool want = top > m_run + 8.f;
                    if (__any_sync(0xffffffffu, want)) {
                        float alpha = 1.f;
                        if (want) {
                            const float next = fminf(top, kTopScore);
                            alpha = ex2(m_run - next);
                            m_run = next;
                            l_run *= alpha;
                        }
                        if (i >= 2) {
                            // The stream's last product must have left O.
                            ok = ring_wait(ring, &bars.pv_done[(g - 2) & 3], ((g - 2) >> 2) & 1, budget_ns);
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < DV; c += 16) {
                                uint32_t o[16];
                                tmem_ld16(tO + DV * x + c, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                tmem_st16(tO + DV * x + c, o);
                            }
                        }
                        weigh_all(m_run == -INFINITY ? 0.f : m_run);
                    }
                    tmem_st32(tS, pk);
                    l_run += sum;
                    tmem_st_wait();
                }
                tc_fence_before();
                warp_arrive(&bars.p_full[b]);
            }
            g0 += tiles;
            if (!ok) break;

            // ------------------------------------- the two streams joined
            // The statistics of the piece before have been read.
            if (p > 0 && !ring_wait(ring, &bars.o_free, (p - 1) & 1, budget_ns)) break;
            stat[x][r] = make_float2(m_run, l_run);
            // Cleared for the next piece but one: read for the last time two pieces
            // ago, and not written before both have met for this one.
            if (threadIdx.x == 0) odd[(p + 2) & 3] = 0;
            warp_arrive(&bars.met);
            if (!ring_wait(ring, &bars.met, p & 1, budget_ns)) break;
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
            const bool extra = odd[p & 3] != 0 && put;
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
                            const int pg = a.table[size_t(at.b) * a.g.M + (j >> a.g.page_log2)];
                            if (!page_ok(pg, a.g.P)) continue;
                            const size_t row = (size_t(pg) * a.g.Hkv + hk) * page + (j & (page - 1));
                            float dot = 0.f;
                            for (int c = 0; c < a.d; ++c)
                                dot = fmaf(__bfloat162float(Q[(size_t(at.row) + r) * a.d + c]),
                                           __bfloat162float(Kp[row * a.d + c]), dot);
                            const float wgt = ex2(dot * scale_log2 - Z);
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                const float v = c0 + e < a.dv ? __bfloat162float(Vp[row * a.dv + c0 + e]) : 0.f;
                                if (!isfinite(v)) y[e] += wgt * v;
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
