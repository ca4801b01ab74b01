// decode_ring.cuh -- the stream of key tiles that the decode kernels consume: a
// ring of shared-memory stages of 64 keys, filled page by page with the TMA by
// one or two warps that run ahead of the others, across the borders of pieces.
//
// A stage is panels of 64 rows of 128 bytes (64 bf16 or 32 fp32 columns) in the
// TMA's 128-byte swizzle: the K panels, then the V panels. The producers alone
// know the split of the call; the leading one leaves beside each stage what the
// consumers need: which keys are there, and with the first tile of a piece the
// piece, and where a kernel asks for it the query rows.
//
// Every wait in the ring is bounded and on an mbarrier. One that runs out sets the
// abort flag, which ends every other wait, and each warp leaves its loop; the block
// and cluster barriers behind the loops are reached on every way.
#pragma once

#include "decode.cuh"

namespace attn {
namespace paged {

constexpr int kPanelBytes = kTileKeys * 128;

enum : int { kFirst = 1, kLast = 2, kStop = 4, kStarts = 8, kEnds = 16 };

struct Stage {
    unsigned long long present;      // keys of the tile that exist
    int flags;                       // kFirst, kLast: tile of its piece; kStop: no tile, the end;
                                     // kStarts, kEnds: the piece of its item
    // with kFirst
    int row, rows;                   // first query row of the item in Q, O and LSE, and how many
    int i0;                          // the first row's query
    int len, nq, t0, tiles;          // its first key tile, and how many
    int b, item, last;               // for the item's head: last, CTA of its last piece
};

template <int kStages, int kGroups>
struct Ring {
    uint64_t full[kStages], empty[kStages];
    uint64_t joint[kGroups][2];      // where the warps of a group meet when a piece ends
    Stage stage[kStages];
    int abort;
};

// Warp-wide wait; false once the call is being abandoned. The bound is counted
// with the SM's clock: reading the global timer costs some thousand cycles, which
// every wait that does not succeed at once would pay.
template <typename RingT>
__device__ __forceinline__ bool ring_wait(RingT& ring, uint64_t* bar, uint32_t parity, unsigned long long budget_ns) {
    volatile int* abort = &ring.abort;
    const uint32_t at = smem_addr(bar);
    bool ok = mbar_try_wait(at, parity);
    if (!ok) {
        const long long from = clock64();
        for (uint32_t turn = 1; !ok; ++turn) {
            ok = mbar_try_wait(at, parity);
            // Two cycles a nanosecond: no SM clock is above 2 GHz. (At a lower clock
            // the bound is longer by as much.)
            if (!ok && (turn & 15u) == 0u && (*abort || (unsigned long long)(clock64() - from) > 2 * budget_ns)) break;
        }
    }
    if (__all_sync(0xffffffffu, ok)) return true;
    if (*abort == 0) {
        record_device_error(kErrTimeout);
        *abort = 1;
    }
    return false;
}

// One lane arrives for the warp, after all of it.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// Collective over the block. False (for all threads) if an earlier kernel's
// timeout has not been read, in which case the call does nothing.
template <bool kTeamed, int kStages, int kGroups>
__device__ __forceinline__ bool set_up(const Parts& parts, Ring<kStages, kGroups>& ring, const uint8_t* smem,
                                       int consumers, int producers) {
    if (threadIdx.x == 0) {
        if (!kTeamed) parts.head[blockIdx.x].b = -1;
        const bool misaligned = (smem_addr(smem) & 1023u) != 0;
        if (misaligned) record_device_error(kErrTimeout);
        ring.abort = misaligned || *reinterpret_cast<volatile unsigned int*>(&g_device_error) != 0;
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&ring.full[s], producers);
            mbar_init(&ring.empty[s], consumers);
        }
        for (int x = 0; x < kGroups; ++x) {
            mbar_init(&ring.joint[x][0], consumers / kGroups);
            mbar_init(&ring.joint[x][1], consumers / kGroups);
        }
        fence_mbar_init();
    }
    __syncthreads();
    const bool skip = ring.abort != 0;
    __syncthreads();                                // every thread has read the flag
    if (!kTeamed) grid_launch_dependents();         // the join may set up meanwhile
    return !skip;
}

// What a producer warp loads. One warp issues a copy in about 100 cycles, and a
// tile of small pages takes many (16 of 16 tokens at d = 128): where a CTA has
// an SM to itself, K and V have a warp each (8 sequences of 17000 tokens, 20
// query rows, pages of 16: 123 us with one, 107 with two; in fp32, 4 rows of 32768
// tokens, 191 and 167), and with two row groups also where two CTAs share it (d =
// 64: 8 x 16500 tokens, 24 rows, pages of 64: 63.7 us with one, 60.0 with two; 4 x
// 28000, 21 rows, pages of 8: 77.1 and 64.4; 200 of 30 to 400, 20 rows: 40.5 and 41.1).
enum class Loads { kBoth, kKeys, kValues };

// A producer warp; the one of K, or of both, leads. A tile is 64 / box pages (box
// = min(page, 64) tokens, one lane each); 32 table entries are held across the
// warp and the next 32 are on the way, as are those of the next piece while this
// one's tiles are issued. C: the kernel's configuration; Q: the query rows, which
// come beside a piece's first tile if it wants them (kQPitch); begin(piece):
// called by the warp when a piece begins, with its description, false to give up.
template <typename C, Loads kLoads, typename RingT, typename W, typename F>
__device__ __forceinline__ void produce(const CUtensorMap* tmK, const CUtensorMap* tmV, const DecodeArgs& a,
                                        const __nv_bfloat16* Q, W& w, RingT& ring, uint8_t* smem,
                                        unsigned long long budget_ns, F&& begin) {
    constexpr int kStages = C::kStages;
    constexpr bool kLead = kLoads != Loads::kValues;
    constexpr int kK = kLoads != Loads::kValues ? C::kKPanels : 0, kV = kLoads != Loads::kKeys ? C::kVPanels : 0;
    const int lane = threadIdx.x & 31;
    const int page_log2 = a.g.page_log2, page = 1 << page_log2;
    const int box_log2 = min(page_log2, 6), box = 1 << box_log2, boxes = kTileKeys >> box_log2;
    if (lane == 0) {
        prefetch_tensor_map(tmK);
        prefetch_tensor_map(tmV);
    }
    int n = 0, s = 0;                               // tiles issued, stage of the next
    uint32_t parity = 1;                            // of the empty barriers: the first round passes
    bool going = true;
    // A piece, the first entries of its table row, and its number of pages.
    struct Ahead {
        Piece p;
        const int* row;
        int base, last, held, ahead;
        bool some;
    };
    auto next = [&] {
        Ahead x;
        x.some = w.next(a, &x.p);
        if (!x.some) return x;
        x.row = a.table + size_t(x.p.b) * a.g.M;
        x.last = pages_of(x.p.len, page_log2);
        x.base = (x.p.t0 * kTileKeys) >> page_log2;
        x.held = x.base + lane < x.last ? x.row[x.base + lane] : -1;
        x.ahead = x.base + 32 + lane < x.last ? x.row[x.base + 32 + lane] : -1;
        return x;
    };
    Ahead now = next(), then = now;
    for (; going && now.some; now = then) {
        const Piece& p = now.p;
        const int hk = a.row_tiles == 1 ? p.item : p.item / a.row_tiles;
        const int r0 = (p.item - hk * a.row_tiles) * a.tile_rows;
        Stage d;
        d.present = 0;
        d.flags = kFirst | (p.t0 == 0 ? kStarts : 0) | (p.t1 == p.tiles ? kEnds : 0);
        d.row = int(row_base(a, p.b, hk)) + r0;
        d.rows = min(a.tile_rows, a.rows - r0);
        d.i0 = a.n == 1 ? 0 : r0 % a.n;
        d.len = p.len;
        d.nq = p.nq;
        d.t0 = p.t0;
        d.tiles = p.t1 - p.t0;
        d.b = p.b;
        d.item = p.item;
        d.last = (d.flags & kStarts) && !(d.flags & kEnds) ? w.owner(p.end - 1) : 0;
        if (kLead && !begin(d)) {
            going = false;
            break;
        }
        constexpr bool with_q = kLead && C::kQPitch > 0;
        for (int t = p.t0; t < p.t1; ++t, ++n) {
            const int k0 = t * kTileKeys, first = k0 >> page_log2;
            if (first - now.base >= 32) {
                now.base += 32;
                now.held = now.ahead;
                now.ahead = now.base + 32 + lane < now.last ? now.row[now.base + 32 + lane] : -1;
            }
            const int key = k0 + (lane << box_log2);
            const int entry = __shfl_sync(0xffffffffu, now.held, (key >> page_log2) - now.base);
            const bool load = lane < boxes && key < p.len && page_ok(entry, a.g.P);
            const unsigned loads = __ballot_sync(0xffffffffu, load);
            if (!ring_wait(ring, &ring.empty[s], parity, budget_ns)) {
                going = false;
                break;
            }
            if (lane == 0) {
                if (kLead) {
                    unsigned long long keys = ~0ull;
                    if (loads != (1u << boxes) - 1u) {
                        const unsigned long long one = box == 64 ? ~0ull : (1ull << box) - 1ull;
                        keys = 0;
                        for (int x = 0; x < boxes; ++x)
                            if (loads >> x & 1) keys |= one << (x << box_log2);
                    }
                    if (p.len - k0 < kTileKeys) keys &= p.len > k0 ? (1ull << (p.len - k0)) - 1ull : 0ull;
                    Stage& st = ring.stage[s];
                    if (t == p.t0) st = d;
                    st.present = keys;
                    st.flags = (t == p.t0 ? d.flags : 0) | (t == p.t1 - 1 ? kLast : 0);
                }
                mbar_arrive_expect_tx(&ring.full[s], __popc(loads) * box * (kK + kV) * 128 +
                                                         (with_q && t == p.t0 ? d.rows * a.d * 2 : 0));
            }
            __syncwarp();
            if constexpr (with_q) {
                // Row r begins 16 r bytes into its place and ends at its start.
                if (t == p.t0 && lane < d.rows) {
                    uint8_t* dst = smem + C::kOffQ + s * C::kQBytes + lane * C::kQPitch;
                    const __nv_bfloat16* src = Q + (size_t(d.row) + lane) * a.d;
                    const int turn = (lane * 16) & (C::kQPitch - 1), first = min(a.d * 2, C::kQPitch - turn);
                    bulk_load(dst + turn, src, first, &ring.full[s]);
                    if (first < a.d * 2) bulk_load(dst, src + first / 2, a.d * 2 - first, &ring.full[s]);
                }
            }
            if (load) {
                uint8_t* dst = smem + s * C::kStageBytes + (lane << box_log2) * 128;
                const int z = entry * a.g.Hkv + hk, y = key & (page - 1);
#pragma unroll
                for (int x = 0; x < kK; ++x)
                    tma_load_3d(dst + x * kPanelBytes, tmK, &ring.full[s], C::kPanelCols * x, y, z);
#pragma unroll
                for (int x = 0; x < kV; ++x)
                    tma_load_3d(dst + C::kKBytes + x * kPanelBytes, tmV, &ring.full[s], C::kPanelCols * x, y, z);
            }
            if (++s == kStages) {
                s = 0;
                parity ^= 1;
            }
            // Once the stages are on the way, or with the piece's last tile.
            if (t == min(p.t1, p.t0 + kStages) - 1) then = next();
        }
    }
    const bool stopped = going && ring_wait(ring, &ring.empty[s], parity, budget_ns);
    if (stopped && lane == 0) {
        if (kLead) ring.stage[s].flags = kStop;
        mbar_arrive(&ring.full[s]);
    }
    // No copy may be in flight into shared memory that the CTA gives back. (The
    // stage that the end took was empty, and its barrier has moved on.)
    for (int x = max(0, n - kStages + (stopped ? 1 : 0)); x < n; ++x)
        (void)mbar_wait_timed(&ring.full[x % kStages], (x / kStages) & 1, budget_ns);
}

// The query rows into L1, ahead of the warps that will read them.
template <typename T>
__device__ __forceinline__ bool prefetch_rows(const T* Q, int q_row, int rows, int d) {
    const char* q = reinterpret_cast<const char*>(Q + size_t(q_row) * d);
    for (int x = (threadIdx.x & 31) * 128; x < rows * d * int(sizeof(T)); x += 32 * 128)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(q + x));
    return true;
}

// What a consumer keeps of the piece it is at.
struct At {
    int row, rows, i0, nq, flags;
    int b, item, last;
};
template <typename RingT>
__device__ __forceinline__ At piece_at(const RingT& ring, int s) {
    const Stage& st = ring.stage[s];
    return At{st.row, st.rows, st.i0, st.nq, st.flags, st.b, st.item, st.last};
}
// The query that row r of the item belongs to.
__device__ __forceinline__ int query_of(const DecodeArgs& a, const At& at, int r) {
    return a.n == 1 ? 0 : (at.i0 + r) % a.n;
}
__device__ __forceinline__ void note_head(const Parts& parts, const At& at) {
    if ((at.flags & (kStarts | kEnds)) == kStarts)
        parts.head[blockIdx.x] = Head{at.b, at.item, at.last, at.nq};
}

}  // namespace paged
}  // namespace attn
