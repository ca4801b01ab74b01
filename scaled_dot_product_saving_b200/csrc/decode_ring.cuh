// decode_ring.cuh -- the stream of key tiles that the decode kernels consume: a
// ring of shared-memory stages of 64 keys, filled page by page with the TMA by
// one warp that runs ahead of the others, across the borders of pieces.
//
// A stage is panels of 64 rows of 128 bytes (64 bf16 or 32 fp32 columns) in the
// TMA's 128-byte swizzle: the K panels, then the V panels.
#pragma once

#include "decode.cuh"

namespace attn {
namespace paged {

constexpr int kPanelBytes = kTileKeys * 128;

template <int kStages>
struct Ring {
    uint64_t full[kStages], empty[kStages];
    unsigned long long present[kStages];           // keys of the stage that exist
    int abort;
};

// A wait that runs out sets the abort flag, after which every wait returns at
// once: each role goes through its loops without data, so that no thread stays
// behind at a barrier, and the error word tells the host.
template <int kStages>
__device__ __forceinline__ void ring_wait(Ring<kStages>& ring, uint64_t* bar, uint32_t parity,
                                          unsigned long long budget_ns) {
    volatile int* abort = &ring.abort;
    if (!mbar_wait(bar, parity, abort, budget_ns)) {
        record_device_error(kErrTimeout);
        *abort = 1;
    }
}

// Collective over the block: barriers, the CTA's share of the work, and no head
// yet. False (for all threads) if an earlier kernel's timeout has not been
// read, in which case the call does nothing.
template <int kStages>
__device__ __forceinline__ bool set_up(const DecodeArgs& a, const Parts& parts, Ring<kStages>& ring,
                                       const uint8_t* smem, int consumers, long long* scratch, long long* found,
                                       Walker* w) {
    if (threadIdx.x == 0) {
        parts.head[blockIdx.x].b = -1;
        const bool misaligned = (smem_addr(smem) & 1023u) != 0;
        if (misaligned) record_device_error(kErrTimeout);
        ring.abort = misaligned || *reinterpret_cast<volatile unsigned int*>(&g_device_error) != 0;
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&ring.full[s], 1);
            mbar_init(&ring.empty[s], consumers);
        }
        fence_mbar_init();
    }
    w->start(a, scratch, found);                    // ends with a barrier
    const bool skip = ring.abort != 0;
    __syncthreads();                                // every thread has read the flag
    grid_launch_dependents();                       // the join may set up meanwhile
    return !skip;
}

// The producer warp. A tile is 64 / box pages (box = min(page, 64) tokens, one
// lane each); 32 table entries are held across the warp and the next 32 are on
// the way. C: the kernel's configuration.
template <typename C, int kStages>
__device__ __forceinline__ void produce(const CUtensorMap* tmK, const CUtensorMap* tmV, const DecodeArgs& a,
                                        Walker w, Ring<kStages>& ring, uint8_t* smem,
                                        unsigned long long budget_ns) {
    const int lane = threadIdx.x & 31;
    const int page_log2 = a.g.page_log2, page = 1 << page_log2;
    const int box_log2 = min(page_log2, 6), box = 1 << box_log2, boxes = kTileKeys >> box_log2;
    if (lane == 0) {
        prefetch_tensor_map(tmK);
        prefetch_tensor_map(tmV);
    }
    int n = 0;                                      // tiles issued
    Piece p;
    while (w.next(a, &p)) {
        const int hk = p.item / a.row_tiles;
        const int* row = a.table + size_t(p.b) * a.g.M;
        const int last = pages_of(p.len, page_log2);
        int base = (p.t0 * kTileKeys) >> page_log2;
        int held = base + lane < last ? row[base + lane] : -1;
        int ahead = base + 32 + lane < last ? row[base + 32 + lane] : -1;
        for (int t = p.t0; t < p.t1; ++t, ++n) {
            const int k0 = t * kTileKeys, first = k0 >> page_log2;
            if (first - base >= 32) {
                base += 32;
                held = ahead;
                ahead = base + 32 + lane < last ? row[base + 32 + lane] : -1;
            }
            const int key = k0 + (lane << box_log2);
            const int entry = __shfl_sync(0xffffffffu, held, (key >> page_log2) - base);
            const bool load = lane < boxes && key < p.len && page_ok(entry, a.g.P);
            const unsigned loads = __ballot_sync(0xffffffffu, load);
            const int s = n % kStages;
            if (n >= kStages) ring_wait(ring, &ring.empty[s], (n / kStages - 1) & 1, budget_ns);
            const bool go = __all_sync(0xffffffffu, !*reinterpret_cast<volatile int*>(&ring.abort));
            if (lane == 0) {
                unsigned long long keys = ~0ull;
                if (loads != (1u << boxes) - 1u) {
                    const unsigned long long one = box == 64 ? ~0ull : (1ull << box) - 1ull;
                    keys = 0;
                    for (int x = 0; x < boxes; ++x)
                        if (loads >> x & 1) keys |= one << (x << box_log2);
                }
                if (p.len - k0 < kTileKeys) keys &= p.len > k0 ? (1ull << (p.len - k0)) - 1ull : 0ull;
                ring.present[s] = keys;
                mbar_arrive_expect_tx(&ring.full[s], go ? __popc(loads) * box * (C::kKPanels + C::kVPanels) * 128 : 0);
            }
            __syncwarp();
            if (load && go) {
                uint8_t* dst = smem + s * C::kStageBytes + (lane << box_log2) * 128;
                const int z = entry * a.g.Hkv + hk, y = key & (page - 1);
#pragma unroll
                for (int x = 0; x < C::kKPanels; ++x)
                    tma_load_3d(dst + x * kPanelBytes, tmK, &ring.full[s], C::kPanelCols * x, y, z);
#pragma unroll
                for (int x = 0; x < C::kVPanels; ++x)
                    tma_load_3d(dst + C::kKBytes + x * kPanelBytes, tmV, &ring.full[s], C::kPanelCols * x, y, z);
            }
        }
    }
    // No copy may be in flight into shared memory that the CTA gives back.
    for (int x = max(0, n - kStages); x < n; ++x)
        (void)mbar_wait_timed(&ring.full[x % kStages], (x / kStages) & 1, budget_ns);
}

}  // namespace paged
}  // namespace attn
