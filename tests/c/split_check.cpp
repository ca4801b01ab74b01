// The split of a decode call over CTAs (csrc/paged.cuh), run on the host: every key
// tile of every item is taken once, pieces of an item lie in consecutive CTAs, the
// last of them is the one that its first piece names; and lengths that change
// between two reads lead to no index past the arrays.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <utility>
#include <vector>

#define __device__
#define __forceinline__ inline
#define __restrict__
using std::max;
using std::min;
struct Dim { int x; };
static Dim threadIdx{0}, blockIdx{0}, blockDim{32}, gridDim{1};
static int reads_past, shrink_after = -1, g_B;
static const int* g_lens;
// Reads of lengths are counted; after `shrink_after` of them the lengths are `later`.
static std::vector<int> later;
static int g_reads;
inline int __ldg(const int* p) {
    const long long i = p - g_lens;
    if (g_lens && i >= 0 && i < 4 * g_B + 64) {
        if (i >= g_B) { ++reads_past; return 0; }
        if (shrink_after >= 0 && g_reads++ >= shrink_after) return later[i];
    }
    return *p;
}
inline int __shfl_sync(unsigned, int v, int) { return v; }
inline long long __shfl_sync(unsigned, long long v, int) { return v; }
template <typename T> T __shfl_up_sync(unsigned, T v, int) { return v; }
inline unsigned __ballot_sync(unsigned, bool v) { return v ? 1u : 0u; }
inline int __ffs(unsigned v) { return __builtin_ffs(int(v)); }
inline void __syncthreads() {}
#define asm
#define volatile(...) ((void)0)
#define __shared__
#include "paged.cuh"
#undef asm
#undef volatile

using namespace attn::paged;

// A warp's lanes share the sequences; here one walker does what lane and warp do.
static bool start(Walker& w, const DecodeArgs& a) {
    long long total = 0;
    for (int b = 0; b < a.g.B; ++b) total += Walker::units_of(a, b);
    w.ctas = int(min((long long)gridDim.x, max(1ll, total)));
    w.q = divide(total, w.ctas);
    w.r = total - w.q * w.ctas;
    const long long c = blockIdx.x;
    w.left = c < w.ctas ? w.q + (c < w.r ? 1 : 0) : 0;
    w.pos = w.q * c + min(c, w.r);
    long long x = 0;
    w.b = w.left > 0 ? sequence_of([&](int k) { return Walker::units_of(a, k); }, 0, a.g.B, w.pos, &x) : 0;
    w.off = w.pos - x;
    return w.left > 0;
}

#define CHECK(c) do { if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); return 1; } } while (0)

int main() {
    std::srand(7);
    for (int round = 0; round < 3000; ++round) {
        const int B = 1 + std::rand() % 9, n = 1 + std::rand() % 3, tiles_max = 1 + std::rand() % 40;
        std::vector<int> lens(4 * B + 64, 0), nq(B);
        for (int b = 0; b < B; ++b) {
            lens[b] = std::rand() % (64 * tiles_max);
            nq[b] = std::rand() % (n + 1);
        }
        g_lens = lens.data();
        g_B = B;
        shrink_after = -1;
        reads_past = 0;
        DecodeArgs a{};
        a.g = Geometry{B, 64 * tiles_max / 8 + 1, 1 << 20, 1 + std::rand() % 4, 3};
        a.lens = lens.data();
        a.q_len = nq.data();
        a.n = n;
        a.row_tiles = 1 + std::rand() % 3;
        gridDim.x = 1 + std::rand() % 60;
        struct At { int cta, last; };
        std::map<std::pair<int, int>, std::vector<std::pair<Piece, At>>> items;
        for (blockIdx.x = 0; blockIdx.x < gridDim.x; ++blockIdx.x) {
            Walker w;
            if (!start(w, a)) continue;
            Piece p;
            while (w.next(a, &p)) items[{p.b, p.item}].push_back({p, At{blockIdx.x, w.owner(p.end - 1)}});
        }
        size_t want = 0;
        for (int b = 0; b < B; ++b) want += nq[b] > 0 ? a.g.Hkv * a.row_tiles : 0;
        CHECK(items.size() == want && reads_past == 0);
        for (auto& it : items) {
            auto& v = it.second;
            const Piece& f = v[0].first;
            CHECK(f.t0 == 0 && v.back().first.t1 == f.tiles && f.tiles == tiles_of(lens[f.b]));
            CHECK(v[0].second.last == v.back().second.cta);
            CHECK(pieces_of(Head{f.b, it.first.second, v[0].second.last, f.nq}, v[0].second.cta, gridDim.x) == int(v.size()));
            for (size_t i = 1; i < v.size(); ++i)
                CHECK(v[i].first.t0 == v[i - 1].first.t1 && v[i].second.cta == v[i - 1].second.cta + 1);
        }
        // Lengths that change after some reads: no bounds hold but those of the arrays.
        later.assign(B, 0);
        for (int b = 0; b < B; ++b) later[b] = std::rand() % 3 ? 0 : std::rand() % (64 * tiles_max);
        const int after = std::rand() % (2 * B + 1);
        for (blockIdx.x = 0; blockIdx.x < gridDim.x; ++blockIdx.x) {
            shrink_after = after;
            g_reads = 0;
            Walker w;
            if (!start(w, a)) continue;
            Piece p;
            while (w.next(a, &p)) {
                const int last = w.owner(p.end - 1);
                CHECK(p.b < B && p.item < a.g.Hkv * a.row_tiles && p.t0 < p.t1 && p.t1 <= p.tiles);
                const int pieces = pieces_of(Head{p.b, p.item, last, p.nq}, blockIdx.x, gridDim.x);
                CHECK(pieces >= 0 && blockIdx.x + pieces <= gridDim.x);
            }
            CHECK(w.b <= B && reads_past == 0);
        }
    }
    std::printf("split_check ok\n");
    return 0;
}
