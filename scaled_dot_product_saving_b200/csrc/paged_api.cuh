// paged_api.cuh -- the entry points of the paged key-value cache (part of the
// one translation unit that attn.cu compiles): argument checks, workspaces and
// launches of decode.cuh and cache.cuh.
#pragma once

namespace {

namespace pg = attn::paged;

constexpr int kMmaRows = 32;            // bf16 on mma.sync up to here (see decode_rows)
// Most CTAs of a decode call, and most CTAs times query rows of an item: what the
// workspace has slots for, on up to kSms SMs (three CTAs an SM for items of 16 rows,
// two for 32, one for 128; decode_stream checks each kernel's).
constexpr int kSms = 148;
constexpr int kDecodeCtas = 3 * kSms, kDecodeRows = 64 * kSms, kDecodeWideRows = pg::kWideRows * kSms;
inline int decode_sms() { return std::min(sm_count(), kSms); }

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Bytes [p, p + n) that a call reads or writes.
struct Region {
    const void* p;
    size_t n;
};
inline bool overlap(const Region& a, const Region& b) {
    const char* x = static_cast<const char*>(a.p);
    const char* y = static_cast<const char*>(b.p);
    return a.p && b.p && a.n && b.n && x < y + b.n && y < x + a.n;
}
// No written region may touch another written or read one. in_place holds the
// read regions that the written region of the same index may equal.
template <size_t W, size_t R>
bool apart(const Region (&written)[W], const Region (&read)[R], const Region* in_place, size_t pairs) {
    for (size_t i = 0; i < W; ++i) {
        for (size_t j = i + 1; j < W; ++j)
            if (overlap(written[i], written[j])) return false;
        for (size_t j = 0; j < R; ++j)
            if (overlap(written[i], read[j])) return false;
        for (size_t j = 0; j < pairs; ++j)
            if (overlap(written[i], in_place[j]) && !(i == j && written[i].p == in_place[j].p)) return false;
    }
    return true;
}

// Widths of a row, which is whole 16 bytes.
attn_status_t check_widths(int d, int dv, attn_dtype_t dtype) {
    if (d > pg::kMaxWidth || dv > pg::kMaxWidth) return ATTN_ERR_UNSUPPORTED;
    const int es = dtype == ATTN_F32 ? 4 : 2;
    return d * es % 16 || dv * es % 16 ? ATTN_ERR_SHAPE : ATTN_OK;
}

// Kernels number pages, tokens and what lies a tile or a block past them in 32 bits.
bool books_fit(int B, int max_pages, int num_pages, int page_log2) {
    return num_pages <= (1 << 30) && static_cast<long long>(B) * max_pages < (1ll << 31) &&
           max_pages <= ((1 << 30) >> page_log2);
}

attn_status_t check_cache(int B, int Hkv, int d, int dv, int num_pages, int page, int max_pages,
                          attn_dtype_t dtype, pg::Geometry* g) {
    if (dtype != ATTN_F32 && dtype != ATTN_BF16) return ATTN_ERR_DTYPE;
    if (B < 1 || Hkv < 1 || d < 1 || dv < 1 || num_pages < 1 || page < 1 || max_pages < 1)
        return ATTN_ERR_SHAPE;
    int log2 = 0;
    while ((1 << log2) < page && log2 < 30) ++log2;
    if ((1 << log2) != page || log2 < pg::kMinPageLog2 || log2 > pg::kMaxPageLog2) return ATTN_ERR_UNSUPPORTED;
    const attn_status_t widths = check_widths(d, dv, dtype);
    if (widths != ATTN_OK) return widths;
    if (static_cast<long long>(num_pages) * Hkv >= (1ll << 31) || !books_fit(B, max_pages, num_pages, log2))
        return ATTN_ERR_SHAPE;
    *g = pg::Geometry{B, max_pages, num_pages, Hkv, log2};
    return ATTN_OK;
}

size_t pool_bytes(const pg::Geometry& g, int width, attn_dtype_t dtype) {
    return (static_cast<size_t>(g.P) * g.Hkv << g.page_log2) * width * (dtype == ATTN_F32 ? 4 : 2);
}

// A programmatic dependent of the kernel before it on the stream: its launch
// overlaps that one. Not while tracing, which would count the overlap twice.
template <typename... P, typename... A>
bool launch_dependent(void (*kern)(P...), dim3 grid, int threads, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = g_trace.on ? 0 : 1;
    if (cudaLaunchKernelEx(&cfg, kern, P(args)...) == cudaSuccess) return true;
    (void)cudaGetLastError();
    return false;
}

// ------------------------------------------------------------------ decode
struct DecodeWorkspace {
    size_t o_off, ml_off, head_off, total;
};
DecodeWorkspace carve_decode(int dv, long long rows_per_head) {
    DecodeWorkspace w;
    const size_t rows = 2ull * (rows_per_head > kMmaRows ? kDecodeWideRows : kDecodeRows);
    w.o_off = 0;
    w.ml_off = round_up(rows * dv * sizeof(float), 256);
    w.head_off = w.ml_off + round_up(rows * 2 * sizeof(float), 256);
    w.total = w.head_off + round_up(kDecodeCtas * sizeof(pg::Head), 256);
    return w;
}

attn_status_t check_decode(int B, int H, int Hkv, int n, int d, int dv, attn_dtype_t dtype) {
    if (dtype != ATTN_F32 && dtype != ATTN_BF16) return ATTN_ERR_DTYPE;
    if (B < 1 || H < 1 || Hkv < 1 || n < 1 || d < 1 || dv < 1 || H % Hkv) return ATTN_ERR_SHAPE;
    if (static_cast<double>(B) * H * n > 1073741824.0) return ATTN_ERR_SHAPE;
    return check_widths(d, dv, dtype);
}

attn_status_t decode_simt(const pg::DecodeArgs& a, const void* Q, const void* Kp, const void* Vp, void* O,
                          float* LSE, const pg::Parts& parts, int* grid, cudaStream_t st) {
    const int smem = pg::simt_smem_bytes(a.d, a.dv);
    if (cudaFuncSetAttribute(pg::decode_simt, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return ATTN_ERR_CUDA;
    *grid = 2 * decode_sms();
    return traced(ATTN_KERNEL_DECODE_SIMT, st, [&] {
        using T = __nv_bfloat16;
        pg::decode_simt<<<*grid, pg::kSimtThreads, smem, st>>>(a, static_cast<const T*>(Q), static_cast<const T*>(Kp),
                                                               static_cast<const T*>(Vp), static_cast<T*>(O), LSE,
                                                               parts);
        return launched();
    });
}

template <typename T>
attn_status_t decode_join(const pg::DecodeArgs& a, void* O, float* LSE, const pg::Parts& parts, int grid,
                          cudaStream_t st) {
    // Warps per row: an item of few rows may come in many pieces (one key head,
    // a long sequence), and few rows leave room for them.
    constexpr int kWarps = pg::kJoinThreads / 32;
    const int rows = std::min(a.rows, a.tile_rows);
    const int split = rows <= 4 ? 4 : rows <= 8 ? 2 : 1;
    const dim3 blocks(grid, (rows * split + kWarps - 1) / kWarps);
    return traced(ATTN_KERNEL_DECODE_JOIN, st, [&] {
        return launch_dependent(pg::decode_join<T>, blocks, pg::kJoinThreads, st, a, static_cast<T*>(O), LSE, parts,
                                split)
                   ? launched()
                   : ATTN_ERR_CUDA;
    });
}

// The kernels that stream tiles with the TMA. C: the kernel's configuration; T:
// the element type, whose columns the maps' 128-byte rows hold. teams: 0, or one
// team for each of so many items.
template <typename C, typename T, typename Kern, typename... More>
attn_status_t decode_stream(Kern kern, int kernel_id, pg::DecodeArgs& a, const void* Q, const void* Kp,
                            const void* Vp, void* O, float* LSE, const pg::Parts& parts, int* grid, int teams,
                            cudaStream_t st, const More&... more) {
    static_assert(C::kCtasPerSm * kSms <= kDecodeCtas, "the workspace holds a head for each CTA");
    static_assert(C::kCtasPerSm * C::kTileRows * kSms <= (C::kTileRows == pg::kWideRows ? kDecodeWideRows : kDecodeRows),
                  "... and two pieces");
    a.tile_rows = C::kTileRows;
    a.row_tiles = (a.rows + a.tile_rows - 1) / a.tile_rows;
    CUtensorMap mk, mv;
    const int page = 1 << a.g.page_log2, heads = a.g.P * a.g.Hkv, box = std::min(page, pg::kTileKeys);
    constexpr auto type = sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    if (!make_map_typed(&mk, Kp, a.d, page, heads, type, sizeof(T), C::kPanelCols, box) ||
        !make_map_typed(&mv, Vp, a.dv, page, heads, type, sizeof(T), C::kPanelCols, box))
        return ATTN_ERR_CUDA;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes) != cudaSuccess)
        return ATTN_ERR_CUDA;
    *grid = teams > 0 ? teams * pg::kTeam : C::kCtasPerSm * decode_sms();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(*grid);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = pg::kTeam;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = teams > 0 ? 1 : 0;
    return traced(kernel_id, st, [&] {
        if (cudaLaunchKernelEx(&cfg, kern, mk, mv, a, static_cast<const T*>(Q), static_cast<T*>(O), LSE, parts,
                               kWaitBudgetNs, more...) != cudaSuccess) {
            (void)cudaGetLastError();
            return ATTN_ERR_CUDA;
        }
        return launched();
    });
}

template <int DK, int DV, int R>
attn_status_t decode_tc(pg::DecodeArgs& a, const void* Q, const void* Kp, const void* Vp, void* O, float* LSE,
                        const pg::Parts& parts, int* grid, cudaStream_t st) {
    using C = pg::DecodeCfg<DK, DV, R, false>;
    if constexpr (R == 1) {
        // Teams where their CTAs are all resident at once and no sequence can be
        // longer than 8 tiles for each of a team's CTAs: one launch instead of two.
        // (Up to 16 rows: one item a key head.)
        const long long items = 1ll * a.g.B * a.g.Hkv;
        if (items * pg::kTeam <= C::kCtasPerSm * sm_count() &&
            (1ll * a.g.M << a.g.page_log2) <= 8 * pg::kTeam * pg::kTileKeys) {
            const attn_status_t s = decode_stream<pg::DecodeCfg<DK, DV, R, true>, __nv_bfloat16>(
                pg::decode_tc<DK, DV, R, true>, ATTN_KERNEL_DECODE_TENSOR, a, Q, Kp, Vp, O, LSE, parts, grid,
                int(items), st);
            *grid = 0;                                     // nothing to join
            return s;
        }
    }
    return decode_stream<C, __nv_bfloat16>(pg::decode_tc<DK, DV, R, false>, ATTN_KERNEL_DECODE_TENSOR, a, Q, Kp, Vp, O,
                                           LSE, parts, grid, 0, st);
}

template <int DK, int DV>
attn_status_t decode_wide(pg::DecodeArgs& a, const void* Q, const void* Kp, const void* Vp, void* O, float* LSE,
                          const pg::Parts& parts, int* grid, cudaStream_t st) {
    using C = pg::DecodeWideCfg<DK, DV>;
    CUtensorMap mq;
    if (!make_map_rows(&mq, Q, a.d, a.g.B * a.H * a.n, a.d, 64, pg::kWideRows)) return ATTN_ERR_CUDA;
    return decode_stream<C, __nv_bfloat16>(pg::decode_wide<DK, DV>, ATTN_KERNEL_DECODE_WIDE, a, Q, Kp, Vp, O, LSE, parts,
                                           grid, 0, st, mq, static_cast<const __nv_bfloat16*>(Kp),
                                           static_cast<const __nv_bfloat16*>(Vp));
}

template <int DK, int DV, int RB, int R>
attn_status_t decode_f32(pg::DecodeArgs& a, const void* Q, const void* Kp, const void* Vp, void* O, float* LSE,
                         const pg::Parts& parts, int* grid, cudaStream_t st) {
    return decode_stream<pg::DecodeF32Cfg<DK, DV, RB, R>, float>(pg::decode_f32<DK, DV, RB, R>, ATTN_KERNEL_DECODE_F32, a,
                                                                 Q, Kp, Vp, O, LSE, parts, grid, 0, st);
}

// Query rows of an item: as many of a key head's as there are, up to 128 (bf16,
// tcgen05 above 32) or 16 (fp32), since every item reads its keys again. 8 x 32768
// tokens, 32 rows: tcgen05 takes 180 us and mma.sync 210 at d = 128, 140 and 105 at d
// = 64; 64 sequences of 100 to 3000 tokens, 24 rows: 98 and 76, 73 and 42; 200 of 30 to
// 400, 32 rows, d = 128: 115 and 82. At d = 128 the times cross with the lengths,
// which the host does not know, and not with the rows: 20, 24, 28 and 32 are within
// 4 % of each other.
template <int DK, int DV>
attn_status_t decode_rows(pg::DecodeArgs& a, const void* Q, const void* Kp, const void* Vp, void* O, float* LSE,
                          const pg::Parts& parts, int* grid, bool f32, cudaStream_t st) {
    if (f32) {
        if (a.rows <= 4) return decode_f32<DK, DV, 4, 1>(a, Q, Kp, Vp, O, LSE, parts, grid, st);
        if (a.rows <= 8) return decode_f32<DK, DV, 8, 1>(a, Q, Kp, Vp, O, LSE, parts, grid, st);
        return decode_f32<DK, DV, 8, 2>(a, Q, Kp, Vp, O, LSE, parts, grid, st);
    }
    if (a.rows <= 16) return decode_tc<DK, DV, 1>(a, Q, Kp, Vp, O, LSE, parts, grid, st);
    if (a.rows <= kMmaRows) return decode_tc<DK, DV, 2>(a, Q, Kp, Vp, O, LSE, parts, grid, st);
    return decode_wide<DK, DV>(a, Q, Kp, Vp, O, LSE, parts, grid, st);
}

// ------------------------------------------------------------------- books
struct CacheWorkspace {
    size_t after_off, start_off, base_off, key_off, stage_off, moves_off, total;
};
CacheWorkspace carve_cache(int B, int max_pages, int num_pages) {
    CacheWorkspace w;
    const auto ints = [](size_t n) { return round_up(n * sizeof(int), 256); };
    w.after_off = ints(pg::kCtlWords);
    w.start_off = w.after_off + ints(B);
    w.base_off = w.start_off + ints(B);
    w.key_off = w.base_off + ints(num_pages);
    w.stage_off = w.key_off + ints(num_pages);
    w.moves_off = w.stage_off + ints(static_cast<size_t>(B) * max_pages);
    w.total = w.moves_off + round_up(std::max<size_t>(B, num_pages) * sizeof(pg::Move), 256);
    return w;
}

pg::Books books(const pg::Geometry& g, const int* table, const int* lens, const int* ref, int* table_out,
                int* lens_out, int* ref_out, int* info, void* workspace) {
    const CacheWorkspace w = carve_cache(g.B, g.M, g.P);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const auto at = [&](size_t off) { return reinterpret_cast<int*>(ws + off); };
    return pg::Books{g, table, lens, ref, table_out, lens_out, ref_out, info, at(0), at(w.after_off),
                     at(w.start_off), at(w.base_off), at(w.key_off), at(w.stage_off),
                     reinterpret_cast<pg::Move*>(ws + w.moves_off)};
}

// One cluster of kBookCtas CTAs.
template <typename... P, typename... A>
attn_status_t launch_books(void (*kern)(P...), cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(pg::kBookCtas);
    cfg.blockDim = dim3(pg::kBookThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = pg::kBookCtas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return traced(ATTN_KERNEL_CACHE_BOOKS, st, [&] {
        if (cudaLaunchKernelEx(&cfg, kern, P(args)...) != cudaSuccess) {
            (void)cudaGetLastError();
            return ATTN_ERR_CUDA;
        }
        return launched();
    });
}

// The books, and the copies that they ask for: at most `spans` (see cache.cuh).
template <typename Kern, typename A>
attn_status_t books_and_rows(Kern kern, void (*copy)(pg::Books, pg::Rows), const pg::Books& k, pg::Rows r,
                             unsigned long long spans, cudaStream_t st, A&& launch) {
    r.here = spans <= pg::kHereSpans && (copy == pg::move_rows || r.flat);
    attn_status_t s = launch(kern, r);
    if (s != ATTN_OK || r.here) {
        if (s == ATTN_OK) g_last_launches = 1;
        return s;
    }
    // A warp per span, up to 8 blocks an SM for new rows, whose warps pass over
    // padding on their way (prompts of 1 to 2000 in 4096 rows: 30.2 us with 8, 30.8
    // with 16, 31.9 with 32, 38.2 with 64); up to 32 for pages, which are all whole
    // (17,400 pages: 104.9, 98.9, 97.5, 96.6).
    const int grid = grid_for(static_cast<size_t>(spans), pg::kCopyThreads / 32,
                              sm_count() * (copy == pg::append_rows ? 8 : 32));
    s = traced(ATTN_KERNEL_CACHE_ROWS, st, [&] {
        return launch_dependent(copy, dim3(grid), pg::kCopyThreads, st, k, r) ? launched() : ATTN_ERR_CUDA;
    });
    if (s == ATTN_OK) g_last_launches = 2;
    return s;
}

}  // namespace

extern "C" {

size_t attn_decode_workspace_size(int B, int H, int Hkv, int n, int d, int dv, attn_dtype_t dtype) {
    if (check_decode(B, H, Hkv, n, d, dv, dtype) != ATTN_OK) return 0;
    return carve_decode(dv, 1ll * H / Hkv * n).total;
}

attn_status_t attn_decode(const void* Q, const void* K_pages, const void* V_pages, const int* table,
                          const int* lens, const int* q_len, void* O, float* LSE, void* workspace,
                          size_t workspace_bytes, int B, int H, int Hkv, int n, int d, int dv,
                          int num_pages, int page, int max_pages, attn_dtype_t dtype, int causal,
                          float scale, void* stream) {
    pg::Geometry g;
    attn_status_t s = check_decode(B, H, Hkv, n, d, dv, dtype);
    if (s == ATTN_OK) s = check_cache(B, Hkv, d, dv, num_pages, page, max_pages, dtype, &g);
    if (s != ATTN_OK) return s;
    if (!std::isfinite(scale * kLog2e)) return ATTN_ERR_SHAPE;      // the kernels' factor: base 2
    if (!Q || !K_pages || !V_pages || !table || !lens || !O || !LSE) return ATTN_ERR_NULL;
    if (!aligned16(Q) || !aligned16(K_pages) || !aligned16(V_pages) || !aligned16(O) || !aligned16(LSE) ||
        !aligned4(table) || !aligned4(lens) || !aligned4(q_len))
        return ATTN_ERR_ALIGN;
    const DecodeWorkspace w = carve_decode(dv, 1ll * H / Hkv * n);
    if (!workspace || workspace_bytes < w.total) return ATTN_ERR_WORKSPACE;
    if (!aligned16(workspace)) return ATTN_ERR_ALIGN;

    // bf16 runs on the tensor cores, fp32 on the CUDA cores; attn_set_path holds here too.
    const bool f32 = dtype == ATTN_F32;
    if (g_path == ATTN_PATH_TENSOR && f32) return ATTN_ERR_UNSUPPORTED;
    pg::DecodeArgs a{g, table, lens, q_len, H, n, d, dv, H / Hkv * n, pg::kRows, 0, causal != 0, scale};
    a.row_tiles = (a.rows + a.tile_rows - 1) / a.tile_rows;      // the kernels' tiles may differ by a factor of 4
    // The kernel numbers its units (key tiles of all items) times CTAs in 64 bits.
    if (4.0 * B * Hkv * a.row_tiles * ((static_cast<double>(max_pages) * page) / pg::kTileKeys + 1 + pg::kItemUnits) >=
        9007199254740992.0)
        return ATTN_ERR_SHAPE;
    const size_t es = dtype == ATTN_F32 ? 4 : 2, rows = static_cast<size_t>(B) * H * n;
    const Region written[] = {{O, rows * dv * es}, {LSE, rows * 4}, {workspace, w.total}};
    const Region read[] = {{Q, rows * d * es}, {K_pages, pool_bytes(g, d, dtype)},
                           {V_pages, pool_bytes(g, dv, dtype)}, {table, static_cast<size_t>(B) * max_pages * 4},
                           {lens, static_cast<size_t>(B) * 4}, {q_len, static_cast<size_t>(B) * 4}};
    if (!apart(written, read, nullptr, 0)) return ATTN_ERR_ALIAS;

    cudaStream_t st = as_stream(stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const pg::Parts parts{reinterpret_cast<float*>(ws + w.o_off), reinterpret_cast<float*>(ws + w.ml_off),
                          reinterpret_cast<pg::Head*>(ws + w.head_off)};
    int grid = 0;
    if (!f32 && g_path == ATTN_PATH_SIMT)
        s = decode_simt(a, Q, K_pages, V_pages, O, LSE, parts, &grid, st);
    else if (d <= 64)
        s = dv <= 64 ? decode_rows<64, 64>(a, Q, K_pages, V_pages, O, LSE, parts, &grid, f32, st)
                     : decode_rows<64, 128>(a, Q, K_pages, V_pages, O, LSE, parts, &grid, f32, st);
    else
        s = dv <= 64 ? decode_rows<128, 64>(a, Q, K_pages, V_pages, O, LSE, parts, &grid, f32, st)
                     : decode_rows<128, 128>(a, Q, K_pages, V_pages, O, LSE, parts, &grid, f32, st);
    const bool join = grid > 0;
    if (s == ATTN_OK && join)
        s = f32 ? decode_join<float>(a, O, LSE, parts, grid, st) : decode_join<__nv_bfloat16>(a, O, LSE, parts, grid, st);
    if (s == ATTN_OK) g_last_launches = join ? 2 : 1;
    return s;
}

size_t attn_cache_workspace_size(int B, int max_pages, int num_pages) {
    if (B < 1 || max_pages < 1 || num_pages < 1 || !books_fit(B, max_pages, num_pages, pg::kMinPageLog2)) return 0;
    return carve_cache(B, max_pages, num_pages).total;
}

attn_status_t attn_cache_append(const void* K, const void* V, void* K_pages, void* V_pages, const int* table,
                                const int* lens, const int* ref, const int* new_len, int* table_out,
                                int* lens_out, int* ref_out, int* info, void* workspace,
                                size_t workspace_bytes, int B, int Hkv, int n, int d, int dv, int num_pages,
                                int page, int max_pages, attn_dtype_t dtype, void* stream) {
    pg::Geometry g;
    attn_status_t s = check_cache(B, Hkv, d, dv, num_pages, page, max_pages, dtype, &g);
    if (s != ATTN_OK) return s;
    // The copy kernel numbers spans of at least one row, of K and of V, below 2^31.
    if (n < 1 || 2.0 * B * Hkv * n >= 2147483648.0) return ATTN_ERR_SHAPE;
    if (!K || !V || !K_pages || !V_pages || !table || !lens || !ref || !table_out || !lens_out || !ref_out || !info)
        return ATTN_ERR_NULL;
    if (!aligned16(K) || !aligned16(V) || !aligned16(K_pages) || !aligned16(V_pages) || !aligned4(table) ||
        !aligned4(lens) || !aligned4(ref) || !aligned4(new_len) || !aligned4(table_out) || !aligned4(lens_out) ||
        !aligned4(ref_out) || !aligned4(info))
        return ATTN_ERR_ALIGN;
    const CacheWorkspace w = carve_cache(B, max_pages, num_pages);
    if (!workspace || workspace_bytes < w.total) return ATTN_ERR_WORKSPACE;
    if (!aligned16(workspace)) return ATTN_ERR_ALIGN;
    const int es = dtype == ATTN_F32 ? 4 : 2;
    const size_t rows = static_cast<size_t>(B) * Hkv * n, tb = static_cast<size_t>(B) * max_pages * 4,
                 lb = static_cast<size_t>(B) * 4, rb = static_cast<size_t>(num_pages) * 4;
    const Region written[] = {{table_out, tb}, {lens_out, lb}, {ref_out, rb}, {info, 12}, {workspace, w.total},
                              {K_pages, pool_bytes(g, d, dtype)}, {V_pages, pool_bytes(g, dv, dtype)}};
    const Region read[] = {{K, rows * d * es}, {V, rows * dv * es}, {new_len, lb}};
    const Region in_place[] = {{table, tb}, {lens, lb}, {ref, rb}};
    if (!apart(written, read, in_place, 3)) return ATTN_ERR_ALIAS;

    cudaStream_t st = as_stream(stream);
    const pg::Books k = books(g, table, lens, ref, table_out, lens_out, ref_out, info, workspace);
    pg::Rows r = pg::Rows::of_new(K_pages, V_pages, d * es / 16, dv * es / 16, B, Hkv, n);
    r.K = static_cast<const uint4*>(K);
    r.V = static_cast<const uint4*>(V);
    r.new_len = new_len;
    const unsigned long long spans = r.flat ? r.spans.d : 1ull * r.spans.d * B * Hkv;
    return books_and_rows(pg::append_books, pg::append_rows, k, r, spans, st, [&](auto kern, const pg::Rows& x) {
        return launch_books(kern, st, k, x);
    });
}

attn_status_t attn_cache_fork(void* K_pages, void* V_pages, const int* table, const int* lens, const int* ref,
                              const int* src, const int* keep, int* table_out, int* lens_out, int* ref_out,
                              int* info, void* workspace, size_t workspace_bytes, int B, int Hkv, int d, int dv,
                              int num_pages, int page, int max_pages, attn_dtype_t dtype, void* stream) {
    pg::Geometry g;
    attn_status_t s = check_cache(B, Hkv, d, dv, num_pages, page, max_pages, dtype, &g);
    if (s != ATTN_OK) return s;
    if (B > (1 << 29)) return ATTN_ERR_SHAPE;              // the kernel ranks sequences up to 2 B
    if (!K_pages || !V_pages || !table || !lens || !ref || !src || !table_out || !lens_out || !ref_out || !info)
        return ATTN_ERR_NULL;
    if (!aligned16(K_pages) || !aligned16(V_pages) || !aligned4(table) || !aligned4(lens) || !aligned4(ref) ||
        !aligned4(src) || !aligned4(keep) || !aligned4(table_out) || !aligned4(lens_out) || !aligned4(ref_out) ||
        !aligned4(info))
        return ATTN_ERR_ALIGN;
    const CacheWorkspace w = carve_cache(B, max_pages, num_pages);
    if (!workspace || workspace_bytes < w.total) return ATTN_ERR_WORKSPACE;
    if (!aligned16(workspace)) return ATTN_ERR_ALIGN;
    const size_t tb = static_cast<size_t>(B) * max_pages * 4, lb = static_cast<size_t>(B) * 4,
                 rb = static_cast<size_t>(num_pages) * 4;
    const Region written[] = {{table_out, tb}, {lens_out, lb}, {ref_out, rb}, {info, 12}, {workspace, w.total},
                              {K_pages, pool_bytes(g, d, dtype)}, {V_pages, pool_bytes(g, dv, dtype)}};
    const Region read[] = {{src, lb}, {keep, lb}};
    const Region in_place[] = {{table, tb}, {lens, lb}, {ref, rb}};
    if (!apart(written, read, in_place, 3)) return ATTN_ERR_ALIAS;

    cudaStream_t st = as_stream(stream);
    const pg::Books k = books(g, table, lens, ref, table_out, lens_out, ref_out, info, workspace);
    const int es = dtype == ATTN_F32 ? 4 : 2;
    const pg::Rows r = pg::Rows::of(K_pages, V_pages, d * es / 16, dv * es / 16, page, Hkv, 1, false);
    return books_and_rows(pg::fork_books, pg::move_rows, k, r, 1ull * B * Hkv * r.spans.d, st,
                          [&](auto kern, const pg::Rows& x) { return launch_books(kern, st, k, src, keep, x); });
}

attn_status_t attn_cache_compact(void* K_pages, void* V_pages, const int* table, const int* lens,
                                 const int* ref, int* table_out, int* ref_out, int* remap, int* info,
                                 void* workspace, size_t workspace_bytes, int B, int Hkv, int d, int dv,
                                 int num_pages, int page, int max_pages, attn_dtype_t dtype, void* stream) {
    pg::Geometry g;
    attn_status_t s = check_cache(B, Hkv, d, dv, num_pages, page, max_pages, dtype, &g);
    if (s != ATTN_OK) return s;
    if (!K_pages || !V_pages || !table || !lens || !ref || !table_out || !ref_out || !remap || !info)
        return ATTN_ERR_NULL;
    if (!aligned16(K_pages) || !aligned16(V_pages) || !aligned4(table) || !aligned4(lens) || !aligned4(ref) ||
        !aligned4(table_out) || !aligned4(ref_out) || !aligned4(remap) || !aligned4(info))
        return ATTN_ERR_ALIGN;
    const CacheWorkspace w = carve_cache(B, max_pages, num_pages);
    if (!workspace || workspace_bytes < w.total) return ATTN_ERR_WORKSPACE;
    if (!aligned16(workspace)) return ATTN_ERR_ALIGN;
    const size_t tb = static_cast<size_t>(B) * max_pages * 4, lb = static_cast<size_t>(B) * 4,
                 rb = static_cast<size_t>(num_pages) * 4;
    const Region written[] = {{table_out, tb}, {ref_out, rb}, {remap, rb}, {info, 12}, {workspace, w.total},
                              {K_pages, pool_bytes(g, d, dtype)}, {V_pages, pool_bytes(g, dv, dtype)}};
    const Region read[] = {{lens, lb}};
    const Region in_place[] = {{table, tb}, {ref, rb}};
    if (!apart(written, read, in_place, 2)) return ATTN_ERR_ALIAS;

    cudaStream_t st = as_stream(stream);
    const pg::Books k = books(g, table, lens, ref, table_out, nullptr, ref_out, info, workspace);
    const int es = dtype == ATTN_F32 ? 4 : 2;
    const pg::Rows r = pg::Rows::of(K_pages, V_pages, d * es / 16, dv * es / 16, page, Hkv, 1, false);
    return books_and_rows(pg::compact_books, pg::move_rows, k, r, 1ull * (num_pages / 2) * Hkv * r.spans.d, st,
                          [&](auto kern, const pg::Rows& x) { return launch_books(kern, st, k, remap, x); });
}

}  // extern "C"
