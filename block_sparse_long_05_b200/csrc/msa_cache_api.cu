// msa_cache_api.cu -- the C ABI of the paged-cache operators (declared in
// include/msa.h): argument validation, workspace layout, tensor maps and
// dispatch.  No computation happens here.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/msa.h"
#include "cache.h"
#include "msa_common.cuh"
#include "tmap.h"

using namespace msa;

namespace {

constexpr size_t kStatusBytes = 256;
static_assert(kWsHeader == MSA_WORKSPACE_HEADER_BYTES, "header documented in msa.h");

struct CacheWs {
    size_t part_o, part_lse, total;
};

CacheWs cache_layout(int d) {
    // pieces of the split kernel, or of the chunk kernel: the calls that launch
    // both run them one after the other
    const size_t split = static_cast<size_t>(2) * kSplitMaxCtas * kSplitMaxRows;
    const size_t chunk = static_cast<size_t>(2) * kChunkMaxCtas * kChunkRows;
    const size_t rows = split > chunk ? split : chunk;
    CacheWs w;
    w.part_o = kWsHeader;
    w.part_lse = align_up(w.part_o + rows * d * 4, 256);
    w.total = align_up(w.part_lse + rows * 4, 256);
    return w;
}

msa_status check_cache(int Hkv, int d, int block, int num_pages) {
    if (Hkv < 1 || d < 1 || block < 1 || num_pages < 1) return MSA_ERR_INVALID_ARG;
    if (!(d == 64 || d == 128)) return MSA_ERR_UNSUPPORTED;
    if (!(block == 32 || block == 64 || block % 128 == 0)) return MSA_ERR_UNSUPPORTED;
    if (static_cast<long long>(num_pages) * block >= (1ll << 31)) return MSA_ERR_UNSUPPORTED;
    return MSA_OK;
}

bool step_fits(int page_stride, int Bt, int total, int block) {
    return static_cast<long long>(page_stride) * block < (1ll << 30) && total < (1 << 30) && Bt < (1 << 24);
}

msa_status check_step(const int32_t *page_table, int page_stride, const int32_t *cu,
                      const int32_t *kv_len, int Bt, int total, int block) {
    if (!page_table || !cu || !kv_len || page_stride < 1 || Bt < 1 || total < 0)
        return MSA_ERR_INVALID_ARG;
    if (!aligned4(page_table) || !aligned4(cu) || !aligned4(kv_len)) return MSA_ERR_INVALID_ARG;
    return step_fits(page_stride, Bt, total, block) ? MSA_OK : MSA_ERR_UNSUPPORTED;
}

msa_status check_ws(const void *ws, size_t bytes, size_t need) {
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255) != 0 || bytes < need)
        return MSA_ERR_WORKSPACE;
    return MSA_OK;
}

// Row stride of a packed bf16 tensor whose rows are read in 16-byte pieces.
bool good_stride(long long stride, long long row) { return stride >= row && stride % 8 == 0; }

StepMap step_of(const int32_t *page_table, int page_stride, int num_pages, const int32_t *cu,
                const int32_t *kv_len, int Bt, int total, int block) {
    StepMap s;
    s.pm = PageMap{page_table, page_stride, num_pages};
    s.cu = cu;
    s.kv_len = kv_len;
    s.Bt = Bt;
    s.total = total;
    s.block = block;
    return s;
}

bool scales_ok(const void *ks, const void *vs) { return ks && vs && aligned16(ks) && aligned16(vs); }

msa_status append_impl(const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                       const void *k_idx, int64_t k_idx_stride, void *k_pages, void *v_pages,
                       float *k_scales, float *v_scales, void *k_idx_pages,
                       const int32_t *page_table, int page_stride, int num_pages,
                       const int32_t *cu, const int32_t *kv_len, int Bt, int total, int Hkv, int d,
                       int d_idx, int block, void *ws, size_t ws_bytes, void *stream, bool i8) {
    if (!k || !v || !k_pages || !v_pages) return MSA_ERR_INVALID_ARG;
    msa_status s = check_cache(Hkv, d, block, num_pages);
    if (s != MSA_OK) return s;
    if ((s = check_step(page_table, page_stride, cu, kv_len, Bt, total, block)) != MSA_OK) return s;
    if (i8 && !scales_ok(k_scales, v_scales)) return MSA_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_pages) || !aligned16(v_pages))
        return MSA_ERR_INVALID_ARG;
    const long long row = static_cast<long long>(Hkv) * d;
    if (!good_stride(k_stride, row) || !good_stride(v_stride, row)) return MSA_ERR_INVALID_ARG;
    if ((k_idx == nullptr) != (k_idx_pages == nullptr)) return MSA_ERR_INVALID_ARG;
    if (k_idx) {
        if (d_idx < 1) return MSA_ERR_INVALID_ARG;
        if (!(d_idx == 64 || d_idx == 128)) return MSA_ERR_UNSUPPORTED;
        if (!aligned16(k_idx) || !aligned16(k_idx_pages) || !good_stride(k_idx_stride, d_idx))
            return MSA_ERR_INVALID_ARG;
    }
    // pieces of the step are numbered with 31 bits
    if (total * (row / 4) >= (1ll << 31)) return MSA_ERR_UNSUPPORTED;
    if ((s = check_ws(ws, ws_bytes, kStatusBytes)) != MSA_OK) return s;
    if (total == 0) return MSA_OK;
    CacheStore c;
    c.k = k_pages;
    c.v = v_pages;
    c.k_scales = i8 ? k_scales : nullptr;
    c.v_scales = i8 ? v_scales : nullptr;
    c.Hkv = Hkv;
    c.d = d;
    const cudaError_t e = launch_kv_append(
        step_of(page_table, page_stride, num_pages, cu, kv_len, Bt, total, block), c, k, k_stride,
        v, v_stride, k_idx, k_idx_stride, k_idx_pages, k_idx ? d_idx : 0, static_cast<int *>(ws),
        static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

msa_status gather_impl(const void *k_pages, const void *v_pages, const float *k_scales,
                       const float *v_scales, const int32_t *page_table, int page_stride,
                       int num_pages, const int32_t *cu, const int32_t *kv_len, void *k, void *v,
                       int Bt, int total, int Hkv, int d, int block, void *ws, size_t ws_bytes,
                       void *stream, bool i8) {
    if (!k || !v || !k_pages || !v_pages) return MSA_ERR_INVALID_ARG;
    msa_status s = check_cache(Hkv, d, block, num_pages);
    if (s != MSA_OK) return s;
    if ((s = check_step(page_table, page_stride, cu, kv_len, Bt, total, block)) != MSA_OK) return s;
    if (i8 && !scales_ok(k_scales, v_scales)) return MSA_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_pages) || !aligned16(v_pages))
        return MSA_ERR_INVALID_ARG;
    if (total * (static_cast<long long>(Hkv) * d / 4) >= (1ll << 31)) return MSA_ERR_UNSUPPORTED;
    if ((s = check_ws(ws, ws_bytes, kStatusBytes)) != MSA_OK) return s;
    if (total == 0) return MSA_OK;
    CacheStore c;
    c.k = const_cast<void *>(k_pages);
    c.v = const_cast<void *>(v_pages);
    c.k_scales = i8 ? const_cast<float *>(k_scales) : nullptr;
    c.v_scales = i8 ? const_cast<float *>(v_scales) : nullptr;
    c.Hkv = Hkv;
    c.d = d;
    const cudaError_t e =
        launch_kv_gather(step_of(page_table, page_stride, num_pages, cu, kv_len, Bt, total, block),
                         c, k, v, static_cast<int *>(ws), static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

// K or V tensor map over a page store: rows of all pages, `box_rows` rows of
// one head per box (64 bf16 or a whole row of codes wide).
bool store_map(CUtensorMap *m, const void *pages, int num_pages, int block, int Hkv, int d,
               int box_rows, bool i8) {
    const int eb = i8 ? 1 : 2;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(Hkv),
                                static_cast<cuuint64_t>(num_pages) * block};
    const cuuint64_t str[2] = {static_cast<cuuint64_t>(d) * eb, static_cast<cuuint64_t>(Hkv) * d * eb};
    const cuuint32_t box[3] = {i8 ? static_cast<cuuint32_t>(d) : 64u, 1u, static_cast<cuuint32_t>(box_rows)};
    return make_tmap(m, pages, 3, dims, str, box,
                     i8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                     i8 && d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

// Which kernels take a step: the split one, the chunk one, or in a batch the
// chunk kernel the sequences with more than kSplitMaxRows rows (tokens * G) and
// the split kernel the others.  It depends on these sizes alone, and only on
// those that the host knows; the lengths are in device memory.
struct Choice {
    bool chunk;
    int rows;         // rows of a sequence and kv head, for the split kernel
    long long tiles;  // row tiles of the split kernel, at most
    long long keys;   // key tiles of a row tile, at most
};
// max_q: rows of the longest sequence, as far as the caller knows.  span: keys
// of a context, as wide as its page-table row (or the selected blocks).
Choice choose(int Bt, int total, int max_q, int G, int Hkv, long long span, int window, int sinks,
              bool sparse) {
    Choice c;
    // (a hint below the average is wrong)
    const long long mean = (static_cast<long long>(total) + Bt - 1) / Bt;
    const long long most = (max_q > mean ? max_q : mean) * G;
    c.rows = most <= kSplitMaxRows ? static_cast<int>(most) : kSplitMaxRows + 1;
    c.keys = span / kSplitKeys + 1;
    const long long near = (static_cast<long long>(window) + sinks) / kSplitKeys + 4;
    if (window && c.keys > near) c.keys = near;
    c.tiles = static_cast<long long>(total) * G / kSplitMaxRows + Bt;
    // Sequences with many rows go to the chunk kernel, unless the whole step is
    // small: it takes 14 us or more where the split kernel, 16 rows at a time, has
    // done with a few hundred tiles.  Measured with page tables as wide as the
    // contexts (bf16, d 128, G 4; split against chunk): 64 rows over 500 keys, 8 kv
    // heads: 14 / 23 us; 20 over 2000: 26 / 27; 200 over 200: 21 / 20; 500 over 500,
    // 2 kv heads: 18 / 24, 8 kv heads: 53 / 25; 64 over 4000: 45 / 38.  (Behind a wider
    // table the same contexts count as longer ones, and their steps go to the chunk
    // kernel earlier.)  A hint that is too low costs time, not rows.
    c.chunk = c.rows > kSplitMaxRows && !sparse && c.tiles * Hkv * (c.keys + 2) > 1536;
    return c;
}

// Shared by the dense and the sparse entry: `a` has everything but the
// workspace regions and the scale of the scores.
// max_q: rows of the longest sequence, as far as the caller knows.
msa_status attend(PagedAttn &a, const void *k_pages, const void *v_pages, int num_pages, int max_q,
                  void *ws, void *stream) {
    const CacheWs L = cache_layout(a.c.d);
    unsigned char *base = static_cast<unsigned char *>(ws);
    a.part_o = reinterpret_cast<float *>(base + L.part_o);
    a.part_lse = reinterpret_cast<float *>(base + L.part_lse);
    a.counters = reinterpret_cast<int *>(base + kStatusBytes);
    a.status = static_cast<int *>(ws);
    a.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(a.c.d));
    const int sms = num_sms_current();
    if (sms <= 0) return MSA_ERR_CUDA;
    const bool i8 = a.c.k_scales != nullptr;
    // kv heads whose CTAs share a run: as many as may be; `all`: so that none of
    // that many CTAs is left over, if several can (chunks of 8 kv heads on 148 SMs:
    // 8 heads in step, on 144, took 2% longer than 4; one by itself 9% with int8)
    auto share = [&](int all) {
        int most = 1, even = 1;
        for (int h = 1; h <= a.c.Hkv && h <= kSplitMaxHeads; ++h) {
            if (a.c.Hkv % h) continue;
            most = h;
            if (all % h == 0) even = h;
        }
        a.heads = even > 1 ? even : most;
        a.groups = a.c.Hkv / a.heads;
    };
    a.by_g = Divisor(a.G);
    a.by_block = Divisor(a.step.block);
    const int box = split_box_rows(a.step.block);
    CUtensorMap tk, tv;
    if (!store_map(&tk, k_pages, num_pages, a.step.block, a.c.Hkv, a.c.d, box, i8) ||
        !store_map(&tv, v_pages, num_pages, a.step.block, a.c.Hkv, a.c.d, box, i8))
        return MSA_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const long long span = a.ids ? static_cast<long long>(a.K) * a.step.block
                                 : static_cast<long long>(a.step.pm.stride) * a.step.block;
    const Choice how = choose(a.step.Bt, a.step.total, max_q, a.G, a.c.Hkv, span, a.window, a.sinks,
                              a.ids != nullptr);
    const bool chunk = how.chunk;
    share(chunk ? sms : 0);
    // work units are numbered with 31 bits
    const long long all = static_cast<long long>(a.step.total) * a.G;
    const long long row_tiles = chunk ? all / kChunkRows + 2ll * a.step.Bt : 2 * how.tiles;
    if (row_tiles * a.groups * (how.keys + 8) >= (1ll << 31)) return MSA_ERR_UNSUPPORTED;
    cudaError_t e = cudaSuccess;
    if (chunk) {
        a.row_lo = a.step.Bt > 1 ? kSplitMaxRows + 1 : 0;
        e = launch_chunk_attn(a, tk, tv, sms, st);
        a.row_lo = 0;
        a.row_hi = kSplitMaxRows;
        share(0);
    }
    if (e == cudaSuccess && (!chunk || a.step.Bt > 1))
        e = launch_split_attn(a, how.rows, tk, tv, sms, st);
    return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

// (positions stay below 2^30, so a longer window hides nothing)
int clamp_window(int window) { return window < (1 << 30) ? window : 1 << 30; }
int clamp_sinks(int window, int sinks) { return !window ? 0 : sinks < (1 << 30) ? sinks : 1 << 30; }
// Without a hint one sequence may have all the rows.
int known_rows(int max_q, int total) { return max_q > 0 && max_q < total ? max_q : total; }

msa_status attn_impl(const void *q, int64_t q_stride, const void *k_pages, const void *v_pages,
                     const float *k_scales, const float *v_scales, const int32_t *page_table,
                     int page_stride, int num_pages, const int32_t *cu, const int32_t *kv_len,
                     void *out, float *lse, int Bt, int total, int max_q, int Hq, int Hkv, int d,
                     int block, int window, int sinks, void *ws, size_t ws_bytes, void *stream,
                     bool i8) {
    if (!q || !k_pages || !v_pages || !out || !lse) return MSA_ERR_INVALID_ARG;
    msa_status s = check_cache(Hkv, d, block, num_pages);
    if (s != MSA_OK) return s;
    if (Hq < 1 || Hq % Hkv != 0 || max_q < 0 || window < 0 || sinks < 0) return MSA_ERR_INVALID_ARG;
    if ((s = check_step(page_table, page_stride, cu, kv_len, Bt, total, block)) != MSA_OK) return s;
    if (i8 && !scales_ok(k_scales, v_scales)) return MSA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out) || !aligned4(lse))
        return MSA_ERR_INVALID_ARG;
    if (!good_stride(q_stride, static_cast<long long>(Hq) * d)) return MSA_ERR_INVALID_ARG;
    if (static_cast<long long>(total) * Hq >= (1ll << 31)) return MSA_ERR_UNSUPPORTED;
    if ((s = check_ws(ws, ws_bytes, cache_layout(d).total)) != MSA_OK) return s;
    if (total == 0) return MSA_OK;
    PagedAttn a;
    a.step = step_of(page_table, page_stride, num_pages, cu, kv_len, Bt, total, block);
    a.c.k_scales = i8 ? const_cast<float *>(k_scales) : nullptr;
    a.c.v_scales = i8 ? const_cast<float *>(v_scales) : nullptr;
    a.c.Hkv = Hkv;
    a.c.d = d;
    a.q = q;
    a.q_stride = q_stride;
    a.out = out;
    a.lse = lse;
    a.Hq = Hq;
    a.G = Hq / Hkv;
    a.window = clamp_window(window);
    a.sinks = clamp_sinks(window, sinks);
    return attend(a, k_pages, v_pages, num_pages, known_rows(max_q, total), ws, stream);
}

}  // namespace

extern "C" {

size_t msa_cache_workspace_size(int Hq, int Hkv, int d) {
    if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || !(d == 64 || d == 128)) return 0;
    return cache_layout(d).total;
}

msa_status msa_kv_append(const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                         const void *k_idx, int64_t k_idx_stride, void *k_pages, void *v_pages,
                         void *k_idx_pages, const int32_t *page_table, int page_stride,
                         int num_pages, const int32_t *cu, const int32_t *kv_len, int Bt,
                         int total, int Hkv, int d, int d_idx, int block, void *workspace,
                         size_t workspace_bytes, void *stream) {
    return append_impl(k, k_stride, v, v_stride, k_idx, k_idx_stride, k_pages, v_pages, nullptr,
                       nullptr, k_idx_pages, page_table, page_stride, num_pages, cu, kv_len, Bt,
                       total, Hkv, d, d_idx, block, workspace, workspace_bytes, stream, false);
}

msa_status msa_kv_append_i8(const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                            const void *k_idx, int64_t k_idx_stride, int8_t *k_pages,
                            int8_t *v_pages, float *k_scales, float *v_scales, void *k_idx_pages,
                            const int32_t *page_table, int page_stride, int num_pages,
                            const int32_t *cu, const int32_t *kv_len, int Bt, int total, int Hkv,
                            int d, int d_idx, int block, void *workspace, size_t workspace_bytes,
                            void *stream) {
    return append_impl(k, k_stride, v, v_stride, k_idx, k_idx_stride, k_pages, v_pages, k_scales,
                       v_scales, k_idx_pages, page_table, page_stride, num_pages, cu, kv_len, Bt,
                       total, Hkv, d, d_idx, block, workspace, workspace_bytes, stream, true);
}

msa_status msa_kv_gather(const void *k_pages, const void *v_pages, const int32_t *page_table,
                         int page_stride, int num_pages, const int32_t *cu, const int32_t *kv_len,
                         void *k, void *v, int Bt, int total, int Hkv, int d, int block,
                         void *workspace, size_t workspace_bytes, void *stream) {
    return gather_impl(k_pages, v_pages, nullptr, nullptr, page_table, page_stride, num_pages, cu,
                       kv_len, k, v, Bt, total, Hkv, d, block, workspace, workspace_bytes, stream,
                       false);
}

msa_status msa_kv_gather_i8(const int8_t *k_pages, const int8_t *v_pages, const float *k_scales,
                            const float *v_scales, const int32_t *page_table, int page_stride,
                            int num_pages, const int32_t *cu, const int32_t *kv_len, void *k,
                            void *v, int Bt, int total, int Hkv, int d, int block, void *workspace,
                            size_t workspace_bytes, void *stream) {
    return gather_impl(k_pages, v_pages, k_scales, v_scales, page_table, page_stride, num_pages,
                       cu, kv_len, k, v, Bt, total, Hkv, d, block, workspace, workspace_bytes,
                       stream, true);
}

int msa_attn_paged_kernels(int Bt, int total, int max_q, int Hq, int Hkv, int block,
                           int page_stride, int window, int sinks) {
    if (Bt < 1 || total < 1 || max_q < 0 || Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || page_stride < 1 ||
        window < 0 || sinks < 0 || check_cache(Hkv, 128, block, 1) != MSA_OK ||
        !step_fits(page_stride, Bt, total, block) || static_cast<long long>(total) * Hq >= (1ll << 31))
        return 0;
    const Choice c = choose(Bt, total, known_rows(max_q, total), Hq / Hkv, Hkv,
                            static_cast<long long>(page_stride) * block, clamp_window(window),
                            clamp_sinks(window, sinks), false);
    return (!c.chunk || Bt > 1 ? MSA_KERNEL_SPLIT : 0) | (c.chunk ? MSA_KERNEL_CHUNK : 0);
}

msa_status msa_attn_paged(const void *q, int64_t q_stride, const void *k_pages,
                          const void *v_pages, const int32_t *page_table, int page_stride,
                          int num_pages, const int32_t *cu, const int32_t *kv_len, void *out,
                          float *lse, int Bt, int total, int max_q, int Hq, int Hkv, int d,
                          int block, int window, int sinks, void *workspace,
                          size_t workspace_bytes, void *stream) {
    return attn_impl(q, q_stride, k_pages, v_pages, nullptr, nullptr, page_table, page_stride,
                     num_pages, cu, kv_len, out, lse, Bt, total, max_q, Hq, Hkv, d, block, window,
                     sinks, workspace, workspace_bytes, stream, false);
}

msa_status msa_attn_paged_i8(const void *q, int64_t q_stride, const int8_t *k_pages,
                             const int8_t *v_pages, const float *k_scales, const float *v_scales,
                             const int32_t *page_table, int page_stride, int num_pages,
                             const int32_t *cu, const int32_t *kv_len, void *out, float *lse,
                             int Bt, int total, int max_q, int Hq, int Hkv, int d, int block,
                             int window, int sinks, void *workspace, size_t workspace_bytes,
                             void *stream) {
    return attn_impl(q, q_stride, k_pages, v_pages, k_scales, v_scales, page_table, page_stride,
                     num_pages, cu, kv_len, out, lse, Bt, total, max_q, Hq, Hkv, d, block, window,
                     sinks, workspace, workspace_bytes, stream, true);
}

msa_status msa_sparse_attn_paged_i8(const void *q, const int8_t *k_pages, const int8_t *v_pages,
                                    const float *k_scales, const float *v_scales,
                                    const int32_t *page_table, int page_stride, int num_pages,
                                    const int32_t *ids, void *out, float *lse, int Bt, int T,
                                    int Hq, int Hkv, int d, int block, int K, void *workspace,
                                    size_t workspace_bytes, void *stream) {
    if (!q || !k_pages || !v_pages || !page_table || !ids || !out || !lse)
        return MSA_ERR_INVALID_ARG;
    msa_status s = check_cache(Hkv, d, block, num_pages);
    if (s != MSA_OK) return s;
    if (Hq < 1 || Hq % Hkv != 0 || Bt < 1 || T < 1 || K < 1 || page_stride < 1)
        return MSA_ERR_INVALID_ARG;
    if (page_stride < (static_cast<long long>(T) + block - 1) / block) return MSA_ERR_INVALID_ARG;
    if (K > kMaxK || T >= (1 << 30) || static_cast<long long>(K) * block >= (1ll << 30) ||
        static_cast<long long>(Bt) * Hq >= (1ll << 31))
        return MSA_ERR_UNSUPPORTED;
    if (!scales_ok(k_scales, v_scales) || !aligned16(q) || !aligned16(k_pages) ||
        !aligned16(v_pages) || !aligned16(out) || !aligned4(lse) || !aligned4(ids) ||
        !aligned4(page_table))
        return MSA_ERR_INVALID_ARG;
    if ((s = check_ws(workspace, workspace_bytes, cache_layout(d).total)) != MSA_OK) return s;
    PagedAttn a;
    a.step = step_of(page_table, page_stride, num_pages, nullptr, nullptr, Bt, Bt, block);
    a.c.k_scales = const_cast<float *>(k_scales);
    a.c.v_scales = const_cast<float *>(v_scales);
    a.c.Hkv = Hkv;
    a.c.d = d;
    a.q = q;
    a.q_stride = static_cast<long long>(Hq) * d;
    a.out = out;
    a.lse = lse;
    a.Hq = Hq;
    a.G = Hq / Hkv;
    a.ids = ids;
    a.K = K;
    a.T = T;
    return attend(a, k_pages, v_pages, num_pages, 1, workspace, stream);
}

}  // extern "C"
