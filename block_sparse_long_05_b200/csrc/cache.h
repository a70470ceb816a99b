// cache.h -- internal launchers of the paged-cache operators (append, gather,
// attention over pages).  Not part of the ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "msa_common.cuh"

namespace msa {

// One step of a batch: packed rows cu[b] .. cu[b+1]-1 belong to sequence b,
// the i-th of them at position kv_len[b] - (cu[b+1] - cu[b]) + i of its
// context.  All arrays are in device memory, so a captured step follows the
// lengths that the buffers hold when it is replayed.
struct StepMap {
    PageMap pm;
    const int32_t *cu = nullptr;      // [Bt + 1]
    const int32_t *kv_len = nullptr;  // [Bt]
    int Bt = 0;
    int total = 0;  // packed rows in the buffers (>= cu[Bt])
    int block = 0;
};

// Page stores of one cache.  Scales (8-bit codes only): fp32 [pages][Hkv][block].
struct CacheStore {
    void *k = nullptr, *v = nullptr;
    float *k_scales = nullptr, *v_scales = nullptr;  // nullptr: bf16 values
    int Hkv = 0, d = 0;
};

// New rows (bf16, [total] rows of Hkv * d values every k_stride / v_stride
// elements) into the pages, with index keys [total][d_idx] where d_idx > 0.
cudaError_t launch_kv_append(const StepMap &step, const CacheStore &c, const void *k,
                             long long k_stride, const void *v, long long v_stride,
                             const void *k_idx, long long k_idx_stride, void *k_idx_pages,
                             int d_idx, int *status, cudaStream_t st);
// Cached rows back to packed bf16 [total][Hkv][d].
cudaError_t launch_kv_gather(const StepMap &step, const CacheStore &c, void *k_out, void *v_out,
                             int *status, cudaStream_t st);

// Division of n < 2^31 by a number that the host knows.
struct Divisor {
    uint32_t d, mul, shift;
    explicit Divisor(uint32_t by = 1) : d(by), mul(0), shift(0) {
        while (shift < 31 && (1u << shift) < by) ++shift;
        // ceil(2^(31 + shift) / by): exact quotients below 2^31
        mul = static_cast<uint32_t>(((1ull << (31 + shift)) + by - 1) / by);
    }
    __host__ __device__ __forceinline__ uint32_t quotient(uint32_t n) const {
        return static_cast<uint32_t>((static_cast<uint64_t>(n) * mul) >> 31 >> shift);
    }
};

// Attention over pages.
struct PagedAttn {
    StepMap step;
    CacheStore c;
    const void *q = nullptr;
    long long q_stride = 0;  // elements between packed rows of q
    void *out = nullptr;     // bf16 [total][Hq][d]
    float *lse = nullptr;    // fp32 [total][Hq]
    int Hq = 0, G = 0;
    int heads = 1;           // kv heads that share a run of key tiles (divides Hkv)
    int groups = 1;          // Hkv / heads
    Divisor by_g, by_block;  // G, rows per page
    int row_lo = 0, row_hi = 0x7FFFFFFF;  // rows (tokens * G) of the sequences that a launch takes
    int window = 0, sinks = 0;       // window 0: every key up to the query's position
    const int32_t *ids = nullptr;    // sparse branch: [Bt][K] selected blocks (one row each)
    int K = 0, T = 0;                // sparse branch: selection width, common length
    float scale_log2 = 0.f;          // log2(e) / sqrt(d)
    float *part_o = nullptr;         // split pieces, fp32 [pieces][rows][d]
    float *part_lse = nullptr;       // their log2-domain lse [pieces][rows]
    int *counters = nullptr;         // finished pieces per run: zero between calls
    int *status = nullptr;
};

constexpr int kSplitKeys = 128;      // keys per tile of the split kernel
constexpr int kSplitMaxRows = 16;    // query rows per tile, at most
constexpr int kSplitMaxCtas = kWsCounters;  // CTAs of the split kernel (workspace bound)
constexpr int kSplitMaxHeads = 16;   // kv heads whose CTAs share a run of key tiles, at most

// Rows of the K / V tensor map boxes of the split kernel.
inline int split_box_rows(int block) { return block < kSplitKeys ? block : kSplitKeys; }
// rows: query rows that a (sequence, kv head) pair has, as far as the caller
// knows; it chooses the tile height.
cudaError_t launch_split_attn(const PagedAttn &a, int rows, const CUtensorMap &tk,
                              const CUtensorMap &tv, int num_sms, cudaStream_t st);

constexpr int kChunkRows = 256;     // query rows per CTA of the chunk kernel
constexpr int kChunkMaxCtas = 256;  // its CTAs, at most (workspace bound)
cudaError_t launch_chunk_attn(const PagedAttn &a, const CUtensorMap &tk, const CUtensorMap &tv,
                              int num_sms, cudaStream_t st);

}  // namespace msa
