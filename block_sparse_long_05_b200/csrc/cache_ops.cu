// cache_ops.cu -- writing the paged cache and reading it back.
//
//   append  bf16:  page row <- new row
//           int8:  per (token, kv head) row x of d values, in fp32:
//                      amax = max |x_i|,  inv = 127 / amax,
//                      code_i = rint(x_i * inv),  scale = amax / 127
//                  so the row reads back as code_i * scale with an error of at
//                  most half a step, amax / 254 (and the rounding of inv).
//                  A row whose amax is below 2^-100 is stored as zeros (127 /
//                  amax would overflow); a row that holds an infinity or a NaN
//                  is stored with codes 0 and scale NaN, so that it reads back
//                  as NaN instead of as values that look sound.
//   gather  packed bf16 rows <- code_i * scale, rounded once (int8), or a copy.
//
// Both are bound by HBM: bytes per value are 2 + 1 (int8) or 2 + 2 (bf16).
// A thread moves 16-byte pieces and issues kPieces loads before it uses any;
// the page of each token is looked up once per token of the CTA's run, into
// shared memory, while those loads are in flight.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cache.h"
#include "msa_common.cuh"

namespace msa {

namespace {

constexpr int kThreads = 256;
constexpr int kPieces = 4;                       // 16-byte pieces per thread
constexpr int kRun = kThreads * kPieces;         // pieces per CTA
constexpr int kMaxTokens = kRun / 8 + 2;         // tokens that a run touches (>= 8 pieces each)
constexpr float kTiny = 7.888609e-31f;           // 2^-100

// Page (x) and row in the page (y) that packed row `tok` maps to.  x = -1:
// none, the row lies behind the last sequence; -2: none, its position is
// below 0 or no such page exists (the latter is reported).
__device__ __forceinline__ int2 store_row(const StepMap &s, int tok, int *status) {
    int lo = 0, hi = s.Bt;  // first b with cu[b + 1] > tok
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s.cu[mid + 1] > tok)
            hi = mid;
        else
            lo = mid + 1;
    }
    if (lo >= s.Bt || tok < s.cu[lo]) return make_int2(-1, 0);
    const long long pos = static_cast<long long>(s.kv_len[lo]) - s.cu[lo + 1] + tok;
    if (pos < 0) return make_int2(-2, 0);
    const long long j = pos / s.block;
    int page = -1;
    if (j < s.pm.stride) page = s.pm.table[static_cast<long long>(lo) * s.pm.stride + j];
    if (page < 0 || page >= s.pm.count) {
        atomicOr(status, kDevBadIds);
        return make_int2(-2, 0);
    }
    return make_int2(page, static_cast<int>(pos - j * s.block));
}

__device__ __forceinline__ uint4 ld_once(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ void unpack8(const uint4 &u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

struct AppendArgs {
    StepMap step;
    CacheStore c;
    const __nv_bfloat16 *k, *v, *k_idx;
    long long k_stride, v_stride, k_idx_stride;
    __nv_bfloat16 *k_idx_pages;
    int d_idx;
    int kv_ctas;  // CTAs of K and V; those behind them copy index keys
    int *status;
};

// PPR: 16-byte pieces per (token, head) row of bf16.  A piece's place in the
// step is ((token * 2 + {K, V}) * Hkv + head) * PPR + piece, so a warp holds
// whole rows and reduces amax over PPR lanes.
template <int PPR, bool I8>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const AppendArgs a) {
    __shared__ int2 dest[kMaxTokens];
    const int tid = threadIdx.x;
    const bool index = static_cast<int>(blockIdx.x) >= a.kv_ctas;
    // (the host keeps the number of pieces below 2^31)
    const uint32_t run = (blockIdx.x - (index ? a.kv_ctas : 0)) * kRun;
    const uint32_t ppt = index ? a.d_idx / 8 : 2 * a.c.Hkv * PPR;  // pieces per token
    const uint32_t total = a.step.total * ppt;
    const int tok0 = static_cast<int>(run / ppt);
    const int ntok = static_cast<int>((min(run + kRun, total) - 1) / ppt) - tok0 + 1;
    uint4 x[kPieces];
    int tok[kPieces], rem[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const uint32_t e = run + i * kThreads + tid;
        tok[i] = -1;
        rem[i] = 0;
        x[i] = make_uint4(0, 0, 0, 0);
        if (e >= total) continue;
        tok[i] = static_cast<int>(e / ppt);
        rem[i] = static_cast<int>(e % ppt);
        if (index) {
            x[i] = ld_once(a.k_idx + tok[i] * a.k_idx_stride + rem[i] * 8);
        } else {
            const int half = a.c.Hkv * PPR;
            x[i] = rem[i] < half ? ld_once(a.k + tok[i] * a.k_stride + rem[i] * 8)
                                 : ld_once(a.v + tok[i] * a.v_stride + (rem[i] - half) * 8);
        }
    }
    for (int t = tid; t < ntok; t += kThreads) dest[t] = store_row(a.step, tok0 + t, a.status);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const int2 to = tok[i] >= 0 ? dest[tok[i] - tok0] : make_int2(-1, 0);
        const bool keep = to.x >= 0;
        const long long row = static_cast<long long>(to.x) * a.step.block + to.y;
        if (index) {
            if (keep)
                *reinterpret_cast<uint4 *>(a.k_idx_pages + row * a.d_idx + rem[i] * 8) = x[i];
            continue;
        }
        const int half = a.c.Hkv * PPR;
        const bool is_v = rem[i] >= half;
        const int hp = is_v ? rem[i] - half : rem[i];  // head * PPR + piece
        void *pages = is_v ? a.c.v : a.c.k;
        if (!I8) {
            if (keep) reinterpret_cast<uint4 *>(pages)[row * half + hp] = x[i];
            continue;
        }
        // |x| as 15-bit patterns order like the values, infinities and NaN on top
        uint32_t m = __vmaxu2(__vmaxu2(x[i].x & 0x7FFF7FFFu, x[i].y & 0x7FFF7FFFu),
                              __vmaxu2(x[i].z & 0x7FFF7FFFu, x[i].w & 0x7FFF7FFFu));
#pragma unroll
        for (int o = 1; o < PPR; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const uint32_t top = max(m & 0xFFFFu, m >> 16) << 16;
        const float amax = __uint_as_float(top);
        const bool bad = top >= 0x7F800000u, tiny = amax < kTiny;
        const float inv = bad || tiny ? 0.f : __fdiv_rn(127.f, amax);
        float f[8];
        unpack8(x[i], f);
        uint32_t w[2] = {0, 0};
        if (!bad) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                w[e / 4] |= (static_cast<uint32_t>(__float2int_rn(f[e] * inv)) & 0xFFu) << (8 * (e % 4));
        }
        if (keep) {
            reinterpret_cast<uint2 *>(pages)[row * half + hp] = make_uint2(w[0], w[1]);
            if (hp % PPR == 0) {
                float *scales = is_v ? a.c.v_scales : a.c.k_scales;
                scales[(static_cast<long long>(to.x) * a.c.Hkv + hp / PPR) * a.step.block + to.y] =
                    bad ? __uint_as_float(0x7FC00000u) : tiny ? 0.f : __fdiv_rn(amax, 127.f);
            }
        }
    }
}

struct GatherArgs {
    StepMap step;
    CacheStore c;
    void *k_out, *v_out;
    int *status;
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// PPR: 16-byte pieces per cached (token, head) row.
template <int PPR, bool I8>
__global__ void __launch_bounds__(kThreads) kv_gather_kernel(const GatherArgs a) {
    __shared__ int2 src[kMaxTokens];
    const int tid = threadIdx.x;
    const uint32_t half = a.c.Hkv * PPR, ppt = 2 * half;
    const uint32_t run = blockIdx.x * kRun;  // (the host keeps the number of pieces below 2^31)
    const uint32_t total = a.step.total * ppt;
    const int tok0 = static_cast<int>(run / ppt);
    const int ntok = static_cast<int>((min(run + kRun, total) - 1) / ppt) - tok0 + 1;
    for (int t = tid; t < ntok; t += kThreads) src[t] = store_row(a.step, tok0 + t, a.status);
    __syncthreads();
    uint4 x[kPieces];
    float s[kPieces];
    uint4 *to[kPieces];  // nullptr: not written
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const uint32_t e = run + i * kThreads + tid;
        x[i] = make_uint4(0, 0, 0, 0);
        s[i] = 0.f;
        to[i] = nullptr;
        if (e >= total) continue;
        const uint32_t tok = e / ppt, rem = e % ppt;
        const int2 from = src[tok - tok0];
        if (from.x == -1) continue;  // behind the last sequence: left as it is
        const bool is_v = rem >= half;
        const uint32_t hp = is_v ? rem - half : rem;  // head * PPR + piece
        to[i] = reinterpret_cast<uint4 *>(is_v ? a.v_out : a.k_out) +
                (static_cast<long long>(tok) * half + hp) * (I8 ? 2 : 1);
        if (from.x < 0) continue;  // no such position or page: zeros
        const long long row = static_cast<long long>(from.x) * a.step.block + from.y;
        x[i] = ld_once(reinterpret_cast<const uint4 *>(is_v ? a.c.v : a.c.k) + row * half + hp);
        if (I8)
            s[i] = (is_v ? a.c.v_scales : a.c.k_scales)
                [(static_cast<long long>(from.x) * a.c.Hkv + hp / PPR) * a.step.block + from.y];
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        if (!to[i]) continue;
        if (!I8) {
            *to[i] = x[i];
            continue;
        }
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t o[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float f[4];
#pragma unroll
            for (int b = 0; b < 4; ++b)
                f[b] = static_cast<float>(static_cast<int8_t>(w[q] >> (8 * b))) * s[i];
            o[2 * q] = pack2(f[0], f[1]);
            o[2 * q + 1] = pack2(f[2], f[3]);
        }
        to[i][0] = make_uint4(o[0], o[1], o[2], o[3]);
        to[i][1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

unsigned runs(long long pieces) { return static_cast<unsigned>((pieces + kRun - 1) / kRun); }

}  // namespace

cudaError_t launch_kv_append(const StepMap &step, const CacheStore &c, const void *k,
                             long long k_stride, const void *v, long long v_stride,
                             const void *k_idx, long long k_idx_stride, void *k_idx_pages,
                             int d_idx, int *status, cudaStream_t st) {
    AppendArgs a;
    a.step = step;
    a.c = c;
    a.k = static_cast<const __nv_bfloat16 *>(k);
    a.v = static_cast<const __nv_bfloat16 *>(v);
    a.k_idx = static_cast<const __nv_bfloat16 *>(k_idx);
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.k_idx_stride = k_idx_stride;
    a.k_idx_pages = static_cast<__nv_bfloat16 *>(k_idx_pages);
    a.d_idx = d_idx;
    a.status = status;
    a.kv_ctas = static_cast<int>(runs(static_cast<long long>(step.total) * 2 * c.Hkv * (c.d / 8)));
    const unsigned grid = a.kv_ctas + (d_idx ? runs(static_cast<long long>(step.total) * (d_idx / 8)) : 0u);
    if (c.d == 128) {
        if (c.k_scales) kv_append_kernel<16, true><<<grid, kThreads, 0, st>>>(a);
        else kv_append_kernel<16, false><<<grid, kThreads, 0, st>>>(a);
    } else {
        if (c.k_scales) kv_append_kernel<8, true><<<grid, kThreads, 0, st>>>(a);
        else kv_append_kernel<8, false><<<grid, kThreads, 0, st>>>(a);
    }
    return cudaGetLastError();
}

cudaError_t launch_kv_gather(const StepMap &step, const CacheStore &c, void *k_out, void *v_out,
                             int *status, cudaStream_t st) {
    GatherArgs a;
    a.step = step;
    a.c = c;
    a.k_out = k_out;
    a.v_out = v_out;
    a.status = status;
    const int ppr = c.d * (c.k_scales ? 1 : 2) / 16;
    const unsigned grid = runs(static_cast<long long>(step.total) * 2 * c.Hkv * ppr);
    if (c.k_scales) {
        if (c.d == 128) kv_gather_kernel<8, true><<<grid, kThreads, 0, st>>>(a);
        else kv_gather_kernel<4, true><<<grid, kThreads, 0, st>>>(a);
    } else {
        if (c.d == 128) kv_gather_kernel<16, false><<<grid, kThreads, 0, st>>>(a);
        else kv_gather_kernel<8, false><<<grid, kThreads, 0, st>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace msa
