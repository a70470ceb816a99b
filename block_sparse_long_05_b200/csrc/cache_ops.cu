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
// HBM is what bounds them at best: bytes per value are 2 + 1 (int8) or 2 + 2
// (bf16).  To get there they must be lean: at 6.5 TB/s an SM has about four issue slots per
// 32 values.  A thread moves units of 16 bytes of the store: 8 bf16 values, or
// 16 codes.  Values become codes and codes values by adding a power of two
// whose last mantissa bit counts 1, so that no conversion instruction (a quarter
// of the rate) is needed.  The page of each token is looked up once per token of
// the CTA's run, into shared memory.  Measured: int8 append of 22190 rows (8
// heads, d 128) 32 us = 4.7 TB/s, int8 gather of 131072 rows 134 us = 6.1 TB/s
// in a replayed graph (151 us where its 32 bytes per thread are stored as two
// halves, as for outputs that do not begin on 32 bytes; the append's loads gain
// nothing from it).  The append does not get there at that size: 67% of the issue
// slots are taken, and its warps wait longest at the barrier behind the look-up
// of their rows.  One or four units of codes per thread, or pairs of lanes that
// read 32 bytes side by side and exchange them in registers, were slower.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cache.h"
#include "msa_common.cuh"
#include "ptx_sm100.cuh"

namespace msa {

namespace {

constexpr int kThreads = 256;
template <bool I8>
struct Units {
    static constexpr int VALUES = I8 ? 16 : 8;          // of a unit
    static constexpr int PER = I8 ? 2 : 4;              // units per thread
    static constexpr int RUN = kThreads * PER;          // units per CTA
    static constexpr int TOKENS = RUN / (64 / VALUES) + 2;  // tokens that a run touches, at most
};
constexpr float kTiny = 7.888609e-31f;           // 2^-100
constexpr float kMagic = 12582912.f;             // 1.5 * 2^23

// The step's row offsets in shared memory, unless there are too many: a
// search for a row's sequence is then a chain of shared-memory reads, not of
// trips to L2 (which made an append of 22 K rows twice as long).
constexpr int kSharedSeqs = 1024;
__device__ __forceinline__ const int32_t *share_offsets(const StepMap &s, int32_t *sh) {
    if (s.Bt > kSharedSeqs) return s.cu;
    for (int i = threadIdx.x; i <= s.Bt; i += kThreads) sh[i] = s.cu[i];
    __syncthreads();
    return sh;
}

// Page (x) and row in the page (y) that packed row `tok` maps to.  x = -1:
// none, the row lies behind the last sequence; -2: none, its position is
// below 0 or no such page exists (the latter is reported).
__device__ __forceinline__ int2 store_row(const StepMap &s, const int32_t *cu, int tok, int *status) {
    int lo = 0, hi = s.Bt;  // first b with cu[b + 1] > tok
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid + 1] > tok)
            hi = mid;
        else
            lo = mid + 1;
    }
    if (lo >= s.Bt || tok < cu[lo]) return make_int2(-1, 0);
    const long long pos = static_cast<long long>(s.kv_len[lo]) - cu[lo + 1] + tok;
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

struct AppendArgs {
    StepMap step;
    CacheStore c;
    const __nv_bfloat16 *k, *v, *k_idx;
    long long k_stride, v_stride, k_idx_stride;
    __nv_bfloat16 *k_idx_pages;
    int d_idx;
    int kv_ctas;  // CTAs of K and V; those behind them copy index keys
    Divisor kv_units, idx_units;  // units per token
    int *status;
};

// UPR: units per (token, head) row.  A unit's place in the step is
// ((token * 2 + {K, V}) * Hkv + head) * UPR + unit, so a warp holds whole rows
// and reduces amax over UPR lanes.
template <int UPR, bool I8>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ AppendArgs a) {
    using U = Units<I8>;
    __shared__ int2 dest[U::TOKENS];
    __shared__ int32_t offsets[kSharedSeqs + 1];
    const int tid = threadIdx.x;
    const bool index = static_cast<int>(blockIdx.x) >= a.kv_ctas;
    // (the host keeps the number of units below 2^31)
    const uint32_t run = (blockIdx.x - (index ? a.kv_ctas : 0)) * U::RUN;
    const Divisor &upt = index ? a.idx_units : a.kv_units;
    const uint32_t total = a.step.total * upt.d, half = a.c.Hkv * UPR;
    const int tok0 = static_cast<int>(upt.quotient(run));
    const int ntok = static_cast<int>(upt.quotient(min(run + U::RUN, total) - 1)) - tok0 + 1;
    uint4 x[U::PER][I8 ? 2 : 1];
    int tok[U::PER];
    uint32_t unit[U::PER];
#pragma unroll
    for (int i = 0; i < U::PER; ++i) {
        const uint32_t e = run + i * kThreads + tid;
        tok[i] = -1;
        unit[i] = 0;
#pragma unroll
        for (int k = 0; k < (I8 ? 2 : 1); ++k) x[i][k] = make_uint4(0, 0, 0, 0);
        if (e >= total) continue;
        tok[i] = static_cast<int>(upt.quotient(e));
        unit[i] = e - tok[i] * upt.d;
        const __nv_bfloat16 *src;
        if (index)
            src = a.k_idx + tok[i] * a.k_idx_stride + unit[i] * U::VALUES;
        else if (unit[i] < half)
            src = a.k + tok[i] * a.k_stride + unit[i] * U::VALUES;
        else
            src = a.v + tok[i] * a.v_stride + (unit[i] - half) * U::VALUES;
        x[i][0] = ld_once(src);
        if (I8) x[i][I8] = ld_once(src + 8);
    }
    const int32_t *cu = share_offsets(a.step, offsets);
    for (int t = tid; t < ntok; t += kThreads) dest[t] = store_row(a.step, cu, tok0 + t, a.status);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < U::PER; ++i) {
        const int2 to = tok[i] >= 0 ? dest[tok[i] - tok0] : make_int2(-1, 0);
        const bool keep = to.x >= 0;
        const long long row = static_cast<long long>(to.x) * a.step.block + to.y;
        if (index) {
            if (keep) {
                uint4 *out = reinterpret_cast<uint4 *>(a.k_idx_pages + row * a.d_idx + unit[i] * U::VALUES);
                out[0] = x[i][0];
                if (I8) out[1] = x[i][I8];
            }
            continue;
        }
        const bool is_v = unit[i] >= half;
        const uint32_t hu = is_v ? unit[i] - half : unit[i];  // head * UPR + unit
        void *pages = is_v ? a.c.v : a.c.k;
        if (!I8) {
            if (keep) reinterpret_cast<uint4 *>(pages)[row * half + hu] = x[i][0];
            continue;
        }
        const uint32_t w[8] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w, x[i][I8].x, x[i][I8].y, x[i][I8].z, x[i][I8].w};
        // |x| as 15-bit patterns order like the values, infinities and NaN on top
        uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
        for (int e = 1; e < 8; ++e) m = __vmaxu2(m, w[e] & 0x7FFF7FFFu);
#pragma unroll
        for (int o = 1; o < UPR; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const uint32_t top = max(m & 0xFFFFu, m >> 16) << 16;
        const float amax = __uint_as_float(top);
        const bool bad = top >= 0x7F800000u, tiny = amax < kTiny;
        const float inv = bad || tiny ? 0.f : __fdiv_rn(127.f, amax);
        const uint64_t magic2 = f2_pack(kMagic, kMagic);
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            // (product and sum rounded one by one: rint(x * inv), as documented; packed
            // products were fused into the sums)
            uint32_t y[4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t u = w[2 * e + k];
                float f0, f1;
                f2_unpack(f2_add(f2_pack(__fmul_rn(__uint_as_float(u << 16), inv), __fmul_rn(__uint_as_float(u & 0xFFFF0000u), inv)), magic2), f0, f1);
                y[2 * k] = __float_as_uint(f0);
                y[2 * k + 1] = __float_as_uint(f1);
            }
            o[e] = __byte_perm(__byte_perm(y[0], y[1], 0x0040), __byte_perm(y[2], y[3], 0x0040), 0x5410);
            if (bad) o[e] = 0;
        }
        if (keep) {
            reinterpret_cast<uint4 *>(pages)[row * half + hu] = make_uint4(o[0], o[1], o[2], o[3]);
            if (hu % UPR == 0) {
                float *scales = is_v ? a.c.v_scales : a.c.k_scales;
                scales[(static_cast<long long>(to.x) * a.c.Hkv + hu / UPR) * a.step.block + to.y] =
                    bad ? __uint_as_float(0x7FC00000u) : tiny ? 0.f : __fdiv_rn(amax, 127.f);
            }
        }
    }
}

struct GatherArgs {
    StepMap step;
    CacheStore c;
    void *k_out, *v_out;
    Divisor units;  // per token
    bool wide;      // int8: k_out and v_out on 32 bytes
    int *status;
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <int UPR, bool I8>
__global__ void __launch_bounds__(kThreads) kv_gather_kernel(const __grid_constant__ GatherArgs a) {
    using U = Units<I8>;
    __shared__ int2 src[U::TOKENS];
    __shared__ int32_t offsets[kSharedSeqs + 1];
    const int tid = threadIdx.x;
    const uint32_t half = a.c.Hkv * UPR;
    const uint32_t run = blockIdx.x * U::RUN;  // (the host keeps the number of units below 2^31)
    const uint32_t total = a.step.total * a.units.d;
    const int tok0 = static_cast<int>(a.units.quotient(run));
    const int ntok = static_cast<int>(a.units.quotient(min(run + U::RUN, total) - 1)) - tok0 + 1;
    const int32_t *cu = share_offsets(a.step, offsets);
    for (int t = tid; t < ntok; t += kThreads) src[t] = store_row(a.step, cu, tok0 + t, a.status);
    __syncthreads();
    uint4 x[U::PER];
    float s[U::PER];
    uint4 *to[U::PER];  // nullptr: not written
#pragma unroll
    for (int i = 0; i < U::PER; ++i) {
        const uint32_t e = run + i * kThreads + tid;
        x[i] = make_uint4(0, 0, 0, 0);
        s[i] = 0.f;
        to[i] = nullptr;
        if (e >= total) continue;
        const uint32_t tok = a.units.quotient(e), unit = e - tok * a.units.d;
        const int2 from = src[tok - tok0];
        if (from.x == -1) continue;  // behind the last sequence: left as it is
        const bool is_v = unit >= half;
        const uint32_t hu = is_v ? unit - half : unit;  // head * UPR + unit
        to[i] = reinterpret_cast<uint4 *>(is_v ? a.v_out : a.k_out) + (static_cast<long long>(tok) * half + hu) * (I8 ? 2 : 1);
        if (from.x < 0) continue;  // no such position or page: zeros
        const long long row = static_cast<long long>(from.x) * a.step.block + from.y;
        x[i] = ld_once(reinterpret_cast<const uint4 *>(is_v ? a.c.v : a.c.k) + row * half + hu);
        if (I8)
            s[i] = __ldg((is_v ? a.c.v_scales : a.c.k_scales) +
                         (static_cast<long long>(from.x) * a.c.Hkv + hu / UPR) * a.step.block + from.y);
    }
#pragma unroll
    for (int i = 0; i < U::PER; ++i) {
        if (!to[i]) continue;
        if (!I8) {
            *to[i] = x[i];
            continue;
        }
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        const uint64_t s2 = f2_pack(s[i], s[i]), back = f2_pack(-8388736.f, -8388736.f);
        uint32_t o[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t u = w[q] ^ 0x80808080u;  // code + 128, then 2^23 + that as a float
            float f[4];
            f2_unpack(f2_mul(f2_add(f2_pack(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7540)), __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7541))), back), s2), f[0], f[1]);
            f2_unpack(f2_mul(f2_add(f2_pack(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7542)), __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7543))), back), s2), f[2], f[3]);
            o[2 * q] = pack2(f[0], f[1]);
            o[2 * q + 1] = pack2(f[2], f[3]);
        }
        if (a.wide) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to[i]), "r"(o[0]),
                         "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                         : "memory");
        } else {
            to[i][0] = make_uint4(o[0], o[1], o[2], o[3]);
            to[i][1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
}

template <bool I8>
unsigned runs(long long units) {
    return static_cast<unsigned>((units + Units<I8>::RUN - 1) / Units<I8>::RUN);
}

template <int UPR, bool I8>
cudaError_t run_append(AppendArgs a, int d, cudaStream_t st) {
    constexpr int V = Units<I8>::VALUES;
    const int units = 2 * a.c.Hkv * (d / V);
    a.kv_units = Divisor(units);
    a.kv_ctas = static_cast<int>(runs<I8>(static_cast<long long>(a.step.total) * units));
    unsigned grid = a.kv_ctas;
    if (a.d_idx) {
        a.idx_units = Divisor(a.d_idx / V);
        grid += runs<I8>(static_cast<long long>(a.step.total) * (a.d_idx / V));
    }
    kv_append_kernel<UPR, I8><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <int UPR, bool I8>
cudaError_t run_gather(GatherArgs a, int d, cudaStream_t st) {
    const int units = 2 * a.c.Hkv * (d / Units<I8>::VALUES);
    a.units = Divisor(units);
    kv_gather_kernel<UPR, I8><<<runs<I8>(static_cast<long long>(a.step.total) * units), kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const StepMap &step, const CacheStore &c, const void *k,
                             long long k_stride, const void *v, long long v_stride,
                             const void *k_idx, long long k_idx_stride, void *k_idx_pages,
                             int d_idx, int *status, cudaStream_t st) {
    const AppendArgs a{step, c, static_cast<const __nv_bfloat16 *>(k), static_cast<const __nv_bfloat16 *>(v),
                       static_cast<const __nv_bfloat16 *>(k_idx), k_stride, v_stride, k_idx_stride,
                       static_cast<__nv_bfloat16 *>(k_idx_pages), d_idx, 0, Divisor(1), Divisor(1), status};
    if (c.d == 128) return c.k_scales ? run_append<8, true>(a, 128, st) : run_append<16, false>(a, 128, st);
    return c.k_scales ? run_append<4, true>(a, 64, st) : run_append<8, false>(a, 64, st);
}

cudaError_t launch_kv_gather(const StepMap &step, const CacheStore &c, void *k_out, void *v_out,
                             int *status, cudaStream_t st) {
    const bool wide = ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 31) == 0;
    const GatherArgs a{step, c, k_out, v_out, Divisor(1), wide, status};
    if (c.d == 128) return c.k_scales ? run_gather<8, true>(a, 128, st) : run_gather<16, false>(a, 128, st);
    return c.k_scales ? run_gather<4, true>(a, 64, st) : run_gather<8, false>(a, 64, st);
}

}  // namespace msa
