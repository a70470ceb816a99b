// paged_attn_split.cu -- attention of few query rows over a paged cache
// (single tokens, short chunks, and the sparse branch on int8 pages).
//
// With the rows of one (sequence, kv head) numbered r = i * G + g (token i,
// head g of the group), a tile of R = 8 or 16 rows attends its keys j with
//     s_j = (q . k_j) / sqrt(d),  m = max s_j,  l = sum exp(s_j - m),
//     o = sum exp(s_j - m) v_j / l,  lse = m + ln l,
// in one pass over the keys, 128 at a time, with a running m and l.
//
// Few rows read many keys once, so HBM bounds it, and the instructions spent
// per key come next.  Both products therefore run on the tensor core with the
// keys (then the value columns) as its 128 rows and the query rows as its
// columns, and take K and V as TMA left them in shared memory:
//     S^T [128 keys][rows] = K Q^T,   O^T [d][rows] = V^T P^T.
// A thread then holds one key's scores of all rows, and afterwards one value
// column's sums of all rows, in its own registers.
//
// int8 pages (k_j = code * sk_j, v_j = code * sv_j) are never converted: the
// products are integer ones (exact), of Q and P written in 7-bit digits,
//     q = 2^e (x2 2^14 + x1 2^7 + x0),  |x| <= 64,  e from the row's largest |q|
//     p_j sv_j = 2^(f - 27) (y3 2^21 + y2 2^14 + y1 2^7 + y0),  0 <= y < 128
// each digit a column of its own.  q keeps 20 bits below its row's largest
// value: a bf16 has 8 of its own, so values within 2^12 of the largest are exact,
// and what smaller ones lose moves a score by at most 2^-20 max |q_i| sum |k_i| /
// sqrt(d), 1/32 of what the rounding of one code may have done there.  2^f is the largest power of two <= the row's
// largest p_j sv_j of the tile's 128 keys, so a term keeps 27 bits below the
// largest one beside it: neither a V row of a large scale that this row does not
// see or weigh, nor a key in another tile that draws most of the weight, takes
// bits from the terms that make up the output.  Where the tile's scales lie
// within a factor of 4, as they mostly do, 2^f comes from the row's largest p and
// the largest scale, and a term keeps 23 bits or more; else the warps exchange
// the terms' maxima (in every tile: 192 us instead of 184 on the decode step
// below, and 354 instead of 297 with 16 rows per tile).  sk and the digits'
// weights are applied in fp32.  (A kernel that turned the codes into bf16
// fragments for mma.sync spent 700 instructions per warp on 16 keys and reached
// 2.6 TB/s.)
// bf16 pages take Q as it is and P as two bf16 terms (hi + lo, 15 bits), both
// positive: an infinite value of V times either of them is that infinity.
//
//  - The key tiles of all (sequence, row tile, kv head) segments form one
//    list that is cut into equal runs, one per CTA: a batch with contexts of
//    any lengths keeps every SM streaming to the end.  Up to 16 heads share a
//    run, each with a CTA of its own: a cached token's heads lie side by side
//    in memory (128 bytes each with int8 and d = 128), and the CTAs that read
//    them do it at the same time, which HBM pages and L2 lines reward.
//  - A producer warp keeps a ring of about 100 KB (200 KB with one CTA per
//    SM) filled by TMA, across segment borders, and looks the pages up 32
//    tiles at a time.
//  - Measured, in a replayed graph: one new token of 64 heads on each of 32
//    int8 contexts of up to 32768 keys: 184 us = 5.4 TB/s (at the card's power
//    limit), on bf16 ones 302 us = 6.4 TB/s; 16 selected blocks of 128 keys for
//    each of 32: 33 us = 4.2 TB/s; one context of 4001 bf16 keys: 12.7 us, all of
//    it latency.
//  - A segment that lies in several runs leaves one fp32 piece per run, and the
//    CTA that finishes the last piece merges them in run order.  An atomic
//    counter tells it that it is the last; which CTA that is has no influence
//    on the result.  (A second kernel for the merge cost 4 us of device time
//    and 3 us of launch on a call of 8 us.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cache.h"
#include "msa_common.cuh"
#include "paged_walk.cuh"
#include "ptx_sm100.cuh"

namespace msa {

namespace {

using namespace walk;

constexpr int kCompute = 256;                // warps 0-3 and 4-7, alternate tiles: one key (then
                                             // one value column) per thread
constexpr int kThreads = kCompute + 64;      // warp 8: producer; warp 9: products
constexpr int kOver = 2;    // a segment's start and end cost about as much as two tiles
constexpr int kMinRun = 3;  // units per run, at least
constexpr float kLn2f = 0.6931471805599453f;

// ------------------------------------------------------------ tile geometry
constexpr int round_up(int x, int m) { return (x + m - 1) / m * m; }

template <int D, bool I8, int R>
struct Tile {
    static constexpr int EB = I8 ? 1 : 2;
    static constexpr int ROWB = D * EB < 128 ? D * EB : 128;  // bytes of a shared-memory row
    static constexpr int REGS = D * EB / ROWB;                // 128-byte wide regions
    static constexpr int REGION = kKeys * ROWB;
    static constexpr int BYTES = REGS * REGION;               // K or V of a tile
    static constexpr int STAGE = 2 * BYTES;                   // V, then K
    static constexpr int CTAS = STAGE > 32768 ? 1 : 2;        // per SM
    // columns of the products (a multiple of 16 each): scores, outputs
    static constexpr int NS = I8 ? round_up(3 * R, 16) : round_up(R, 16);
    static constexpr int NO = I8 ? 4 * R : 2 * R;
    static constexpr int QBYTES = NS * D * EB;
    static constexpr int PBYTES = NO * kKeys * EB;
    // the ring takes what the 227 KB of an SM leave
    static constexpr int STAGES = STAGE > 32768 ? 3 : STAGE > 16384 ? (R <= 8 ? 3 : 2) : 5;
    static constexpr int COLS = 2 * (NS + NO);  // both warpgroups
    // maxima of a warp: its rows' scores, then (int8) their weights times V scales, and
    // the least and largest of its V scales, of two tiles
    static constexpr int TW = I8 ? 2 * R + 4 : R + 4;
    static constexpr int TMEM = COLS <= 64 ? 64 : COLS <= 128 ? 128 : 256;
    static_assert(COLS <= 256, "two CTAs share the 512 columns of an SM");
};

struct alignas(16) StageMeta {
    int pos[4];  // first key of each 32-key quarter; -1: nothing there
};

constexpr int kScaleBytes = 2 * kKeys * 4;  // K and V scales of a stage
template <int D, bool I8, int R>
constexpr size_t split_smem_bytes() {
    using T = Tile<D, I8, R>;
    return static_cast<size_t>(T::STAGES) * T::STAGE + round_up(T::QBYTES, 1024) +
           2 * round_up(T::PBYTES, 1024) + (I8 ? T::STAGES * kScaleBytes : 0) + 8 * T::TW * 4 + R * 36 + 16 + T::STAGES * (sizeof(StageMeta) + 16) + 72;
}

// Maximum and minimum over the warp (a NaN counts as absent).
__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float warp_min(float x) {
    float r;
    asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// 4 columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t (&r)[4]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr)
                 : "memory");
}

// x2 2^14 + x1 2^7 + x0 of signed sums (x0, x1 below 2^21).
__device__ __forceinline__ float from_digits(uint32_t x0, uint32_t x1, uint32_t x2) {
    const int lo = static_cast<int>(x1) * 128 + static_cast<int>(x0);
    return fmaf(static_cast<float>(static_cast<int>(x2)), 16384.f, static_cast<float>(lo));
}

// Byte offset of 16-byte piece c of row r of a swizzled region.
template <int ROWB>
__device__ __forceinline__ uint32_t piece_at(uint32_t r, uint32_t c) {
    if (ROWB == 128) return sw128_offset(r, c);
    return r * 64u + ((c ^ ((r >> 1) & 3u)) << 4);
}

// Operand descriptors.  Key-major rows (K, Q, P): the contraction runs along a
// row; V^T: it runs over the rows, and a row holds 64 bf16 or D codes of d.
// With d = 64 the second half of V^T's 128 rows is whatever lies one region
// further (the K tile); its sums are never read.
template <int ROWB>
__device__ __forceinline__ uint64_t row_desc(uint32_t addr) {
    return ROWB == 128 ? sdesc_sw128(addr, 16, 1024) : sdesc_sw64(addr);
}
template <int ROWB, int REGION>
__device__ __forceinline__ uint64_t col_desc(uint32_t addr) {
    if (ROWB == 128) return sdesc_sw128(addr, REGION, 1024);
    return (sdesc_sw64(addr) & ~(0x3FFFull << 16)) | (static_cast<uint64_t>(REGION >> 4) << 16);
}

constexpr uint32_t kIdescAMn = 1u << 15;  // A runs along M in memory

// ===========================================================================
// Merge of the pieces of a segment that begins in run c0:
//   lse = log2 sum 2^lse_p,  out = sum 2^(lse_p - lse) o_p
// by the compute warps: every eighth piece each, 4 rows at a time, a lane
// D / 32 columns of all 4, then over the warps in shared memory (pool: 8 KB,
// tops: 64 floats).
// ===========================================================================
template <int D, int R>
__device__ __noinline__ void merge_pieces(const PagedAttn &a, const RowTile &t, int cu0, int h, int c0,
                                          int pieces, float *pool, float *tops) {
    constexpr int RG = 4, COLS = D / 32, WARPS = kCompute / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int live = min(t.rows - t.r0, R);
    float2 *ml = reinterpret_cast<float2 *>(tops);  // [warp][row] (maximum, sum)
#pragma unroll 1
    for (int rg = 0; rg < live; rg += RG) {
        float acc[RG][COLS], top[RG], sum[RG];
#pragma unroll
        for (int r = 0; r < RG; ++r) {
            top[r] = -INFINITY;
            sum[r] = 0.f;
#pragma unroll
            for (int e = 0; e < COLS; ++e) acc[r][e] = 0.f;
        }
#pragma unroll 1
        for (int p = warp; p < pieces; p += WARPS) {
            const long long row0 = piece_slot(a, c0, p) * R + rg;
            const float lp = lane < RG && rg + lane < live ? __ldcg(a.part_lse + row0 + lane) : -INFINITY;
            float y[RG][COLS];
#pragma unroll
            for (int r = 0; r < RG; ++r)
#pragma unroll
                for (int e = 0; e < COLS; e += 2) {
                    float2 u = make_float2(0.f, 0.f);
                    if (rg + r < live) u = __ldcg(reinterpret_cast<const float2 *>(a.part_o + (row0 + r) * D + lane * 2 + e * 32));
                    y[r][e] = u.x;
                    y[r][e + 1] = u.y;
                }
#pragma unroll
            for (int r = 0; r < RG; ++r) {
                const float l = __shfl_sync(0xFFFFFFFFu, lp, r);
                // (no key of this row in the piece: weight 0, whatever y holds)
                const float g = fmaxf(top[r], l), z = g == -INFINITY ? 0.f : g;
                const float f = ex2_approx(top[r] - z), w = ex2_approx(l - z);
                top[r] = g;
                sum[r] = sum[r] * f + w;
#pragma unroll
                for (int e = 0; e < COLS; ++e) acc[r][e] = acc[r][e] * f + (l == -INFINITY ? 0.f : w * y[r][e]);
            }
        }
        if (lane == 0) {
#pragma unroll
            for (int r = 0; r < RG; ++r) ml[warp * RG + r] = make_float2(top[r], sum[r]);
        }
        named_barrier(1, kCompute);
        constexpr int ROWS = 2;  // rows at a time: [warp][ROWS][D] in the pool
#pragma unroll
        for (int q = 0; q < RG; q += ROWS) {
            if (rg + q >= live) break;
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
#pragma unroll
                for (int e = 0; e < COLS; e += 2)
                    *reinterpret_cast<float2 *>(pool + (warp * ROWS + r) * D + lane * 2 + e * 32) = make_float2(acc[q + r][e], acc[q + r][e + 1]);
            named_barrier(1, kCompute);
            const int r = threadIdx.x / D, col = threadIdx.x % D;
            if (r < ROWS && rg + q + r < live) {
                float g = -INFINITY, s = 0.f, x = 0.f;
#pragma unroll
                for (int w = 0; w < WARPS; ++w) g = fmaxf(g, ml[w * RG + q + r].x);
                const float z = g == -INFINITY ? 0.f : g;
#pragma unroll
                for (int w = 0; w < WARPS; ++w) {
                    const float2 y = ml[w * RG + q + r];
                    const float f = y.x == -INFINITY ? 1.f : ex2_approx(y.x - z);  // (-inf: nothing, or NaN)
                    s += y.y * f;
                    x += pool[(w * ROWS + r) * D + col] * f;
                }
                const int row = t.r0 + rg + q + r, tok = static_cast<int>(a.by_g.quotient(row));
                const long long orow = (static_cast<long long>(cu0) + tok) * a.Hq + static_cast<long long>(h) * a.G + (row - tok * a.G);
                const float inv = s == 0.f ? 0.f : 1.f / s;
                static_cast<__nv_bfloat16 *>(a.out)[orow * D + col] = __float2bfloat16_rn(x * inv);
                if (col == 0) a.lse[orow] = s == 0.f ? -INFINITY : (z + __log2f(s)) * kLn2f;
            }
            named_barrier(1, kCompute);
        }
    }
}

// ===========================================================================
// One run per CTA.
// ===========================================================================
template <int D, bool I8, int R>
__global__ void __launch_bounds__(kThreads, Tile<D, I8, R>::CTAS) split_attn_kernel(
    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
    const __grid_constant__ PagedAttn a) {
    using T = Tile<D, I8, R>;
    extern __shared__ __align__(1024) unsigned char ring[];
    unsigned char *q_s = ring + T::STAGES * T::STAGE;
    unsigned char *p_s = q_s + round_up(T::QBYTES, 1024);
    float *scales = reinterpret_cast<float *>(p_s + 2 * round_up(T::PBYTES, 1024));  // [stage][K, V][128]
    constexpr int TW = T::TW;
    static_assert(2 * round_up(T::PBYTES, 1024) >= 8192 && 8 * TW >= 64, "merge buffers");
    float *tops_s = scales + (I8 ? T::STAGES * 2 * kKeys : 0);     // [warp][TW]
    float *qscale = tops_s + 8 * TW;                               // [R] factor of a row's scores
    float *maxima_s = qscale + R;                                  // [warpgroup][2][R] the rows' m, tile about
    float *sums = maxima_s + 4 * R;                                // [warpgroup][R] the rows' l
    int *rowpos = reinterpret_cast<int *>(sums + 2 * R);           // [R] position, -1: no such row
    int *poison = rowpos + R;                                      // [R] a seen key's sv is not finite
    StageMeta *meta = reinterpret_cast<StageMeta *>(
        (reinterpret_cast<uintptr_t>(poison + R) + 15) & ~static_cast<uintptr_t>(15));
    uint64_t *full = reinterpret_cast<uint64_t *>(meta + T::STAGES);
    uint64_t *empty = full + T::STAGES;
    uint64_t *bar_s = empty + T::STAGES;  // [warpgroup] scores complete
    uint64_t *bar_o = bar_s + 2;          // [warpgroup] outputs complete
    uint64_t *p_ready = bar_s + 4;        // [warpgroup] weights written, scores and last outputs read
    uint64_t *q_ready = bar_s + 6;        // Q of a segment written
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar_s + 7);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    volatile int *last_piece = abort_flag + 1;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < T::STAGES; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_s + i, 1);
            mbar_init(bar_o + i, 1);
            mbar_init(p_ready + i, kCompute / 2);
        }
        mbar_init(q_ready, kCompute);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }
    if (tid < kCompute) {  // rows of the operand buffer that no digit or head ever fills
        for (int e = tid; e < T::QBYTES / 16; e += kCompute) reinterpret_cast<uint4 *>(q_s)[e] = make_uint4(0, 0, 0, 0);
    }
    const Found found = find_run(a, R, kOver, kMinRun);
    if (found.start >= found.work) return;
    if (warp == 9) {
        tmem_alloc(tmem_slot, T::TMEM);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;  // per warpgroup: NS columns of scores, NO of outputs
    Walk walk(a, found, kOver);
    const int block = a.step.block;

    if (warp == 8) {
        // -------------------------------------------------------- producer
        uint32_t it = 0;
        const int box = min(block, kKeys);  // keys per TMA box
        bool ok = true;
        while (ok && walk.next(a, R)) {
            const RowTile t = row_tile(a, walk.s, walk.rt, R);
            const int x1 = min(walk.x1, t.count);
            for (int xb = walk.x0; xb < x1 && ok; xb += 32) {
                // positions and store rows of this lane's tile, by 32-key quarters
                int pos[4] = {-1, -1, -1, -1}, z[4] = {0, 0, 0, 0};
                const int x = xb + lane;
                if (x < x1) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (i > 0 && i * 32 % box != 0) {  // within the box of the quarter before
                            pos[i] = pos[i - 1] < 0 ? -1 : pos[i - 1] + 32;
                            continue;
                        }
                        int p;  // key position of the box
                        if (a.ids) {
                            const int v = x * kKeys + i * 32, slot = a.by_block.quotient(v);
                            const int id = slot < a.K ? a.ids[static_cast<long long>(walk.b) * a.K + slot] : -1;
                            const int N = (a.T + block - 1) / block;
                            if (id < -1 || id >= N) atomicOr(a.status, kDevBadIds);
                            p = id < 0 || id >= N ? -1 : id * block + (v - slot * block);
                            if (p >= a.T) p = -1;
                        } else {
                            p = (x < t.na ? x : x + t.skip) * kKeys + i * 32;
                            // (keys before every row's window: their page may be gone)
                            if (p > t.tmax || p >= walk.s.cap ||
                                (a.window && p + box <= t.tmin - a.window + 1 && p >= a.sinks))
                                p = -1;
                        }
                        if (p < 0) continue;
                        const int j = a.by_block.quotient(p);
                        const int page = a.step.pm.table[static_cast<long long>(walk.b) * a.step.pm.stride + j];
                        if (page < 0 || page >= a.step.pm.count) {
                            atomicOr(a.status, kDevBadIds);
                            continue;
                        }
                        pos[i] = p;
                        z[i] = page * block + (p - j * block);
                    }
                }
                const int m = min(32, x1 - xb);
                for (int y = 0; y < m && ok; ++y) {
                    int p[4], zz[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        p[i] = __shfl_sync(0xFFFFFFFFu, pos[i], y);
                        zz[i] = __shfl_sync(0xFFFFFFFFu, z[i], y);
                    }
                    const int st = it % T::STAGES;
                    if (lane == 0) {
                        if (it >= T::STAGES)
                            ok = mbar_wait(empty + st, ((it / T::STAGES) & 1) ^ 1, abort_flag, a.status);
                        if (ok) {
                            *reinterpret_cast<int4 *>(meta + st) = make_int4(p[0], p[1], p[2], p[3]);
                            unsigned char *dv = ring + st * T::STAGE, *dk = dv + T::BYTES;
                            int boxes = 0;
#pragma unroll
                            for (int i = 0; i < 4; ++i) boxes += i * 32 % box == 0 && p[i] >= 0;
                            if (boxes == 0)
                                mbar_arrive(full + st);
                            else
                                mbar_arrive_expect_tx(full + st, boxes * box * (2 * D * T::EB + (I8 ? 8 : 0)));
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if (i * 32 % box != 0 || p[i] < 0) continue;
#pragma unroll
                                for (int r = 0; r < T::REGS; ++r) {
                                    const uint32_t o = r * T::REGION + i * 32 * T::ROWB;
                                    tma_load_3d(dk + o, &tm_k, full + st, r * 64, walk.h, zz[i]);
                                    tma_load_3d(dv + o, &tm_v, full + st, r * 64, walk.h, zz[i]);
                                }
                                if (I8) {
                                    const int page = static_cast<int>(a.by_block.quotient(zz[i]));
                                    const long long so = (static_cast<long long>(page) * a.c.Hkv + walk.h) * block + (zz[i] - page * block);
                                    bulk_load(scales + (2 * st) * kKeys + i * 32, a.c.k_scales + so, box * 4, full + st);
                                    bulk_load(scales + (2 * st + 1) * kKeys + i * 32, a.c.v_scales + so, box * 4, full + st);
                                }
                            }
                        }
                    }
                    ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
                    if (ok) ++it;
                }
            }
        }
        // after an abort: the copies have landed before the CTA ends
        if (!ok && lane == 0) {
            for (uint32_t i = it > T::STAGES ? it - T::STAGES : 0; i < it; ++i) {
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait(full + i % T::STAGES, (i / T::STAGES) & 1))
                    if (global_timer_ns() - t0 > kWaitLimitNs / 4) break;
            }
        }
        return;
    }

    if (warp == 9) {
        // -------------------------------------------------------- products
        // Tiles alternate between the warpgroups.  S^T of a tile is issued as soon
        // as its keys have landed, before the O^T of the tile before, whose
        // weights the other warpgroup is still at.
        if (lane == 0) {
            constexpr uint32_t idesc_s = I8 ? idesc_s8_s32(128, T::NS) : idesc_bf16_f32(128, T::NS, false);
            constexpr uint32_t idesc_o = (I8 ? idesc_s8_s32(128, T::NO) : idesc_bf16_f32(128, T::NO, false)) | kIdescAMn;
            constexpr int EK = I8 ? 32 : 16;  // contraction of one instruction (32 bytes)
            const uint64_t kd0 = row_desc<T::ROWB>(smem_addr(ring + T::BYTES)), qd0 = row_desc<T::ROWB>(smem_addr(q_s));
            const uint64_t vd0 = col_desc<T::ROWB, T::REGION>(smem_addr(ring)), pd0 = row_desc<128>(smem_addr(p_s));
            uint32_t it = 0, segs = 0;
            bool ok = true;
            auto outputs = [&](uint32_t i) {  // O^T of tile i
                const uint32_t g = i & 1;
                if (!(ok = mbar_wait(p_ready + g, i >> 1 & 1, abort_flag, a.status))) return;
                tc_fence_after();
                const uint32_t st = i % T::STAGES, tmem_o = tmem + g * (T::NS + T::NO) + T::NS;
#pragma unroll
                for (int k = 0; k < kKeys / EK; ++k) {
                    const uint64_t vd = vd0 + st * (T::STAGE >> 4) + ((k * EK * T::ROWB) >> 4);
                    const uint64_t pd = pd0 + ((g * round_up(T::PBYTES, 1024) + (k / 4) * T::NO * 128 + (k % 4) * 32) >> 4);
                    if (I8)
                        umma_i8(tmem_o, vd, pd, idesc_o, k > 0);
                    else
                        umma_bf16(tmem_o, vd, pd, idesc_o, k > 0);
                }
                umma_commit(bar_o + g);
                umma_commit(empty + st);
            };
            while (ok && walk.next(a, R)) {
                const RowTile t = row_tile(a, walk.s, walk.rt, R);
                const int x1 = min(walk.x1, t.count);
                if (x1 <= walk.x0) continue;  // nothing to see: Q is not announced
                ok = mbar_wait(q_ready, segs++ & 1, abort_flag, a.status);
                for (int x = walk.x0; x < x1 && ok; ++x, ++it) {
                    const uint32_t st = it % T::STAGES, tmem_s = tmem + (it & 1) * (T::NS + T::NO);
                    if (!(ok = mbar_wait(full + st, (it / T::STAGES) & 1, abort_flag, a.status))) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < D / EK; ++k) {
                        const uint64_t kd = kd0 + st * (T::STAGE >> 4) + (((k / 4) * T::REGION + (k % 4) * 32) >> 4);
                        const uint64_t qd = qd0 + (((k / 4) * T::NS * 128 + (k % 4) * 32) >> 4);
                        if (I8)
                            umma_i8(tmem_s, kd, qd, idesc_s, k > 0);
                        else
                            umma_bf16(tmem_s, kd, qd, idesc_s, k > 0);
                    }
                    umma_commit(bar_s + (it & 1));
                    if (x > walk.x0) outputs(it - 1);
                }
                if (ok) outputs(it - 1);
            }
        }
        __syncwarp();
        named_barrier(2, kCompute + 32);  // the compute warps have read their last outputs
        tmem_dealloc(tmem, T::TMEM);
        return;
    }

    // ------------------------------------------------------------ warps 0-7
    const uint32_t wg = warp >> 2;  // warpgroup
    const int key = tid & 127, quarter = warp & 3;
    const uint32_t tmem_s = tmem + wg * (T::NS + T::NO) + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t tmem_o = tmem_s + T::NS;
    unsigned char *p_w = p_s + wg * round_up(T::PBYTES, 1024);
    float *tops = tops_s + wg * 4 * TW, *maxima = maxima_s + wg * 2 * R;
    uint32_t it = 0;           // tiles taken (by both warpgroups)
    bool ok = true;            // false: a wait of this thread gave up
    bool dead = false;         // the same for all: no tile is taken any more, but every
                               // barrier is met
    while (walk.next(a, R)) {
        const RowTile t = row_tile(a, walk.s, walk.rt, R);
        const int x1 = min(walk.x1, t.count);
        // ---- Q rows into shared memory, 16 threads per row (8 with d = 64)
        constexpr int TPR = D / 8;
#pragma unroll
        for (int rr = 0; rr < R; rr += kCompute / TPR) {
            const int r = rr + tid / TPR, c = tid % TPR;
            if (R % (kCompute / TPR) != 0 && r >= R) continue;  // (whole warps)
            const int row = t.r0 + r, tok = static_cast<int>(a.by_g.quotient(row));
            uint4 u = make_uint4(0, 0, 0, 0);
            if (row < t.rows)
                u = *reinterpret_cast<const uint4 *>(
                    static_cast<const __nv_bfloat16 *>(a.q) + (walk.s.cu0 + tok) * a.q_stride +
                    (static_cast<long long>(walk.h) * a.G + (row - tok * a.G)) * D + c * 8);
            if (c == 0) {
                rowpos[r] = row < t.rows ? walk.s.off + tok : -1;
                maxima_s[r] = maxima_s[2 * R + r] = -INFINITY;
                if (I8) poison[r] = 0;
            }
            if (!I8) {
                *reinterpret_cast<uint4 *>(q_s + (c / 8) * T::NS * 128 + sw128_offset(r, c % 8)) = u;
            } else {
                // digits of q / 2^e, 2^e the largest power of two <= the row's largest |q|
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
                uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                                      __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
#pragma unroll
                for (int o = 1; o < TPR; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                const uint32_t top = max(m & 0xFFFFu, m >> 16) << 16;
                const uint32_t e = top & 0x7F800000u;
                const bool usable = e != 0 && e != 0x7F800000u;
                // 2^-e as a product, since 2^-127 is subnormal: the biased exponents of the
                // factors add up to 127 + 127 + (127 - biased e)
                const uint32_t e1 = e >> 1 & 0x7F800000u;
                const float inv = usable ? __uint_as_float(0x5F000000u - e1) : 0.f;
                const float inv2 = usable ? __uint_as_float(0x5F800000u - (e - e1)) : 0.f;
                if (c == 0)
                    qscale[r] = e == 0x7F800000u ? __uint_as_float(0x7FC00000u)
                                                 : __uint_as_float(e) * 1.9073486328125e-6f * a.scale_log2;  // 2^-19
                uint32_t d0[2] = {0, 0}, d1[2] = {0, 0}, d2[2] = {0, 0};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float q = __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
                    const int x = usable ? __float2int_rn(q * inv * inv2 * 524288.f) : 0;  // |x| <= 2^20
                    const int y0 = ((x + 64) & 127) - 64, x1_ = (x - y0) >> 7;
                    const int y1 = ((x1_ + 64) & 127) - 64, y2 = (x1_ - y1) >> 7;
                    d0[i / 4] |= (static_cast<uint32_t>(y0) & 0xFFu) << (8 * (i % 4));
                    d1[i / 4] |= (static_cast<uint32_t>(y1) & 0xFFu) << (8 * (i % 4));
                    d2[i / 4] |= (static_cast<uint32_t>(y2) & 0xFFu) << (8 * (i % 4));
                }
                const uint32_t half = (c & 1) * 8;
                *reinterpret_cast<uint2 *>(q_s + piece_at<T::ROWB>(r, c / 2) + half) = make_uint2(d0[0], d0[1]);
                *reinterpret_cast<uint2 *>(q_s + piece_at<T::ROWB>(R + r, c / 2) + half) = make_uint2(d1[0], d1[1]);
                *reinterpret_cast<uint2 *>(q_s + piece_at<T::ROWB>(2 * R + r, c / 2) + half) = make_uint2(d2[0], d2[1]);
            }
        }
        fence_proxy_async_smem();
        if (x1 > walk.x0) mbar_arrive(q_ready);
        named_barrier(1, kCompute);  // rowpos, qscale, maxima

        float o[R], l[R];  // this column's sums, this key lane's weights
#pragma unroll
        for (int r = 0; r < R; ++r) o[r] = l[r] = 0.f;
        const float *m = maxima;  // the rows' running maxima
        const int last = min(t.tmax, walk.s.cap - 1);  // last key that any row sees

        // This thread's key of a tile: its position, whether any row or every row
        // sees it, its scales; read one tile ahead, while the products run.
        int pos = 0;
        bool any = false, every = false, bad_sv = false;
        float sk = 1.f, sv = 1.f;
        auto take_key = [&](uint32_t i) {
            const int st = i % T::STAGES;
            ok = ok && mbar_wait(full + st, (i / T::STAGES) & 1, abort_flag, a.status);
            const int base = ok ? meta[st].pos[quarter] : -1;
            pos = base < 0 ? 0x7FFFFFFF : base + lane;
            any = pos <= last && (!a.window || pos > t.tmin - a.window || pos < a.sinks);
            every = pos <= min(t.tmin, walk.s.cap - 1) && (!a.window || pos > t.tmax - a.window || pos < a.sinks);
            if (I8) {
                sk = scales[2 * st * kKeys + key];
                sv = any ? scales[(2 * st + 1) * kKeys + key] : 0.f;
                bad_sv = !(sv <= 3.4028235e38f);  // inf or NaN
                if (bad_sv) sv = 0.f;
                const float2 ends = make_float2(warp_min(any ? sv : INFINITY), warp_max(sv));
                if (lane == 0) *reinterpret_cast<float2 *>(tops + quarter * TW + 2 * R + (i & 2)) = ends;
            } else if (!any) {
                // a key that no row sees counts nothing, whatever its V row holds
#pragma unroll
                for (int c = 0; c < 8 * T::REGS; ++c)
                    *reinterpret_cast<uint4 *>(ring + st * T::STAGE + c / 8 * T::REGION + key * 128 + ((c + lane) & 7) * 16) =
                        make_uint4(0, 0, 0, 0);
            }
        };
        const uint32_t end = it + max(x1 - walk.x0, 0);  // tiles taken after this segment
        uint32_t i = it + ((it ^ wg) & 1);               // the warpgroup's first tile of it
        if (i < end && !dead) take_key(i);
        for (; i < end && !dead; i += 2) {
            const bool all = __all_sync(0xFFFFFFFFu, every);
            ok = ok && mbar_wait(bar_s + wg, i >> 1 & 1, abort_flag, a.status);
            __syncwarp();
            tc_fence_after();
            float s[R];
#pragma unroll
            for (int r0 = 0; r0 < R; r0 += 4) {
                uint32_t w[I8 ? 3 : 1][4];
#pragma unroll
                for (int k = 0; k < (I8 ? 3 : 1); ++k) tmem_ld4(tmem_s + k * R + r0, w[k]);
                float4 qs = make_float4(a.scale_log2, a.scale_log2, a.scale_log2, a.scale_log2);
                if (I8) qs = *reinterpret_cast<const float4 *>(qscale + r0);
                const float f[4] = {qs.x, qs.y, qs.z, qs.w};
                tmem_wait_ld();
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    s[r0 + r] = I8 ? from_digits(w[0][r], w[I8][r], w[2 * I8][r]) * (f[r] * sk)
                                   : __uint_as_float(w[0][r]) * f[r];
            }
            if (!all) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int tt = rowpos[r];
                    const bool v = pos <= min(tt, walk.s.cap - 1) && (!a.window || pos > tt - a.window || pos < a.sinks);
                    if (I8 && bad_sv && v) poison[r] = 1;
                    s[r] = v ? s[r] : -INFINITY;
                }
            } else if (I8 && bad_sv) {
#pragma unroll
                for (int r = 0; r < R; ++r) poison[r] = 1;
            }
#pragma unroll
            for (int r = 0; r < R; r += 4) {
                const float4 g = make_float4(warp_max(s[r]), warp_max(s[r + 1]), warp_max(s[r + 2]), warp_max(s[r + 3]));
                if (lane == 0) *reinterpret_cast<float4 *>(tops + quarter * TW + r) = g;
            }
            dead = named_barrier_or(3 + wg, 128, !ok);
            if (dead) break;
            // ---- weights, relative to the running maxima
            // int8: V scales within a factor of 4 (the same for all), and the largest one's exponent
            bool alike = false;
            int top_sv = 0;
            if (I8) {
                float lo = INFINITY, hi = 0.f;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float2 ends = *reinterpret_cast<const float2 *>(tops + w * TW + 2 * R + (i & 2));
                    lo = fminf(lo, ends.x);
                    hi = fmaxf(hi, ends.y);
                }
                alike = hi <= 4.f * lo;
                top_sv = __float_as_int(hi) & 0x7F800000;
            }
            // digits of a term p sv of row r, in the unit 2^(f - 127 - 27 + spare) (f: in place of
            // a float's exponent); returns the unit.  Units end at 2^-126.
            auto digits = [&](int r, float term, int f, int spare) -> float {
                f = max(f, 28 << 23);
                const uint32_t y = __float2uint_rn(term * __int_as_float(((281 - spare) << 23) - f));  // below 2^28
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    p_w[sw128_offset(k * R + r, key / 16) + key % 16] = static_cast<unsigned char>(y >> (7 * k) & 0x7Fu);
                return __int_as_float(f - ((27 - spare) << 23));
            };
            float *mnext = maxima + (m == maxima ? R : 0);
            if (key < R)
                mnext[key] = fmaxf(fmaxf(fmaxf(tops[key], tops[TW + key]), fmaxf(tops[2 * TW + key], tops[3 * TW + key])), m[key]);
#pragma unroll
            for (int r0 = 0; r0 < R; r0 += 4) {
                float mo[4], mn[4], mt[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // mt: of this tile
                *reinterpret_cast<float4 *>(mo) = *reinterpret_cast<const float4 *>(m + r0);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float4 g = *reinterpret_cast<const float4 *>(tops + w * TW + r0);
                    mt[0] = fmaxf(mt[0], g.x);
                    mt[1] = fmaxf(mt[1], g.y);
                    mt[2] = fmaxf(mt[2], g.z);
                    mt[3] = fmaxf(mt[3], g.w);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) mn[e] = fmaxf(mo[e], mt[e]);
                if (mn[0] != mo[0] || mn[1] != mo[1] || mn[2] != mo[2] || mn[3] != mo[3]) {  // (the same for all)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float f = mo[e] == -INFINITY ? (l[r0 + e] == 0.f ? 0.f : 1.f) : ex2_approx(mo[e] - mn[e]);
                        o[r0 + e] *= f;
                        l[r0 + e] *= f;
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = r0 + e;
                    const float p = ex2_approx(s[r0 + e] - (mn[e] == -INFINITY ? 0.f : mn[e]));
                    l[r0 + e] += p;
                    if (I8) {
                        s[r0 + e] = p * sv;
                        if (alike) {
                            // p <= 2^(mt - mn), so the terms are below 2^(f + 1) (one bit is spared for the
                            // approximation of p), and the largest is not below 2^(f - 3)
                            const float up = __fadd_ru(fmaxf(mt[e] - mn[e], -127.f), 12582912.f);  // 1.5 2^23: rounds up to an integer
                            s[r0 + e] = digits(r, s[r0 + e], top_sv + static_cast<int>(__float_as_uint(up) << 23), 1);
                        }
                    } else {
                        // hi: the largest bf16 below p (0 for 0, so that masked keys are zeros)
                        const uint32_t u = __float_as_uint(p), h = (u - (u != 0)) & 0xFFFF0000u;
                        const __nv_bfloat16 hi = __ushort_as_bfloat16(static_cast<unsigned short>(h >> 16));
                        const __nv_bfloat16 lo = __float2bfloat16_rn(p - __uint_as_float(h));
                        unsigned char *at = p_w + (key / 64) * T::NO * 128 + key % 8 * 2;
                        *reinterpret_cast<__nv_bfloat16 *>(at + sw128_offset(r, key % 64 / 8)) = hi;
                        *reinterpret_cast<__nv_bfloat16 *>(at + sw128_offset(R + r, key % 64 / 8)) = lo;
                    }
                }
            }
            m = mnext;
            if (I8 && !alike) {
                // the rows' largest terms themselves
#pragma unroll
                for (int r = 0; r < R; r += 4) {
                    const float4 g = make_float4(warp_max(s[r]), warp_max(s[r + 1]), warp_max(s[r + 2]), warp_max(s[r + 3]));
                    if (lane == 0) *reinterpret_cast<float4 *>(tops + quarter * TW + R + r) = g;
                }
                named_barrier(3 + wg, 128);
#pragma unroll
                for (int r = 0; r < R; r += 4) {
                    float g[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const float4 x = *reinterpret_cast<const float4 *>(tops + w * TW + R + r);
                        g[0] = fmaxf(g[0], x.x);
                        g[1] = fmaxf(g[1], x.y);
                        g[2] = fmaxf(g[2], x.z);
                        g[3] = fmaxf(g[3], x.w);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[r + e] = digits(r + e, s[r + e], __float_as_int(g[e]) & 0x7F800000, 0);
                }
            }
            fence_proxy_async_smem();
            tc_fence_before();
            mbar_arrive(p_ready + wg);
            if (i + 2 < end) take_key(i + 2);
            ok = mbar_wait(bar_o + wg, i >> 1 & 1, abort_flag, a.status) && ok;
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int r0 = 0; r0 < R; r0 += 4) {
                uint32_t w[I8 ? 4 : 2][4];
#pragma unroll
                for (int k = 0; k < (I8 ? 4 : 2); ++k) tmem_ld4(tmem_o + k * R + r0, w[k]);
                tmem_wait_ld();
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    o[r0 + r] = I8 ? fmaf(from_digits(w[0][r], w[1][r], w[2 * I8][r] + 128 * w[3 * I8][r]), s[r0 + r], o[r0 + r])
                                   : o[r0 + r] + (__uint_as_float(w[0][r]) + __uint_as_float(w[1][r]));
            }
        }
        it = end;

        // ---- end of the segment: the rows' sums over the key lanes, then both
        // warpgroups' results (merge buffer: the weights', which are all read)
        named_barrier(1, kCompute);  // (both have their last outputs)
        // (halving the rows with each exchange: lane i ends with row i / (32 / R))
#pragma unroll
        for (int k = 16, n = R / 2; k; k >>= 1, n >>= 1) {
            const bool up = lane & k;
            if (n) {
#pragma unroll
                for (int r = 0; r < n; ++r) {
                    const float send = up ? l[r] : l[r + n], keep = up ? l[r + n] : l[r];
                    l[r] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, k);
                }
            } else {
                l[0] += __shfl_xor_sync(0xFFFFFFFFu, l[0], k);
            }
        }
        if (lane % (32 / R) == 0) tops[quarter * TW + lane / (32 / R)] = l[0];
        named_barrier(3 + wg, 128);
        if (key < R) {
            sums[wg * R + key] = (tops[key] + tops[TW + key]) + (tops[2 * TW + key] + tops[3 * TW + key]);
            if (m != maxima) maxima[key] = maxima[R + key];
        }
        float *pool = reinterpret_cast<float *>(p_s);  // [warpgroup][row][column]
        static_assert(2 * T::PBYTES >= 2 * R * 128 * 4, "exchange buffer");
#pragma unroll
        for (int r = 0; r < R; ++r) pool[(wg * R + r) * 128 + key] = o[r];
        named_barrier(1, kCompute);
        const long long prow = walk.slot(found) * R;
#pragma unroll 1
        for (int r = warp; r < R && t.r0 + r < t.rows; r += kCompute / 32) {  // a warp per row
            const float m0 = maxima_s[r], m1 = maxima_s[2 * R + r], l0 = sums[r], l1 = sums[R + r];
            const float top = fmaxf(m0, m1), z = top == -INFINITY ? 0.f : top;
            // (a warpgroup without a key has sums 0; NaN sums stay)
            const float f0 = m0 == -INFINITY ? 1.f : ex2_approx(m0 - z), f1 = m1 == -INFINITY ? 1.f : ex2_approx(m1 - z);
            const float sum = l0 * f0 + l1 * f1;
            float inv = sum == 0.f ? 0.f : 1.f / sum;
            if (I8 && poison[r]) inv = __uint_as_float(0x7FC00000u);
            const float lse2 = sum == 0.f ? -INFINITY : z + __log2f(sum);
            const int row = t.r0 + r, tok = static_cast<int>(a.by_g.quotient(row));
            const long long orow = (static_cast<long long>(walk.s.cu0) + tok) * a.Hq + static_cast<long long>(walk.h) * a.G + (row - tok * a.G);
#pragma unroll
            for (int c = 2 * lane; c < D; c += 64) {
                const float2 x = *reinterpret_cast<const float2 *>(pool + r * 128 + c), y = *reinterpret_cast<const float2 *>(pool + (R + r) * 128 + c);
                const float u = (x.x * f0 + y.x * f1) * inv, v = (x.y * f0 + y.y * f1) * inv;
                if (walk.whole)
                    *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(a.out) + orow * D + c) = __floats2bfloat162_rn(u, v);
                else
                    *reinterpret_cast<float2 *>(a.part_o + (prow + r) * D + c) = make_float2(u, v);
            }
            if (lane == 0) {
                if (walk.whole)
                    a.lse[orow] = lse2 * kLn2f;
                else
                    a.part_lse[prow + r] = lse2;
            }
        }
        if (!walk.whole) {
            // the last of the segment's pieces to be finished merges them
            const int c0 = walk.first_run(found), c1 = walk.last_run(found);
            int *counter = a.counters + c0 * a.heads + blockIdx.x % a.heads;
            named_barrier(1, kCompute);
            if (tid == 0) {
                __threadfence();  // (the barrier has ordered the other threads' writes before it)
                *last_piece = atomicAdd(counter, 1) == c1 - c0;
            }
            named_barrier(1, kCompute);
            if (*last_piece) {
                __threadfence();
                merge_pieces<D, R>(a, t, walk.s.cu0, walk.h, c0, c1 - c0 + 1, reinterpret_cast<float *>(p_s), tops_s);
                if (tid == 0) *counter = 0;  // as the next call expects it
            }
        } else {
            named_barrier(1, kCompute);  // tops and the Q buffer are free
        }
    }
    tc_fence_before();
    named_barrier(2, kCompute + 32);
}

template <int D, bool I8, int R>
cudaError_t launch(const PagedAttn &a, const CUtensorMap &tk, const CUtensorMap &tv, int num_sms,
                   cudaStream_t st) {
    using T = Tile<D, I8, R>;
    constexpr size_t smem = split_smem_bytes<D, I8, R>();
    static_assert(T::CTAS * (smem + 1024) <= 228 * 1024, "shared memory of an SM");
    const cudaError_t e = cudaFuncSetAttribute(
        split_attn_kernel<D, I8, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    const int ctas = T::CTAS * num_sms < kSplitMaxCtas ? T::CTAS * num_sms : kSplitMaxCtas;
    split_attn_kernel<D, I8, R><<<ctas / a.heads * a.heads, kThreads, smem, st>>>(tk, tv, a);
    return cudaGetLastError();
}

template <int D, bool I8>
cudaError_t launch_rows(const PagedAttn &a, int rows, const CUtensorMap &tk, const CUtensorMap &tv,
                        int num_sms, cudaStream_t st) {
    if (rows <= 8) return launch<D, I8, 8>(a, tk, tv, num_sms, st);
    return launch<D, I8, 16>(a, tk, tv, num_sms, st);
}

}  // namespace

cudaError_t launch_split_attn(const PagedAttn &a, int rows, const CUtensorMap &tk,
                              const CUtensorMap &tv, int num_sms, cudaStream_t st) {
    if (a.c.d == 128)
        return a.c.k_scales ? launch_rows<128, true>(a, rows, tk, tv, num_sms, st)
                            : launch_rows<128, false>(a, rows, tk, tv, num_sms, st);
    return a.c.k_scales ? launch_rows<64, true>(a, rows, tk, tv, num_sms, st)
                        : launch_rows<64, false>(a, rows, tk, tv, num_sms, st);
}

}  // namespace msa
