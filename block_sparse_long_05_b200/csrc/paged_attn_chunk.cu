// paged_attn_chunk.cu -- attention of a chunk of new tokens over a paged cache
// (more than 16 query rows per sequence and kv head; formulas as in
// paged_attn_split.cu).
//
// The matrix products bound it: 4 d flops per (row, key).  A CTA takes 256 rows
// (i * G + g, token i, head g) of one kv head as two tiles of 128 and walks the
// keys 128 at a time:
//     S = Q K^T (tensor memory), P = 2^(S c - m) in bf16 over S, O += P V
// with the two row tiles half a step apart, so that one tile's products run
// while the other tile is in its softmax.  Both products read K and V from
// shared memory as TMA left them; P never leaves tensor memory.  Two warpgroups
// share a row tile, 64 of the 128 keys each: a thread has half a row of S, in
// two passes of 32 scores (first the maximum, then the weights), and takes no
// shuffles.  The running reference m may lag behind the maximum, since weights
// and sums are floating point numbers: it is raised, and O rescaled, only when
// a score passes it by 2^8, which one vote per tile finds out.  (Weights are
// 256 at most, so that values of V up to 2^100 stay in the range of fp32.)
//
// int8 pages: eight warps turn the codes into bf16 tiles (exact) ahead of the
// products; the scales sk multiply the scores and sv the weights in fp32.
//
// P (with int8 pages: P times sv) is rounded to bf16, a relative error of at most
// 2^-8 per weight, averaged over the keys; the sum l takes the unrounded values.
// The output's own rounding is as large, and a second term would double the
// second product.
//
// The work is cut into equal runs of key tiles, one CTA per SM (paged_walk.cuh).
// Segments in several runs leave fp32 pieces that a second kernel merges.  At a
// segment's end the next one's Q is on its way, and its first products run,
// before this one's outputs are written.
//
// Measured, in a replayed graph: 2048 tokens of 32 heads over 32768 keys, bf16,
// d 128: 1.26 ms = 0.85 PFLOP/s, 51% of a large library product, 14 us of it the
// merge (at the card's power limit, 1540 MHz in a loop; 1.08 ms before it is
// reached); 8192 tokens in a window of 1024: 215 us = 0.60 PFLOP/s of visible
// pairs (int8: 334 us); six int8 contexts of up to 12007 keys with 2215 new
// tokens of 64 heads: 0.88 ms = 0.62 PFLOP/s.  A step of a row tile takes about 4100 clocks: 1700 until the scores
// of the next 128 keys are there (its own two products and the other tile's,
// 512 clocks each, and the way there), 500 for the maximum, 150 for the vote,
// 1450 for the weights.  S and P share columns, and with O they fill tensor
// memory, so the next scores cannot be computed ahead.  With int8 the scales and
// the conversion take shared memory's time: 6300 clocks.
// Slower: weights kept in registers in one pass (1225 against 1184 us; the loop
// no longer fits the instruction cache), a part of the exponentials as
// polynomials (+2% with an eighth of them, +7% with a half), two steps of P
// (bf16 -1%, int8 +6%), a fourth stage for int8 tiles instead of buffers for
// their codes (+3%).
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

constexpr int kRows = kChunkRows;
constexpr int kOver = 4;       // a segment's start and end cost about as much as two to four
                               // tiles (2, 3 and 6 here are within 1%)
constexpr int kMinRun = 5;     // units per run, at least
constexpr int kMetaSlots = 8;  // tiles whose positions and scales are kept: more than
                               // the rings of K and V tiles hold at a time
constexpr float kLag = 8.f;    // powers of two by which a weight may pass 1
constexpr float kLn2f = 0.6931471805599453f;

template <int D, bool I8>
struct Chunk {
    static constexpr int REGS = D / 64;            // 128-byte wide regions of a bf16 tile
    static constexpr int TILE = REGS * 128 * 128;  // bf16 tile: 128 rows
    static constexpr int RAW = 128 * D;            // tile of codes
    static constexpr int STAGES = I8 ? (D == 128 ? 3 : 6) : (D == 128 ? 5 : 8);  // bf16 tiles of K or V
    static constexpr int RAWS = I8 ? (D == 128 ? 3 : 4) : 0;                     // tiles of codes
    // warps 0-15: softmax; 16-23: int8 conversion; then a producer and a product
    // warp, and two that fill up their warpgroup.  Registers per thread: at launch
    // THREADS * LAUNCH of the SM's 65536, then split anew.
    static constexpr int CONV = I8 ? 8 : 0;
    static constexpr int THREADS = I8 ? 896 : 640;
    static constexpr int LAUNCH = I8 ? 72 : 96;
    static constexpr int REST = I8 ? 40 : 64;
    static constexpr int SOFTMAX = I8 ? 96 : 104;
    static_assert(512 * SOFTMAX + (THREADS - 512) * REST <= THREADS * LAUNCH && THREADS * LAUNCH <= 65536, "registers");
};

struct alignas(16) TileMeta {
    int pos;    // first key
    int valid;  // bit i: keys 32 i .. 32 i + 31 are there
    int pad[2];
};

template <int D, bool I8>
constexpr size_t chunk_smem_bytes() {
    using C = Chunk<D, I8>;
    return static_cast<size_t>(2 + C::STAGES) * C::TILE + C::RAWS * (C::RAW + 1024) +
           kMetaSlots * (sizeof(TileMeta) + 8 + (I8 ? 1024 : 0)) + 2048 +
           (2 * C::STAGES + 2 * C::RAWS + 9) * 8 + 64;
}

// 16 bytes to shared memory, zeros if they are not there.
__device__ __forceinline__ void cp_async16(void *dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ uint32_t bf2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Two signed bytes (the low bytes of the 16-bit halves of x) as bf16, exactly:
// 128 + (low 7 bits), minus 128, or minus 256 where the sign bit is set.
// 0x4300 is 128 in bf16, whose last mantissa bit counts 1; the byte's sign bit
// falls on the lowest exponent bit, and 0x4380 is 256.
__device__ __forceinline__ uint32_t s8x2_bf16(uint32_t x) {
    const uint32_t hi = (x & 0x007F007Fu) | 0x43004300u, lo = (x & 0x00800080u) | 0x43004300u;
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&hi),
                                     *reinterpret_cast<const __nv_bfloat162 *>(&lo));
    return *reinterpret_cast<const uint32_t *>(&r);
}

template <int D, bool I8>
__global__ void __launch_bounds__(Chunk<D, I8>::THREADS, 1) chunk_attn_kernel(
    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
    const __grid_constant__ PagedAttn a) {
    using C = Chunk<D, I8>;
    constexpr int EB = I8 ? 1 : 2;
    constexpr int RS = C::RAWS > 0 ? C::RAWS : 1;
    extern __shared__ __align__(1024) unsigned char q_s[];  // [row tile]
    unsigned char *ring = q_s + 2 * C::TILE;             // [stage]
    unsigned char *raw = ring + C::STAGES * C::TILE;     // [raw stage]
    float *raw_sc = reinterpret_cast<float *>(raw + C::RAWS * C::RAW);   // [raw stage][K, V][128]
    float *scales = raw_sc + C::RAWS * 256;                              // [slot][K, V][128]
    float *halves = scales + (I8 ? kMetaSlots * 256 : 0);  // [row tile][half][row]: maxima, then sums
    TileMeta *meta = reinterpret_cast<TileMeta *>(halves + 512);
    uint64_t *meta_full = reinterpret_cast<uint64_t *>(meta + kMetaSlots);
    uint64_t *full = meta_full + kMetaSlots, *empty = full + C::STAGES;
    uint64_t *raw_full = empty + C::STAGES, *raw_empty = raw_full + C::RAWS;
    uint64_t *bar_s = raw_empty + C::RAWS;  // [row tile] scores complete
    uint64_t *bar_o = bar_s + 2;            // [row tile] outputs complete
    uint64_t *p_ready = bar_s + 4;          // [row tile] weights written
    uint64_t *q_ready = bar_s + 6;          // [row tile] Q of a segment written
    uint64_t *edge = bar_s + 8;             // a V tile that gets zeros
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar_s + 9);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kProducer = 16 + C::CONV, kProducts = kProducer + 1;
    if (tid == 0) {
        for (int i = 0; i < kMetaSlots; ++i) mbar_init(meta_full + i, I8 ? 128 : 1);
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(full + i, I8 ? 256 : 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < C::RAWS; ++i) {
            mbar_init(raw_full + i, 1);
            mbar_init(raw_empty + i, 256);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_s + i, 1);
            mbar_init(bar_o + i, 1);
            mbar_init(p_ready + i, 256);
            mbar_init(q_ready + i, 256);
        }
        mbar_init(edge, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }
    const Found found = find_run(a, kRows, kOver, kMinRun);
    if (found.start >= found.work) return;
    if (warp == kProducts) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;  // S / P of the row tiles, then O of the row tiles: 128 columns each
    Walk walk(a, found, kOver);
    const int block = a.step.block;
    // (each branch begins with its warpgroup's register request)
    if (warp >= 16) {
        if (I8 && warp < kProducer) {
            fewer_registers<C::REST>();
            // -------------------------------------------------------- int8 -> bf16
            // Thread: half a row of the tile; rows of 16-byte pieces, swizzled on both
            // sides so that eight neighbouring rows fall on different banks.
            const int r = tid & 127, half = warp >> 2 & 1;
            uint32_t e = 0, slot = 0;
            bool ok = true;
            auto convert = [&](bool is_v) {
                const uint32_t rs = e % RS, st = e % C::STAGES;
                ok = mbar_wait(raw_full + rs, (e / RS) & 1, abort_flag, a.status);
                if (ok && e >= static_cast<uint32_t>(C::STAGES))
                    ok = mbar_wait(empty + st, ((e / C::STAGES) & 1) ^ 1, abort_flag, a.status);
                if (!ok) return;
                const unsigned char *src = raw + rs * C::RAW;
                unsigned char *dst = ring + st * C::TILE;
                if (!is_v && half == 0) {
                    float *sc = scales + slot % kMetaSlots * 256;
                    sc[r] = raw_sc[rs * 256 + r];
                    sc[128 + r] = raw_sc[rs * 256 + 128 + r];
                    mbar_arrive(meta_full + slot % kMetaSlots);
                    ++slot;
                }
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const int p = half * (D / 32) + i;
                    const uint32_t at = D == 128 ? sw128_offset(r, p) : r * 64u + ((p ^ ((r >> 1) & 3u)) << 4);
                    const uint4 u = *reinterpret_cast<const uint4 *>(src + at);
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
                    uint32_t o[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        o[2 * k] = s8x2_bf16(__byte_perm(w[k], 0, 0x1100));
                        o[2 * k + 1] = s8x2_bf16(__byte_perm(w[k], 0, 0x3322));
                    }
                    unsigned char *to = dst + p / 4 * 16384;
                    *reinterpret_cast<uint4 *>(to + sw128_offset(r, p % 4 * 2)) = make_uint4(o[0], o[1], o[2], o[3]);
                    *reinterpret_cast<uint4 *>(to + sw128_offset(r, p % 4 * 2 + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
                }
                fence_proxy_async_smem();
                mbar_arrive(full + st);
                mbar_arrive(raw_empty + rs);
                ++e;
            };
            while (ok && walk.next(a, kRows)) {
                const RowTile t = row_tile(a, walk.s, walk.rt, kRows);
                const int n = min(walk.x1, t.count) - walk.x0;
                for (int x = 0; x < n && ok; ++x) {
                    convert(false);
                    if (x > 0 && ok) convert(true);
                }
                if (n > 0 && ok) convert(true);
            }
            return;
        }
        fewer_registers<C::REST>();
        if (warp == kProducer) {
            // -------------------------------------------------------- producer
            // Order of the tiles: K 0, then K x + 1 and V x in turn.
            uint32_t e = 0, edges = 0;  // tiles issued; V tiles with zeros
            uint32_t slot = 0;          // key tiles announced
            const int box = min(block, kKeys);
            bool ok = true;
            // One tile of K or V: keys at pos.. (valid quarters), store rows z.  Some
            // row of the segment sees the keys below hi that are sinks or from lo on.
            auto load = [&](bool is_v, int pos, int valid, const int (&z)[4], int h, int lo, int hi, uint32_t sl) {
                const uint32_t st = e % (I8 ? RS : C::STAGES), ph = e / (I8 ? RS : C::STAGES);
                uint64_t *fb = I8 ? raw_full + st : full + st;
                unsigned char *dst = I8 ? raw + st * C::RAW : ring + st * C::TILE;
                // rows of V that no row may use are zeroed (bf16: they may hold anything,
                // and 0 times it need not be 0)
                const bool zeros = !I8 && is_v && (valid != 15 || pos + kKeys > hi || (pos < lo && pos + kKeys > a.sinks));
                if (lane == 0) {
                    if (e >= static_cast<uint32_t>(I8 ? RS : C::STAGES))
                        ok = mbar_wait((I8 ? raw_empty : empty) + st, (ph & 1) ^ 1, abort_flag, a.status);
                    if (ok) {
                        if (!is_v) {
                            meta[sl % kMetaSlots].pos = pos;
                            meta[sl % kMetaSlots].valid = valid;
                            if (!I8) mbar_arrive(meta_full + sl % kMetaSlots);
                        }
                        uint64_t *tb = zeros ? edge : fb;
                        int boxes = 0;
#pragma unroll
                        for (int i = 0; i < 4; ++i) boxes += i * 32 % box == 0 && (valid >> i & 1);
                        if (boxes == 0)
                            mbar_arrive(tb);
                        else
                            mbar_arrive_expect_tx(tb, boxes * box * (D * EB + (I8 && !is_v ? 8 : 0)));
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (i * 32 % box != 0 || !(valid >> i & 1)) continue;
                            if (I8) {
                                tma_load_3d(dst + i * 32 * D, is_v ? &tm_v : &tm_k, tb, 0, h, z[i]);
                                if (!is_v) {
                                    const int page = static_cast<int>(a.by_block.quotient(z[i]));
                                    const long long so = (static_cast<long long>(page) * a.c.Hkv + h) * block + (z[i] - page * block);
                                    bulk_load(raw_sc + st * 256 + i * 32, a.c.k_scales + so, box * 4, tb);
                                    bulk_load(raw_sc + st * 256 + 128 + i * 32, a.c.v_scales + so, box * 4, tb);
                                }
                            } else {
#pragma unroll
                                for (int r = 0; r < C::REGS; ++r)
                                    tma_load_3d(dst + r * 16384 + i * 4096, is_v ? &tm_v : &tm_k, tb, r * 64, h, z[i]);
                            }
                        }
                        if (zeros) ok = mbar_wait(edge, edges & 1, abort_flag, a.status);
                    }
                }
                ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
                if (ok && zeros) {
                    ++edges;
                    mbar_try_wait(edge, (edges - 1) & 1);  // (complete: orders this lane's writes behind the copy's)
                    for (int r = lane; r < kKeys; r += 32) {
                        const int p = pos + r;
                        if ((valid >> (r / 32) & 1) && p < hi && (p >= lo || p < a.sinks)) continue;
#pragma unroll
                        for (int c = 0; c < 8 * C::REGS; ++c)
                            *reinterpret_cast<uint4 *>(dst + c / 8 * 16384 + r * 128 + ((c + lane) & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(fb);
                }
                if (ok) ++e;
            };
            while (ok && walk.next(a, kRows)) {
                const RowTile t = row_tile(a, walk.s, walk.rt, kRows);
                const int x1 = min(walk.x1, t.count);
                const int hi = min(t.tmax + 1, walk.s.cap);
                const int lo = a.window ? t.tmin - a.window + 1 : 0;
                int vp = 0, vv = 0, vz[4] = {0, 0, 0, 0};  // the V tile that follows the next K tile
                for (int xb = walk.x0; xb < x1 && ok; xb += 32) {
                    int pos = 0, valid = 0, z[4] = {0, 0, 0, 0};
                    const int x = xb + lane;
                    if (x < x1) {
                        pos = (x < t.na ? x : x + t.skip) * kKeys;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (i > 0 && i * 32 % box != 0) {
                                valid |= (valid >> (i - 1) & 1) << i;
                                continue;
                            }
                            const int p = pos + i * 32;
                            // (keys before every row's window: their page may be gone)
                            if (p >= hi || (p + box <= lo && p >= a.sinks)) continue;
                            const int j = a.by_block.quotient(p);
                            const int page = a.step.pm.table[static_cast<long long>(walk.b) * a.step.pm.stride + j];
                            if (page < 0 || page >= a.step.pm.count) {
                                atomicOr(a.status, kDevBadIds);
                                continue;
                            }
                            valid |= 1 << i;
                            z[i] = page * block + (p - j * block);
                        }
                    }
                    const int m = min(32, x1 - xb);
                    for (int y = 0; y < m && ok; ++y) {
                        const int p = __shfl_sync(0xFFFFFFFFu, pos, y), v = __shfl_sync(0xFFFFFFFFu, valid, y);
                        int zz[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) zz[i] = __shfl_sync(0xFFFFFFFFu, z[i], y);
                        load(false, p, v, zz, walk.h, lo, hi, slot);
                        ++slot;
                        if (xb + y > walk.x0 && ok) load(true, vp, vv, vz, walk.h, lo, hi, 0);
                        vp = p;
                        vv = v;
#pragma unroll
                        for (int i = 0; i < 4; ++i) vz[i] = zz[i];
                    }
                }
                if (ok && x1 > walk.x0) load(true, vp, vv, vz, walk.h, lo, hi, 0);
            }
            // after an abort: the copies have landed before the CTA ends
            if (!ok && lane == 0) {
                const uint32_t n = I8 ? RS : C::STAGES;
                for (uint32_t i = e > n ? e - n : 0; i < e; ++i) {
                    const uint64_t t0 = global_timer_ns();
                    while (!mbar_try_wait((I8 ? raw_full : full) + i % n, (i / n) & 1))
                        if (global_timer_ns() - t0 > kWaitLimitNs / 4) break;
                }
            }
            return;
        }

        if (warp == kProducts) {
            // -------------------------------------------------------- products
            if (lane == 0) {
                constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, false), idesc_o = idesc_bf16_f32(128, D, true);
                const uint64_t q0 = sdesc_sw128(smem_addr(q_s), 16, 1024), k0 = sdesc_sw128(smem_addr(ring), 16, 1024);
                const uint64_t v0 = sdesc_sw128(smem_addr(ring), 16384, 1024);
                uint32_t e = 0, nq[2] = {0, 0}, np[2] = {0, 0};  // ring tiles taken; Q and weights awaited
                bool ok = true;
                auto scores = [&](int t, uint32_t st) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t o = (k / 4) * 16384 + (k % 4) * 32;
                        umma_bf16(tmem + t * 128, q0 + ((t * C::TILE + o) >> 4), k0 + ((st * C::TILE + o) >> 4), idesc_s, k > 0);
                    }
                    umma_commit(bar_s + t);
                };
                while (ok && walk.next(a, kRows)) {
                    const RowTile rt = row_tile(a, walk.s, walk.rt, kRows);
                    const int n = min(walk.x1, rt.count) - walk.x0;
                    const int tiles = rt.rows - rt.r0 > 128 ? 2 : 1;
                    if (n <= 0) continue;
                    for (int t = 0; t < tiles && ok; ++t) ok = mbar_wait(q_ready + t, nq[t]++ & 1, abort_flag, a.status);
                    if (!ok) break;
                    uint32_t st = e % C::STAGES;
                    if (!(ok = mbar_wait(full + st, (e / C::STAGES) & 1, abort_flag, a.status))) break;
                    tc_fence_after();
                    for (int t = 0; t < tiles; ++t) scores(t, st);
                    umma_commit(empty + st);
                    ++e;
                    for (int x = 0; x < n && ok; ++x) {
                        const bool more = x + 1 < n;
                        const uint32_t ek = e, ev = more ? e + 1 : e;
                        const uint32_t sk = ek % C::STAGES, sv = ev % C::STAGES;
                        if (!(ok = mbar_wait(full + sv, (ev / C::STAGES) & 1, abort_flag, a.status))) break;
                        for (int t = 0; t < tiles; ++t) {
                            if (!(ok = mbar_wait(p_ready + t, np[t]++ & 1, abort_flag, a.status))) break;
                            tc_fence_after();
#pragma unroll
                            for (int k = 0; k < kKeys / 16; ++k)
                                umma_bf16_tmem_a(tmem + 256 + t * 128, tmem + t * 128 + (k / 4) * 64 + (k % 4) * 8,
                                                 v0 + ((sv * C::TILE + k * 16 * 128) >> 4), idesc_o, x > 0 || k > 0);
                            umma_commit(bar_o + t);
                            if (more) {
                                if (t == 0 && !(ok = mbar_wait(full + sk, (ek / C::STAGES) & 1, abort_flag, a.status))) break;
                                tc_fence_after();
                                scores(t, sk);
                            }
                        }
                        if (!ok) break;
                        umma_commit(empty + sv);
                        if (more) umma_commit(empty + sk);
                        e = ev + 1;
                    }
                }
            }
            __syncwarp();
            named_barrier(2, 512 + 32);  // the softmax warps have read their last outputs
            tmem_dealloc(tmem, 512);
            return;
        }

        return;
    }

    more_registers<C::SOFTMAX>();
    // ------------------------------------------------------------ softmax
    // Two warpgroups per row tile, 64 of a tile's 128 keys each; a thread has a
    // row.  Its weights go over the first half of its own score columns.
    const int t = warp >> 3, half = warp >> 2 & 1, row = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tmem_s = tmem + t * 128 + half * 64 + lanes, tmem_o = tmem + 256 + t * 128 + half * (D / 2) + lanes;
    const uint64_t c2 = f2_pack(a.scale_log2, a.scale_log2);
    float *mine_x = halves + (t * 2 + half) * 128 + row;
    const float *other_x = halves + (t * 2 + (half ^ 1)) * 128 + row;
    uint32_t slot = 0, n_s = 0;  // key tiles; products awaited
    bool ok = true;
    // Q rows of the segment's tile to shared memory, if the segment has keys: the
    // copies are started, and announced later
    auto start_q = [&]() -> bool {
        const RowTile rt = row_tile(a, walk.s, walk.rt, kRows);
        const int first = rt.r0 + t * 128;
        if ((t == 1 && rt.rows <= first) || min(walk.x1, rt.count) <= walk.x0) return false;
        constexpr int PPR = D / 8, STEP = 256 / PPR;
        const int c = row % PPR, r0 = (row + half * 128) / PPR;
        const int step_tok = a.by_g.quotient(STEP), step_g = STEP - step_tok * a.G;
        int tok = a.by_g.quotient(first + r0), g = first + r0 - tok * a.G;
        const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(a.q) + walk.s.cu0 * a.q_stride +
                                   static_cast<long long>(walk.h) * a.G * D + c * 8;
#pragma unroll
        for (int i = 0; i < PPR / 2; ++i) {
            const bool there = first + r0 + i * STEP < rt.rows;  // (zeros otherwise)
            cp_async16(q_s + t * C::TILE + (c / 8) * 16384 + sw128_offset(r0 + i * STEP, c % 8),
                       there ? src + tok * a.q_stride + g * D : src, there);
            tok += step_tok;
            g += step_g;
            if (g >= a.G) {
                g -= a.G;
                ++tok;
            }
        }
        return true;
    };
    auto announce_q = [&]() {
        cp_async_wait_all();
        fence_proxy_async_smem();
        mbar_arrive(q_ready + t);
    };
    bool more = walk.next(a, kRows);
    if (more && start_q()) announce_q();
    while (more) {
        const RowTile rt = row_tile(a, walk.s, walk.rt, kRows);
        const int x0 = walk.x0, x1 = min(walk.x1, rt.count);
        const bool idle = t == 1 && rt.rows - rt.r0 <= 128;  // no rows in this tile
        const int first = rt.r0 + t * 128;                   // first row of the tile
        const int mine = first + row, tok = static_cast<int>(a.by_g.quotient(mine));
        const bool live = mine < rt.rows;
        const int tpos = live ? min(walk.s.off + tok, walk.s.cap - 1) : -1;  // last key that the row sees
        const int wpos = a.window && live ? walk.s.off + tok - a.window : -1;  // a key at or before it is out,
                                                                               // unless a sink
        // the tile's rows, for the choice of the masked path
        const int tmin = min(walk.s.off + static_cast<int>(a.by_g.quotient(first)), walk.s.cap - 1);
        const int tmax = walk.s.off + static_cast<int>(a.by_g.quotient(min(first + 128, rt.rows) - 1));

        const bool any = x1 > x0, whole = walk.whole;
        const long long prow = walk.slot(found) * kRows + t * 128 + row;
        const long long orow = (static_cast<long long>(walk.s.cu0) + tok) * a.Hq + static_cast<long long>(walk.h) * a.G + (mine - tok * a.G);
        more = walk.next(a, kRows);  // (here, where the first scores are awaited)

        float m = -INFINITY, l = 0.f;
        for (int x = x0; x < x1; ++x, ++slot) {
            if (idle || !ok) continue;
            ok = mbar_wait(meta_full + slot % kMetaSlots, (slot / kMetaSlots) & 1, abort_flag, a.status) &&
                 mbar_wait(bar_s + t, n_s & 1, abort_flag, a.status);
            __syncwarp();
            tc_fence_after();
            const int pos = meta[slot % kMetaSlots].pos, valid = meta[slot % kMetaSlots].valid;
            const float *sk = scales + slot % kMetaSlots * 256 + half * 64, *sv = sk + 128;
            const bool masked = valid != 15 || pos + kKeys - 1 > tmin ||
                                (a.window && pos <= tmax - a.window && pos + kKeys > a.sinks);
            // 32 scores, times sk; keys that the row does not see are -inf
            auto scores = [&](int c, uint32_t(&y)[32]) {
                tmem_ld32(tmem_s + c * 32, y);
                tmem_wait_ld();
                if (I8) {
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 k4 = *reinterpret_cast<const float4 *>(sk + c * 32 + i);
                        float f0, f1, f2, f3;
                        f2_unpack(f2_mul(f2_pack(__uint_as_float(y[i]), __uint_as_float(y[i + 1])), f2_pack(k4.x, k4.y)), f0, f1);
                        f2_unpack(f2_mul(f2_pack(__uint_as_float(y[i + 2]), __uint_as_float(y[i + 3])), f2_pack(k4.z, k4.w)), f2, f3);
                        y[i] = __float_as_uint(f0);
                        y[i + 1] = __float_as_uint(f1);
                        y[i + 2] = __float_as_uint(f2);
                        y[i + 3] = __float_as_uint(f3);
                    }
                }
            };
            // keys of the 32 that the row sees, one bit each
            auto visible = [&](int c) -> uint32_t {
                auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; };
                const int k0 = pos + half * 64 + c * 32;
                uint32_t bits = below(tpos + 1 - k0);
                if (a.window) bits &= ~below(wpos + 1 - k0) | below(a.sinks - k0);
                return valid >> (half * 2 + c) & 1 ? bits : 0u;
            };
            // (at a mask's edge most warps have 32 keys that all rows see)
            auto mask = [&](uint32_t bits, uint32_t(&y)[32]) {
                if (!__any_sync(0xFFFFFFFFu, bits != 0xFFFFFFFFu)) return;
#pragma unroll
                for (int i = 0; i < 32; ++i) y[i] = bits >> i & 1 ? y[i] : 0xFF800000u;
            };
            // ---- the row's maximum
            float g = -INFINITY;
            // (not unrolled: copies of the body run slower, for want of instruction cache)
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
                uint32_t y[32];
                scores(c, y);
                if (masked) mask(visible(c), y);
                float g4[4] = {g, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < 32; i += 8)
#pragma unroll
                    for (int k = 0; k < 4; ++k) g4[k] = fmax3(g4[k], __uint_as_float(y[i + k]), __uint_as_float(y[i + 4 + k]));
                g = fmaxf(fmax3(g4[0], g4[1], g4[2]), g4[3]);
            }
            g *= a.scale_log2;
            // Weights and sums are floating point numbers, so the reference m may lag
            // behind the maximum: it is raised (with O and l) when a score of some row of
            // the tile passes it by 2^kLag, and at first.
            if (named_barrier_or(3 + t, 256, g > m + kLag || !ok)) {
                *mine_x = g;
                named_barrier(3 + t, 256);
                const float mn = fmaxf(m, fmaxf(g, *other_x));
                const float f = m == -INFINITY ? 1.f : ex2_approx(m - mn);  // (nothing, or NaN, so far)
                m = mn;
                l *= f;
                if (x > x0) {  // O of the tiles before, complete by now or soon
                    ok = ok && mbar_wait(bar_o + t, (n_s - 1) & 1, abort_flag, a.status);
                    __syncwarp();
                    tc_fence_after();
#pragma unroll 1
                    for (int k = 0; k < D / 2; k += 16) {
                        uint32_t w[16];
                        tmem_ld16(tmem_o + k, w);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * f);
                        tmem_st16(tmem_o + k, w);
                    }
                }
                // (*other_x is read before it is written again: a whole tile lies between)
                if (named_barrier_or(3 + t, 256, !ok)) {
                    ok = false;
                    continue;
                }
            }
            // ---- the weights, over score columns that have been read
            const float mr = m == -INFINITY ? 0.f : m;
            const uint64_t nm = f2_pack(-mr, -mr);
            uint64_t la = f2_pack(0.f, 0.f), lb = la;
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
                uint32_t y[32], w[16];
                scores(c, y);
                uint32_t bits = 0xFFFFFFFFu;
                if (masked) mask(bits = visible(c), y);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float e0, e1;
                    f2_unpack(f2_fma(f2_pack(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1])), c2, nm), e0, e1);
                    uint64_t p = f2_pack(ex2_approx(e0), ex2_approx(e1));  // (masked columns: 0)
                    if (i & 1)
                        lb = f2_add(lb, p);
                    else
                        la = f2_add(la, p);
                    if (I8) {
                        const float2 s2 = *reinterpret_cast<const float2 *>(sv + c * 32 + 2 * i);
                        p = f2_mul(p, f2_pack(s2.x, s2.y));
                    }
                    float p0, p1;
                    f2_unpack(p, p0, p1);
                    w[i] = bf2(p0, p1);
                }
                if (I8 && masked) {  // a masked key's scale may hold anything
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        w[i] &= (bits >> (2 * i) & 1 ? 0x0000FFFFu : 0u) | (bits >> (2 * i + 1) & 1 ? 0xFFFF0000u : 0u);
                }
                tmem_st16(tmem_s + c * 16, w);
            }
            float l0, l1, l2, l3;
            f2_unpack(la, l0, l1);
            f2_unpack(lb, l2, l3);
            l += (l0 + l1) + (l2 + l3);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(p_ready + t);
            ++n_s;
        }
        // the next segment's Q (the last scores of this one are complete), so that
        // its first products run beside these outputs
        const bool fetched = more && start_q();
        if (idle) {
            if (fetched) announce_q();
            continue;
        }

        // ---- outputs: final, or a piece; half of the columns each
        *mine_x = l;
        named_barrier(3 + t, 256);
        l += *other_x;
        if (any) ok = ok && mbar_wait(bar_o + t, (n_s - 1) & 1, abort_flag, a.status);
        __syncwarp();
        tc_fence_after();
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const float lse2 = l == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m) + __log2f(l);
#pragma unroll 1
        for (int c = 0; c < D / 2; c += 32) {
            uint32_t o[32];
            __syncwarp();
            tmem_ld32(tmem_o + c, o);
            tmem_wait_ld();
            if (fetched && c == 0) announce_q();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(any ? __uint_as_float(o[i]) * inv : 0.f);
            const int col = half * (D / 2) + c;
            if (whole) {
                // two lanes write 32 bytes of a row at a time: first of the even
                // lane's row, then of the odd one's
                const bool odd = lane & 1;
                const long long other = __shfl_xor_sync(0xFFFFFFFFu, live ? orow : -1ll, 1);
                const long long rows2[2] = {odd ? other : live ? orow : -1ll, odd ? live ? orow : -1ll : other};
#pragma unroll
                for (int i = 0; i < 32; i += 16) {
                    uint32_t w[8], x[4];
#pragma unroll
                    for (int k = 0; k < 8; ++k) w[k] = bf2(__uint_as_float(o[i + 2 * k]), __uint_as_float(o[i + 2 * k + 1]));
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[k] = __shfl_xor_sync(0xFFFFFFFFu, odd ? w[k] : w[4 + k], 1);
                    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + col + i + odd * 8;
                    if (rows2[0] >= 0)
                        *reinterpret_cast<uint4 *>(out + rows2[0] * D) =
                            odd ? make_uint4(x[0], x[1], x[2], x[3]) : make_uint4(w[0], w[1], w[2], w[3]);
                    if (rows2[1] >= 0)
                        *reinterpret_cast<uint4 *>(out + rows2[1] * D) =
                            odd ? make_uint4(w[4], w[5], w[6], w[7]) : make_uint4(x[0], x[1], x[2], x[3]);
                }
            } else if (live) {
                uint4 *out = reinterpret_cast<uint4 *>(a.part_o + prow * D + col);
#pragma unroll
                for (int i = 0; i < 8; ++i) out[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
        }
        if (live && half == 0) {
            if (whole)
                a.lse[orow] = lse2 * kLn2f;
            else
                a.part_lse[prow] = lse2;
        }
        tc_fence_before();
        ok = !named_barrier_or(3 + t, 256, !ok);  // (sums are read before the next segment's maxima)
    }
    named_barrier(2, 512 + 32);
}

// ===========================================================================
// Merge of the segments that lie in several runs: CTAs (c, *) take the segment
// that begins in run c and goes on into run c + 1, if there is one, 64 rows
// each, 8 per warp:  lse = log2 sum 2^lse_p,  out = sum 2^(lse_p - lse) o_p.
// ===========================================================================
constexpr int kMergeThreads = 256, kMergeRows = 64;  // 8 rows per warp

template <int D>
__global__ void __launch_bounds__(kMergeThreads) chunk_merge_kernel(const __grid_constant__ PagedAttn a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the pieces come from the previous kernel
    constexpr int COLS = D / 32, RW = kMergeRows * 32 / kMergeThreads;
    Found f = find_run(a, kRows, kOver, kMinRun, true);
    const int start = f.start;
    if (f.start >= f.work || f.run >= f.work - f.start) return;
    const int next = f.start + f.run;
    // the segment of the run's last unit
    f.start = next - 1;
    Walk walk(a, f, kOver);
    walk.end = next;
    if (!walk.next(a, kRows) || walk.tile0 < start || walk.end0 <= next) return;  // begun earlier, or ends here
    f.start = start;
    const int c0 = walk.first_run(f), pieces = walk.last_run(f) - c0 + 1;
    const int lane = threadIdx.x & 31, r0 = blockIdx.y * kMergeRows + (threadIdx.x >> 5) * RW;
    const int rows = min(walk.s.n * a.G - walk.rt * kRows, kRows);
    if (r0 >= rows) return;
    float acc[RW][COLS], top[RW], sum[RW];
#pragma unroll
    for (int r = 0; r < RW; ++r) {
        top[r] = -INFINITY;
        sum[r] = 0.f;
#pragma unroll
        for (int e = 0; e < COLS; ++e) acc[r][e] = 0.f;
    }
#pragma unroll 2
    for (int p = 0; p < pieces; ++p) {
        const long long row0 = piece_slot(a, c0, p) * kRows + r0;
        const float lp = lane < RW && r0 + lane < rows ? a.part_lse[row0 + lane] : -INFINITY;
        float y[RW][COLS];
#pragma unroll
        for (int r = 0; r < RW; ++r)
#pragma unroll
            for (int e = 0; e < COLS; e += 2) {
                float2 u = make_float2(0.f, 0.f);
                if (r0 + r < rows) u = *reinterpret_cast<const float2 *>(a.part_o + (row0 + r) * D + lane * 2 + e * 32);
                y[r][e] = u.x;
                y[r][e + 1] = u.y;
            }
#pragma unroll
        for (int r = 0; r < RW; ++r) {
            const float l = __shfl_sync(0xFFFFFFFFu, lp, r);
            const float g = fmaxf(top[r], l), z = g == -INFINITY ? 0.f : g;
            const float fo = ex2_approx(top[r] - z), w = ex2_approx(l - z);
            top[r] = g;
            sum[r] = sum[r] * fo + w;
#pragma unroll
            for (int e = 0; e < COLS; ++e) acc[r][e] = acc[r][e] * fo + (l == -INFINITY ? 0.f : w * y[r][e]);
        }
    }
#pragma unroll
    for (int r = 0; r < RW; ++r) {
        if (r0 + r >= rows) break;
        const int mine = walk.rt * kRows + r0 + r, tok = static_cast<int>(a.by_g.quotient(mine));
        const long long orow = (static_cast<long long>(walk.s.cu0) + tok) * a.Hq + static_cast<long long>(walk.h) * a.G + (mine - tok * a.G);
        const float inv = sum[r] == 0.f ? 0.f : 1.f / sum[r];
#pragma unroll
        for (int e = 0; e < COLS; e += 2)
            *reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(a.out) + orow * D + lane * 2 + e * 32) =
                bf2(acc[r][e] * inv, acc[r][e + 1] * inv);
        if (lane == 0) a.lse[orow] = sum[r] == 0.f ? -INFINITY : ((top[r] == -INFINITY ? 0.f : top[r]) + __log2f(sum[r])) * kLn2f;
    }
}

template <int D, bool I8>
cudaError_t launch(const PagedAttn &a, const CUtensorMap &tk, const CUtensorMap &tv, int num_sms,
                   cudaStream_t st) {
    constexpr size_t smem = chunk_smem_bytes<D, I8>();
    static_assert(smem <= 227 * 1024, "shared memory of a CTA");
    cudaError_t e = cudaFuncSetAttribute(chunk_attn_kernel<D, I8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    const int ctas = (num_sms < kChunkMaxCtas ? num_sms : kChunkMaxCtas) / a.heads * a.heads;
    chunk_attn_kernel<D, I8><<<ctas, Chunk<D, I8>::THREADS, smem, st>>>(tk, tv, a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, kRows / kMergeRows);
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, chunk_merge_kernel<D>, a);
}

}  // namespace

cudaError_t launch_chunk_attn(const PagedAttn &a, const CUtensorMap &tk, const CUtensorMap &tv,
                              int num_sms, cudaStream_t st) {
    if (a.c.d == 128)
        return a.c.k_scales ? launch<128, true>(a, tk, tv, num_sms, st) : launch<128, false>(a, tk, tv, num_sms, st);
    return a.c.k_scales ? launch<64, true>(a, tk, tv, num_sms, st) : launch<64, false>(a, tk, tv, num_sms, st);
}

}  // namespace msa
