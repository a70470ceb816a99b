// paged_attn_split.cu -- attention of few query rows over a paged cache
// (single tokens, short chunks, and the sparse branch on int8 pages).
//
// With the rows of one (sequence, kv head) numbered r = i * G + g (token i,
// head g of the group), a tile of 16 rows attends its keys j with
//     s_j = (q . k_j) / sqrt(d),  m = max s_j,  l = sum exp(s_j - m),
//     o = sum exp(s_j - m) v_j / l,  lse = m + ln l,
// in one pass over the keys with a running m and l.  With int8 pages k_j =
// code_j * sk_j and v_j = code_j * sv_j: the codes enter the matrix products
// exactly (a signed byte fits bf16), sk_j scales the scores and sv_j the
// weights, both in fp32, so no dequantised value is rounded.
//
// Few rows read many keys once, so HBM bounds it: 16 rows x 64 keys need
// 48 mma per warp for 8 KB (bf16) or 4 KB (int8) of K and V.  Therefore
//  - the key tiles of all (sequence, row tile, kv head) segments form one
//    list that is cut into equal runs, one per CTA, two CTAs per SM: a batch
//    with contexts of any lengths keeps every SM streaming to the end;
//  - a producer warp keeps a ring of about 100 KB per CTA filled by TMA,
//    across segment borders, and looks the pages up 32 tiles at a time;
//  - four warps take 16 keys of a 64-key tile each, with their own m, l and
//    o in registers, and meet only at the end of a segment;
//  - a segment that lies in several runs leaves one fp32 piece per run, which
//    the combine kernel (programmatic dependent launch) merges in run order:
//    no atomics, the same result every time.
// The weights enter the second product as two bf16 terms (hi + lo, 16 bits
// of mantissa): the matrix unit is idle most of the time here, and the
// output then carries its own final rounding only.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cache.h"
#include "msa_common.cuh"
#include "ptx_sm100.cuh"

namespace msa {

namespace {

constexpr int kComputeWarps = 4;
constexpr int kSplitThreads = 32 * (kComputeWarps + 1);
constexpr int kTileRows = kSplitTileRows, kKeys = kSplitKeys;
constexpr int kMinRun = 2;  // tiles per run: below it a combine costs more than the run saves
constexpr float kLn2f = 0.6931471805599453f;

// ------------------------------------------------------------ the work list
// Sequence b of a step, in rows and key tiles.
struct Seq {
    int cu0;      // first packed row
    int n;        // tokens
    int off;      // position of token 0 (may be negative)
    int cap;      // keys that the page table can hold
    int nt;       // row tiles
    int nk;       // key tiles per row tile (upper bound over the row tiles)
};

__device__ __forceinline__ Seq seq_of(const PagedAttn &a, int b) {
    Seq s;
    if (a.ids) {  // sparse branch: the tiles of K selected blocks, one row per sequence
        s.cu0 = b;
        s.n = 1;
        s.off = a.T - 1;
        s.cap = a.T;
        s.nk = (a.K * a.step.block + kKeys - 1) / kKeys;
    } else {
        const int c0 = min(max(a.step.cu[b], 0), a.step.total);
        const int c1 = min(max(a.step.cu[b + 1], c0), a.step.total);
        s.cu0 = c0;
        s.n = c1 - c0;
        s.cap = a.step.pm.stride * a.step.block;
        const int len = max(a.step.kv_len[b], 0), kv = min(len, s.cap);
        s.off = len - s.n;
        s.nk = (kv + kKeys - 1) / kKeys;
        if (a.window) {
            const int span = min(s.n, kTileRows / a.G + 2);  // tokens of a row tile
            const int near = (a.window + span) / kKeys + 3;
            s.nk = min(s.nk, near + (min(a.sinks, kv) + kKeys - 1) / kKeys);
        }
        s.nk = max(s.nk, 1);  // rows without a key are written too
    }
    s.nt = (s.n * a.G + kTileRows - 1) / kTileRows;
    return s;
}

__device__ __forceinline__ long long seq_work(const PagedAttn &a, const Seq &s) {
    return static_cast<long long>(s.nt) * a.c.Hkv * s.nk;
}

// Row tile rt of a sequence: positions of its rows and its key tiles.  Tile
// x is at key (x < na ? x : x + skip) * 64, for x < count.
struct RowTile {
    int r0;          // first row
    int rows;        // rows of the sequence
    int tmin, tmax;  // positions of its first and last row
    int na, skip, count;
};

__device__ __forceinline__ RowTile row_tile(const PagedAttn &a, const Seq &s, int rt) {
    RowTile t;
    t.rows = s.n * a.G;
    t.r0 = rt * kTileRows;
    t.tmin = s.off + t.r0 / a.G;
    t.tmax = s.off + (min(t.r0 + kTileRows, t.rows) - 1) / a.G;
    t.na = t.skip = 0;
    if (a.ids) {
        t.count = s.nk;
        return t;
    }
    const int end = min(t.tmax + 1, s.cap);
    t.count = end > 0 ? (end + kKeys - 1) / kKeys : 0;
    if (a.window) {
        const int lo = max(t.tmin - a.window + 1, 0) / kKeys;
        t.na = min((min(a.sinks, max(end, 0)) + kKeys - 1) / kKeys, lo);
        t.skip = lo - t.na;
        t.count = max(t.count - t.skip, 0);
    }
    return t;
}

// Exclusive prefix of the work over the sequences: total, and the sequence
// and offset that hold unit u.  All threads of the CTA; blockDim <= 256.
struct Found {
    int b;
    long long off;
};
__device__ long long total_work(const PagedAttn &a, long long *sm) {
    long long w = 0;
    for (int b = threadIdx.x; b < a.step.Bt; b += blockDim.x) {
        const Seq s = seq_of(a, b);
        w += seq_work(a, s);
        // a context longer than its page-table row: the keys past it do not exist
        if (s.off + s.n > s.cap) atomicOr(a.status, kDevBadIds);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) w += __shfl_xor_sync(0xFFFFFFFFu, w, o);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = w;
    __syncthreads();
    long long sum = 0;
    for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) sum += sm[i];
    __syncthreads();
    return sum;
}
__device__ Found find_unit(const PagedAttn &a, long long u, long long *sm) {
    // sm: [0..7] warp sums, [8] sequence, [9] offset
    long long base = 0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    for (int b0 = 0; b0 < a.step.Bt; b0 += blockDim.x) {
        const int b = b0 + threadIdx.x;
        const long long w = b < a.step.Bt ? seq_work(a, seq_of(a, b)) : 0;
        long long p = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xFFFFFFFFu, p, o);
            if (lane >= o) p += y;
        }
        if (lane == 31) sm[warp] = p;
        __syncthreads();
        long long before = base, chunk = 0;
        for (int i = 0; i < nw; ++i) {
            if (i < warp) before += sm[i];
            chunk += sm[i];
        }
        const long long first = before + p - w;
        if (u >= first && u < first + w) {
            sm[8] = b;
            sm[9] = u - first;
        }
        base += chunk;
        __syncthreads();
        if (u < base) break;
    }
    Found f;
    f.b = static_cast<int>(sm[8]);
    f.off = sm[9];
    __syncthreads();
    return f;
}

__device__ __forceinline__ long long run_length(long long work, int ctas) {
    const long long per = (work + ctas - 1) / ctas;
    return per > kMinRun ? per : kMinRun;
}

// A run's segments in order: sequence, row tile, kv head, key tiles [x0, x1).
struct Walk {
    Seq s;
    int b, rt, h, x0, x1;
    long long pos, end, off;
    __device__ __forceinline__ Walk(const Found &f, long long start, long long stop)
        : b(f.b), pos(start), end(stop), off(f.off) {}
    __device__ __forceinline__ bool next(const PagedAttn &a) {
        if (pos >= end) return false;
        s = seq_of(a, b);
        while (off >= seq_work(a, s)) {  // (only after a step; bounded by Bt)
            off = 0;
            if (++b >= a.step.Bt) return false;
            s = seq_of(a, b);
        }
        const long long seg = off / s.nk;
        x0 = static_cast<int>(off - seg * s.nk);
        rt = static_cast<int>(seg / a.c.Hkv);
        h = static_cast<int>(seg - static_cast<long long>(rt) * a.c.Hkv);
        const long long left = end - pos;
        x1 = left < s.nk - x0 ? x0 + static_cast<int>(left) : s.nk;
        pos += x1 - x0;
        off += x1 - x0;
        return true;
    }
};

// ------------------------------------------------------------ tile geometry
template <int D, bool I8>
struct Tile {
    static constexpr int ROWB = D * (I8 ? 1 : 2) < 128 ? D * (I8 ? 1 : 2) : 128;  // smem row
    static constexpr int REGS = D * (I8 ? 1 : 2) / ROWB;  // 128-byte wide regions
    static constexpr int REGION = kKeys * ROWB;
    static constexpr int BYTES = REGS * REGION;           // K or V of 64 keys
    static constexpr int STAGE = 2 * BYTES;
    static constexpr int STAGES = STAGE >= 32768 ? 3 : STAGE >= 16384 ? 6 : 8;
    static constexpr int CW = I8 ? D / 8 : 8;  // columns of V per thread group and region
    static constexpr int NT = D / 8;           // 8-column tiles of O
    static constexpr int KST = D / 16;         // k-steps of q . k
};

struct alignas(8) StageMeta {
    int pos[2];  // first key of each 32-key half; -1: nothing there
};

constexpr int kMergeBytes = kComputeWarps * kTileRows * 32 * 4;

template <int D, bool I8>
constexpr size_t split_smem_bytes() {
    using T = Tile<D, I8>;
    return 1024 + static_cast<size_t>(T::STAGES) * (T::STAGE + sizeof(StageMeta) + 16 + (I8 ? 512 : 0)) +
           kMergeBytes + kComputeWarps * kTileRows * 8 + 256;
}

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            smem_addr(dst)),
        "l"(src), "r"(bytes), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t bf2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Two signed bytes (in the low bytes of the 16-bit halves of x) as bf16, both
// exact: 128 + (low 7 bits) minus 128, or minus 256 where the sign bit is
// set.  0x4300 is 128 in bf16, its last mantissa bit counts 1, and the sign
// bit of the byte falls on the lowest exponent bit (0x4380 is 256).
__device__ __forceinline__ uint32_t s8x2_bf16(uint32_t x) {
    const uint32_t hi = (x & 0x007F007Fu) | 0x43004300u, lo = (x & 0x00800080u) | 0x43004300u;
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&hi),
                                     *reinterpret_cast<const __nv_bfloat162 *>(&lo));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Offset of 16-byte piece c of row r of a tile region.
template <int ROWB>
__device__ __forceinline__ uint32_t piece_at(uint32_t r, uint32_t c) {
    if (ROWB == 128) return sw128_offset(r, c);
    return r * 64u + ((c ^ ((r >> 1) & 3u)) << 4);  // 64-byte swizzle
}

// ===========================================================================
// One run per CTA.  Warp 4: producer; warps 0-3: 16 keys of each tile.
// In an mma fragment a thread (gq = lane / 4, c = lane % 4) holds rows gq and
// gq + 8.  The order of the d values over the k-steps, and of the columns of
// V over the 8-column tiles, is chosen so that a thread reads K and V in
// 16-byte pieces without bank conflicts: K pieces 2c and 2c + 1 of its key
// (Q is loaded in the same order), V pieces gq of its four keys, whose values
// are paired key by key by byte permutes.
// ===========================================================================
template <int D, bool I8>
__global__ void __launch_bounds__(kSplitThreads, 2) split_attn_kernel(
    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
    const __grid_constant__ PagedAttn a) {
    using T = Tile<D, I8>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *ring = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    float *merge = reinterpret_cast<float *>(ring + T::STAGES * T::STAGE);  // [warp][row][32]
    float2 *ml = reinterpret_cast<float2 *>(merge + kMergeBytes / 4);       // [warp][row] (m, l)
    float *scales = reinterpret_cast<float *>(ml + kComputeWarps * kTileRows);  // [stage][2][64]
    uint64_t *full = reinterpret_cast<uint64_t *>(scales + (I8 ? T::STAGES * 128 : 0));
    uint64_t *empty = full + T::STAGES;
    StageMeta *meta = reinterpret_cast<StageMeta *>(empty + T::STAGES);
    long long *scan = reinterpret_cast<long long *>(meta + T::STAGES);  // [10]
    volatile int *abort_flag = reinterpret_cast<volatile int *>(scan + 10);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < T::STAGES; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, kComputeWarps);
        }
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }
    const long long work = total_work(a, scan);
    const long long run = run_length(work, gridDim.x);
    const long long start = run * blockIdx.x, stop = min(start + run, work);
    if (start >= stop) return;
    Walk walk(find_unit(a, start, scan), start, stop);
    const int block = a.step.block;

    if (warp == kComputeWarps) {
        // -------------------------------------------------------- producer
        uint32_t it = 0;
        const int half = min(block, kKeys);  // keys per TMA box
        bool ok = true;
        while (ok && walk.next(a)) {
            const RowTile t = row_tile(a, walk.s, walk.rt);
            const int x1 = min(walk.x1, t.count);
            for (int xb = walk.x0; xb < x1 && ok; xb += 32) {
                // page and position of this lane's tile (two boxes with 32-key blocks)
                int pos[2] = {-1, -1}, z[2] = {0, 0};
                const int x = xb + lane;
                if (x < x1) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (i == 1 && block >= kKeys) {
                            pos[1] = pos[0] < 0 ? -1 : pos[0] + 32;
                            break;
                        }
                        int p;  // key position of the box
                        if (a.ids) {
                            const int v = x * kKeys + i * 32, slot = v / block;
                            const int id = slot < a.K ? a.ids[static_cast<long long>(walk.b) * a.K + slot] : -1;
                            const int N = (a.T + block - 1) / block;
                            if (id < -1 || id >= N) atomicOr(a.status, kDevBadIds);
                            p = id < 0 || id >= N ? -1 : id * block + (v - slot * block);
                            if (p >= a.T) p = -1;
                        } else {
                            p = (x < t.na ? x : x + t.skip) * kKeys + i * 32;
                            if (p > t.tmax || p >= walk.s.cap) p = -1;
                        }
                        if (p < 0) continue;
                        const int j = p / block;
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
                for (int y = 0; y < m; ++y) {
                    const int p0 = __shfl_sync(0xFFFFFFFFu, pos[0], y), p1 = __shfl_sync(0xFFFFFFFFu, pos[1], y);
                    const int z0 = __shfl_sync(0xFFFFFFFFu, z[0], y), z1 = __shfl_sync(0xFFFFFFFFu, z[1], y);
                    const int st = it % T::STAGES;
                    if (lane == 0) {
                        if (it >= T::STAGES)
                            ok = mbar_wait(empty + st, ((it / T::STAGES) & 1) ^ 1, abort_flag, a.status);
                        if (ok) {
                            meta[st].pos[0] = p0;
                            meta[st].pos[1] = p1;
                            unsigned char *dk = ring + st * T::STAGE, *dv = dk + T::BYTES;
                            const int boxes = (p0 >= 0) + (half < kKeys && p1 >= 0);
                            if (boxes == 0) {
                                mbar_arrive(full + st);
                            } else {
                                mbar_arrive_expect_tx(full + st, boxes * half * (2 * D * (I8 ? 1 : 2) + (I8 ? 8 : 0)));
                                for (int i = 0; i < kKeys / half; ++i) {
                                    if ((i ? p1 : p0) < 0) continue;
                                    const int zz = i ? z1 : z0;
#pragma unroll
                                    for (int r = 0; r < T::REGS; ++r) {
                                        const uint32_t o = r * T::REGION + i * half * T::ROWB;
                                        tma_load_3d(dk + o, &tm_k, full + st, r * 64, walk.h, zz);
                                        tma_load_3d(dv + o, &tm_v, full + st, r * 64, walk.h, zz);
                                    }
                                    if (I8) {
                                        const int page = zz / block;
                                        const long long so = (static_cast<long long>(page) * a.c.Hkv + walk.h) * block + (zz - page * block);
                                        bulk_load(scales + st * 128 + i * half, a.c.k_scales + so, half * 4, full + st);
                                        bulk_load(scales + st * 128 + 64 + i * half, a.c.v_scales + so, half * 4, full + st);
                                    }
                                }
                            }
                        }
                    }
                    ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
                    if (!ok) break;
                    ++it;
                }
            }
        }
        // the copies have landed before the CTA ends (after an abort; otherwise
        // the compute warps have seen them all)
        if (!ok && lane == 0) {
            for (uint32_t i = it > T::STAGES ? it - T::STAGES : 0; i < it; ++i) {
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait(full + i % T::STAGES, (i / T::STAGES) & 1))
                    if (global_timer_ns() - t0 > kWaitLimitNs / 4) break;
            }
        }
        return;
    }

    // ------------------------------------------------------------ compute
    const int gq = lane >> 2, c = lane & 3;
    uint32_t it = 0;
    bool ok = true;  // false: a wait gave up; the warps still meet at every barrier
    while (walk.next(a)) {
        const RowTile t = row_tile(a, walk.s, walk.rt);
        const int x1 = min(walk.x1, t.count);
        const bool whole = walk.x0 == 0 && walk.x1 == walk.s.nk;
        // this thread's two rows: positions (-1: no such row) and Q fragments
        int tpos[2];
        uint32_t qf[T::KST][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = t.r0 + gq + 8 * i;
            const int tok = r / a.G;
            tpos[i] = r < t.rows ? walk.s.off + tok : -1;
            const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) +
                                     (walk.s.cu0 + tok) * a.q_stride +
                                     (static_cast<long long>(walk.h) * a.G + (r - tok * a.G)) * D;
            if (!I8) {
#pragma unroll
                for (int p = 0; p < T::KST / 2; ++p) {  // piece 2c + p % 2 of region p / 2
                    uint4 u = make_uint4(0, 0, 0, 0);
                    if (r < t.rows) u = *reinterpret_cast<const uint4 *>(q + (p / 2) * 64 + (2 * c + p % 2) * 8);
                    qf[2 * p][i] = u.x;
                    qf[2 * p][2 + i] = u.y;
                    qf[2 * p + 1][i] = u.z;
                    qf[2 * p + 1][2 + i] = u.w;
                }
            } else {
#pragma unroll
                for (int p = 0; p < T::KST / 2; ++p) {  // 8 of the 16 values of a piece of codes
                    const int piece = D == 128 ? 2 * c + p / 2 : c;
                    uint4 u = make_uint4(0, 0, 0, 0);
                    if (r < t.rows) u = *reinterpret_cast<const uint4 *>(q + piece * 16 + (p % 2) * 8);
                    qf[2 * p][i] = u.x;
                    qf[2 * p][2 + i] = u.y;
                    qf[2 * p + 1][i] = u.z;
                    qf[2 * p + 1][2 + i] = u.w;
                }
            }
        }
        float o[T::NT][4];
#pragma unroll
        for (int j = 0; j < T::NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        const int last = min(t.tmax, walk.s.cap - 1);  // last key that any row sees

        for (int x = walk.x0; x < x1 && ok; ++x, ++it) {
            const int st = it % T::STAGES;
            if (lane == 0) ok = mbar_wait(full + st, (it / T::STAGES) & 1, abort_flag, a.status);
            ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
            if (!ok) break;
            // (every lane observes the phase itself, which orders its reads)
            mbar_try_wait(full + st, (it / T::STAGES) & 1);
            const int base = meta[st].pos[warp >> 1];
            const int p0 = base + (warp & 1) * 16;  // first of this warp's 16 keys
            const unsigned char *ks = ring + st * T::STAGE, *vs = ks + T::BYTES;
            const bool none = base < 0 || p0 > last ||
                              (a.window && p0 >= a.sinks && p0 + 15 <= t.tmin - a.window);
            if (!none) {
                const bool all = p0 + 15 <= min(t.tmin, walk.s.cap - 1) &&
                                 (!a.window || p0 > t.tmax - a.window || p0 + 15 < a.sinks);
                float s[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    s[h][0] = s[h][1] = s[h][2] = s[h][3] = 0.f;
                    const uint32_t key = warp * 16 + h * 8 + gq;
                    if (!I8) {
#pragma unroll
                        for (int p = 0; p < T::KST / 2; ++p) {
                            const uint4 u = *reinterpret_cast<const uint4 *>(
                                ks + (p / 2) * T::REGION + piece_at<T::ROWB>(key, 2 * c + p % 2));
                            mma16816(s[h], qf[2 * p][0], qf[2 * p][1], qf[2 * p][2], qf[2 * p][3], u.x, u.y);
                            mma16816(s[h], qf[2 * p + 1][0], qf[2 * p + 1][1], qf[2 * p + 1][2], qf[2 * p + 1][3], u.z, u.w);
                        }
                    } else {
#pragma unroll
                        for (int p = 0; p < T::KST / 4; ++p) {
                            const uint4 u = *reinterpret_cast<const uint4 *>(
                                ks + piece_at<T::ROWB>(key, D == 128 ? 2 * c + p : c));
                            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t b0 = s8x2_bf16(__byte_perm(w[e], 0, 0x1100));
                                const uint32_t b1 = s8x2_bf16(__byte_perm(w[e], 0, 0x3322));
                                const int k = 4 * p + e;
                                mma16816(s[h], qf[k][0], qf[k][1], qf[k][2], qf[k][3], b0, b1);
                            }
                        }
                    }
                }
                // scores in log2 units; masked ones are -inf whatever the key held
                bool seen[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float2 sk = make_float2(1.f, 1.f);
                    if (I8) sk = *reinterpret_cast<const float2 *>(scales + st * 128 + warp * 16 + h * 8 + 2 * c);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float y = s[h][e] * a.scale_log2;
                        if (I8) y *= e & 1 ? sk.y : sk.x;
                        bool v = true;
                        if (!all) {
                            const int pos = p0 + h * 8 + 2 * c + (e & 1), tt = tpos[e >> 1];
                            v = pos <= min(tt, walk.s.cap - 1) &&
                                (!a.window || pos > tt - a.window || pos < a.sinks);
                        }
                        seen[h][e] = v;
                        s[h][e] = v ? y : -INFINITY;
                    }
                }
                float g[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    g[i] = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1]));
                    g[i] = fmaxf(g[i], __shfl_xor_sync(0xFFFFFFFFu, g[i], 1));
                    g[i] = fmaxf(g[i], __shfl_xor_sync(0xFFFFFFFFu, g[i], 2));
                }
                // the reference m only has to keep the weights in range: it is
                // raised (and o, l rescaled) when a score passes it by 2^8
                if (__any_sync(0xFFFFFFFFu, g[0] > m[0] + 8.f || g[1] > m[1] + 8.f)) {
                    float f[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float mn = fmaxf(m[i], g[i]);
                        f[i] = m[i] == -INFINITY ? 0.f : ex2_approx(m[i] - mn);
                        m[i] = mn;
                        l[i] *= f[i];
                    }
#pragma unroll
                    for (int j = 0; j < T::NT; ++j) {
                        o[j][0] *= f[0];
                        o[j][1] *= f[0];
                        o[j][2] *= f[1];
                        o[j][3] *= f[1];
                    }
                }
                uint32_t hi[4], lo[4];  // A fragments of the weights
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float2 sv = make_float2(1.f, 1.f);
                    if (I8) sv = *reinterpret_cast<const float2 *>(scales + st * 128 + 64 + warp * 16 + h * 8 + 2 * c);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float mr = m[i] == -INFINITY ? 0.f : m[i];
                        float w0 = ex2_approx(s[h][2 * i] - mr), w1 = ex2_approx(s[h][2 * i + 1] - mr);
                        l[i] += w0 + w1;
                        if (I8) {  // (a masked key's scale may hold anything)
                            w0 = seen[h][2 * i] ? w0 * sv.x : 0.f;
                            w1 = seen[h][2 * i + 1] ? w1 * sv.y : 0.f;
                        }
                        const uint32_t p = bf2(w0, w1);
                        hi[2 * h + i] = p;
                        lo[2 * h + i] = bf2(w0 - __uint_as_float(p << 16), w1 - __uint_as_float(p & 0xFFFF0000u));
                    }
                }
                // keys that no row of the tile sees count nothing, whatever their V rows hold
                uint32_t keep[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int pos = p0 + (e >> 1) * 8 + 2 * c + (e & 1);
                    const bool v = all || (pos <= last && (!a.window || pos > t.tmin - a.window || pos < a.sinks));
                    keep[e] = v ? 0xFFFFFFFFu : 0u;
                }
                const uint32_t row = warp * 16 + 2 * c;
#pragma unroll
                for (int r = 0; r < (I8 ? 1 : T::REGS); ++r) {
                    uint4 u[4];
                    const unsigned char *vr = vs + r * T::REGION;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t k = row + (e >> 1) * 8 + (e & 1);
                        if (I8 && D == 64) {
                            const uint2 y = *reinterpret_cast<const uint2 *>(vr + piece_at<T::ROWB>(k, gq >> 1) + (gq & 1) * 8);
                            u[e] = make_uint4(y.x, y.y, 0, 0);
                        } else {
                            u[e] = *reinterpret_cast<const uint4 *>(vr + piece_at<T::ROWB>(k, gq));
                        }
                        if (!I8) {
                            u[e].x &= keep[e];
                            u[e].y &= keep[e];
                            u[e].z &= keep[e];
                            u[e].w &= keep[e];
                        }
                    }
                    const uint32_t w[4][4] = {{u[0].x, u[0].y, u[0].z, u[0].w},
                                              {u[1].x, u[1].y, u[1].z, u[1].w},
                                              {u[2].x, u[2].y, u[2].z, u[2].w},
                                              {u[3].x, u[3].y, u[3].z, u[3].w}};
#pragma unroll
                    for (int j = 0; j < T::CW; ++j) {
                        uint32_t b0, b1;
                        if (!I8) {
                            const uint32_t sel = j & 1 ? 0x7632 : 0x5410;
                            b0 = __byte_perm(w[0][j / 2], w[1][j / 2], sel);
                            b1 = __byte_perm(w[2][j / 2], w[3][j / 2], sel);
                        } else {
                            const uint32_t e = j & 3, sel = e | (e << 4) | ((4 + e) << 8) | ((4 + e) << 12);
                            b0 = s8x2_bf16(__byte_perm(w[0][j / 4], w[1][j / 4], sel));
                            b1 = s8x2_bf16(__byte_perm(w[2][j / 4], w[3][j / 4], sel));
                        }
                        float(&acc)[4] = o[r * 8 + j];
                        mma16816(acc, hi[0], hi[1], hi[2], hi[3], b0, b1);
                        mma16816(acc, lo[0], lo[1], lo[2], lo[3], b0, b1);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + st);
        }

        // ---- the four warps' results of the segment, merged
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 1);
            l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 2);
            if (c == 0) ml[warp * kTileRows + gq + 8 * i] = make_float2(m[i], l[i]);
        }
        named_barrier(1, 32 * kComputeWarps);
        float f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kComputeWarps; ++w) top = fmaxf(top, ml[w * kTileRows + gq + 8 * i].x);
            f[i] = m[i] == -INFINITY ? (l[i] == 0.f ? 0.f : 1.f) : ex2_approx(m[i] - top);
        }
        // this thread's row and 4 columns of each 32-column round
        const int row = tid >> 3, n = tid & 7;
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kComputeWarps; ++w) top = fmaxf(top, ml[w * kTileRows + row].x);
#pragma unroll
        for (int w = 0; w < kComputeWarps; ++w) {
            const float2 y = ml[w * kTileRows + row];
            sum += y.x == -INFINITY ? y.y : y.y * ex2_approx(y.x - top);
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const float lse2 = sum == 0.f ? -INFINITY : (top == -INFINITY ? 0.f : top) + __log2f(sum);
        const int r = t.r0 + row, tok = r / a.G;
        const bool live = r < t.rows;
        const long long orow = (static_cast<long long>(walk.s.cu0) + tok) * a.Hq + static_cast<long long>(walk.h) * a.G + (r - tok * a.G);
        const long long prow = (2ll * blockIdx.x + (walk.pos - (walk.x1 - walk.x0) == start ? 0 : 1)) * kTileRows + row;
        if (n == 0 && live) {
            if (whole)
                a.lse[orow] = lse2 * kLn2f;
            else
                a.part_lse[prow] = lse2;
        }
#pragma unroll
        for (int q = 0; q < T::NT / 4; ++q) {
            // columns of 8-column tiles 4q .. 4q + 3: value e of group n is column
            // (region) * 64 + n * CW + (first of the four) + e
            float *mine = merge + (warp * kTileRows + gq) * 32 + 2 * c * 4;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    *reinterpret_cast<float4 *>(mine + i * 8 * 32 + k * 4) =
                        make_float4(o[4 * q][2 * i + k] * f[i], o[4 * q + 1][2 * i + k] * f[i],
                                    o[4 * q + 2][2 * i + k] * f[i], o[4 * q + 3][2 * i + k] * f[i]);
            named_barrier(1, 32 * kComputeWarps);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kComputeWarps; ++w) {
                const float4 y = *reinterpret_cast<const float4 *>(merge + (w * kTileRows + row) * 32 + n * 4);
                acc.x += y.x;
                acc.y += y.y;
                acc.z += y.z;
                acc.w += y.w;
            }
            const int col = I8 ? n * T::CW + 4 * q : (q / 2) * 64 + n * 8 + (q % 2) * 4;
            if (live) {
                if (whole)
                    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + orow * D + col) =
                        make_uint2(bf2(acc.x * inv, acc.y * inv), bf2(acc.z * inv, acc.w * inv));
                else
                    *reinterpret_cast<float4 *>(a.part_o + prow * D + col) =
                        make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
            }
            named_barrier(1, 32 * kComputeWarps);
        }
    }
}

// ===========================================================================
// Merge of the segments that lie in several runs: CTA c takes the segment
// that begins in run c and goes on into run c + 1, if there is one.  Its
// pieces are the last one of run c and the first ones of the runs behind it.
//   lse = log2 sum 2^lse_p,  out = sum 2^(lse_p - lse) o_p
// ===========================================================================
constexpr int kCombineThreads = 256;

template <int D>
__global__ void __launch_bounds__(kCombineThreads) split_combine_kernel(const __grid_constant__ PagedAttn a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the pieces come from the previous kernel
    __shared__ long long scan[10];
    __shared__ float wt[32][kTileRows];
    const long long work = total_work(a, scan);
    const long long run = run_length(work, gridDim.x);
    const long long first = run * blockIdx.x, next = first + run;
    if (next >= work) return;
    const Found at = find_unit(a, next - 1, scan);
    const Seq s = seq_of(a, at.b);
    const long long seg = at.off / s.nk;
    const long long seg0 = next - 1 - (at.off - seg * s.nk), seg1 = seg0 + s.nk;
    if (seg0 < first || seg1 <= next) return;  // begun earlier, or ends here
    const int rt = static_cast<int>(seg / a.c.Hkv), h = static_cast<int>(seg - static_cast<long long>(rt) * a.c.Hkv);
    const int pieces = static_cast<int>((seg1 - 1) / run - blockIdx.x) + 1;
    const long long slot0 = 2ll * blockIdx.x + (seg0 == first ? 0 : 1);
    auto slot = [&](int p) { return p == 0 ? slot0 : 2ll * (blockIdx.x + p); };

    constexpr int COLS = D / 16;  // columns per thread
    const int row = threadIdx.x >> 4, col = (threadIdx.x & 15) * COLS;
    float acc[COLS];
#pragma unroll
    for (int e = 0; e < COLS; ++e) acc[e] = 0.f;
    float top = -INFINITY, sum = 0.f;
    for (int p0 = 0; p0 < pieces; p0 += 32) {
        const int m = min(32, pieces - p0);
        __syncthreads();
        for (int e = threadIdx.x; e < m * kTileRows; e += kCombineThreads)
            wt[e / kTileRows][e % kTileRows] = a.part_lse[slot(p0 + e / kTileRows) * kTileRows + e % kTileRows];
        __syncthreads();
        float g = top;
        for (int p = 0; p < m; ++p) g = fmaxf(g, wt[p][row]);
        const float f = top == -INFINITY ? 0.f : ex2_approx(top - g);
        sum *= f;
#pragma unroll
        for (int e = 0; e < COLS; ++e) acc[e] *= f;
        top = g;
#pragma unroll 4
        for (int p = 0; p < m; ++p) {
            const float lp = wt[p][row];
            if (lp == -INFINITY) continue;  // a piece without a key for this row
            const float w = ex2_approx(lp - top);
            const float4 *src = reinterpret_cast<const float4 *>(a.part_o + (slot(p0 + p) * kTileRows + row) * D + col);
            sum += w;
#pragma unroll
            for (int e = 0; e < COLS / 4; ++e) {
                const float4 y = src[e];
                acc[4 * e] += w * y.x;
                acc[4 * e + 1] += w * y.y;
                acc[4 * e + 2] += w * y.z;
                acc[4 * e + 3] += w * y.w;
            }
        }
    }
    const int r = rt * kTileRows + row;
    if (r >= s.n * a.G) return;
    const int tok = r / a.G;
    const long long orow = (static_cast<long long>(s.cu0) + tok) * a.Hq + static_cast<long long>(h) * a.G + (r - tok * a.G);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + orow * D + col;
#pragma unroll
    for (int e = 0; e < COLS; e += 4)
        *reinterpret_cast<uint2 *>(out + e) = make_uint2(bf2(acc[e] * inv, acc[e + 1] * inv),
                                                         bf2(acc[e + 2] * inv, acc[e + 3] * inv));
    if (col == 0) a.lse[orow] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * kLn2f;
}

template <int D, bool I8>
cudaError_t launch(const PagedAttn &a, const CUtensorMap &tk, const CUtensorMap &tv, int ctas,
                   cudaStream_t st) {
    constexpr size_t smem = split_smem_bytes<D, I8>();
    cudaError_t e = cudaFuncSetAttribute(split_attn_kernel<D, I8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    split_attn_kernel<D, I8><<<ctas, kSplitThreads, smem, st>>>(tk, tv, a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kCombineThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, split_combine_kernel<D>, a);
}

}  // namespace

cudaError_t launch_split_attn(const PagedAttn &a, const CUtensorMap &tk, const CUtensorMap &tv,
                              int num_sms, cudaStream_t st) {
    const int ctas = 2 * num_sms < kSplitMaxCtas ? 2 * num_sms : kSplitMaxCtas;
    if (a.c.d == 128)
        return a.c.k_scales ? launch<128, true>(a, tk, tv, ctas, st) : launch<128, false>(a, tk, tv, ctas, st);
    return a.c.k_scales ? launch<64, true>(a, tk, tv, ctas, st) : launch<64, false>(a, tk, tv, ctas, st);
}

}  // namespace msa
