// paged_walk.cuh -- the work list of the attention kernels over pages: the key
// tiles of all (sequence, row tile, kv head) segments in one order, cut into
// equal runs, one per CTA.  Kernel code only.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "cache.h"
#include "msa_common.cuh"

namespace msa {

namespace walk {

constexpr int kKeys = kSplitKeys;  // keys per tile

// Sequence b of a step, in rows and key tiles.
struct Seq {
    int cu0;      // first packed row
    int n;        // tokens
    int off;      // position of token 0 (may be negative)
    int cap;      // keys that the page table can hold
    int nt;       // row tiles
    int nk;       // key tiles per row tile (upper bound over the row tiles)
};

__device__ __forceinline__ Seq seq_of(const PagedAttn &a, int b, int R) {
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
            const int span = min(s.n, R / a.G + 2);  // tokens of a row tile
            const int near = (a.window + span) / kKeys + 3;
            s.nk = min(s.nk, near + (min(a.sinks, kv) + kKeys - 1) / kKeys);
        }
        s.nk = max(s.nk, 1);  // rows without a key are written too
    }
    const int rows = s.n * a.G;
    // (a mixed batch is shared between two kernels by the rows of a sequence)
    s.nt = rows < a.row_lo || rows > a.row_hi ? 0 : (rows + R - 1) / R;
    return s;
}

__device__ __forceinline__ long long seq_work(const PagedAttn &a, const Seq &s) {
    return static_cast<long long>(s.nt) * (a.c.Hkv / a.heads) * s.nk;
}

// Row tile rt of a sequence: positions of its rows and its key tiles.  Tile
// x is at key (x < na ? x : x + skip) * 64, for x < count.
struct RowTile {
    int r0;          // first row
    int rows;        // rows of the sequence
    int tmin, tmax;  // positions of its first and last row
    int na, skip, count;
};

__device__ __forceinline__ RowTile row_tile(const PagedAttn &a, const Seq &s, int rt, int R) {
    RowTile t;
    t.rows = s.n * a.G;
    t.r0 = rt * R;
    t.tmin = s.off + t.r0 / a.G;
    t.tmax = s.off + (min(t.r0 + R, t.rows) - 1) / a.G;
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

// Where a run begins: sequence and offset in it.  CTAs blockIdx.x / heads share
// a run of at least `least` tiles.  All threads of the CTA take
// part; blockDim is a multiple of 32 and at most 512.
struct Found {
    int b;
    long long off;
    long long work;   // tiles of the step
    long long start;  // first tile of this CTA's run
    long long run;    // tiles per run
};

__device__ __forceinline__ long long run_length(long long work, int ctas, int least) {
    const long long per = (work + ctas - 1) / ctas;
    return per > least ? per : least;
}

// sm: [0..15] warp sums, [16] sequence, [17] offset
__device__ __forceinline__ Found find_run(const PagedAttn &a, int R, int least, long long *sm) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const int Bt = a.step.Bt, chunks = (Bt + blockDim.x - 1) / blockDim.x;
    auto work_of = [&](int b) -> long long {
        if (b >= Bt) return 0;
        const Seq s = seq_of(a, b, R);
        // a context longer than its page-table row: the keys past it do not exist
        if (s.off + s.n > s.cap) atomicOr(a.status, kDevBadIds);
        return seq_work(a, s);
    };
    Found f;
    f.b = 0;
    f.off = f.work = 0;
    // one chunk of sequences (the usual case): its work stays in a register;
    // otherwise a first sweep adds up and a second one searches
    long long w = work_of(threadIdx.x);
    for (int c = 1; c < chunks; ++c) w += work_of(c * blockDim.x + threadIdx.x);
    const long long mine = w;
#pragma unroll
    for (int o = 16; o; o >>= 1) w += __shfl_xor_sync(0xFFFFFFFFu, w, o);
    if (lane == 0) sm[warp] = w;
    __syncthreads();
    for (int i = 0; i < nw; ++i) f.work += sm[i];
    f.run = run_length(f.work, gridDim.x / a.heads, least);
    f.start = f.run * (blockIdx.x / a.heads);
    if (f.start >= f.work) return f;
    long long base = 0;
    for (int c = 0; c < chunks; ++c) {
        const long long x = chunks == 1 ? mine : work_of(c * blockDim.x + threadIdx.x);
        long long p = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xFFFFFFFFu, p, o);
            if (lane >= o) p += y;
        }
        __syncthreads();
        if (lane == 31) sm[warp] = p;
        __syncthreads();
        long long before = base, all = 0;
        for (int i = 0; i < nw; ++i) {
            if (i < warp) before += sm[i];
            all += sm[i];
        }
        const long long first = before + p - x;
        if (f.start >= first && f.start < first + x) {
            sm[16] = c * static_cast<int>(blockDim.x) + threadIdx.x;
            sm[17] = f.start - first;
        }
        base += all;
        if (f.start < base) break;
    }
    __syncthreads();
    f.b = static_cast<int>(sm[16]);
    f.off = sm[17];
    return f;
}

// A run's segments in order: sequence, row tile, kv head, key tiles [x0, x1).
struct Walk {
    Seq s;
    int b, rt, h, x0, x1;
    long long pos, end, off;
    __device__ __forceinline__ explicit Walk(const Found &f)
        : b(f.b), pos(f.start), end(min(f.start + f.run, f.work)), off(f.off) {}
    __device__ __forceinline__ bool next(const PagedAttn &a, int R) {
        if (pos >= end) return false;
        s = seq_of(a, b, R);
        while (off >= seq_work(a, s)) {  // (only after a step; bounded by Bt)
            off = 0;
            if (++b >= a.step.Bt) return false;
            s = seq_of(a, b, R);
        }
        const long long seg = off / s.nk;
        const int chunks = a.c.Hkv / a.heads;
        x0 = static_cast<int>(off - seg * s.nk);
        const int y = static_cast<int>(seg / chunks);
        h = static_cast<int>(seg - static_cast<long long>(y) * chunks) * a.heads + blockIdx.x % a.heads;
        // last, first, last but one, ...: in a causal chunk late row tiles have more
        // keys than early ones, and a run of several gets its share of both
        rt = y & 1 ? y / 2 : s.nt - 1 - y / 2;
        const long long left = end - pos;
        x1 = left < s.nk - x0 ? x0 + static_cast<int>(left) : s.nk;
        pos += x1 - x0;
        off += x1 - x0;
        return true;
    }
};

}  // namespace walk

}  // namespace msa
