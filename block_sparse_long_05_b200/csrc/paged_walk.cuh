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

// Work of a sequence in units: its key tiles, and `over` more per segment for
// what a segment costs beside them (reading Q, writing the output).
__device__ __forceinline__ long long seq_work(const PagedAttn &a, const Seq &s, int over) {
    return static_cast<long long>(s.nt) * (a.c.Hkv / a.heads) * (s.nk + over);
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
// a run of at least `least` units.  All threads of the CTA take
// part; blockDim is a multiple of 32 and at most 512.
struct Found {
    int b;
    long long off;
    long long work;   // units of the step
    long long start;  // first unit of this CTA's run
    long long run;    // units per run
};

__device__ __forceinline__ long long run_length(long long work, int ctas, int least) {
    const long long per = (work + ctas - 1) / ctas;
    return per > least ? per : least;
}

// sm: [0..15] warp sums, [16] sequence, [17] offset
// `end`: the place of the run's last unit instead of its first one.
__device__ __forceinline__ Found find_run(const PagedAttn &a, int R, int over, int least, long long *sm, bool end = false) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const int Bt = a.step.Bt, chunks = (Bt + blockDim.x - 1) / blockDim.x;
    auto work_of = [&](int b) -> long long {
        if (b >= Bt) return 0;
        const Seq s = seq_of(a, b, R);
        // a context longer than its page-table row: the keys past it do not exist
        if (s.off + s.n > s.cap) atomicOr(a.status, kDevBadIds);
        return seq_work(a, s, over);
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
    const long long u = end ? min(f.start + f.run, f.work) - 1 : f.start;
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
        if (u >= first && u < first + x) {
            sm[16] = c * static_cast<int>(blockDim.x) + threadIdx.x;
            sm[17] = u - first;
        }
        base += all;
        if (u < base) break;
    }
    __syncthreads();
    f.b = static_cast<int>(sm[16]);
    f.off = sm[17];
    return f;
}

// A run's pieces of segments in order: sequence, row tile, kv head, key tiles
// [x0, x1).  A segment's extra units come before its tiles; a run that ends
// among them has no piece of it.
struct Walk {
    Seq s;
    int b, rt, h, x0, x1;
    bool whole;            // all tiles of the segment
    long long tile0, end0;  // units of the segment's first tile, and behind its last one
    long long pos, end, off;
    int over;
    __device__ __forceinline__ Walk(const Found &f, int over_)
        : b(f.b), pos(f.start), end(min(f.start + f.run, f.work)), off(f.off), over(over_) {}
    __device__ __forceinline__ bool next(const PagedAttn &a, int R) {
        while (pos < end) {
            s = seq_of(a, b, R);
            while (off >= seq_work(a, s, over)) {  // (only after a step; bounded by Bt)
                off = 0;
                if (++b >= a.step.Bt) return false;
                s = seq_of(a, b, R);
            }
            const int chunks = a.c.Hkv / a.heads, units = s.nk + over;
            int seg, u0;  // segment of the sequence, unit of the segment
            if (off >> 31) {
                const long long y = off / units;
                seg = static_cast<int>(y);
                u0 = static_cast<int>(off - y * units);
            } else {
                seg = static_cast<int>(off) / units;
                u0 = static_cast<int>(off) - seg * units;
            }
            const int y = seg / chunks;
            h = (seg - y * chunks) * a.heads + blockIdx.x % a.heads;
            // last, first, last but one, ...: in a causal chunk late row tiles have more
            // keys than early ones, and a run of several gets its share of both
            rt = y & 1 ? y / 2 : s.nt - 1 - y / 2;
            const long long left = end - pos;
            const int u1 = left < units - u0 ? u0 + static_cast<int>(left) : units;
            tile0 = pos - u0 + over;
            end0 = pos - u0 + units;
            pos += u1 - u0;
            off += u1 - u0;
            if (u1 <= over) continue;
            x0 = max(u0 - over, 0);
            x1 = u1 - over;
            whole = x0 == 0 && x1 == s.nk;
            return true;
        }
        return false;
    }
    // Where the piece goes that is not the whole segment (per row tile and
    // head): a run has at most one that goes on from the run before (slot 0) and
    // one that goes on into the next run (slot 1).
    __device__ __forceinline__ long long slot(const Found &f) const {
        return 2ll * blockIdx.x + (tile0 >= f.start ? 1 : 0);
    }
    // First and last run with a piece of the segment.
    __device__ __forceinline__ int first_run(const Found &f) const { return static_cast<int>(tile0 / f.run); }
    __device__ __forceinline__ int last_run(const Found &f) const { return static_cast<int>((end0 - 1) / f.run); }
};

// Slot of piece p of a segment that begins in run c0 (its heads' CTAs share it).
__device__ __forceinline__ long long piece_slot(const PagedAttn &a, int c0, int p) {
    return 2ll * ((c0 + p) * a.heads + blockIdx.x % a.heads) + (p == 0 ? 1 : 0);
}

}  // namespace walk

}  // namespace msa
