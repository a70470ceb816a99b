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
constexpr int kAlignUnits = 10;    // units that a run may grow by to end with a segment

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
            const int span = min(s.n, static_cast<int>(a.by_g.quotient(R)) + 2);  // tokens of a row tile
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
// what a segment costs beside them (reading Q, writing the output).  (The host
// keeps the units of a step below 2^31.)
__device__ __forceinline__ int seq_work(const PagedAttn &a, const Seq &s, int over) {
    return s.nt * a.groups * (s.nk + over);
}

// Row tile rt of a sequence: positions of its rows and its key tiles.  Tile
// x is at key (x < na ? x : x + skip) * 128, for x < count.
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
    t.tmin = s.off + static_cast<int>(a.by_g.quotient(t.r0));
    t.tmax = s.off + static_cast<int>(a.by_g.quotient(min(t.r0 + R, t.rows) - 1));
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
        // (a window may begin behind the last key that the page table holds)
        t.count = t.na + max(t.count - lo, 0);
    }
    return t;
}

// Where a run begins: sequence (and what seq_of says of it) and offset in it.
// CTAs blockIdx.x / heads share a run of at least `least` units.
struct Found {
    Seq s;
    int b, off;
    int work;   // units of the step
    int start;  // first unit of this CTA's run
    int run;    // units per run
};

// Every warp finds out for itself (one round of loads and shuffles for up to 32
// sequences, no barrier).  `end`: the place of the run's last unit instead of
// its first one.
__device__ __forceinline__ Found find_run(const PagedAttn &a, int R, int over, int least, bool end = false) {
    const int lane = threadIdx.x & 31, Bt = a.step.Bt;
    Found f;
    int work = 0, most = 0, fewest = 0x7FFFFFFF;
    Seq s = {};
    int w = 0;
    for (int b0 = 0; b0 < Bt; b0 += 32) {
        w = 0;
        if (b0 + lane < Bt) {
            s = seq_of(a, b0 + lane, R);
            w = seq_work(a, s, over);
            // a context longer than its page-table row: the keys past it do not exist
            if (s.off + s.n > s.cap) atomicOr(a.status, kDevBadIds);
            if (w) {
                most = max(most, s.nk + over);
                fewest = min(fewest, s.nk + over);
            }
        }
        work += __reduce_add_sync(0xFFFFFFFFu, w);
    }
    f.work = work;
    const int ctas = gridDim.x / a.heads;
    f.run = max((work + ctas - 1) / ctas, least);
    // Segments of one size: runs of whole segments, if they are not much longer,
    // need no merge (which costs about as much as ten tiles).
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    fewest = __reduce_min_sync(0xFFFFFFFFu, fewest);
    if (most == fewest) {
        const int whole = (f.run + most - 1) / most * most;
        if (whole <= f.run + kAlignUnits) f.run = whole;
    }
    // (below 2^31 too: whole runs that start inside the work)
    const int c = blockIdx.x / a.heads;
    f.start = c <= work / f.run ? c * f.run : work;
    f.b = f.off = 0;
    if (f.start >= work) return f;
    const int u = end ? min(work - f.start, f.run) - 1 + f.start : f.start;
    int base = 0;
    for (int b0 = 0; b0 < Bt; b0 += 32) {
        if (Bt > 32) {
            w = 0;
            if (b0 + lane < Bt) {
                s = seq_of(a, b0 + lane, R);
                w = seq_work(a, s, over);
            }
        }
        int p = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, p, o);
            if (lane >= o) p += y;
        }
        // the first sequence whose end lies behind u
        const uint32_t behind = __ballot_sync(0xFFFFFFFFu, base + p > u);
        if (behind) {
            const int l = __ffs(behind) - 1;
            f.b = b0 + l;
            f.off = u - __shfl_sync(0xFFFFFFFFu, base + p - w, l);
            f.s.cu0 = __shfl_sync(0xFFFFFFFFu, s.cu0, l);
            f.s.n = __shfl_sync(0xFFFFFFFFu, s.n, l);
            f.s.off = __shfl_sync(0xFFFFFFFFu, s.off, l);
            f.s.cap = __shfl_sync(0xFFFFFFFFu, s.cap, l);
            f.s.nt = __shfl_sync(0xFFFFFFFFu, s.nt, l);
            f.s.nk = __shfl_sync(0xFFFFFFFFu, s.nk, l);
            break;
        }
        base += __shfl_sync(0xFFFFFFFFu, p, 31);
    }
    return f;
}

// A run's pieces of segments in order: sequence, row tile, kv head, key tiles
// [x0, x1).  A segment's extra units come before its tiles; a run that ends
// among them has no piece of it.
struct Walk {
    Seq s;
    int b, rt, h, x0, x1;
    bool whole;       // all tiles of the segment
    int tile0, end0;  // units of the segment's first tile, and behind its last one
    int pos, end;
    int y, g, u0;     // the next segment: row tile in the order below, group of heads; its next unit
    int over, hi;     // hi: this CTA's head of those that share the run
    __device__ __forceinline__ Walk(const PagedAttn &a, const Found &f, int over_)
        : s(f.s), b(f.b), pos(f.start), end(f.run < f.work - f.start ? f.start + f.run : f.work),
          over(over_), hi(blockIdx.x % a.heads) {
        const int units = s.nk + over, seg = f.off / units;
        u0 = f.off - seg * units;
        y = seg / a.groups;
        g = seg - y * a.groups;
    }
    __device__ __forceinline__ bool next(const PagedAttn &a, int R) {
        while (pos < end) {
            while (y >= s.nt) {  // (only after a step; bounded by Bt)
                y = g = 0;
                if (++b >= a.step.Bt) return false;
                s = seq_of(a, b, R);
            }
            const int units = s.nk + over, from = u0;
            h = g * a.heads + hi;
            // last, first, last but one, ...: in a causal chunk late row tiles have more
            // keys than early ones, and a run of several gets its share of both
            rt = y & 1 ? y / 2 : s.nt - 1 - y / 2;
            const int u1 = min(u0 + end - pos, units);
            tile0 = pos - u0 + over;
            end0 = pos - u0 + units;
            pos += u1 - u0;
            u0 = u1 == units ? 0 : u1;
            if (u1 == units && ++g == a.groups) {
                g = 0;
                ++y;
            }
            if (u1 <= over) continue;
            x0 = max(from - over, 0);
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
    __device__ __forceinline__ int first_run(const Found &f) const { return tile0 / f.run; }
    __device__ __forceinline__ int last_run(const Found &f) const { return (end0 - 1) / f.run; }
};

// Slot of piece p of a segment that begins in run c0 (its heads' CTAs share it).
__device__ __forceinline__ long long piece_slot(const PagedAttn &a, int c0, int p) {
    return 2ll * ((c0 + p) * a.heads + blockIdx.x % a.heads) + (p == 0 ? 1 : 0);
}

}  // namespace walk

}  // namespace msa
