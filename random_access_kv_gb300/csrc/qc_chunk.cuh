// What the kernels of attention of chunks share: a sequence and its masks, the division of the work, and the parts that
// are joined.
//
// A job is one (sequence, key/value head, run of ROWS query rows); row r of a sequence's head is new token r / group,
// query head r % group of that head. A job's places come in tiles of 128, from the first that any of its rows sees
// to the last. All tiles of all jobs, in order, are dealt to the units (pairs of CTAs) in runs of equal length,
// so that sequences of unlike lengths fill the card evenly; a unit may end one job and begin the next. A job that lies
// within one unit's run is written out by it. Of any other, each unit leaves its part in the workspace, with a
// line that says whose it is, and the parts are added in order.
#pragma once

#include <cuda_runtime.h>

#include "qc_internal.h"

namespace qc {

constexpr int kChunkTile = 128;

struct Sequence {
    int len, news;          // cached and new tokens
    int prefix;             // places that all its rows see, at most len + news
    int first;              // row of its first new token
};

// Sequence b's, clamped to what the call allows.
__device__ __forceinline__ Sequence sequence(const Chunk &p, int b, bool tell) {
    const int n = (int)p.n_tokens;
    int from = __ldg(p.starts + b), to = __ldg(p.starts + b + 1), len = __ldg(p.lens + b);
    if (from < 0 || to < from || to > n || to - from > p.max_new || len < 0 || len > p.max_len) {
        if (tell) atomicOr(p.flags, QC_FLAG_RANGE);
        from = min(max(from, 0), n);
        to = min(max(to, from), n);
        to = from + min(to - from, p.max_new);
        len = min(max(len, 0), p.max_len);
    }
    Sequence s;
    s.len = len;
    s.news = to - from;
    s.prefix = p.prefix ? min(__ldg(p.prefix + b), len + s.news) : 0;
    s.first = from;
    return s;
}

// The places lo .. hi - 1 that the row at place t sees.
__device__ __forceinline__ int2 sees(const Chunk &p, const Sequence &s, int t) {
    return make_int2(p.window && t + 1 > p.window ? t + 1 - p.window : 0, max(t + 1, s.prefix));
}

// Tiles from x to y - 1 that rows r0 .. r0 + n - 1 of a head see; none where there are no such rows.
__device__ __forceinline__ int2 tiles_of_rows(const Chunk &p, const Sequence &s, int r0, int n) {
    const int rows = s.news * p.group;
    if (r0 >= rows) return make_int2(0, 0);
    const int i0 = r0 / p.group, i1 = (min(r0 + n, rows) - 1) / p.group;
    return make_int2(sees(p, s, s.len + i0).x / kChunkTile, (sees(p, s, s.len + i1).y + kChunkTile - 1) / kChunkTile);
}

__device__ __forceinline__ int runs_of(const Chunk &p, const Sequence &s, int rows) { return (s.news * p.group + rows - 1) / rows; }

// A unit's place in the order of tiles.
struct ChunkWalk {
    int b, kv, run;         // sequence, head, run of rows
    Sequence s;
    int first, last;        // the job's tiles: first .. last - 1
    int tile;
    int64_t left;           // tiles that the unit still has, this one included

    // The unit's steps of this job: tile .. end() - 1; the job's first step is its last tile.
    __device__ __forceinline__ int end() const { return left < last - tile ? tile + (int)left : last; }
    // The tile of a step, and the step of a tile.
    __device__ __forceinline__ int place(int step) const { return first + last - 1 - step; }
    template <int ROWS>
    __device__ __forceinline__ void enter(const Chunk &p) {
        const int2 t = tiles_of_rows(p, s, run * ROWS, ROWS);
        first = t.x;
        last = t.y;
        tile = first;
    }
    // On to the next job's first tile. left is 0 at the end of the unit's run.
    template <int ROWS>
    __device__ __forceinline__ void next(const Chunk &p) {
        left -= end() - tile;
        if (left <= 0) return;
        if (++run >= runs_of(p, s, ROWS)) {
            run = 0;
            if (++kv >= p.g.heads) {
                kv = 0;
                do {
                    if (++b >= p.n_seq) {
                        left = 0;
                        return;
                    }
                    s = sequence(p, b, false);
                } while (!s.news);
            }
        }
        enter<ROWS>(p);
    }
};

__device__ __forceinline__ int64_t warp_sum(int64_t x) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}
__device__ __forceinline__ int64_t warp_upto(int64_t x, int lane) {
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, m);
        if (lane >= m) x += y;
    }
    return x;
}
__device__ __forceinline__ Sequence of_lane(const Sequence &s, int l) {
    Sequence r;
    r.len = __shfl_sync(0xffffffffu, s.len, l);
    r.news = __shfl_sync(0xffffffffu, s.news, l);
    r.prefix = __shfl_sync(0xffffffffu, s.prefix, l);
    r.first = __shfl_sync(0xffffffffu, s.first, l);
    return r;
}

// Tiles of one head of this lane's sequence (one warp). Few runs are counted by the lane, many by the warp.
template <int ROWS>
__device__ __forceinline__ int64_t head_tiles(const Chunk &p, const Sequence &s, int lane) {
    const int runs = runs_of(p, s, ROWS);
    int64_t sum = 0;
    if (runs <= 4)
        for (int i = 0; i < runs; ++i) {
            const int2 t = tiles_of_rows(p, s, i * ROWS, ROWS);
            sum += t.y - t.x;
        }
    for (uint32_t many = __ballot_sync(0xffffffffu, runs > 4); many; many &= many - 1) {
        const int l = __ffs(many) - 1;
        const Sequence o = of_lane(s, l);
        const int n = runs_of(p, o, ROWS);
        int64_t mine = 0;
        for (int i = lane; i < n; i += 32) {
            const int2 t = tiles_of_rows(p, o, i * ROWS, ROWS);
            mine += t.y - t.x;
        }
        mine = warp_sum(mine);
        if (lane == l) sum = mine;
    }
    return sum;
}

__device__ __forceinline__ Sequence sequence_or_none(const Chunk &p, int b, bool tell) {
    return b < p.n_seq ? sequence(p, b, tell) : Sequence{0, 0, 0, 0};
}

// Unit `unit` of `units`' run (one warp). tell: what is out of range is reported.
template <int ROWS>
__device__ __forceinline__ ChunkWalk find_run(const Chunk &p, int unit, int units, bool tell, int lane) {
    int64_t total = 0;
    for (int b = 0; b < p.n_seq; b += 32) total += head_tiles<ROWS>(p, sequence_or_none(p, b + lane, tell), lane);
    total = warp_sum(total) * p.g.heads;
    const int64_t per = (total + units - 1) / units;
    int64_t at = per * unit;
    ChunkWalk w = {};
    w.left = at < total ? (total - at < per ? total - at : per) : 0;
    if (w.left <= 0) return w;
    for (int b0 = 0; b0 < p.n_seq; b0 += 32) {
        const Sequence s = sequence_or_none(p, b0 + lane, false);
        const int64_t one = head_tiles<ROWS>(p, s, lane), mine = one * p.g.heads, upto = warp_upto(mine, lane);
        const uint32_t past = __ballot_sync(0xffffffffu, upto > at);
        if (!past) {
            at -= __shfl_sync(0xffffffffu, upto, 31);
            continue;
        }
        const int l = __ffs(past) - 1;
        at -= __shfl_sync(0xffffffffu, upto - mine, l);
        const int64_t head = __shfl_sync(0xffffffffu, one, l);
        w.b = b0 + l;
        w.s = of_lane(s, l);
        w.kv = (int)(at / head);
        at -= w.kv * head;
        const int runs = runs_of(p, w.s, ROWS);
        for (int i0 = 0; i0 < runs; i0 += 32) {
            const int2 t = tiles_of_rows(p, w.s, (i0 + lane) * ROWS, ROWS);
            const int64_t n = i0 + lane < runs ? t.y - t.x : 0, to = warp_upto(n, lane);
            const uint32_t here = __ballot_sync(0xffffffffu, to > at);
            if (here) {
                const int k = __ffs(here) - 1;
                at -= __shfl_sync(0xffffffffu, to - n, k);
                w.run = i0 + k;
                break;
            }
            at -= __shfl_sync(0xffffffffu, to, 31);
        }
        w.enter<ROWS>(p);
        w.tile += (int)at;
        return w;
    }
    w.left = 0;             // not reached: at < total
    return w;
}

// The workspace: for each of 2 units' parts a line, then values [rows][d], then (reference, sum) [rows]. A unit's first
// job is part 2 unit, the last one of its run, if that is another, part 2 unit + 1. A unit's lines are emptied before
// anything of it can give up, and written when all of its copies are under way: so a line is this call's, or empty.
struct PartLine {
    int b, kv, run;
    int what;               // 0: no part; else kHolds, with kOpens where it has the job's first tile, kCloses its last
};
enum { kHolds = 1, kOpens = 2, kCloses = 4 };

struct ChunkParts {
    PartLine *lines;
    float *values;
    float2 *ml;
    int rows, d;
    __device__ __forceinline__ float *row(int64_t part, int r) const { return values + (part * rows + r) * d; }
    __device__ __forceinline__ float2 *stat(int64_t part, int r) const { return ml + part * rows + r; }
};
inline int64_t chunk_parts_bytes(int64_t units, int rows, int d) { return 2 * units * (16 + rows * ((int64_t)d * 4 + 8)); }
inline ChunkParts chunk_parts_at(void *ws, int64_t units, int rows, int d) {
    ChunkParts r;
    r.lines = (PartLine *)ws;
    r.values = (float *)(r.lines + 2 * units);
    r.ml = (float2 *)(r.values + 2 * units * rows * d);
    r.rows = rows;
    r.d = d;
    return r;
}

// What the host settles of a call.
struct ChunkPlan {
    int device;
    int units;
    int raw;                // stages of codes as the pages hold them
    int smem;
};

// A call's kernel (qc_chunk_tc.cuh), by format and head dimension.
constexpr int kChunkRows = 512;         // of a job
template <int FMT, int D>
cudaError_t launch_chunk_tc(const qc_ctx *c, int type, const Chunk &p, cudaStream_t s);
int chunk_units(const qc_ctx *c, int64_t n_seq, int64_t n_tokens, int group, int64_t max_len, int64_t max_new);
cudaError_t launch_chunk_join(const Chunk &p, const ChunkParts &parts, int type, int units, cudaStream_t s);

}  // namespace qc
