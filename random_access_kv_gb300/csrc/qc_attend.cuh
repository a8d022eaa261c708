// What the attention kernels of the quantised cache share: the division of the work, and the joining of
// its parts.
//
// A job is one (sequence, key/value head, tile of query rows); row r of a sequence's head is node r /
// group, query head r % group of that head. A job's places come in tiles of a kernel's own length. All
// tiles of all jobs, in order, are dealt to the units (warps or CTAs) in runs of equal length, so that sequences of
// unlike lengths fill the card evenly; a unit may end one job and begin the next. A job that lies within
// one unit's run is written out by it. Of any other, each unit leaves its part (running maximum m, sum l,
// and weighted values, all float32) in the workspace, and `join_parts` adds the parts in order.
#pragma once

#include <atomic>
#include <type_traits>

#include "fq_sm100.cuh"
#include "qc_formats.cuh"

namespace qc {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Lengths of sequence b, clamped to what the call allows.
__device__ __forceinline__ int2 lengths(const Attend &p, int b, bool tell) {
    int len = __ldg(p.lens + b), nodes = p.nodes ? __ldg(p.nodes + b) : p.n_nodes;
    if (len < 0 || len > p.max_len || nodes < 0 || nodes > p.n_nodes) {
        if (tell) atomicOr(p.flags, QC_FLAG_RANGE);
        len = min(max(len, 0), (int)p.max_len);
        nodes = min(max(nodes, 0), p.n_nodes);
    }
    return make_int2(len, nodes);
}

__device__ __forceinline__ int tiles_of(int2 n, int tile) { return n.y ? (n.x + n.y + tile - 1) / tile : 0; }

// Tiles of one job of every sequence, summed (one warp).
__device__ __forceinline__ int64_t all_tiles(const Attend &p, int tile, int lane) {
    int64_t sum = 0;
    for (int b = lane; b < p.n_seq; b += 32) sum += tiles_of(lengths(p, b, false), tile);
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    return sum;
}

// A unit's place in the order of tiles.
struct Walk {
    int b, job, tile;       // sequence, job within it (head * row tiles + row tile), tile within the job
    int tiles;              // tiles of the job
    int2 n;                 // lengths of the sequence
    int64_t left;           // tiles that the unit still has, this one included
};

// Fills `before` (one warp).
__device__ __forceinline__ void write_before(const Attend &p, int64_t *before, int jobs, int tile, int lane) {
    int64_t base = 0;
    for (int b0 = 0; b0 < p.n_seq; b0 += 32) {
        const int b = b0 + lane;
        const int64_t mine = b < p.n_seq ? (int64_t)tiles_of(lengths(p, b, true), tile) * jobs : 0;
        int64_t upto = mine;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, upto, m);
            if (lane >= m) upto += o;
        }
        if (b < p.n_seq) before[b] = base + upto - mine;
        base += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (lane == 0) before[p.n_seq] = base;
}

// The place of tile `at` (one warp; at < total). jobs: jobs per sequence.
__device__ __forceinline__ Walk find(const Attend &p, int64_t at, int64_t left, int jobs, int tile, int lane) {
    Walk w = {};
    w.left = left;
    if (left <= 0) return w;
    for (int b0 = 0;; b0 += 32) {
        const int b = b0 + lane;
        const int2 n = b < p.n_seq ? lengths(p, b, false) : make_int2(0, 0);
        const int64_t mine = (int64_t)tiles_of(n, tile) * jobs;
        int64_t upto = mine;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, upto, m);
            if (lane >= m) upto += o;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, upto > at);
        if (past) {
            const int l = __ffs(past) - 1;
            w.b = b0 + l;
            const int64_t start = __shfl_sync(0xffffffffu, upto - mine, l);
            w.n.x = __shfl_sync(0xffffffffu, n.x, l);
            w.n.y = __shfl_sync(0xffffffffu, n.y, l);
            w.tiles = tiles_of(w.n, tile);
            w.job = (int)((at - start) / w.tiles);
            w.tile = (int)((at - start) - (int64_t)w.job * w.tiles);
            return w;
        }
        at -= __shfl_sync(0xffffffffu, upto, 31);
        if (b0 + 32 >= p.n_seq) {       // not reached: at < total
            w.left = 0;
            return w;
        }
    }
}

// The next job's first tile. False at the end of the unit's run.
__device__ __forceinline__ bool next_job(const Attend &p, Walk &w, int jobs, int tile) {
    if (w.left <= 0) return false;
    w.tile = 0;
    if (++w.job < jobs) return true;
    w.job = 0;
    while (++w.b < p.n_seq) {
        w.n = lengths(p, w.b, false);
        w.tiles = tiles_of(w.n, tile);
        if (w.tiles) return true;
    }
    w.left = 0;
    return false;
}

// Tiles per unit, and so the unit of a tile.
__device__ __forceinline__ int64_t run_length(int64_t total, int units) { return (total + units - 1) / units; }

// The workspace: `before` [n_seq + 1], the tiles of the jobs before each sequence (and of all), and the
// parts. unit c's first job (it may have begun in an earlier unit) is part 2 c, the job
// at the end of its run part 2 c + 1 when that is another one. Per part: values [rows][d], then for
// all parts (m, l) [rows].
struct Parts {
    int64_t *before;
    float *values;
    float2 *ml;
    int rows, d;
    __device__ __forceinline__ float *row(int64_t part, int r) const { return values + (part * rows + r) * d; }
    __device__ __forceinline__ float2 *stat(int64_t part, int r) const { return ml + part * rows + r; }
};
inline int64_t before_bytes(int64_t n_seq) { return (n_seq * 8 + 8 + 15) / 16 * 16; }
inline int64_t workspace_bytes(int64_t n_seq, int64_t parts, int rows, int d) {
    return before_bytes(n_seq) + parts * rows * ((int64_t)d * 4 + 8);
}
inline Parts parts_at(void *ws, int64_t n_seq, int64_t parts, int rows, int d) {
    Parts r;
    r.before = (int64_t *)ws;
    r.values = (float *)((char *)ws + before_bytes(n_seq));
    r.ml = (float2 *)(r.values + parts * rows * d);
    r.rows = rows;
    r.d = d;
    return r;
}

// Lets a kernel use `bytes` of shared memory on the current device: asked for once per kernel and device (`done`: a
// bit per device).
template <typename Kernel>
inline cudaError_t allow_smem(Kernel *kernel, int bytes, int device, std::atomic<uint64_t> &done) {
    const uint64_t bit = 1ull << (device & 63);
    if (device < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Joins the parts of every job that lies in several units, and writes the zeros of sequences without tiles.
cudaError_t launch_join(const Attend &p, const Parts &parts, int type, int row_tiles, int tile, int units, cudaStream_t s);

// The kernels (qc_attend_rows.cuh, qc_attend_tc.cu).
template <int D>
cudaError_t attend_rows_d(const qc_ctx *c, int type, const Attend &p, cudaStream_t s);
template <int D>
int64_t rows_workspace_d(const qc_ctx *c, int rows, int64_t n_seq, int n_nodes, int64_t max_len);
template <>
cudaError_t attend_rows_d<64>(const qc_ctx *c, int type, const Attend &p, cudaStream_t s);
template <>
cudaError_t attend_rows_d<128>(const qc_ctx *c, int type, const Attend &p, cudaStream_t s);
template <>
int64_t rows_workspace_d<64>(const qc_ctx *c, int rows, int64_t n_seq, int n_nodes, int64_t max_len);
template <>
int64_t rows_workspace_d<128>(const qc_ctx *c, int rows, int64_t n_seq, int n_nodes, int64_t max_len);
cudaError_t launch_attend_tc(const qc_ctx *c, int type, const Attend &p, cudaStream_t s);
int64_t tc_workspace(const qc_ctx *c, int64_t n_seq, int n_nodes, int n_q_heads, int64_t max_len);

// N consecutive results of a row to their type; 16-byte stores where N allows.
template <typename T, int N>
__device__ __forceinline__ void store_row(T *out, const float *v) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        if constexpr (sizeof(T) == 2 && std::is_same<T, __half>::value) {
            const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    if constexpr (N % 8 == 0) {
#pragma unroll
        for (int i = 0; i < N / 8; ++i)
            reinterpret_cast<uint4 *>(out)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else if constexpr (N == 4) {
        *reinterpret_cast<uint2 *>(out) = make_uint2(w[0], w[1]);
    } else {
        *reinterpret_cast<uint32_t *>(out) = w[0];
    }
}

}  // namespace qc
