// Attention of chunks over the quantised cache: the size of a call's division, and the joining of the parts that it
// leaves.
//
// The division follows lengths that only the device knows: all tiles of all (run of rows, head) jobs, as the rows' windows and the
// prefixes leave them, are dealt to the pairs of CTAs in equal runs. A pair's open jobs at either end go to the workspace: the
// float32 outputs of their own places, and the sums of weights beside them. The joining launch starts while the first still runs, and
// adds them, each by its share of the weights, in the order of the units, so that results do not depend on timing. A unit's rows are shared out over several blocks too, two to
// a warp, since few units may hold all open jobs.
#include <math.h>

#include "qc_attend.cuh"
#include "qc_chunk.cuh"

namespace qc {
namespace {

constexpr int kThreads = 256;

// The unit that opens a job which others go on with adds that job's parts up: each warp a row at a time, its parts in
// the order of the units.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) chunk_join(const Chunk p, const ChunkParts parts, int units) {
    constexpr int N = D / 32;
    fq::sm100::griddep_wait();
    const int unit = blockIdx.x, lane = threadIdx.x & 31;
    // a unit's open job is the last of its run
    int64_t first = 2 * (int64_t)unit + 1;
    PartLine line = parts.lines[first];
    if (!line.what) line = parts.lines[--first];
    if (!(line.what & kOpens) || (line.what & kCloses)) return;
    // a line leads to rows of the call's own tensors or nowhere, whatever the workspace holds
    if (line.b < 0 || line.b >= p.n_seq || line.kv < 0 || line.kv >= p.g.heads) return;
    const Sequence s = sequence(p, line.b, false);
    if (line.run < 0 || line.run >= runs_of(p, s, parts.rows)) return;
    int last = unit + 1;
    while (last < units - 1 && !(parts.lines[2 * (int64_t)last].what & kCloses)) ++last;
    const int rows = min(s.news * p.group - line.run * parts.rows, parts.rows);
    for (int r = (int)blockIdx.y * (kThreads / 32) + (threadIdx.x >> 5); r < rows; r += (int)gridDim.y * (kThreads / 32)) {
        auto part_of = [&](int c) { return c == unit ? first : 2 * (int64_t)c; };
        auto stat = [&](int c) { return c <= last ? *parts.stat(part_of(c), r) : make_float2(-INFINITY, 0.f); };
        // lane i has the sums of the i-th part, and of every 32nd from there
        const float2 mine = stat(unit + lane);
        float m = mine.x, l = 0.f, o[N] = {};
        for (int c = unit + 32 + lane; c <= last; c += 32) m = fmaxf(m, stat(c).x);
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
        const float ref = m == -INFINITY ? 0.f : m;
        // a part's sum of weights in the largest reference's unit, as two factors: either may be far from 1
        auto weight = [&](float2 st) {
            const float t = st.x - ref, a = fmaxf(t, -100.f);
            return make_float2(exp2f(a), exp2f(t - a) * st.y);
        };
        float2 w = weight(mine);
        l = w.x * w.y;
        for (int c = unit + 32 + lane; c <= last; c += 32) {
            const float2 x = weight(stat(c));
            l = fmaf(x.x, x.y, l);
        }
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
        const float by = l != 0.f ? 1.f / l : 0.f;                  // a NaN goes out
        for (int c0 = unit; c0 <= last; c0 += 32) {
            if (c0 > unit) w = weight(stat(c0 + lane));
            const float share = w.y * by;
            const int n = min(last - c0 + 1, 32);
#pragma unroll 4
            for (int i = 0; i < n; ++i) {
                const float *v = parts.row(part_of(c0 + i), r) + lane * N;
                const float a = __shfl_sync(0xffffffffu, w.x, i), b = __shfl_sync(0xffffffffu, share, i);
#pragma unroll
                for (int k = 0; k < N; ++k) o[k] = fmaf(v[k] * a, b, o[k]);
            }
        }
        const int at = line.run * parts.rows + r, token = at / p.group;
        const int64_t out_row = (int64_t)(s.first + token) * p.n_q_heads + line.kv * p.group + (at - token * p.group);
        store_row<T, N>(static_cast<T *>(p.out) + out_row * D + lane * N, o);
        if (p.lse && lane == 0) p.lse[out_row] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
    }
}

template <typename T>
cudaError_t join(const Chunk &p, const ChunkParts &parts, int units, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)units - 1, (unsigned)parts.rows / (2 * kThreads / 32));       // two rows to a warp
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (p.g.d == 64) return cudaLaunchKernelEx(&cfg, chunk_join<T, 64>, p, parts, units);
    return cudaLaunchKernelEx(&cfg, chunk_join<T, 128>, p, parts, units);
}

}  // namespace

cudaError_t launch_chunk_join(const Chunk &p, const ChunkParts &parts, int type, int units, cudaStream_t s) {
    return type == QC_F16 ? join<__half>(p, parts, units, s) : join<__nv_bfloat16>(p, parts, units, s);
}

// Pairs of CTAs: as many as the card has, or as there may be tiles.
int chunk_units(const qc_ctx *c, int64_t n_seq, int64_t n_tokens, int group, int64_t max_len, int64_t max_new) {
    const int64_t one = n_tokens < max_new ? n_tokens : max_new, pairs = c->num_sms / 2;
    const int64_t tiles = (max_len + one + kChunkTile - 1) / kChunkTile + 1;
    // runs of rows: full ones, and one that is not for each sequence
    const int64_t runs = n_tokens * group / kChunkRows + (n_seq < n_tokens ? n_seq : n_tokens);
    if (runs >= pairs || tiles >= pairs || runs * tiles * c->heads >= pairs) return (int)pairs;
    return (int)(runs * tiles * c->heads < 1 ? 1 : runs * tiles * c->heads);
}

int64_t chunk_workspace(const qc_ctx *c, int64_t n_seq, int64_t n_tokens, int n_q_heads, int64_t max_len, int64_t max_new) {
    if (n_seq == 0 || n_tokens == 0 || max_new == 0) return 0;
    return chunk_parts_bytes(chunk_units(c, n_seq, n_tokens, n_q_heads / c->heads, max_len, max_new), kChunkRows, c->d);
}

cudaError_t launch_chunk(const qc_ctx *c, int type, const Chunk &p, cudaStream_t s) {
    if (c->d == 64)
        return c->fmt == QC_INT8   ? launch_chunk_tc<QC_INT8, 64>(c, type, p, s)
               : c->fmt == QC_E4M3 ? launch_chunk_tc<QC_E4M3, 64>(c, type, p, s)
                                   : launch_chunk_tc<QC_E2M1, 64>(c, type, p, s);
    return c->fmt == QC_INT8   ? launch_chunk_tc<QC_INT8, 128>(c, type, p, s)
           : c->fmt == QC_E4M3 ? launch_chunk_tc<QC_E4M3, 128>(c, type, p, s)
                               : launch_chunk_tc<QC_E2M1, 128>(c, type, p, s);
}

}  // namespace qc
