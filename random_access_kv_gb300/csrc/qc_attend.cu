// Attention over the quantised cache: choice of the kernel, and the joining of the parts that it leaves.
#include <math.h>

#include "qc_attend.cuh"

namespace qc {
namespace {

constexpr int kThreads = 128;

// One warp per query row. Rows of jobs within one CTA are done already; the others' parts lie in
// consecutive CTAs: part 2 c + 1 of the first (part 2 c if the job begins its run), part 2 c of the rest.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) join_parts(const Attend p, const Parts parts, int row_tiles, int tile, int ctas) {
    fq::sm100::griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int R = p.n_nodes * p.group;
    if (row >= (int64_t)p.n_seq * p.g.heads * R) return;
    const int r = (int)(row % R), h = (int)(row / R % p.g.heads), b = (int)(row / R / p.g.heads);
    const int jobs = p.g.heads * row_tiles, rt = r / parts.rows, rr = r - rt * parts.rows;
    const int2 n = lengths(p, b, false);
    const int tiles = tiles_of(n, tile);
    const int64_t out_row = ((int64_t)b * p.n_nodes + r / p.group) * p.n_q_heads + h * p.group + r % p.group;
    float m = -INFINITY, l = 0.f;
    float o[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
    if (tiles && r / p.group < n.y) {
        const int64_t before = parts.before[b], total = parts.before[p.n_seq];
        const int64_t per = run_length(total, ctas);
        const int64_t first = before + (int64_t)(h * row_tiles + rt) * tiles;
        const int64_t c0 = first / per, c1 = (first + tiles - 1) / per;
        if (c0 == c1) return;
        const int64_t p0 = 2 * c0 + (first == c0 * per ? 0 : 1);
        for (int64_t c = c0; c <= c1; ++c) m = fmaxf(m, parts.stat(c == c0 ? p0 : 2 * c, rr)->x);
        const float ref = m == -INFINITY ? 0.f : m;
        for (int64_t c = c0; c <= c1; ++c) {
            const int64_t at = c == c0 ? p0 : 2 * c;
            const float2 s = *parts.stat(at, rr);
            const float w = exp2f(s.x - ref);
            l = fmaf(s.y, w, l);
            const float *v = parts.row(at, rr) + lane * (D / 32);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) o[i] = fmaf(v[i], w, o[i]);
        }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    T *out = static_cast<T *>(p.out) + out_row * D + lane * (D / 32);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] *= inv;
    store_row<T, D / 32>(out, o);
    if (p.lse && lane == 0) p.lse[out_row] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

template <typename T, int D>
cudaError_t join(const Attend &p, const Parts &parts, int row_tiles, int tile, int ctas, cudaStream_t s) {
    const int64_t rows = (int64_t)p.n_seq * p.n_nodes * p.n_q_heads;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((rows + kThreads / 32 - 1) / (kThreads / 32)));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_parts<T, D>, p, parts, row_tiles, tile, ctas);
}

}  // namespace

cudaError_t launch_join(const Attend &p, const Parts &parts, int type, int row_tiles, int tile, int ctas, cudaStream_t s) {
    if (type == QC_F16)
        return p.g.d == 64 ? join<__half, 64>(p, parts, row_tiles, tile, ctas, s)
                           : join<__half, 128>(p, parts, row_tiles, tile, ctas, s);
    return p.g.d == 64 ? join<__nv_bfloat16, 64>(p, parts, row_tiles, tile, ctas, s)
                       : join<__nv_bfloat16, 128>(p, parts, row_tiles, tile, ctas, s);
}

int64_t attend_workspace(const qc_ctx *c, int64_t n_seq, int n_nodes, int n_q_heads, int64_t max_len) {
    return rows_workspace(c, n_seq, n_nodes, n_q_heads, max_len);
}

cudaError_t launch_attend(const qc_ctx *c, int type, const Attend &p, cudaStream_t s) {
    return launch_attend_rows(c, type, p, s);
}

}  // namespace qc
