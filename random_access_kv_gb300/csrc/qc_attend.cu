// Attention over the quantised cache: choice of the kernel, and the joining of the parts that it leaves.
#include <math.h>

#include "qc_attend.cuh"

namespace qc {
namespace {

constexpr int kThreads = 128;

template <int N>
__device__ __forceinline__ void load_row(const float *p, float (&v)[N]) {
    if constexpr (N == 4) {
        const float4 x = *reinterpret_cast<const float4 *>(p);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
        const float2 x = *reinterpret_cast<const float2 *>(p);
        v[0] = x.x, v[1] = x.y;
    }
}

// One warp per query row. Rows of jobs within one unit are done already; the others' parts lie in
// consecutive units: part 2 c + 1 of the first (part 2 c if the job begins its run), part 2 c of the rest.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) join_parts(const Attend p, const Parts parts, int row_tiles, int tile, int units) {
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
        const int64_t per = run_length(total, units);
        const int64_t first = before + (int64_t)(h * row_tiles + rt) * tiles;
        const int64_t c0 = first / per, c1 = (first + tiles - 1) / per;
        if (c0 == c1) return;
        const int64_t p0 = 2 * c0 + (first == c0 * per ? 0 : 1);
        // all parts' maxima first, a lane each; then the values, several loads under way
        for (int64_t c = c0 + lane; c <= c1; c += 32) m = fmaxf(m, parts.stat(c == c0 ? p0 : 2 * c, rr)->x);
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
        const float ref = m == -INFINITY ? 0.f : m;
        for (int64_t cb = c0; cb <= c1; cb += 32) {
            const int n = (int)(c1 - cb + 1 < 32 ? c1 - cb + 1 : 32);
            float2 st = make_float2(-INFINITY, 0.f);
            if (lane < n) st = *parts.stat(cb + lane == c0 ? p0 : 2 * (cb + lane), rr);
            const float w = exp2f(st.x - ref);
            l += st.y * w;                      // this lane's parts
            for (int i0 = 0; i0 < n; i0 += 8) {
                float v[8][D / 32], wi[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int64_t c = cb + i0 + i;
                    wi[i] = __shfl_sync(0xffffffffu, w, (i0 + i) & 31);
                    if (i0 + i < n) {
                        load_row<D / 32>(parts.row(c == c0 ? p0 : 2 * c, rr) + lane * (D / 32), v[i]);
                    } else {
                        wi[i] = 0.f;
#pragma unroll
                        for (int j = 0; j < D / 32; ++j) v[i][j] = 0.f;
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) o[j] = fmaf(v[i][j], wi[i], o[j]);
            }
        }
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;      // a NaN goes out
    T *out = static_cast<T *>(p.out) + out_row * D + lane * (D / 32);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] *= inv;
    store_row<T, D / 32>(out, o);
    if (p.lse && lane == 0) p.lse[out_row] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

template <typename T, int D>
cudaError_t join(const Attend &p, const Parts &parts, int row_tiles, int tile, int units, cudaStream_t s) {
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
    return cudaLaunchKernelEx(&cfg, join_parts<T, D>, p, parts, row_tiles, tile, units);
}

}  // namespace

cudaError_t launch_join(const Attend &p, const Parts &parts, int type, int row_tiles, int tile, int units, cudaStream_t s) {
    if (type == QC_F16)
        return p.g.d == 64 ? join<__half, 64>(p, parts, row_tiles, tile, units, s)
                           : join<__half, 128>(p, parts, row_tiles, tile, units, s);
    return p.g.d == 64 ? join<__nv_bfloat16, 64>(p, parts, row_tiles, tile, units, s)
                       : join<__nv_bfloat16, 128>(p, parts, row_tiles, tile, units, s);
}

namespace {

// Which kernel. qc_attend_tc.cu pays 128 rows' tensor-core time and one thread's softmax per row whatever the
// rows' number, qc_attend_rows.cuh its conversion and products anew for every 24 or 32 rows: the first is for more
// than 32. Below about a thousand places rows whose weight lies on few places are likely, and qc_attend_rows.cuh
// follows their light weights further; that costs time where rows are many. Here (qc_attend_tc.cu) and there, us:
//   int8, bf16, d = 128, 16 x 16,384, 20 rows: 283 and 178; 32: 289 and 246; 36: 290 and 344;
//   the same in e2m1, 36 rows: 289 and 368; in fp16 queries, int8, 36 rows: 336 and 436;
//   e4m3, fp16, d = 64, 8 sequences of 4,096 places at most, 32 rows: 41 and 40; 40: 30 and 35; 128: 38 and 101;
//   e2m1, fp16, d = 128, 32 sequences of 32,768 places at most, 4 rows: 632 and 203; int8, bf16, 256 rows, 8 x 32,768:
//   392 and 1,669; 256 rows, 8 x 960 places: 51 and 138 (below the rule's bound: the second runs).
bool many_rows(int64_t max_len, int n_nodes, int rows) { return rows > 32 && max_len + n_nodes >= 1024; }

}  // namespace

// Of these sizes and of all smaller ones, whichever kernel they go to.
int64_t attend_workspace(const qc_ctx *c, int64_t n_seq, int n_nodes, int n_q_heads, int64_t max_len) {
    const int rows = n_nodes * (n_q_heads / c->heads);
    if (n_seq == 0) return 0;
    const int64_t few = c->d == 64 ? rows_workspace_d<64>(c, rows, n_seq, n_nodes, max_len) : rows_workspace_d<128>(c, rows, n_seq, n_nodes, max_len);
    const int64_t many = many_rows(max_len, n_nodes, rows) ? tc_workspace(c, n_seq, n_nodes, n_q_heads, max_len) : 0;
    return few > many ? few : many;
}

cudaError_t launch_attend(const qc_ctx *c, int type, const Attend &p, cudaStream_t s) {
    if (many_rows(p.max_len, p.n_nodes, p.n_nodes * p.group)) return launch_attend_tc(c, type, p, s);
    return c->d == 64 ? attend_rows_d<64>(c, type, p, s) : attend_rows_d<128>(c, type, p, s);
}

}  // namespace qc
