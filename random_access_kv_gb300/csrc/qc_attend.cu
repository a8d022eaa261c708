// Attention of drafted tokens over the quantised cache: one warp per query row.
//
// A lane holds d / 32 elements of the query; every place that the row sees costs one dot product over
// the warp, one step of the running maximum and sum, and d / 32 multiply-adds per lane.
#include <math.h>

#include "qc_formats.cuh"

namespace qc {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(__half *p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

template <int FMT>
__device__ __forceinline__ float element(const Geometry &g, const unsigned char *part, int which, int t, int e) {
    const int byte = t * g.row + (FMT == QC_E2M1 ? e / 2 : e);
    const uint32_t c = part[g.codes(which) + piece_at(byte >> 4) * 16 + (byte & 15)];
    if constexpr (FMT == QC_INT8) return (float)(signed char)c;
    if constexpr (FMT == QC_E4M3) return e4m3_value(c);
    const uint32_t h = half2_e2m1(e & 1 ? c >> 4 : c & 15u);
    const float sb = e4m3_value(part[g.block_scales(which) + t * g.blocks + e / 16]);
    return __half2float(__ushort_as_half((unsigned short)h)) * 16384.f * sb;
}

template <typename T, int D, int FMT>
__global__ void __launch_bounds__(kThreads) attend(const Attend p) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (row >= (int64_t)p.n_seq * p.n_nodes * p.n_q_heads) return;
    const int head = (int)(row % p.n_q_heads), node = (int)(row / p.n_q_heads % p.n_nodes);
    const int b = (int)(row / p.n_q_heads / p.n_nodes), kv = head / p.group;
    int len = p.lens[b], nodes = p.nodes ? p.nodes[b] : p.n_nodes;
    if (len < 0 || len > p.max_len || nodes < 0 || nodes > p.n_nodes) {
        if (lane == 0) atomicOr(p.flags, QC_FLAG_RANGE);
        len = min(max(len, 0), (int)p.max_len);
        nodes = min(max(nodes, 0), p.n_nodes);
    }
    const T *q = static_cast<const T *>(p.q) + b * p.q_seq + node * p.q_node + head * p.q_head;
    float qv[E], o[E];
    for (int i = 0; i < E; ++i) qv[i] = to_float(q[i * 32 + lane]), o[i] = 0.f;
    float m = -INFINITY, l = 0.f;
    const uint32_t *tree = p.tree ? p.tree + ((int64_t)b * p.n_nodes + node) * p.words : nullptr;
    const int end = node < nodes ? len + nodes : 0;
    for (int t = 0; t < end; ++t) {
        if (t >= len) {
            const int j = t - len;
            if (tree ? !((tree[j >> 5] >> (j & 31)) & 1u) : j > node) continue;
        }
        const int64_t page = p.table[b * p.table_stride + (t >> p.g.shift)];
        if (page < 0 || page >= p.n_pages) {
            if (lane == 0) atomicOr(p.flags, QC_FLAG_RANGE);
            continue;
        }
        const unsigned char *part = p.pages + (page * p.g.heads + kv) * (int64_t)p.g.part;
        const int at = t & (p.g.page - 1);
        float s = 0.f;
        for (int i = 0; i < E; ++i) s += qv[i] * element<FMT>(p.g, part, 0, at, i * 32 + lane);
        for (int x = 16; x >= 1; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= reinterpret_cast<const float *>(part + p.g.scales(0))[at] * p.scale;
        const float m2 = fmaxf(m, s), w = expf(s - m2), old = expf(m - m2);
        const float vs = reinterpret_cast<const float *>(part + p.g.scales(1))[at] * w;
        l = l * old + w;
        for (int i = 0; i < E; ++i) o[i] = o[i] * old + vs * element<FMT>(p.g, part, 1, at, i * 32 + lane);
        m = m2;
    }
    T *out = static_cast<T *>(p.out) + row * D;
    for (int i = 0; i < E; ++i) put(out + i * 32 + lane, l > 0.f ? o[i] / l : 0.f);
    if (p.lse && lane == 0) p.lse[row] = l > 0.f ? m + logf(l) : -INFINITY;
}

template <typename T, int D>
cudaError_t launch(const qc_ctx *c, const Attend &p, cudaStream_t s) {
    const int64_t rows = (int64_t)p.n_seq * p.n_nodes * p.n_q_heads, blocks = (rows + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    if (c->fmt == QC_INT8)
        attend<T, D, QC_INT8><<<(unsigned)blocks, kThreads, 0, s>>>(p);
    else if (c->fmt == QC_E4M3)
        attend<T, D, QC_E4M3><<<(unsigned)blocks, kThreads, 0, s>>>(p);
    else
        attend<T, D, QC_E2M1><<<(unsigned)blocks, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

int64_t attend_workspace(const qc_ctx *, int64_t, int, int, int64_t) { return 0; }

cudaError_t launch_attend(const qc_ctx *c, int type, const Attend &p, cudaStream_t s) {
    if (type == QC_F16) return c->d == 64 ? launch<__half, 64>(c, p, s) : launch<__half, 128>(c, p, s);
    return c->d == 64 ? launch<__nv_bfloat16, 64>(c, p, s) : launch<__nv_bfloat16, 128>(c, p, s);
}

}  // namespace qc
