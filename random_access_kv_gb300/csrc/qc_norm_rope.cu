// Norm of each head and its rotation by position, in one pass over the rows.
//
//   y = x * rsqrt(mean(x^2) + eps) * w;  (a, b) -> (a cos - b sin, b cos + a sin) on the first `rot`.
//
// Bound by memory: each element is read once and written once for about eight operations. A row is held by d
// / 8 lanes, two groups of four elements each; its mean square is a butterfly over those lanes. Where the
// pairs lie half the rotated part apart, a lane's second group holds its first group's partners, so that
// the rotation takes no exchange. A warp keeps its token's cosines and sines in registers and takes several
// heads of the token with them, their loads under way together. 32,768 tokens of 32 + 8 heads of 128 (fp16):
// 119 us, 5.8 TB/s, 85 % of the card's copy rate; 128 us without the streaming hints, 153 us with eight
// neighbouring elements to a lane and an exchange between lanes. Few tokens are bound by the launch.
#include "qc_formats.cuh"

namespace qc {
namespace {

constexpr int kThreads = 128;

template <typename T, int D, bool INTER, int U>
__global__ void __launch_bounds__(kThreads) norm_rope(const NormRope p, int q_chunks) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kHeads = kRows * U;
    const int lane = threadIdx.x & 31, sub = lane / kLanes, i8 = lane % kLanes;
    const int64_t token = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (token >= p.n) return;
    const bool is_k = (int)blockIdx.y >= q_chunks;
    const Heads t = is_k ? p.k : p.q;
    const int h0 = ((int)blockIdx.y - (is_k ? q_chunks : 0)) * kHeads + sub;
    // the lane's groups of four: a pair's two halves, or neighbours
    const int rot = p.rot, half = rot >> 1;
    const bool turned = 8 * i8 < rot, apart = !INTER && turned;
    const int ea = apart ? 4 * i8 : 8 * i8, eb = apart ? half + 4 * i8 : 8 * i8 + 4;

    Four<T> in[U][2];
    const T *x = static_cast<const T *>(t.x) + token * t.token;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = h0 + u * kRows;
        if (h < t.heads) {
            in[u][0].load(x + h * t.head + ea, U > 1);
            in[u][1].load(x + h * t.head + eb, U > 1);
        }
    }
    bool in_table = true;
    float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (rot) {
        const int64_t pos = __ldg(p.pos + token);
        in_table = pos >= 0 && pos < p.max_pos;
        if (!in_table && lane == 0) atomicOr(p.flags, QC_FLAG_RANGE);
        if (in_table && turned) {
            const float *row = p.table + pos * rot + 4 * i8;
            c = __ldg(reinterpret_cast<const float4 *>(row));
            s = __ldg(reinterpret_cast<const float4 *>(row + half));
        }
    }
    float w[8];
    if (t.w) {
        Four<float> r;
        r.load(t.w + ea);
        r.get(w);
        r.load(t.w + eb);
        r.get(w + 4);
    }
    T *out = static_cast<T *>(t.out) + token * t.out_token;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = h0 + u * kRows;
        const bool there = h < t.heads;
        float v[8];
        if (there) {
            in[u][0].get(v);
            in[u][1].get(v + 4);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.f;
        }
        if (t.w) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(v[i], v[i], sum);
#pragma unroll
            for (int m = kLanes / 2; m >= 1; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
            const float r = rsqrtf(sum * (1.f / D) + p.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = v[i] * r * w[i];
        }
        if (turned) {
            const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float &a = INTER ? v[2 * i] : v[i], &b = INTER ? v[2 * i + 1] : v[4 + i];
                const float a0 = a, b0 = b;
                a = a0 * cs[i] - b0 * sn[i];
                b = b0 * cs[i] + a0 * sn[i];
            }
        }
        if (!in_table) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.f;
        }
        if (there) {
            Four<T>::store(out + h * t.out_head + ea, v, U > 1);
            Four<T>::store(out + h * t.out_head + eb, v + 4, U > 1);
        }
    }
}

template <typename T, int D, bool INTER, int U>
cudaError_t launch(const NormRope &p, cudaStream_t s) {
    constexpr int kHeads = 32 / (D / 8) * U;
    const int qc = (p.q.heads + kHeads - 1) / kHeads, kc = (p.k.heads + kHeads - 1) / kHeads;
    const int64_t blocks = (p.n + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    norm_rope<T, D, INTER, U><<<dim3((unsigned)blocks, (unsigned)(qc + kc)), kThreads, 0, s>>>(p, qc);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t pick(const qc_ctx *c, const NormRope &p, cudaStream_t s) {
    // Few rows: one per lane group, as many warps as there are. Many: four, so that a warp has four
    // loads under way and reads its token's table row once for all of them.
    const int64_t rows = p.n * (p.q.heads + p.k.heads);
    const bool many = rows * (D / 8) > (int64_t)c->num_sms * 2048;
    if (p.interleaved) return many ? launch<T, D, true, 4>(p, s) : launch<T, D, true, 1>(p, s);
    return many ? launch<T, D, false, 4>(p, s) : launch<T, D, false, 1>(p, s);
}

template <typename T>
cudaError_t pick_d(const qc_ctx *c, const NormRope &p, cudaStream_t s) {
    return c->d == 64 ? pick<T, 64>(c, p, s) : pick<T, 128>(c, p, s);
}

}  // namespace

cudaError_t launch_norm_rope(const qc_ctx *c, int type, const NormRope &p, cudaStream_t s) {
    return type == QC_F16 ? pick_d<__half>(c, p, s) : type == QC_BF16 ? pick_d<__nv_bfloat16>(c, p, s) : pick_d<float>(c, p, s);
}

}  // namespace qc
