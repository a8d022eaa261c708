// Norm of each head and its rotation by position, in one pass over the rows.
//
//   y = x * rsqrt(mean(x^2) + eps) * w;  (a, b) -> (a cos - b sin, b cos + a sin) on the first `rot`.
//
// Bound by memory: each element is read once and written once for about eight operations. A row is
// held by d / 8 lanes, eight consecutive elements (16 bytes of a 16-bit type) each; its mean square is
// a butterfly over those lanes. A warp keeps its token's cosines and sines in registers and takes
// several heads of the token with them.
#include "qc_formats.cuh"

namespace qc {
namespace {

constexpr int kThreads = 128;

// One lane's eight cosines and sines, in the order of its elements (pairs of neighbours: four of each).
struct Turn {
    float c[8], s[8];
};

template <typename T, int D, bool INTER, int U>
__global__ void __launch_bounds__(kThreads) norm_rope(const NormRope p, int q_chunks, int k_chunks) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kHeads = kRows * U;
    const int lane = threadIdx.x & 31, sub = lane / kLanes, e0 = (lane % kLanes) * 8;
    const int chunks = q_chunks + k_chunks;
    const int64_t task = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t token = task / chunks;
    if (token >= p.n) return;
    int chunk = (int)(task - token * chunks);
    const bool is_k = chunk >= q_chunks;
    if (is_k) chunk -= q_chunks;
    const Heads &t = is_k ? p.k : p.q;
    const int h0 = chunk * kHeads + sub;

    Eight<T> in[U];
    const T *x = static_cast<const T *>(t.x) + token * t.token + e0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = h0 + u * kRows;
        if (h < t.heads) in[u].load(x + h * t.head);
    }

    const int rot = p.rot, half = rot >> 1;
    bool in_table = true;
    Turn turn;
    const bool turned = e0 < rot;
    if (rot) {
        const int64_t pos = __ldg(p.pos + token);
        in_table = pos >= 0 && pos < p.max_pos;
        if (!in_table && lane == 0) atomicOr(p.flags, QC_FLAG_RANGE);
        if (in_table && turned) {
            const float *row = p.table + pos * rot;
            if constexpr (INTER) {
                const float4 c = __ldg(reinterpret_cast<const float4 *>(row + e0 / 2));
                const float4 s = __ldg(reinterpret_cast<const float4 *>(row + half + e0 / 2));
                turn.c[0] = c.x, turn.c[1] = c.y, turn.c[2] = c.z, turn.c[3] = c.w;
                turn.s[0] = s.x, turn.s[1] = s.y, turn.s[2] = s.z, turn.s[3] = s.w;
            } else {
                // the second half of the rotated elements adds its partner with the other sign
                const bool second = e0 >= half;
                const int i0 = second ? e0 - half : e0;
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    const float4 c = __ldg(reinterpret_cast<const float4 *>(row + i0 + i));
                    const float4 s = __ldg(reinterpret_cast<const float4 *>(row + half + i0 + i));
                    const float sign = second ? 1.f : -1.f;
                    turn.c[i] = c.x, turn.c[i + 1] = c.y, turn.c[i + 2] = c.z, turn.c[i + 3] = c.w;
                    turn.s[i] = sign * s.x, turn.s[i + 1] = sign * s.y, turn.s[i + 2] = sign * s.z,
                    turn.s[i + 3] = sign * s.w;
                }
            }
        }
    }
    float w[8];
    if (t.w) {
        Eight<float> r;
        r.load(t.w + e0);
        r.get(w);
    }
    // lane that holds the other halves of this lane's pairs (itself beyond the rotated elements)
    const int away = half / 8;
    const int partner = !turned ? lane : e0 >= half ? lane - away : lane + away;

    T *out = static_cast<T *>(t.out) + token * t.out_token + e0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = h0 + u * kRows;
        const bool there = h < t.heads;
        float v[8];
        if (there) {
            in[u].get(v);
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
        if (rot) {
            if constexpr (INTER) {
                if (turned && in_table) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float a = v[2 * i], b = v[2 * i + 1];
                        v[2 * i] = a * turn.c[i] - b * turn.s[i];
                        v[2 * i + 1] = b * turn.c[i] + a * turn.s[i];
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float other = __shfl_sync(0xffffffffu, v[i], partner);
                    if (turned && in_table) v[i] = v[i] * turn.c[i] + other * turn.s[i];
                }
            }
            if (!in_table) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = 0.f;
            }
        }
        if (there) Eight<T>::store(out + h * t.out_head, v);
    }
}

template <typename T, int D, bool INTER, int U>
cudaError_t launch(const NormRope &p, cudaStream_t s) {
    constexpr int kHeads = 32 / (D / 8) * U;
    const int qc = (p.q.heads + kHeads - 1) / kHeads, kc = (p.k.heads + kHeads - 1) / kHeads;
    const int64_t blocks = (p.n * (qc + kc) + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    norm_rope<T, D, INTER, U><<<(unsigned)blocks, kThreads, 0, s>>>(p, qc, kc);
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
