// Rows in and out of the quantised cache.
//
// Bound by memory: a write reads each row once and writes 1/2 to 1/8 of it, a read the reverse. A row is held
// by d / 8 lanes, eight elements each. For a write its largest magnitude is a butterfly over those lanes (over
// two lanes for a block of e2m1); a lane's eight codes go out as one 8-byte (4-byte) store, so a row's codes
// make one full line (half a line). A warp takes U rows per lane group, of consecutive tokens and one head
// (which lie one after another in a page), all their loads under way together; neighbouring blocks take
// neighbouring heads. 32,768 tokens of 8 heads of 128 (bf16, e2m1): written in 57 us (3.0 TB/s; bound by issue
// slots, 84 %: four exact divisions a row or block, and the search for the largest magnitude), read in 40 us (4.4
// TB/s); a random read of 104,864 tokens (int8 to fp16) in 141 us (4.6 TB/s).
#include "qc_formats.cuh"

namespace qc {
namespace {

constexpr int kThreads = 128;

// Byte offset, within a head's part of a page, of the codes of elements e0 .. e0 + 7 of token t.
template <int FMT>
__device__ __forceinline__ int code_at(const Geometry &g, int which, int t, int e0) {
    const int byte = t * g.row + (FMT == QC_E2M1 ? e0 / 2 : e0);
    return g.codes(which) + piece_at(byte >> 4) * 16 + (byte & 15);
}

// What a block works on: blockIdx.x = (token group, head), blockIdx.y = keys or values.
template <int D, int U, int E>
struct Task {               // E elements of a row to a lane
    static constexpr int kLanes = D / E, kRows = 32 / kLanes;
    int lane, e0, h;
    int64_t token;          // of u = 0; the next ones kRows apart
    __device__ __forceinline__ Task(const Rows &p) {
        lane = threadIdx.x & 31;
        e0 = lane % kLanes * E;
        const uint32_t group = blockIdx.x / (uint32_t)p.g.heads;
        h = (int)(blockIdx.x - group * (uint32_t)p.g.heads);
        token = ((int64_t)group * (kThreads / 32) + (threadIdx.x >> 5)) * (U * kRows) + lane / kLanes;
    }
};

template <typename T, int D, int FMT, int U>
__global__ void __launch_bounds__(kThreads) write_rows(const Rows p) {
    const Task<D, U, 8> k(p);
    constexpr int kLanes = D / 8, kRows = 32 / kLanes;
    const int which = blockIdx.y, e0 = k.e0;
    const T *x = static_cast<const T *>(which ? p.v : p.k) + k.h * (which ? p.v_head : p.k_head) + e0;
    const int64_t stride = which ? p.v_token : p.k_token;
    Eight<T> in[U];
    int64_t slots[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t token = k.token + u * kRows;
        slots[u] = -1;
        if (token < p.n) {
            slots[u] = __ldg(p.slots + token);
            in[u].load(x + token * stride);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const bool there = k.token + u * kRows < p.n;
        const int64_t slot = slots[u];
        float v[8];
        if (there) {
            in[u].get(v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.f;
        }
        // largest magnitude, NaN included: of magnitudes as integers, which order as the floats do
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
        const uint32_t pair = max(top, __shfl_xor_sync(0xffffffffu, top, 1));     // a block of 16
        top = pair;
#pragma unroll
        for (int m = kLanes / 2; m >= 2; m >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
        if (!there || slot == -1) continue;
        if (slot < 0 || slot >= p.slots_end) {
            if (e0 == 0) atomicOr(p.flags, QC_FLAG_RANGE);
            continue;
        }
        const bool finite = top < 0x7f800000u;
        if (!finite && e0 == 0) atomicOr(p.flags, QC_FLAG_NONFINITE);
        const float A = __uint_as_float(top);
        const bool zero = !finite || A < kLeast;
        const float scale = zero ? 0.f : __fdiv_rn(A, kTop<FMT>);
        const float up = zero ? 0.f : __fdiv_rn(kTop<FMT>, A);
        unsigned char *part = p.pages + ((slot >> p.g.shift) * p.g.heads + k.h) * (int64_t)p.g.part;
        const int t = (int)(slot & (p.g.page - 1));
        float y[8];
        if constexpr (FMT == QC_E2M1) {
            uint32_t sb = 0;
            float by = 0.f;
            if (!zero) {
                sb = e4m3x2(__fmul_rn(__uint_as_float(pair), __fdiv_rn(448.f, A)), 0.f) & 0xffu;
                by = sb ? __fdiv_rn(up, e4m3_value(sb)) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = zero ? 0.f : __fmul_rn(v[i], by);
            *reinterpret_cast<uint32_t *>(part + code_at<FMT>(p.g, which, t, e0)) = codes_e2m1(y);
            if ((k.lane & 1) == 0) part[p.g.block_scales(which) + t * p.g.blocks + e0 / 16] = (unsigned char)sb;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = zero ? 0.f : __fmul_rn(v[i], up);
            *reinterpret_cast<uint2 *>(part + code_at<FMT>(p.g, which, t, e0)) =
                FMT == QC_INT8 ? codes_int8(y) : codes_e4m3(y);
        }
        if (e0 == 0) reinterpret_cast<float *>(part + p.g.scales(which))[t] = scale;
    }
}

// A lane takes 16 elements here (a 16-byte piece, or a block of e2m1): twice the bytes under way of eight.
template <typename T, int D, int FMT, int U>
__global__ void __launch_bounds__(kThreads) read_rows(const Rows p) {
    const Task<D, U, 16> k(p);
    constexpr int kRows = 32 / (D / 16);
    const int which = blockIdx.y, e0 = k.e0;
    T *out = static_cast<T *>(which ? p.v_out : p.k_out);
    if (!out) return;
    int64_t slots[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t token = k.token + u * kRows;
        slots[u] = token < p.n ? __ldg(p.slots + token) : -1;
    }
    uint4 c[U];
    uint32_t block[U];
    float scale[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        c[u] = make_uint4(0, 0, 0, 0);
        block[u] = 0;
        scale[u] = 0.f;
        if (slots[u] >= 0 && slots[u] < p.slots_end) {
            const unsigned char *part = p.pages + ((slots[u] >> p.g.shift) * p.g.heads + k.h) * (int64_t)p.g.part;
            const int t = (int)(slots[u] & (p.g.page - 1));
            const unsigned char *at = part + code_at<FMT>(p.g, which, t, e0);
            if constexpr (FMT == QC_E2M1) {
                const uint2 w = *reinterpret_cast<const uint2 *>(at);
                c[u].x = w.x, c[u].y = w.y;
                block[u] = part[p.g.block_scales(which) + t * p.g.blocks + e0 / 16];
            } else {
                c[u] = *reinterpret_cast<const uint4 *>(at);
            }
            scale[u] = reinterpret_cast<const float *>(part + p.g.scales(which))[t];
        } else if (slots[u] != -1 && e0 == 0) {
            atomicOr(p.flags, QC_FLAG_RANGE);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t token = k.token + u * kRows;
        if (token >= p.n) continue;
        const bool held = slots[u] >= 0 && slots[u] < p.slots_end;
        const float sb = FMT == QC_E2M1 ? e4m3_value(block[u]) : 0.f;
        T *to = out + (token * p.g.heads + k.h) * D + e0;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float v[8];
            if constexpr (FMT == QC_E2M1)
                values<FMT>(make_uint2(half ? c[u].y : c[u].x, 0), sb, v);
            else
                values<FMT>(half ? make_uint2(c[u].z, c[u].w) : make_uint2(c[u].x, c[u].y), sb, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = held ? v[i] * scale[u] : 0.f;
            Eight<T>::store(to + 8 * half, v);
        }
    }
}

template <typename T, int D, int FMT, int U, bool WRITE>
cudaError_t launch(const Rows &p, cudaStream_t s) {
    constexpr int kPerBlock = kThreads / 32 * (32 / (D / (WRITE ? 8 : 16))) * U;
    const int64_t blocks = (p.n + kPerBlock - 1) / kPerBlock * p.g.heads;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)blocks, 2);
    if constexpr (WRITE)
        write_rows<T, D, FMT, U><<<grid, kThreads, 0, s>>>(p);
    else
        read_rows<T, D, FMT, U><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T, int D, int FMT>
cudaError_t pick_u(const qc_ctx *c, const Rows &p, bool write, cudaStream_t s) {
    // Few rows: one per lane group, as many warps as there are. Many: four, for four loads under way (a random read
    // of 104,864 tokens: 170 us with one, 141 with four, 158 with eight).
    const bool many = p.n * p.g.heads * (D / 8) > (int64_t)c->num_sms * 2048;
    if (write) return many ? launch<T, D, FMT, 4, true>(p, s) : launch<T, D, FMT, 1, true>(p, s);
    return many ? launch<T, D, FMT, 4, false>(p, s) : launch<T, D, FMT, 1, false>(p, s);
}

template <typename T>
cudaError_t pick(const qc_ctx *c, const Rows &p, bool write, cudaStream_t s) {
    if (c->d == 64)
        return c->fmt == QC_INT8   ? pick_u<T, 64, QC_INT8>(c, p, write, s)
               : c->fmt == QC_E4M3 ? pick_u<T, 64, QC_E4M3>(c, p, write, s)
                                   : pick_u<T, 64, QC_E2M1>(c, p, write, s);
    return c->fmt == QC_INT8   ? pick_u<T, 128, QC_INT8>(c, p, write, s)
           : c->fmt == QC_E4M3 ? pick_u<T, 128, QC_E4M3>(c, p, write, s)
                               : pick_u<T, 128, QC_E2M1>(c, p, write, s);
}

cudaError_t run(const qc_ctx *c, int type, const Rows &p, bool write, cudaStream_t s) {
    return type == QC_F16    ? pick<__half>(c, p, write, s)
           : type == QC_BF16 ? pick<__nv_bfloat16>(c, p, write, s)
                             : pick<float>(c, p, write, s);
}

}  // namespace

cudaError_t launch_write(const qc_ctx *c, int type, const Rows &p, cudaStream_t s) { return run(c, type, p, true, s); }
cudaError_t launch_read(const qc_ctx *c, int type, const Rows &p, cudaStream_t s) { return run(c, type, p, false, s); }

}  // namespace qc
