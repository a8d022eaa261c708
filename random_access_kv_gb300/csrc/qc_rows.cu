// Rows in and out of the quantised cache.
//
// Bound by memory: a write reads each row once and writes 1/2 to 1/8 of it, a read the reverse. A row
// is held by d / 8 lanes, eight elements each. For a write its largest magnitude is a butterfly over
// those lanes (over two lanes for a block of e2m1); a lane's eight codes go out as one 8-byte (4-byte)
// store, so a row's codes make one full line (half a line).
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

template <typename T, int D, int FMT>
__global__ void __launch_bounds__(kThreads) write_rows(const Rows p) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes;
    const int lane = threadIdx.x & 31, e0 = (lane % kLanes) * 8;
    const int64_t row = ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kRows + lane / kLanes;
    // row = (token, k or v, head)
    const int per = 2 * p.g.heads;
    const int64_t token = row / per;
    const int rest = (int)(row - token * per), which = rest >= p.g.heads, h = which ? rest - p.g.heads : rest;
    const bool there = token < p.n;
    const int64_t slot = there ? __ldg(p.slots + token) : -1;
    float v[8];
    if (there) {
        Eight<T> r;
        r.load(static_cast<const T *>(which ? p.v : p.k) + token * (which ? p.v_token : p.k_token) +
               h * (which ? p.v_head : p.k_head) + e0);
        r.get(v);
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
    if (!there || slot == -1) return;
    if (slot < 0 || slot >= p.slots_end) {
        if (e0 == 0) atomicOr(p.flags, QC_FLAG_RANGE);
        return;
    }
    const bool finite = top < 0x7f800000u;
    if (!finite && e0 == 0) atomicOr(p.flags, QC_FLAG_NONFINITE);
    const float A = __uint_as_float(top);
    const bool zero = !finite || A < kLeast;
    const float scale = zero ? 0.f : __fdiv_rn(A, kTop<FMT>);
    const float up = zero ? 0.f : __fdiv_rn(kTop<FMT>, A);
    unsigned char *part = p.pages + ((slot >> p.g.shift) * p.g.heads + h) * (int64_t)p.g.part;
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
        if ((lane & 1) == 0) part[p.g.block_scales(which) + t * p.g.blocks + e0 / 16] = (unsigned char)sb;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = zero ? 0.f : __fmul_rn(v[i], up);
        *reinterpret_cast<uint2 *>(part + code_at<FMT>(p.g, which, t, e0)) =
            FMT == QC_INT8 ? codes_int8(y) : codes_e4m3(y);
    }
    if (e0 == 0) reinterpret_cast<float *>(part + p.g.scales(which))[t] = scale;
}

template <typename T, int D, int FMT>
__global__ void __launch_bounds__(kThreads) read_rows(const Rows p) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes;
    const int lane = threadIdx.x & 31, e0 = (lane % kLanes) * 8;
    const int64_t row = ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kRows + lane / kLanes;
    const int per = 2 * p.g.heads;
    const int64_t token = row / per;
    if (token >= p.n) return;
    const int rest = (int)(row - token * per), which = rest >= p.g.heads, h = which ? rest - p.g.heads : rest;
    T *out = static_cast<T *>(which ? p.v_out : p.k_out);
    if (!out) return;
    const int64_t slot = __ldg(p.slots + token);
    float v[8];
    if (slot < 0 || slot >= p.slots_end) {
        if (slot != -1 && e0 == 0) atomicOr(p.flags, QC_FLAG_RANGE);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
    } else {
        const unsigned char *part = p.pages + ((slot >> p.g.shift) * p.g.heads + h) * (int64_t)p.g.part;
        const int t = (int)(slot & (p.g.page - 1));
        const unsigned char *at = part + code_at<FMT>(p.g, which, t, e0);
        uint2 c;
        float block = 0.f;
        if constexpr (FMT == QC_E2M1) {
            c = make_uint2(*reinterpret_cast<const uint32_t *>(at), 0);
            block = e4m3_value(part[p.g.block_scales(which) + t * p.g.blocks + e0 / 16]);
        } else {
            c = *reinterpret_cast<const uint2 *>(at);
        }
        const float scale = reinterpret_cast<const float *>(part + p.g.scales(which))[t];
        values<FMT>(c, block, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= scale;
    }
    Eight<T>::store(out + (token * p.g.heads + h) * D + e0, v);
}

template <typename T, int D, int FMT>
cudaError_t launch(const Rows &p, bool write, cudaStream_t s) {
    constexpr int kPerBlock = kThreads / 32 * (32 / (D / 8));
    const int64_t blocks = (p.n * 2 * p.g.heads + kPerBlock - 1) / kPerBlock;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    if (write)
        write_rows<T, D, FMT><<<(unsigned)blocks, kThreads, 0, s>>>(p);
    else
        read_rows<T, D, FMT><<<(unsigned)blocks, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t pick(const qc_ctx *c, const Rows &p, bool write, cudaStream_t s) {
    if (c->d == 64)
        return c->fmt == QC_INT8   ? launch<T, 64, QC_INT8>(p, write, s)
               : c->fmt == QC_E4M3 ? launch<T, 64, QC_E4M3>(p, write, s)
                                   : launch<T, 64, QC_E2M1>(p, write, s);
    return c->fmt == QC_INT8   ? launch<T, 128, QC_INT8>(p, write, s)
           : c->fmt == QC_E4M3 ? launch<T, 128, QC_E4M3>(p, write, s)
                               : launch<T, 128, QC_E2M1>(p, write, s);
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
