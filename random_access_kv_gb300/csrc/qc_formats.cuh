// Device helpers of the quantised cache: rows of fp16, bf16 or fp32 in and out of registers, and the
// three code formats of include/qcache.h.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "qc_internal.h"

namespace qc {

// Eight consecutive elements of a row held by one lane, as they lie in memory.
template <typename T>
struct Eight;
template <>
struct Eight<__half> {
    uint4 r;
    __device__ __forceinline__ void load(const __half *p) { r = *(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
    static __device__ __forceinline__ void store(__half *p, const float (&v)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Eight<__nv_bfloat16> {
    uint4 r;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { r = *(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&v)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = *(reinterpret_cast<const float4 *>(p));
        b = *(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    static __device__ __forceinline__ void store(float *p, const float (&v)[8]) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
};

// Four consecutive elements. once: they are touched a single time, and need not stay in the second-level cache.
template <typename T>
struct Four;
template <>
struct Four<__half> {
    uint2 r;
    __device__ __forceinline__ void load(const __half *p, bool once = false) {
        r = once ? __ldcs(reinterpret_cast<const uint2 *>(p)) : *reinterpret_cast<const uint2 *>(p);
    }
    __device__ __forceinline__ void get(float *v) const {
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&r.x)), b = __half22float2(*reinterpret_cast<const __half2 *>(&r.y));
        v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
    }
    static __device__ __forceinline__ void store(__half *p, const float *v, bool once = false) {
        const __half2 a = __floats2half2_rn(v[0], v[1]), b = __floats2half2_rn(v[2], v[3]);
        const uint2 w = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
        if (once)
            __stcs(reinterpret_cast<uint2 *>(p), w);
        else
            *reinterpret_cast<uint2 *>(p) = w;
    }
};
template <>
struct Four<__nv_bfloat16> {
    uint2 r;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p, bool once = false) {
        r = once ? __ldcs(reinterpret_cast<const uint2 *>(p)) : *reinterpret_cast<const uint2 *>(p);
    }
    __device__ __forceinline__ void get(float *v) const {
        v[0] = __uint_as_float(r.x << 16), v[1] = __uint_as_float(r.x & 0xffff0000u);
        v[2] = __uint_as_float(r.y << 16), v[3] = __uint_as_float(r.y & 0xffff0000u);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float *v, bool once = false) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
        const uint2 w = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
        if (once)
            __stcs(reinterpret_cast<uint2 *>(p), w);
        else
            *reinterpret_cast<uint2 *>(p) = w;
    }
};
template <>
struct Four<float> {
    float4 r;
    __device__ __forceinline__ void load(const float *p, bool once = false) {
        r = once ? __ldcs(reinterpret_cast<const float4 *>(p)) : *reinterpret_cast<const float4 *>(p);
    }
    __device__ __forceinline__ void get(float *v) const { v[0] = r.x, v[1] = r.y, v[2] = r.z, v[3] = r.w; }
    static __device__ __forceinline__ void store(float *p, const float *v, bool once = false) {
        const float4 w = make_float4(v[0], v[1], v[2], v[3]);
        if (once)
            __stcs(reinterpret_cast<float4 *>(p), w);
        else
            *reinterpret_cast<float4 *>(p) = w;
    }
};

// Eight floats, already in a code's units, to codes (round to nearest even, largest code beyond the
// range): 8 bytes for the 8-bit formats, 4 for e2m1.
__device__ __forceinline__ uint2 codes_int8(const float (&y)[8]) {
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = (uint32_t)__float2int_rn(y[i]) & 0xffu;
    return make_uint2(b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24, b[4] | b[5] << 8 | b[6] << 16 | b[7] << 24);
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint2 codes_e4m3(const float (&y)[8]) {
    return make_uint2(e4m3x2(y[0], y[1]) | e4m3x2(y[2], y[3]) << 16, e4m3x2(y[4], y[5]) | e4m3x2(y[6], y[7]) << 16);
}
__device__ __forceinline__ uint32_t codes_e2m1(const float (&y)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    return r;
}

// Codes as fp16 pairs. Each 8- or 4-bit value is a fp16 value times a power of two, so moving its
// bits to fp16's places converts it exactly, subnormal codes included:
//   int8  u = code ^ 0x80: 0x6400 | u is 1024 + u, and 1152 is subtracted;
//   e4m3  (bias 7, 3 fraction bits):  sign << 8, rest << 7 gives value * 2^-8  (fp16's bias is 15);
//   e2m1  (bias 1, 1 fraction bit):   sign << 12, rest << 9 gives value * 2^-14.
// `x` holds one code in the low byte (e2m1: low nibble) of each half.
__device__ __forceinline__ uint32_t half2_int8(uint32_t x) {        // x: bytes already ^ 0x80
    const uint32_t h = x | 0x64006400u;
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&h), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t half2_e4m3(uint32_t x) { return (x & 0x00800080u) << 8 | (x & 0x007f007fu) << 7; }
__device__ __forceinline__ uint32_t half2_e2m1(uint32_t x) { return (x & 0x00080008u) << 12 | (x & 0x00070007u) << 9; }

__device__ __forceinline__ float e4m3_value(uint32_t byte) {
    const uint32_t h = half2_e4m3(byte);
    return __half2float(__ushort_as_half((unsigned short)h)) * 256.f;
}

__device__ __forceinline__ float2 float2_of(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2 *>(&h)); }

// Eight codes to float32, without the row's scale: int8 and e4m3 from 8 bytes; e2m1 from the low word,
// times its block scale.
template <int FMT>
__device__ __forceinline__ void values(uint2 c, float block, float (&v)[8]) {
    if constexpr (FMT == QC_E2M1) {
        const float up = block * 16384.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t b = c.x >> (8 * i);
            const float2 f = float2_of(half2_e2m1((b & 0xfu) | (b & 0xf0u) << 12));
            v[2 * i] = f.x * up;
            v[2 * i + 1] = f.y * up;
        }
    } else {
        const uint32_t flip = FMT == QC_INT8 ? 0x80808080u : 0u;
        const uint32_t w[2] = {c.x ^ flip, c.y ^ flip};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = __byte_perm(w[i >> 1], 0, i & 1 ? 0x4342 : 0x4140);
            const float2 f = float2_of(FMT == QC_INT8 ? half2_int8(x) : half2_e4m3(x));
            const float up = FMT == QC_INT8 ? 1.f : 256.f;
            v[2 * i] = f.x * up;
            v[2 * i + 1] = f.y * up;
        }
    }
}

// Where 16-byte piece p of a run of codes lies.
__device__ __forceinline__ int piece_at(int p) { return p ^ ((p >> 3) & 7); }

// Largest code value that a row's largest magnitude maps to, block scale included.
template <int FMT>
constexpr float kTop = FMT == QC_INT8 ? 127.f : FMT == QC_E4M3 ? 448.f : 2688.f;
constexpr float kLeast = 7.8886090522101181e-31f;   // 2^-100: rows below hold zeros

}  // namespace qc
