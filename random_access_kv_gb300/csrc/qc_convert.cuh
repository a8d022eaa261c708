// Codes to tensor-core operands, and the small arithmetic that both attention kernels use.
#pragma once

#include "qc_attend.cuh"

namespace qc {

// One lane of a converged warp. Unlike a test of the lane's number it tells the compiler that what follows is
// one thread's, so that the tensor cores' operands go to uniform registers without a loop over lanes.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// x, or NaN for an infinity: of a query, whose product with a code may be a plain infinity or none, so that every
// score of its row is a NaN.
__device__ __forceinline__ float finite_or_nan(float x) { return fmaf(x, 0.f, x); }

__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __half2 r = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    const __half2 r = __hmax2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Two e4m3 codes (low half of x) as fp16.
__device__ __forceinline__ uint32_t cvt_e4m3(uint32_t x) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(x));
    return r;
}
// Eight e2m1 codes as fp16, neighbours together.
__device__ __forceinline__ void cvt_e2m1(uint32_t x, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\tcvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(x));
}
// A block scale (e4m3 byte, in the low byte) in both halves.
__device__ __forceinline__ uint32_t both_e4m3(uint32_t byte) { return cvt_e4m3(byte | byte << 8); }

__device__ __forceinline__ uint32_t sub1152(uint32_t x) {
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&x), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// The least power of two that is not below x > 0 (0 for 0).
__device__ __forceinline__ float power_above(float x) {
    const uint32_t b = __float_as_uint(x);
    return b == 0 ? 0.f : __uint_as_float(min((b + 0x007fffffu) & 0xff800000u, 0x7f000000u));
}

// Which of the 32 places from node j0 on (negative: the prefix) node `node` sees, a bit each.
__device__ __forceinline__ uint32_t window(const Attend &p, const uint32_t *tree, int node, int nodes, int j0) {
    if (j0 <= -32) return 0xffffffffu;
    const int k = j0 >> 5;          // -1: the prefix
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int at = k + i, last = node - 32 * at;
        if (tree)
            w[i] = at < 0 ? 0xffffffffu : at < p.words ? __ldg(tree + at) : 0u;
        else
            w[i] = last >= 31 ? 0xffffffffu : last < 0 ? 0u : (2u << last) - 1u;
    }
    const uint32_t bits = __funnelshift_r(w[0], w[1], j0 & 31);
    const int there = nodes - j0;
    return there >= 32 ? bits : there <= 0 ? 0u : bits & ((1u << there) - 1u);
}

}  // namespace qc
