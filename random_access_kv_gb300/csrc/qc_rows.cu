// Rows in and out of the quantised cache.
//
// Bound by memory: a write reads each row once and writes 1/2 to 1/8 of it, a read the reverse. A row is held
// by d / 16 lanes, 16 elements each: a 16-byte piece of codes, or a block of e2m1 (of eight elements a lane, as it
// was: a write of 32,768 tokens 57 us against 38, a random read of 104,864 141 against 103; two divisions fewer, two
// steps fewer of the search for the largest magnitude, and twice the bytes under way). For a write the largest
// magnitude is a butterfly over those lanes. A warp takes U rows per lane group, of consecutive tokens and one head
// (which lie one after another in a page), all their loads under way together; neighbouring blocks take
// neighbouring heads. 32,768 tokens of 8 heads of 128 (bf16, e2m1): written in 38 us (4.5 TB/s; bound by issue
// slots, 83 %: the largest magnitude, exact products and conversions), read in 33 us (5.2 TB/s); a random read of
// 104,864 tokens (int8 to fp16) in 103 us (6.3 TB/s).
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

// 16 elements go out. wide: the address is a multiple of 32, and 32 bytes go in one store (a random read of 104,864
// tokens: 103 us, against 110 with two of 16 bytes).
template <typename T>
__device__ __forceinline__ void store16(T *p, const float (&v)[2][8], bool wide) {
    constexpr int kWords = 4 * (int)sizeof(T);
    alignas(16) uint32_t w[kWords];
    Eight<T>::store(reinterpret_cast<T *>(w), v[0]);
    Eight<T>::store(reinterpret_cast<T *>(w) + 8, v[1]);
    uint32_t *to = reinterpret_cast<uint32_t *>(p);
#pragma unroll
    for (int i = 0; i < kWords; i += 8) {
        if (wide) {
            asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]),
                         "r"(w[i + 4]), "r"(w[i + 5]), "r"(w[i + 6]), "r"(w[i + 7]), "l"(to + i)
                         : "memory");
        } else {
            reinterpret_cast<uint4 *>(to + i)[0] = reinterpret_cast<const uint4 *>(w + i)[0];
            reinterpret_cast<uint4 *>(to + i)[1] = reinterpret_cast<const uint4 *>(w + i)[1];
        }
    }
}

// What a block works on: blockIdx.x = (token group, head), blockIdx.y = keys or values.
template <int D, int U>
struct Task {
    static constexpr int kLanes = D / 16, kRows = 32 / kLanes;
    int lane, e0, h;
    int64_t token;          // of u = 0; the next ones kRows apart
    __device__ __forceinline__ Task(const Rows &p) {
        lane = threadIdx.x & 31;
        e0 = lane % kLanes * 16;
        const uint32_t group = blockIdx.x / (uint32_t)p.g.heads;
        h = (int)(blockIdx.x - group * (uint32_t)p.g.heads);
        token = ((int64_t)group * (kThreads / 32) + (threadIdx.x >> 5)) * (U * kRows) + lane / kLanes;
    }
};

template <typename T, int D, int FMT, int U>
__global__ void __launch_bounds__(kThreads) write_rows(const Rows p) {
    const Task<D, U> k(p);
    constexpr int kLanes = D / 16, kRows = 32 / kLanes;
    const int which = blockIdx.y, e0 = k.e0;
    const T *x = static_cast<const T *>(which ? p.v : p.k) + k.h * (which ? p.v_head : p.k_head) + e0;
    const int64_t stride = which ? p.v_token : p.k_token;
    Eight<T> in[U][2];
    int64_t slots[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t token = k.token + u * kRows;
        slots[u] = -1;
        if (token < p.n) {
            slots[u] = __ldg(p.slots + token);
            in[u][0].load(x + token * stride);
            in[u][1].load(x + token * stride + 8);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const bool there = k.token + u * kRows < p.n;
        const int64_t slot = slots[u];
        float v[2][8];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (there) {
                in[u][half].get(v[half]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[half][i] = 0.f;
            }
        }
        // largest magnitude, NaN included: of magnitudes as integers, which order as the floats do
        uint32_t block = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) block = max(block, __float_as_uint(v[i >> 3][i & 7]) & 0x7fffffffu);
        uint32_t top = block;
#pragma unroll
        for (int m = kLanes / 2; m >= 1; m >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
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
        float by = zero ? 0.f : __fdiv_rn(kTop<FMT>, A);
        unsigned char *part = p.pages + ((slot >> p.g.shift) * p.g.heads + k.h) * (int64_t)p.g.part;
        const int t = (int)(slot & (p.g.page - 1));
        if constexpr (FMT == QC_E2M1) {
            uint32_t sb = 0;
            if (!zero) {
                sb = e4m3x2(__fmul_rn(__uint_as_float(block), __fdiv_rn(448.f, A)), 0.f) & 0xffu;
                by = sb ? __fdiv_rn(by, e4m3_value(sb)) : 0.f;
            }
            part[p.g.block_scales(which) + t * p.g.blocks + e0 / 16] = (unsigned char)sb;
        }
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[half][i] = zero ? 0.f : __fmul_rn(v[half][i], by);
        unsigned char *to = part + code_at<FMT>(p.g, which, t, e0);
        if constexpr (FMT == QC_E2M1) {
            *reinterpret_cast<uint2 *>(to) = make_uint2(codes_e2m1(v[0]), codes_e2m1(v[1]));
        } else {
            const uint2 a = FMT == QC_INT8 ? codes_int8(v[0]) : codes_e4m3(v[0]), b = FMT == QC_INT8 ? codes_int8(v[1]) : codes_e4m3(v[1]);
            *reinterpret_cast<uint4 *>(to) = make_uint4(a.x, a.y, b.x, b.y);
        }
        if (e0 == 0) reinterpret_cast<float *>(part + p.g.scales(which))[t] = scale;
    }
}

template <typename T, int D, int FMT, int U>
__global__ void __launch_bounds__(kThreads) read_rows(const Rows p) {
    const Task<D, U> k(p);
    constexpr int kRows = 32 / (D / 16);
    const int which = blockIdx.y, e0 = k.e0;
    T *out = static_cast<T *>(which ? p.v_out : p.k_out);
    if (!out) return;
    const bool wide = reinterpret_cast<uintptr_t>(out) % 32 == 0;       // a row is a multiple of 128 bytes
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
        float v[2][8];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if constexpr (FMT == QC_E2M1)
                values<FMT>(make_uint2(half ? c[u].y : c[u].x, 0), sb, v[half]);
            else
                values<FMT>(half ? make_uint2(c[u].z, c[u].w) : make_uint2(c[u].x, c[u].y), sb, v[half]);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[half][i] = held ? v[half][i] * scale[u] : 0.f;
        }
        store16(out + (token * p.g.heads + k.h) * D + e0, v, wide);
    }
}

template <typename T, int D, int FMT, int U, bool WRITE>
cudaError_t launch(const Rows &p, cudaStream_t s) {
    constexpr int kPerBlock = kThreads / 32 * (32 / (D / 16)) * U;
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
    // Few rows: one per lane group, as many warps as there are. Many: two, for two loads under way (a random read of
    // 104,864 tokens: 113 us with one, 103 with two, 110 with three; a write of 32,768 tokens 48, 38 and 38).
    const bool many = p.n * p.g.heads * (D / 16) > (int64_t)c->num_sms * 2048;
    if (write) return many ? launch<T, D, FMT, 2, true>(p, s) : launch<T, D, FMT, 1, true>(p, s);
    return many ? launch<T, D, FMT, 2, false>(p, s) : launch<T, D, FMT, 1, false>(p, s);
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
