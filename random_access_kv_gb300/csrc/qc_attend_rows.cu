// Attention over the quantised cache for few query rows per key/value head (single tokens, chains,
// small trees).
//
// What bounds it: the pages, read once. A producer warp copies tiles of 64 places from the pages, as
// they lie, to a ring of shared-memory stages with bulk asynchronous copies (one per page part, so the
// copies of several tiles are under way at any time); the consumer warps turn codes into tensor-core
// fragments in registers.
//
// Products. Codes are exact in fp16, and so are e2m1 codes times their e4m3 block scale (5 bits), so
// the products q . code are exact and summed in float32; the row's scale multiplies the score
// afterwards. A bf16 query row is brought into fp16's range by a power of two (8 bits fit 11). For the
// values, the weight p_t times the row's scale is the operand: w_t = p_t * (s_t / ref) * 2^14, ref a
// power of two, the running bound of the scales seen. p_t <= 1, so w_t <= 2^14 keeps fp16's 11 bits over
// 28 binades; `slice` says what becomes of lighter weights.
//
// Order of elements. A sum over d may take them in any order as long as both operands do: lane c of a
// quad takes elements c d / 4 .. of a key, so one 16-byte load feeds four (e2m1: eight) steps. For the
// values lane group g takes elements g d / 8 .., one per 8-wide tile of the output, and pairs of places
// are put together by byte permutes; there is no transposed copy of the values. The pages' swizzle
// keeps these loads free of bank conflicts, with places assigned to columns as `place` says.
#include <math.h>

#include "qc_attend.cuh"

namespace qc {
namespace {

using namespace fq::sm100;

constexpr int kTile = 64;               // places per stage
constexpr int kSlices = 4;              // warps that share a stage, 16 places each
constexpr int kRows = 16;               // query rows of a warp
constexpr float kWeight = 16384.f;      // 2^14
constexpr float kLeastNormal = 6.103515625e-05f;    // 2^-14, fp16's
constexpr float kLift = 16777216.f;     // 2^24
constexpr float kThin = 16.f;           // a quarter of a row's sum of weights, the heaviest being 1

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
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

template <int FMT, int D>
struct Shape {
    static constexpr int kRow = FMT == QC_E2M1 ? D / 2 : D;             // bytes of a row's codes
    static constexpr int kBlocks = FMT == QC_E2M1 ? D / 16 : 0;
    static constexpr int kStage = 2 * kTile * (kRow + 4 + kBlocks);     // bytes of a tile
    // Place (0 .. 15 of a slice) of column n of 8-wide score tile u.
    static __device__ __forceinline__ int place(int u, int n) {
        if constexpr (kRow == 128) return 8 * u + n;
        if constexpr (kRow == 64) return 4 * (n >> 1) + 2 * u + (n & 1);
        return (n >> 1) + 4 * (2 * u + (n & 1));
    }
};

struct Plan {
    int row_tiles;      // tiles of `rows` rows per head
    int row_warps;      // warps' row tiles of 16 in a CTA (1 or 2)
    int stages;
    int ctas;
    int smem;
};

struct Shared {
    uint64_t full[16], empty[16];
    uint32_t bad[16];           // per stage: sixteenths of the tile whose page does not exist
    Walk start;
    uint32_t fail;
};

// One thread's share of a slice's offsets within a stage.
template <int FMT, int D>
struct Offsets {
    using S = Shape<FMT, D>;
    int k[2][S::kRow == 128 ? 2 : 1];   // keys' codes: of column g of tile u
    int v[4];                           // values' codes: of the lane's four places
    int ks[4], vs[4];                   // scales of the lane's four places
    int kb[2], vb[4];                   // block scales
    __device__ __forceinline__ void set(int slice, int page, int g, int c) {
        const int sub_tokens = page < kTile ? page : kTile;
        const int t0 = slice * 16, base = t0 / sub_tokens * (2 * sub_tokens * (S::kRow + 4 + S::kBlocks)), at = t0 % sub_tokens;
        const int vcodes = base + sub_tokens * S::kRow, scales = base + 2 * sub_tokens * S::kRow;
        const int blocks = scales + 8 * sub_tokens;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int t = at + S::place(u, g);
#pragma unroll
            for (int h = 0; h < (S::kRow == 128 ? 2 : 1); ++h) {
                const int byte = t * S::kRow + c * (S::kRow / 4) + 16 * h;
                k[u][h] = base + piece_at(byte >> 4) * 16 + (byte & 15);
            }
            kb[u] = blocks + t * S::kBlocks + c * (S::kBlocks / 4);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int tv = at + S::place(u, 2 * c + e), byte = tv * S::kRow + g * (S::kRow / 8);
                v[2 * u + e] = vcodes + piece_at(byte >> 4) * 16 + (byte & 15);
                ks[2 * u + e] = scales + tv * 4;
                vs[2 * u + e] = scales + (sub_tokens + tv) * 4;
                vb[2 * u + e] = blocks + (sub_tokens + tv) * S::kBlocks + g * S::kBlocks / 8;
            }
        }
    }
};

template <int N>
__device__ __forceinline__ void load_words(const unsigned char *p, uint32_t (&w)[N]) {
    if constexpr (N == 4) {
        const uint4 r = *reinterpret_cast<const uint4 *>(p);
        w[0] = r.x, w[1] = r.y, w[2] = r.z, w[3] = r.w;
    } else if constexpr (N == 2) {
        const uint2 r = *reinterpret_cast<const uint2 *>(p);
        w[0] = r.x, w[1] = r.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    }
}

// Scores of the slice: s[u][e] row g, s[u][2 + e] row g + 8, place(u, 2 c + e), before any scale.
template <int FMT, int D>
__device__ __forceinline__ void scores(const unsigned char *st, const Offsets<FMT, D> &o, const uint32_t (&qa)[D / 16][4],
                                       float (&s)[2][4]) {
    using S = Shape<FMT, D>;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[u][i] = 0.f;
        if constexpr (FMT == QC_E2M1) {
            uint32_t w[D / 32];
            load_words(st + o.k[u][0], w);
            uint32_t sb[D / 64];
#pragma unroll
            for (int i = 0; i < D / 64; ++i) sb[i] = both_e4m3(st[o.kb[u] + i]);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                uint32_t h[4];
                cvt_e2m1(w[i], h);
                mma(s[u], qa[2 * i], mul2(h[0], sb[i / 2]), mul2(h[1], sb[i / 2]));
                mma(s[u], qa[2 * i + 1], mul2(h[2], sb[i / 2]), mul2(h[3], sb[i / 2]));
            }
        } else {
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
                uint32_t w[4];
                load_words(st + o.k[u][h], w);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (FMT == QC_INT8) {
                        const uint32_t x = w[i] ^ 0x80808080u;
                        mma(s[u], qa[4 * h + i], half2_int8(__byte_perm(x, 0x64646464u, 0x4140)),
                            half2_int8(__byte_perm(x, 0x64646464u, 0x4342)));
                    } else {
                        mma(s[u], qa[4 * h + i], cvt_e4m3(w[i]), cvt_e4m3(w[i] >> 16));
                    }
                }
            }
        }
    }
}

// out[nt] += weights (a) times the slice's values. keep: which of the lane's four places exist (only
// asked when MASK; the others' bytes may be anything, NaN codes included, and count as zeros).
template <int FMT, int D, bool MASK>
__device__ __forceinline__ void add_values(const unsigned char *st, const Offsets<FMT, D> &o, const uint32_t (&a)[4], uint32_t keep,
                                           float (&out)[D / 8][4]) {
    using S = Shape<FMT, D>;
    constexpr int W = S::kRow / 32;                     // words of a place in a lane
    uint32_t w[4][W];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        load_words(st + o.v[i], w[i]);
        if (MASK && !((keep >> i) & 1u)) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[i][j] = 0;
        }
    }
    if constexpr (FMT == QC_E2M1) {
        uint32_t sb[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t x = st[o.vb[2 * i]], y = st[o.vb[2 * i + 1]];
            if (MASK && !((keep >> (2 * i)) & 1u)) x = 0;
            if (MASK && !((keep >> (2 * i + 1)) & 1u)) y = 0;
            sb[i] = cvt_e4m3(x | y << 8);
        }
#pragma unroll
        for (int j = 0; j < W; ++j) {
            uint32_t h[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) cvt_e2m1(w[i][j], h[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                mma(out[8 * j + 2 * e], a, mul2(__byte_perm(h[0][e], h[1][e], 0x5410), sb[0]),
                    mul2(__byte_perm(h[2][e], h[3][e], 0x5410), sb[1]));
                mma(out[8 * j + 2 * e + 1], a, mul2(__byte_perm(h[0][e], h[1][e], 0x7632), sb[0]),
                    mul2(__byte_perm(h[2][e], h[3][e], 0x7632), sb[1]));
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j) {
            if constexpr (FMT == QC_INT8) {
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i][j] ^= 0x80808080u;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t pick = e | (4 + e) << 8;             // byte e of both, in the even bytes
                    const uint32_t x = __byte_perm(w[0][j], w[1][j], pick), y = __byte_perm(w[2][j], w[3][j], pick);
                    mma(out[4 * j + e], a, half2_int8(x & 0x00ff00ffu), half2_int8(y & 0x00ff00ffu));
                }
            } else {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint32_t h[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) h[i] = cvt_e4m3(e ? w[i][j] >> 16 : w[i][j]);
                    mma(out[4 * j + 2 * e], a, __byte_perm(h[0], h[1], 0x5410), __byte_perm(h[2], h[3], 0x5410));
                    mma(out[4 * j + 2 * e + 1], a, __byte_perm(h[0], h[1], 0x7632), __byte_perm(h[2], h[3], 0x7632));
                }
            }
        }
    }
}

// The softmax state of a warp's 16 rows: a thread holds rows g and g + 8.
template <int D>
struct State {
    float m[2], l[2];       // maximum (base-2 units), this thread's share of the sum
    float ref;              // power of two, bound of the values' scales; 0: none yet
    float o[D / 8][4];
    __device__ __forceinline__ void clear() {
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
        ref = 0.f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    }
};

__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}

// The least power of two that is not below x > 0 (0 for 0).
__device__ __forceinline__ float power_above(float x) {
    const uint32_t b = __float_as_uint(x);
    return b == 0 ? 0.f : __uint_as_float(min((b + 0x007fffffu) & 0xff800000u, 0x7f000000u));
}

// seen: what the lane's eight scores see, bit 4 r + 2 u + e for row g + 8 r, place(u, 2 c + e); bit 8 + 2 u + e:
// the place exists.
template <int FMT, int D, bool MASK>
__device__ __forceinline__ void slice(const unsigned char *st, const Offsets<FMT, D> &of, const uint32_t (&qa)[D / 16][4],
                                      const float (&up)[2], uint32_t seen, State<D> &z) {
    float s[2][4];
    scores<FMT, D>(st, of, qa, s);
    float top[2] = {-INFINITY, -INFINITY}, vs[4], vtop = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float ks = *reinterpret_cast<const float *>(st + of.ks[i]);
        vs[i] = *reinterpret_cast<const float *>(st + of.vs[i]);
        if (MASK && !((seen >> (8 + i)) & 1u)) vs[i] = 0.f;
        vtop = fmaxf(vtop, vs[i]);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float &x = s[i >> 1][2 * r + (i & 1)];
            x *= ks * up[r];
            if (MASK && !((seen >> (4 * r + i)) & 1u)) x = -INFINITY;
            top[r] = fmaxf(top[r], x);
        }
    }
    vtop = quad_max(vtop);
    top[0] = quad_max(top[0]);
    top[1] = quad_max(top[1]);
    if (__any_sync(0xffffffffu, top[0] > z.m[0] || top[1] > z.m[1] || vtop > z.ref)) {
        const float ref = fmaxf(z.ref, power_above(vtop));
        const float shrink = ref > 0.f ? z.ref / ref : 0.f;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float m = fmaxf(z.m[r], top[r]);
            const float old = m == -INFINITY ? 1.f : ex2(z.m[r] - m);
            z.m[r] = m;
            z.l[r] *= old;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                z.o[i][2 * r] *= old * shrink;
                z.o[i][2 * r + 1] *= old * shrink;
            }
        }
        z.ref = ref;
    }
    const float unit = z.ref > 0.f ? kWeight / z.ref : 0.f;
    float wt[2][2][2];
    bool light = false;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const float m = z.m[r] == -INFINITY ? 0.f : z.m[r];
        const bool thin = z.l[r] < kThin;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float q = ex2(s[u][2 * r + e] - m);
                z.l[r] += q;
                wt[r][u][e] = q * (vs[2 * u + e] * unit);
                light |= thin && wt[r][u][e] < kLeastNormal && wt[r][u][e] > 0.f;
            }
        }
    }
    // Weights below fp16's normals lose bits. That shows only where every heavier place holds an exact
    // zero, so only in rows whose weight lies on few places ("thin"); their light weights are added in a
    // pass of their own, scaled up, with the sums scaled along (powers of two: exact).
    light = __any_sync(0xffffffffu, light);
    uint32_t a[4];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int u = 0; u < 2; ++u) a[2 * u + r] = pack2(wt[r][u][0], wt[r][u][1]);
    if (light) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int u = 0; u < 2; ++u)
                a[2 * u + r] = pack2(wt[r][u][0] < kLeastNormal ? 0.f : wt[r][u][0], wt[r][u][1] < kLeastNormal ? 0.f : wt[r][u][1]);
    }
#pragma unroll 1
    for (int pass = 0;; ++pass) {
        add_values<FMT, D, MASK>(st, of, a, seen >> 8, z.o);
        if (!light) break;
        const float by = pass ? 1.f / kLift : kLift;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) z.o[i][0] *= by, z.o[i][1] *= by, z.o[i][2] *= by, z.o[i][3] *= by;
        if (pass) break;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int u = 0; u < 2; ++u)
                a[2 * u + r] = pack2(wt[r][u][0] < kLeastNormal ? wt[r][u][0] * kLift : 0.f,
                                     wt[r][u][1] < kLeastNormal ? wt[r][u][1] * kLift : 0.f);
    }
}

// Copies tile `tile` of a job's pages to a stage (one warp). entry: lane i's page of the tile's i-th part.
template <int FMT, int D>
__device__ __forceinline__ void fetch(const Attend &p, const Walk &w, int kv, int entry, unsigned char *stage, uint64_t *full,
                                      uint32_t *bad, int lane) {
    using S = Shape<FMT, D>;
    const int sub = p.g.page < kTile ? p.g.page : kTile, parts = kTile / sub;
    const int end = w.n.x + w.n.y;
    const bool mine = lane < parts && w.tile * kTile + lane * sub < end;
    const bool good = mine && entry >= 0 && entry < p.n_pages;
    const uint32_t have = __ballot_sync(0xffffffffu, good), missing = __ballot_sync(0xffffffffu, mine && !good);
    constexpr int kPer = 2 * (S::kRow + 4 + S::kBlocks);        // bytes of a place
    if (lane == 0) {
        if (missing) atomicOr(p.flags, QC_FLAG_RANGE);
        uint32_t m = 0;
        for (int i = 0; i < parts; ++i)
            if ((missing >> i) & 1u) m |= ((1u << (sub / 16)) - 1u) << (i * sub / 16);
        *bad = m;
        mbar_arrive_expect_tx(full, __popc(have) * sub * kPer);
    }
    __syncwarp();
    const unsigned char *head = p.pages + ((int64_t)entry * p.g.heads + kv) * (int64_t)p.g.part;
    if (p.g.page <= kTile) {
        if (good) bulk_g2s(stage + lane * sub * kPer, head, sub * kPer, full);
    } else if (have) {
        // part of a longer page: its six runs, one lane each
        const int64_t h0 = __shfl_sync(0xffffffffu, (long long)(head - p.pages), 0);
        const int t0 = w.tile * kTile & (p.g.page - 1), which = lane & 1, kind = lane >> 1;
        const unsigned char *src = p.pages + h0;
        int dst = 0, bytes = 0;
        if (kind == 0) {
            src += p.g.codes(which) + t0 * S::kRow;
            dst = which * kTile * S::kRow;
            bytes = kTile * S::kRow;
        } else if (kind == 1) {
            src += p.g.scales(which) + t0 * 4;
            dst = 2 * kTile * S::kRow + which * kTile * 4;
            bytes = kTile * 4;
        } else if (kind == 2 && S::kBlocks) {
            src += p.g.block_scales(which) + t0 * S::kBlocks;
            dst = 2 * kTile * (S::kRow + 4) + which * kTile * S::kBlocks;
            bytes = kTile * S::kBlocks;
        }
        if (bytes) bulk_g2s(stage + dst, src, bytes, full);
    }
}

template <typename T>
__device__ __forceinline__ float2 two(const T *p);
template <>
__device__ __forceinline__ float2 two<__half>(const __half *p) {
    return __half22float2(*reinterpret_cast<const __half2 *>(p));
}
template <>
__device__ __forceinline__ float2 two<__nv_bfloat16>(const __nv_bfloat16 *p) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(p));
}

// The query rows g and g + 8 of a warp as fragments; up[r]: what a row's scores are multiplied by beside
// the keys' scales.
template <typename T, int FMT, int D>
__device__ __forceinline__ void load_queries(const Attend &p, const Walk &w, int kv, int r0, int R, int g, int c,
                                             uint32_t (&qa)[D / 16][4], float (&up)[2]) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = r0 + g + 8 * r;
        const bool there = row < R;
        const int node = there ? row / p.group : 0, h = there ? row % p.group : 0;
        const T *q = static_cast<const T *>(p.q) + w.b * p.q_seq + node * p.q_node + (kv * p.group + h) * p.q_head + c * (D / 4);
        float2 v[D / 8];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) v[i] = there ? two(q + 2 * i) : make_float2(0.f, 0.f);
        float down = 1.f;
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) top = fmaxf(top, fmaxf(fabsf(v[i].x), fabsf(v[i].y)));
            top = quad_max(top);
            // largest magnitude to [2^13, 2^14)
            const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -100), 127);
            const float f = __uint_as_float((uint32_t)(13 - e + 127) << 23);
            down = __uint_as_float((uint32_t)(e - 13 + 127) << 23);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) v[i].x *= f, v[i].y *= f;
        }
        up[r] = p.scale * kLog2e * down;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const __half2 x = __floats2half2_rn(v[2 * i + e].x, v[2 * i + e].y);
                qa[i][2 * e + r] = *reinterpret_cast<const uint32_t *>(&x);
            }
        }
    }
}

// What the lane's eight scores of a slice that begins at place t0 see.
template <int FMT, int D>
__device__ __forceinline__ uint32_t seen_bits(const Attend &p, const Walk &w, int t0, uint32_t bad, int r0, int R, int g, int c) {
    if (bad) return 0;
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (t0 + Shape<FMT, D>::place(i >> 1, 2 * c + (i & 1)) < w.n.x + w.n.y) bits |= 256u << i;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = r0 + g + 8 * r, node = row / p.group;
        if (row >= R || node >= w.n.y) continue;
        const uint32_t *tree = p.tree ? p.tree + ((int64_t)w.b * p.n_nodes + node) * p.words : nullptr;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = t0 + Shape<FMT, D>::place(i >> 1, 2 * c + (i & 1)) - w.n.x;
            bool sees = j < 0;
            if (j >= 0 && j < w.n.y) sees = tree ? (__ldg(tree + (j >> 5)) >> (j & 31)) & 1u : j <= node;
            if (sees) bits |= 1u << (4 * r + i);
        }
    }
    return bits;
}

template <typename T, int FMT, int D, int RW>
__global__ void __launch_bounds__(32 * (kSlices * RW + 1), RW == 1 ? 2 : 1)
    attend_rows(const Attend p, const Parts parts, const Plan plan) {
    using S = Shape<FMT, D>;
    constexpr int kWarps = kSlices * RW;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Shared sh;
    __shared__ float2 stat[kWarps][kRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int R = p.n_nodes * p.group, jobs = p.g.heads * plan.row_tiles;
    unsigned char *ring = smem;
    float *sum = reinterpret_cast<float *>(smem + plan.stages * S::kStage);     // [RW][D / 2][32]: joined values

    griddep_wait();
    if (warp == kWarps) {
        const int64_t total = all_tiles(p, kTile, lane) * jobs, per = run_length(total, gridDim.x);
        const int64_t at = per * blockIdx.x, left = at < total ? (total - at < per ? total - at : per) : 0;
        const Walk w = find(p, at, left, jobs, kTile, lane);
        if (blockIdx.x == 0) write_before(p, parts.before, jobs, kTile, lane);
        if (lane == 0) {
            sh.start = w;
            sh.fail = 0;
            for (int i = 0; i < plan.stages; ++i) {
                mbar_init(&sh.full[i], 1);
                mbar_init(&sh.empty[i], kWarps);
            }
            fence_barrier_init();
        }
    }
    __syncthreads();
    Walk w = sh.start;
    int stage = 0;
    uint32_t phase = 0;

    if (warp == kWarps) {
        // ---- producer
        const int sub_shift = p.g.shift < 6 ? p.g.shift : 6, parts_of = kTile >> sub_shift;
        int used = 0;
        bool ok = true;
        while (w.left > 0 && ok) {
            const int kv = w.job / plan.row_tiles;
            const int32_t *row = p.table + w.b * p.table_stride;
            const int end = w.n.x + w.n.y;
            auto entry_of = [&](int tile) {
                const int t = tile * kTile + (lane << sub_shift);
                return lane < parts_of && tile < w.tiles && t < end ? __ldg(row + (t >> p.g.shift)) : -1;
            };
            int entry = entry_of(w.tile);
            for (; w.tile < w.tiles && w.left > 0; ++w.tile, --w.left) {
                const int next = entry_of(w.tile + 1);
                if (used >= plan.stages) {
                    // the ring's earlier content must have been read
                    ok = mbar_wait(&sh.empty[stage], phase ^ 1u);
                    ok = __all_sync(0xffffffffu, ok) && *(volatile uint32_t *)&sh.fail == 0;
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                }
                fetch<FMT, D>(p, w, kv, entry, ring + stage * S::kStage, &sh.full[stage], &sh.bad[stage], lane);
                entry = next;
                ++used;
                if (++stage == plan.stages) stage = 0, phase ^= 1u;
            }
            if (ok) next_job(p, w, jobs, kTile);
        }
        if (!ok) {
            // let the copies under way land before the CTA's shared memory goes
            if (lane == 0) atomicOr(p.flags, QC_FLAG_TIMEOUT), atomicExch(&sh.fail, 1u);
            for (int i = 0; i < plan.stages && i < used; ++i) {
                if (stage == 0) phase ^= 1u;
                stage = (stage ? stage : plan.stages) - 1;
                mbar_wait(&sh.full[stage], phase);
            }
        }
        griddep_launch_dependents();
        return;
    }

    // ---- consumers
    const int g = lane >> 2, c = lane & 3, slice_of = warp & (kSlices - 1), rw = warp / kSlices;
    Offsets<FMT, D> of;
    of.set(slice_of, p.g.page, g, c);
    bool ok = true;
    int segment = 0;
    while (w.left > 0) {
        const int kv = w.job / plan.row_tiles, r0 = (w.job % plan.row_tiles * RW + rw) * kRows;
        const bool whole_before = w.tile == 0;
        uint32_t qa[D / 16][4];
        float up[2];
        load_queries<T, FMT, D>(p, w, kv, r0, R, g, c, qa, up);
        State<D> z;
        z.clear();
        for (; w.tile < w.tiles && w.left > 0; ++w.tile, --w.left) {
            if (ok && !mbar_wait(&sh.full[stage], phase)) ok = false;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const unsigned char *st = ring + stage * S::kStage;
            const uint32_t bad = sh.bad[stage];
            const int t0 = w.tile * kTile + slice_of * 16;
            if (t0 + 16 <= w.n.x && !bad) {
                slice<FMT, D, false>(st, of, qa, up, 0xfffu, z);
            } else if (t0 < w.n.x + w.n.y) {
                const uint32_t seen = seen_bits<FMT, D>(p, w, t0, (bad >> slice_of) & 1u, r0, R, g, c);
                slice<FMT, D, true>(st, of, qa, up, seen, z);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.empty[stage]);
            if (++stage == plan.stages) stage = 0, phase ^= 1u;
        }
        if (!ok) {
            if (lane == 0) atomicOr(p.flags, QC_FLAG_TIMEOUT), atomicExch(&sh.fail, 1u);
        }
        // join the slices' warps: sums of l over the quad, then maxima and values over the warps in order
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            z.l[r] += __shfl_xor_sync(0xffffffffu, z.l[r], 1);
            z.l[r] += __shfl_xor_sync(0xffffffffu, z.l[r], 2);
            if (c == 0) stat[warp][g + 8 * r] = make_float2(z.m[r], z.l[r]);
        }
        ok = named_sync_and(1, 32 * kWarps, ok);        // one that gave up takes the others with it
        float m[2], l[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
#pragma unroll
            for (int i = 0; i < kSlices; ++i) m[r] = fmaxf(m[r], stat[rw * kSlices + i][g + 8 * r].x);
#pragma unroll
            for (int i = 0; i < kSlices; ++i) {
                const float2 x = stat[rw * kSlices + i][g + 8 * r];
                if (x.x != -INFINITY) l[r] += x.y * ex2(x.x - m[r]);
            }
            const float f = z.m[r] == -INFINITY ? 0.f : ex2(z.m[r] - m[r]) * (z.ref * (1.f / kWeight));
#pragma unroll
            for (int i = 0; i < D / 8; ++i) z.o[i][2 * r] *= f, z.o[i][2 * r + 1] *= f;
        }
        float4 *mine = reinterpret_cast<float4 *>(sum + rw * (D / 2) * 32);
        for (int turn = 0; turn < kSlices - 1; ++turn) {
            if (slice_of == turn) {
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    float4 x = make_float4(z.o[i][0], z.o[i][1], z.o[i][2], z.o[i][3]);
                    if (turn) {
                        const float4 y = mine[i * 32 + lane];
                        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
                    }
                    mine[i * 32 + lane] = x;
                }
            }
            named_sync(1, 32 * kWarps);
        }
        if (slice_of == kSlices - 1) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const float4 y = mine[i * 32 + lane];
                z.o[i][0] += y.x, z.o[i][1] += y.y, z.o[i][2] += y.z, z.o[i][3] += y.w;
            }
            const bool whole = whole_before && w.tile == w.tiles;
            // part 2 c: the job that the CTA's run begins with; 2 c + 1: the one it ends with
            const int64_t part = 2 * (int64_t)blockIdx.x + (segment ? 1 : 0);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = r0 + g + 8 * r;
                if (row >= R) continue;
                float v[D / 4];
#pragma unroll
                for (int i = 0; i < D / 8; ++i) v[i] = z.o[i][2 * r], v[D / 8 + i] = z.o[i][2 * r + 1];
                if (whole) {
                    const int node = row / p.group, h = kv * p.group + row % p.group;
                    const bool there = node < w.n.y && l[r] > 0.f;
                    const float inv = there ? 1.f / l[r] : 0.f;
#pragma unroll
                    for (int i = 0; i < D / 4; ++i) v[i] = there ? v[i] * inv : 0.f;
                    const int64_t at = ((int64_t)w.b * p.n_nodes + node) * p.n_q_heads + h;
                    store_row<T, D / 4>(static_cast<T *>(p.out) + at * D + c * (D / 4), v);
                    if (p.lse && c == 0) p.lse[at] = there ? (m[r] + log2f(l[r])) * kLn2 : -INFINITY;
                } else {
                    float4 *to = reinterpret_cast<float4 *>(parts.row(part, rw * kRows + g + 8 * r) + c * (D / 4));
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) to[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    if (c == 0) *parts.stat(part, rw * kRows + g + 8 * r) = make_float2(m[r], l[r]);
                }
            }
        }
        ++segment;
        if (!ok) break;
        next_job(p, w, jobs, kTile);
        named_sync(1, 32 * kWarps);         // stat and sum are free again
    }
}

template <int FMT, int D>
Plan plan_rows(const qc_ctx *c, int rows, int64_t n_seq, int64_t max_len, int n_nodes) {
    using S = Shape<FMT, D>;
    Plan p;
    // Up to 16 rows: one tile of rows, two CTAs on an SM. More: two row tiles share each stage.
    p.row_warps = rows <= kRows ? 1 : 2;
    p.row_tiles = (rows + kRows * p.row_warps - 1) / (kRows * p.row_warps);
    const int per_sm = p.row_warps == 1 ? 2 : 1, room = 216 * 1024 / per_sm - 1024, joined = p.row_warps * kRows * D * 4;
    p.stages = (room - joined) / S::kStage;
    if (p.stages > 12) p.stages = 12;
    p.smem = p.stages * S::kStage + joined;
    p.ctas = per_sm * c->num_sms;
    const int64_t most = n_seq * c->heads * p.row_tiles * ((max_len + n_nodes + kTile - 1) / kTile);
    if (p.ctas > most) p.ctas = (int)most;
    return p;
}

template <int FMT, int D>
int64_t workspace(const qc_ctx *c, int rows, int64_t n_seq, int64_t max_len, int n_nodes) {
    const Plan p = plan_rows<FMT, D>(c, rows, n_seq, max_len, n_nodes);
    return workspace_bytes(n_seq, 2 * (int64_t)p.ctas, p.row_warps * kRows, D);
}

template <typename T, int FMT, int D, int RW>
cudaError_t run(const Plan &plan, const Attend &p, int type, cudaStream_t s) {
    const Parts parts = parts_at(p.workspace, p.n_seq, 2 * (int64_t)plan.ctas, RW * kRows, D);
    static_assert(sizeof(Shared) < 1024, "static shared memory");
    cudaError_t e = cudaFuncSetAttribute(attend_rows<T, FMT, D, RW>, cudaFuncAttributeMaxDynamicSharedMemorySize, plan.smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)plan.ctas);
    cfg.blockDim = dim3(32 * (kSlices * RW + 1));
    cfg.dynamicSmemBytes = plan.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, attend_rows<T, FMT, D, RW>, p, parts, plan);
    if (e != cudaSuccess) return e;
    return launch_join(p, parts, type, plan.row_tiles, kTile, plan.ctas, s);
}

template <int FMT, int D>
cudaError_t pick(const qc_ctx *c, int type, const Attend &p, cudaStream_t s) {
    const Plan plan = plan_rows<FMT, D>(c, p.n_nodes * p.group, p.n_seq, p.max_len, p.n_nodes);
    if (type == QC_F16)
        return plan.row_warps == 1 ? run<__half, FMT, D, 1>(plan, p, type, s) : run<__half, FMT, D, 2>(plan, p, type, s);
    return plan.row_warps == 1 ? run<__nv_bfloat16, FMT, D, 1>(plan, p, type, s) : run<__nv_bfloat16, FMT, D, 2>(plan, p, type, s);
}

}  // namespace

cudaError_t launch_attend_rows(const qc_ctx *c, int type, const Attend &p, cudaStream_t s) {
    if (c->d == 64)
        return c->fmt == QC_INT8   ? pick<QC_INT8, 64>(c, type, p, s)
               : c->fmt == QC_E4M3 ? pick<QC_E4M3, 64>(c, type, p, s)
                                   : pick<QC_E2M1, 64>(c, type, p, s);
    return c->fmt == QC_INT8   ? pick<QC_INT8, 128>(c, type, p, s)
           : c->fmt == QC_E4M3 ? pick<QC_E4M3, 128>(c, type, p, s)
                               : pick<QC_E2M1, 128>(c, type, p, s);
}

int64_t rows_workspace(const qc_ctx *c, int64_t n_seq, int n_nodes, int n_q_heads, int64_t max_len) {
    const int rows = n_nodes * (n_q_heads / c->heads);
    if (n_seq == 0) return 0;
    if (c->d == 64)
        return c->fmt == QC_INT8   ? workspace<QC_INT8, 64>(c, rows, n_seq, max_len, n_nodes)
               : c->fmt == QC_E4M3 ? workspace<QC_E4M3, 64>(c, rows, n_seq, max_len, n_nodes)
                                   : workspace<QC_E2M1, 64>(c, rows, n_seq, max_len, n_nodes);
    return c->fmt == QC_INT8   ? workspace<QC_INT8, 128>(c, rows, n_seq, max_len, n_nodes)
           : c->fmt == QC_E4M3 ? workspace<QC_E4M3, 128>(c, rows, n_seq, max_len, n_nodes)
                               : workspace<QC_E2M1, 128>(c, rows, n_seq, max_len, n_nodes);
}

}  // namespace qc
