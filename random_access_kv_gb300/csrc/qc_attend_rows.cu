// Attention over the quantised cache for few query rows per key/value head (single tokens, chains,
// small trees).
//
// Each of the eight warps on an SM (two CTAs of four, so that every scheduler has two) has a run of tiles of
// 32 places of its own. It copies them from the pages, as they lie, to its ring of shared-memory stages with
// bulk asynchronous copies, two or more tiles ahead, and turns codes into tensor-core fragments in registers.
// Warps never wait for one another; what one leaves unused of the memory's bandwidth, for instance at the
// start of a job, the other seven on its SM take.
//
// What bounds it: in the limit the pages, read once. As measured the schedulers issue every second cycle, two
// warps each, held up by the latency of dependent conversions and products: 4 rows over 32 sequences of up to
// 32,768 places (e2m1, 637 MB) take 226 us, 2.8 TB/s; 20 rows over 16 x 16,384 (int8, 555 MB) 195 us. Twelve
// warps of 168 registers instead of eight of 255 spill: 270 and 216 us when eight took 256 and 212.
//
// Products. Codes are exact in fp16, and so are e2m1 codes times their e4m3 block scale (5 bits), so
// the products q . code are exact and summed in float32; the row's scale multiplies the score
// afterwards. A bf16 query row is brought into fp16's range by a power of two (8 bits fit 11). For the
// values, the weight p_t times the row's scale is the operand: w_t = p_t * (s_t / ref) * 2^12, ref a
// power of two, the running bound of the scales seen. A row's reference m moves only when a score passes
// it by 3 (base 2), to 3 above that score: so p_t <= 2^3 and w_t <= 2^15, the sums are rescaled seldom
// (a first tile's reference serves until a score is 2^6 times heavier), and the maximum is only reduced
// over a row's lanes when it is. w_t keeps fp16's 11 bits down to 2^-14; `add_tile` says what becomes of
// lighter weights.
//
// Order of elements. A sum over d may take them in any order as long as both operands do: lane c of a
// quad takes elements c d / 4 .. of a key, so one 16-byte load feeds four (e2m1: eight) steps. For the
// values lane group g takes elements g d / 8 .., one per 8-wide tile of the output, and pairs of places
// are put together by byte permutes; there is no transposed copy of the values. The pages' swizzle
// keeps these loads free of bank conflicts, with places assigned to columns as `place` says.
#include <math.h>

#include "qc_attend.cuh"
#include "qc_convert.cuh"

namespace qc {
namespace {

using namespace fq::sm100;

constexpr int kTile = 32;               // places per stage
constexpr int kPerSm = 8, kWarps = 4;   // warps on an SM (255 registers and 27 KB each) and of a CTA
constexpr int kRoom = 27 * 1024;
constexpr float kWeight = 4096.f;       // 2^12
constexpr float kLag = 3.f;             // how far (base 2) a score may pass the row's reference
constexpr float kHead = 3.f;            // how far above the largest score a new reference is put
constexpr float kLeastNormal = 6.103515625e-05f;    // 2^-14, fp16's
constexpr float kLift = 16777216.f;     // 2^24
constexpr float kHeavy = 2.44140625e-04f;   // 2^-12
constexpr int kSettled = 12;            // heavy places that a row must have met

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int FMT, int D>
struct Shape {
    static constexpr int kRow = FMT == QC_E2M1 ? D / 2 : D;             // bytes of a row's codes
    static constexpr int kBlocks = FMT == QC_E2M1 ? D / 16 : 0;
    static constexpr int kStage = 2 * kTile * (kRow + 4 + kBlocks);     // bytes of a tile
    // A stage: keys' codes, values' codes, keys' scales, values' scales, keys' block scales, values'.
    static constexpr int kCodes = kTile * kRow, kScales = 2 * kCodes, kBlockScales = kScales + 8 * kTile;
    // Place (0 .. 15 of a half tile) of column n of 8-wide score tile u.
    static __device__ __forceinline__ int place(int u, int n) {
        if constexpr (kRow == 128) return 8 * u + n;
        if constexpr (kRow == 64) return 4 * (n >> 1) + 2 * u + (n & 1);
        return (n >> 1) + 4 * (2 * u + (n & 1));
    }
};

struct Plan {
    int device;
    int row_tiles;      // tiles of 16 MT rows per head
    int mt;             // 16-row tiles of a warp (1 or 2)
    int stages;
    int units;          // warps
    int smem;           // of a warp
};

// One lane's offsets within a stage. Rows of 128 and 64 bytes: the other offsets are these plus
// constants; rows of 32 bytes: the swizzle's phase differs between half tiles.
template <int FMT, int D>
struct Offsets {
    using S = Shape<FMT, D>;
    static constexpr int kK = S::kRow == 128 ? 1 : S::kRow == 64 ? 2 : 4, kV = 2 * kK;
    int k[kK], v[kV];
    static __device__ __forceinline__ int code(int t, int byte, bool short_pages) {
        byte += t * S::kRow;
        if (S::kRow == 32 && short_pages && t >= 16)        // a page of 16 begins its own run
            return 16 * S::kRow + piece_at((byte - 16 * S::kRow) >> 4) * 16 + (byte & 15);
        return piece_at(byte >> 4) * 16 + (byte & 15);
    }
    __device__ __forceinline__ void set(int g, int c, bool short_pages) {
#pragma unroll
        for (int i = 0; i < kK; ++i) k[i] = code(16 * (i >> 1) + S::place(i & 1, g), c * (S::kRow / 4), short_pages);
#pragma unroll
        for (int i = 0; i < kV; ++i)
            v[i] = S::kCodes + code(16 * (i >> 2) + S::place(S::kRow == 128 ? 0 : (i >> 1) & 1, 2 * c + (i & 1)), g * (S::kRow / 8), short_pages);
    }
    __device__ __forceinline__ int key(int x, int u, int h) const {
        if constexpr (S::kRow == 128) return (k[0] ^ (16 * h)) + 1024 * u + 2048 * x;
        if constexpr (S::kRow == 64) return k[u] + 1024 * x;
        return k[2 * x + u];
    }
    __device__ __forceinline__ int value(int x, int u, int e) const {
        if constexpr (S::kRow == 128) return v[e] + 1024 * u + 2048 * x;
        if constexpr (S::kRow == 64) return v[2 * u + e] + 1024 * x;
        return v[4 * x + 2 * u + e];
    }
};

template <int N>
__device__ __forceinline__ void load_words(const unsigned char *p, uint32_t *w) {
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

// The scales of the lane's eight places: [4 x + 2 u + e] is that of place(u, 2 c + e) of half tile x.
template <int ROW>
__device__ __forceinline__ void load_scales(const unsigned char *p, int c, float (&s)[8]) {
    const float *f = reinterpret_cast<const float *>(p);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        if constexpr (ROW == 128) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float2 r = *reinterpret_cast<const float2 *>(f + 16 * x + 8 * u + 2 * c);
                s[4 * x + 2 * u] = r.x;
                s[4 * x + 2 * u + 1] = r.y;
            }
        } else if constexpr (ROW == 64) {
            const float4 r = *reinterpret_cast<const float4 *>(f + 16 * x + 4 * c);
            s[4 * x] = r.x, s[4 * x + 1] = r.y, s[4 * x + 2] = r.z, s[4 * x + 3] = r.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) s[4 * x + i] = f[16 * x + c + 4 * i];
        }
    }
}

// Query fragments: in registers for one row tile; for two in shared memory, lane by lane.
template <int D, int MT>
struct Queries;
template <int D>
struct Queries<D, 1> {
    uint32_t a[D / 16][4];
    __device__ __forceinline__ void put(uint4 *, int, int, int i, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
        a[i][0] = w0, a[i][1] = w1, a[i][2] = w2, a[i][3] = w3;
    }
    __device__ __forceinline__ void get(const uint4 *, int, int, int i, uint32_t (&r)[4]) const {
        r[0] = a[i][0], r[1] = a[i][1], r[2] = a[i][2], r[3] = a[i][3];
    }
};
template <int D>
struct Queries<D, 2> {
    __device__ __forceinline__ void put(uint4 *sm, int lane, int mt, int i, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
        sm[(mt * (D / 16) + i) * 32 + lane] = make_uint4(w0, w1, w2, w3);
    }
    __device__ __forceinline__ void get(const uint4 *sm, int lane, int mt, int i, uint32_t (&r)[4]) const {
        const uint4 v = sm[(mt * (D / 16) + i) * 32 + lane];
        r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
    }
};

// Scores of a tile before any scale: s[mt][2 x + u][2 r + e] of row g + 8 r, place(u, 2 c + e) of half x.
template <int FMT, int D, int MT>
__device__ __forceinline__ void scores(const unsigned char *st, const Offsets<FMT, D> &o, const Queries<D, MT> &q, const uint4 *qs,
                                       int lane, float (&s)[MT][4][4]) {
    using S = Shape<FMT, D>;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n) s[m][n][0] = s[m][n][1] = s[m][n][2] = s[m][n][3] = 0.f;
    constexpr int kChunks = S::kRow == 128 ? 2 : 1, kWords = S::kRow / 16 / kChunks;     // a lane's words per place
    constexpr int kSteps = FMT == QC_E2M1 ? 2 : 1;                                       // 16-wide steps per word
#pragma unroll
    for (int h = 0; h < kChunks; ++h) {
        uint32_t w[4][kWords];
        uint32_t sb[4][2];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            load_words<kWords>(st + o.key(n >> 1, n & 1, h), w[n]);
            if constexpr (FMT == QC_E2M1) {
                const unsigned char *b = st + S::kBlockScales + (16 * (n >> 1) + S::place(n & 1, lane >> 2)) * S::kBlocks + (lane & 3) * (S::kBlocks / 4);
                if constexpr (D == 128) {
                    const uint32_t x = *reinterpret_cast<const uint16_t *>(b);
                    sb[n][0] = cvt_e4m3(__byte_perm(x, 0, 0x4400));
                    sb[n][1] = cvt_e4m3(__byte_perm(x, 0, 0x4411));
                } else {
                    sb[n][0] = both_e4m3(*b);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            uint32_t qa[MT][kSteps][4];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int k = 0; k < kSteps; ++k) q.get(qs, lane, m, (h * kWords + i) * kSteps + k, qa[m][k]);
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                uint32_t b[4];
                if constexpr (FMT == QC_E2M1) {
                    cvt_e2m1(w[n][i], b);
#pragma unroll
                    for (int j = 0; j < 4; ++j) b[j] = mul2(b[j], sb[n][i / 2]);
                } else if constexpr (FMT == QC_INT8) {
                    const uint32_t x = w[n][i] ^ 0x80808080u;
                    b[0] = sub1152(__byte_perm(x, 0x64646464u, 0x4140));
                    b[1] = sub1152(__byte_perm(x, 0x64646464u, 0x4342));
                } else {
                    b[0] = cvt_e4m3(w[n][i]);
                    b[1] = cvt_e4m3(w[n][i] >> 16);
                }
#pragma unroll
                for (int k = 0; k < kSteps; ++k)
#pragma unroll
                    for (int m = 0; m < MT; ++m) mma(s[m][n], qa[m][k], b[2 * k], b[2 * k + 1]);
            }
        }
    }
}

// out[mt][nt] += weights a[mt][x] times the values of half tile x. keep: which of the lane's eight places
// exist (only asked when MASK; the others' bytes may be anything, NaN codes included, and count as zeros).
template <int FMT, int D, int MT, bool MASK>
__device__ __forceinline__ void add_values(const unsigned char *st, const Offsets<FMT, D> &o, const uint32_t (&a)[MT][2][4], int lane,
                                           uint32_t keep, float (&out)[MT][D / 8][4]) {
    using S = Shape<FMT, D>;
    constexpr int W = S::kRow / 32;                     // words of a place in a lane
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        uint32_t w[4][W];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            load_words<W>(st + o.value(x, i >> 1, i & 1), w[i]);
            if (MASK && !((keep >> (4 * x + i)) & 1u)) {
#pragma unroll
                for (int j = 0; j < W; ++j) w[i][j] = 0;
            }
        }
        if constexpr (FMT == QC_E2M1) {
            uint32_t sb[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const unsigned char *b = st + S::kBlockScales + kTile * S::kBlocks + (lane >> 2) * S::kBlocks / 8;
                uint32_t y = b[(16 * x + S::place(i, 2 * (lane & 3))) * S::kBlocks], z = b[(16 * x + S::place(i, 2 * (lane & 3) + 1)) * S::kBlocks];
                if (MASK && !((keep >> (4 * x + 2 * i)) & 1u)) y = 0;
                if (MASK && !((keep >> (4 * x + 2 * i + 1)) & 1u)) z = 0;
                sb[i] = cvt_e4m3(y | z << 8);
            }
#pragma unroll
            for (int j = 0; j < W; ++j) {
                uint32_t h[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) cvt_e2m1(w[i][j], h[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t sel = e & 1 ? 0x7632 : 0x5410;
                    const uint32_t b0 = mul2(__byte_perm(h[0][e / 2], h[1][e / 2], sel), sb[0]);
                    const uint32_t b1 = mul2(__byte_perm(h[2][e / 2], h[3][e / 2], sel), sb[1]);
#pragma unroll
                    for (int m = 0; m < MT; ++m) mma(out[m][8 * j + e], a[m][x], b0, b1);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j) {
                if constexpr (FMT == QC_INT8) {
                    // bytes of two places side by side, then fp16 pairs of (place, next place)
                    const uint32_t y0 = __byte_perm(w[0][j], w[1][j], 0x5140) ^ 0x80808080u, y1 = __byte_perm(w[0][j], w[1][j], 0x7362) ^ 0x80808080u;
                    const uint32_t z0 = __byte_perm(w[2][j], w[3][j], 0x5140) ^ 0x80808080u, z1 = __byte_perm(w[2][j], w[3][j], 0x7362) ^ 0x80808080u;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t sel = e & 1 ? 0x4342 : 0x4140;
                        const uint32_t b0 = sub1152(__byte_perm(e < 2 ? y0 : y1, 0x64646464u, sel));
                        const uint32_t b1 = sub1152(__byte_perm(e < 2 ? z0 : z1, 0x64646464u, sel));
#pragma unroll
                        for (int m = 0; m < MT; ++m) mma(out[m][4 * j + e], a[m][x], b0, b1);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t h[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) h[i] = cvt_e4m3(e ? w[i][j] >> 16 : w[i][j]);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t sel = k ? 0x7632 : 0x5410;
                            const uint32_t b0 = __byte_perm(h[0], h[1], sel), b1 = __byte_perm(h[2], h[3], sel);
#pragma unroll
                            for (int m = 0; m < MT; ++m) mma(out[m][4 * j + 2 * e + k], a[m][x], b0, b1);
                        }
                    }
                }
            }
        }
    }
}

// The softmax state of a warp's rows: a thread holds rows g and g + 8 of each row tile.
template <int D, int MT>
struct State {
    float m[MT][2], l[MT][2];   // reference (base-2 units), this thread's share of the sum
    float ref;                  // power of two, bound of the values' scales; 0: none yet
    int heavy;                  // places of weight kHeavy or more that each row met, 8 bits per row, at most 127
    bool settled;               // kSettled or more for every row of the warp
    float o[MT][D / 8][4];
    __device__ __forceinline__ void clear() {
        ref = 0.f;
        heavy = 0;
        settled = false;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            m[t][0] = m[t][1] = -INFINITY;
            l[t][0] = l[t][1] = 0.f;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.f;
        }
    }
};

__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}

// What a lane's scores see: bit 8 r + 4 x + 2 u + e of row[mt] for row g + 8 r and place(u, 2 c + e) of half
// x; there: the places that exist.
template <int MT>
struct Seen {
    uint32_t row[MT], there;
};

template <int FMT, int D, int MT, bool MASK>
__device__ __forceinline__ void add_tile(const unsigned char *st, const Offsets<FMT, D> &of, const Queries<D, MT> &q, const uint4 *qs,
                                         float up, const float (&down)[MT][2], const Seen<MT> &seen, int lane, State<D, MT> &z) {
    using S = Shape<FMT, D>;
    float s[MT][4][4];
    scores<FMT, D, MT>(st, of, q, qs, lane, s);
    float ks[8], vs[8], vtop = 0.f, top[MT][2];
    load_scales<S::kRow>(st + S::kScales, lane & 3, ks);
    load_scales<S::kRow>(st + S::kScales + 4 * kTile, lane & 3, vs);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        ks[i] *= up;
        if (MASK && !((seen.there >> i) & 1u)) vs[i] = 0.f;
        vtop = fmaxf(vtop, vs[i]);
    }
    bool grows = vtop > z.ref;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float &y = s[t][i >> 1][2 * r + (i & 1)];
                y *= ks[i];
                if (MASK && !((seen.row[t] >> (8 * r + i)) & 1u)) y = -INFINITY;
            }
            float x = fmax3(s[t][0][2 * r], s[t][0][2 * r + 1], s[t][1][2 * r]);
            x = fmax3(x, s[t][1][2 * r + 1], s[t][2][2 * r]);
            x = fmax3(x, s[t][2][2 * r + 1], s[t][3][2 * r]);
            top[t][r] = fmaxf(x, s[t][3][2 * r + 1]) * down[t][r];
            grows |= top[t][r] > z.m[t][r] + kLag;
        }
    }
    if (__any_sync(0xffffffffu, grows)) {
        const float ref = fmaxf(z.ref, power_above(quad_max(vtop)));
        const float shrink = ref > 0.f ? z.ref / ref : 0.f;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float x = quad_max(top[t][r]);
                const float m = x > z.m[t][r] + kLag ? x + kHead : z.m[t][r];
                const float old = m == -INFINITY ? 1.f : ex2(z.m[t][r] - m);
                z.m[t][r] = m;
                z.l[t][r] *= old;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    z.o[t][i][2 * r] *= old * shrink;
                    z.o[t][i][2 * r + 1] *= old * shrink;
                }
            }
        }
        z.ref = ref;
        z.heavy = 0;
        z.settled = false;
    }
    const float unit = z.ref > 0.f ? kWeight / z.ref : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) vs[i] *= unit;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float m = z.m[t][r] == -INFINITY ? 0.f : z.m[t][r];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float &y = s[t][i >> 1][2 * r + (i & 1)];
                y = ex2(fmaf(y, down[t][r], -m));
                z.l[t][r] += y;
                y *= vs[i];
            }
        }
    }
    // Weights below fp16's normals are off by up to 2^-25, which shows only where all heavier places hold
    // an exact zero. Once a row has met a dozen places of weight 2^-12 or more since its reference last
    // moved, no element has only zeros in them and the error is below 2^-11 of the sum. Until then, what
    // the rounding of light weights leaves is added in a pass of its own, scaled up, with the sums scaled
    // along (powers of two: exact).
    bool light = false;
    if (!z.settled) {
        bool few = false;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float least = kLeastNormal;
                int n = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float y = s[t][i >> 1][2 * r + (i & 1)];
                    n += y >= kHeavy;
                    least = fminf(least, y > 0.f ? y : kLeastNormal);
                }
                n += __shfl_xor_sync(0xffffffffu, n, 1);
                n += __shfl_xor_sync(0xffffffffu, n, 2);
                n = min(n + ((z.heavy >> (16 * t + 8 * r)) & 0xff), 127);
                z.heavy = (z.heavy & ~(0xff << (16 * t + 8 * r))) | n << (16 * t + 8 * r);
                few |= n < kSettled;
                light |= n < kSettled && least < kLeastNormal;
            }
        }
        light = __any_sync(0xffffffffu, light);
        z.settled = !__any_sync(0xffffffffu, few);
    }
    uint32_t a[MT][2][4];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                a[t][n >> 1][2 * (n & 1) + r] = pack2(s[t][n][2 * r], s[t][n][2 * r + 1]);
            }
#pragma unroll 1
    for (int pass = 0;; ++pass) {
        add_values<FMT, D, MT, MASK>(st, of, a, lane, seen.there, z.o);
        if (!light) break;
        const float by = pass ? 1.f / kLift : kLift;
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int i = 0; i < D / 8; ++i) z.o[t][i][0] *= by, z.o[t][i][1] *= by, z.o[t][i][2] *= by, z.o[t][i][3] *= by;
        if (pass) break;
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float w0 = s[t][n][2 * r], w1 = s[t][n][2 * r + 1];
                    const float2 had = float2_of(a[t][n >> 1][2 * (n & 1) + r]);
                    a[t][n >> 1][2 * (n & 1) + r] = pack2(w0 < kLeastNormal ? (w0 - had.x) * kLift : 0.f, w1 < kLeastNormal ? (w1 - had.y) * kLift : 0.f);
                }
    }
}

// Copies tile `tile` of a job's pages to a stage (the whole warp): keys' and values' codes, scales and block
// scales; of two pages when pages hold 16 places. entry: lane i's page of the tile's i-th part. Returns the
// halves of the tile whose page does not exist.
template <int FMT, int D>
__device__ __forceinline__ uint32_t fetch(const Attend &p, const Walk &w, int tile, int kv, int entry, unsigned char *stage,
                                          uint64_t *full, int lane) {
    using S = Shape<FMT, D>;
    const bool halves = p.g.page < kTile;
    const int parts = halves ? 2 : 1, places = kTile / parts, at = tile * kTile & (p.g.page - 1);
    const bool mine = lane < parts && tile * kTile + lane * 16 < w.n.x + w.n.y;
    const bool good = mine && entry >= 0 && entry < p.n_pages;
    const uint32_t have = __ballot_sync(0xffffffffu, good), missing = __ballot_sync(0xffffffffu, mine && !good);
    if (missing && lane == 0) atomicOr(p.flags, QC_FLAG_RANGE);
    if (elect_one()) mbar_arrive_expect_tx(full, __popc(have) * places * (S::kStage / kTile));
    for (int i = 0; i < parts; ++i) {
        const int64_t page = __shfl_sync(0xffffffffu, entry, i);
        if ((have >> i) & 1u) {
            const unsigned char *src = p.pages + (page * p.g.heads + kv) * (int64_t)p.g.part;
            if (elect_one()) {
#pragma unroll
                for (int which = 0; which < 2; ++which) {
                    bulk_g2s(stage + which * S::kCodes + i * 16 * S::kRow, src + p.g.codes(which) + at * S::kRow, places * S::kRow, full);
                    bulk_g2s(stage + S::kScales + (which * kTile + i * 16) * 4, src + p.g.scales(which) + at * 4, places * 4, full);
                    if constexpr (S::kBlocks != 0)
                        bulk_g2s(stage + S::kBlockScales + (which * kTile + i * 16) * S::kBlocks, src + p.g.block_scales(which) + at * S::kBlocks,
                                 places * S::kBlocks, full);
                }
            }
        }
    }
    return halves ? missing : missing ? 3u : 0u;
}

// The query rows as fragments; down: the power of two that a row's scores are multiplied by.
template <typename T, int FMT, int D, int MT>
__device__ __forceinline__ void load_queries(const Attend &p, const Walk &w, int kv, int r0, int R, int lane, Queries<D, MT> &qf,
                                             uint4 *qs, float (&down)[MT][2]) {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        uint32_t a[2][D / 8];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = r0 + 16 * t + g + 8 * r;
            const bool there = row < R;
            const int node = there ? row / p.group : 0, h = there ? row % p.group : 0;
            const T *q = static_cast<const T *>(p.q) + w.b * p.q_seq + node * p.q_node + (kv * p.group + h) * p.q_head + c * (D / 4);
            float v[D / 4];
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                Eight<T> e;
                float f[8] = {};
                if (there) {
                    e.load(q + 8 * i);
                    e.get(f);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) v[8 * i + j] = f[j];
            }
            down[t][r] = 1.f;
            if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                float top = 0.f;
#pragma unroll
                for (int i = 0; i < D / 4; ++i) top = fmaxf(top, fabsf(v[i]));
                top = quad_max(top);
                // largest magnitude to [2^13, 2^14)
                const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -100), 127);
                const float f = __uint_as_float((uint32_t)(13 - e + 127) << 23);
                down[t][r] = __uint_as_float((uint32_t)(e - 13 + 127) << 23);
#pragma unroll
                for (int i = 0; i < D / 4; ++i) v[i] *= f;
            }
#pragma unroll
            for (int i = 0; i < D / 8; ++i) a[r][i] = pack2(v[2 * i], v[2 * i + 1]);
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i) qf.put(qs, lane, t, i, a[0][2 * i], a[1][2 * i], a[0][2 * i + 1], a[1][2 * i + 1]);
    }
}

template <int FMT, int D, int MT>
__device__ __forceinline__ Seen<MT> look(const Attend &p, const Walk &w, int t0, uint32_t bad, int r0, int R, int lane) {
    const int g = lane >> 2, c = lane & 3;
    const int exist = w.n.x + w.n.y - t0;
    const uint32_t good = (exist >= 32 ? 0xffffffffu : (1u << max(exist, 0)) - 1u) & ~((bad & 1u ? 0xffffu : 0u) | (bad & 2u ? 0xffff0000u : 0u));
    uint32_t win[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = r0 + 16 * m + g + 8 * r, node = row < R ? row / p.group : 0;
            const uint32_t *tree = p.tree ? p.tree + ((int64_t)w.b * p.n_nodes + node) * p.words : nullptr;
            win[m][r] = window(p, tree, node, w.n.y, t0 - w.n.x);
            if (row >= R || node >= w.n.y) win[m][r] = 0;
        }
    }
    Seen<MT> seen;
    seen.there = 0;
#pragma unroll
    for (int m = 0; m < MT; ++m) seen.row[m] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int at = 16 * (i >> 2) + Shape<FMT, D>::place((i >> 1) & 1, 2 * c + (i & 1));
        seen.there |= ((good >> at) & 1u) << i;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int r = 0; r < 2; ++r) seen.row[m] |= (((win[m][r] & good) >> at) & 1u) << (8 * r + i);
    }
    return seen;
}

template <typename T, int FMT, int D, int MT>
__global__ void __launch_bounds__(32 * kWarps, kPerSm / kWarps) attend_rows(const Attend p, const Parts parts, const Plan plan) {
    using S = Shape<FMT, D>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint64_t bars[kWarps][4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, unit = blockIdx.x * kWarps + warp;
    const int R = p.n_nodes * p.group, jobs = p.g.heads * plan.row_tiles;
    uint64_t *full = bars[warp];
    unsigned char *ring = smem + warp * plan.smem;
    uint4 *qs = reinterpret_cast<uint4 *>(ring + plan.stages * S::kStage);
    if (lane == 0) {
        for (int i = 0; i < plan.stages; ++i) mbar_init(&full[i], 1);
        fence_barrier_init();
    }
    Offsets<FMT, D> of;
    of.set(lane >> 2, lane & 3, p.g.page < kTile);
    __syncwarp();

    griddep_wait();
    const int64_t total = all_tiles(p, kTile, lane) * jobs, per = run_length(total, plan.units), at = per * unit;
    if (unit == 0) write_before(p, parts.before, jobs, kTile, lane);
    Walk w = find(p, at, at < total ? (total - at < per ? total - at : per) : 0, jobs, kTile, lane);
    int stage = 0, segment = 0;
    uint32_t phase = 0;
    const float up = p.scale * kLog2e;
    bool ok = true;
    while (w.left > 0 && ok) {
        const int kv = w.job / plan.row_tiles, r0 = w.job % plan.row_tiles * (16 * MT);
        const int from = w.tile, end = (int)(w.left < w.tiles - from ? from + w.left : w.tiles);
        const int32_t *row = p.table + w.b * p.table_stride;
        auto entry_of = [&](int tile) {
            const int t = tile * kTile + lane * 16;
            return lane < 2 && tile < end && t < w.n.x + w.n.y ? __ldg(row + (t >> p.g.shift)) : -1;
        };
        // the first tiles, then the queries while they travel
        uint32_t bad = 0;       // two bits per stage
        int ahead = from, ahead_stage = stage;
        int entry = entry_of(ahead);
        auto send = [&]() {
            const int next = entry_of(ahead + 1);
            const uint32_t b = fetch<FMT, D>(p, w, ahead, kv, entry, ring + ahead_stage * S::kStage, &full[ahead_stage], lane);
            bad = (bad & ~(3u << (2 * ahead_stage))) | b << (2 * ahead_stage);
            entry = next;
            ++ahead;
            if (++ahead_stage == plan.stages) ahead_stage = 0;
        };
        for (int i = 0; i < plan.stages && ahead < end; ++i) send();
        Queries<D, MT> q;
        float down[MT][2];
        load_queries<T, FMT, D, MT>(p, w, kv, r0, R, lane, q, qs, down);
        __syncwarp();
        State<D, MT> z;
        z.clear();
        int tile = from;
        for (; tile < end; ++tile) {
            ok = __all_sync(0xffffffffu, mbar_wait(&full[stage], phase));
            if (!ok) break;
            const unsigned char *st = ring + stage * S::kStage;
            const int t0 = tile * kTile;
            const uint32_t b = (bad >> (2 * stage)) & 3u;
            if (t0 + kTile <= w.n.x && !b) {
                add_tile<FMT, D, MT, false>(st, of, q, qs, up, down, Seen<MT>{}, lane, z);
            } else {
                add_tile<FMT, D, MT, true>(st, of, q, qs, up, down, look<FMT, D, MT>(p, w, t0, b, r0, R, lane), lane, z);
            }
            __syncwarp();
            if (++stage == plan.stages) stage = 0, phase ^= 1u;
            if (ahead < end) send();
        }
        if (!ok) {
            // let the copies under way land before the CTA's shared memory goes
            if (lane == 0) atomicOr(p.flags, QC_FLAG_TIMEOUT);
            for (; tile < ahead; ++tile) {
                mbar_wait(&full[stage], phase);
                if (++stage == plan.stages) stage = 0, phase ^= 1u;
            }
        }
        const bool whole = from == 0 && end == w.tiles;
        // part 2 c: the job that the warp's run begins with; 2 c + 1: the one it ends with
        const int64_t part = 2 * (int64_t)unit + (segment ? 1 : 0);
        const int g = lane >> 2, c = lane & 3;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float l = z.l[t][r];
                l += __shfl_xor_sync(0xffffffffu, l, 1);
                l += __shfl_xor_sync(0xffffffffu, l, 2);
                const int at_row = 16 * t + g + 8 * r, rr = r0 + at_row;
                if (rr >= R) continue;
                float v[D / 4];
                const float unit = z.ref * (1.f / kWeight);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) v[i] = z.o[t][i][2 * r] * unit, v[D / 8 + i] = z.o[t][i][2 * r + 1] * unit;
                if (whole) {
                    const int node = rr / p.group, h = kv * p.group + rr % p.group;
                    const bool there = node < w.n.y && l > 0.f;
                    const float inv = there ? 1.f / l : 0.f;
#pragma unroll
                    for (int i = 0; i < D / 4; ++i) v[i] = there ? v[i] * inv : 0.f;
                    const int64_t o = ((int64_t)w.b * p.n_nodes + node) * p.n_q_heads + h;
                    store_row<T, D / 4>(static_cast<T *>(p.out) + o * D + c * (D / 4), v);
                    if (p.lse && c == 0) p.lse[o] = there ? (z.m[t][r] + log2f(l)) * kLn2 : -INFINITY;
                } else {
                    float4 *to = reinterpret_cast<float4 *>(parts.row(part, at_row) + c * (D / 4));
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) to[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    if (c == 0) *parts.stat(part, at_row) = make_float2(z.m[t][r], l);
                }
            }
        }
        ++segment;
        w.left -= end - from;
        next_job(p, w, jobs, kTile);
    }
    griddep_launch_dependents();
}

template <int FMT, int D>
Plan plan_rows(const qc_ctx *c, int rows, int64_t n_seq, int64_t max_len, int n_nodes) {
    using S = Shape<FMT, D>;
    Plan p;
    p.device = c->device;
    // Up to 16 rows: one row tile per warp, its queries in registers. More: two, which share the codes'
    // conversion, their queries in shared memory.
    p.mt = rows <= 16 ? 1 : 2;
    p.row_tiles = (rows + 16 * p.mt - 1) / (16 * p.mt);
    const int queries = p.mt == 1 ? 0 : p.mt * 16 * D * 2;
    p.stages = (kRoom - queries) / S::kStage;
    if (p.stages > 4) p.stages = 4;
    p.smem = p.stages * S::kStage + queries;
    p.units = kPerSm * c->num_sms;
    const int64_t most = n_seq * c->heads * p.row_tiles * ((max_len + n_nodes + kTile - 1) / kTile);
    if (p.units > most) p.units = (int)(most + kWarps - 1) / kWarps * kWarps;
    return p;
}

template <int FMT, int D>
int64_t workspace(const qc_ctx *c, int rows, int64_t n_seq, int64_t max_len, int n_nodes) {
    const Plan p = plan_rows<FMT, D>(c, rows, n_seq, max_len, n_nodes);
    return workspace_bytes(n_seq, 2 * (int64_t)p.units, p.mt * 16, D);
}

template <typename T, int FMT, int D, int MT>
cudaError_t run(const Plan &plan, const Attend &p, int type, cudaStream_t s) {
    const Parts parts = parts_at(p.workspace, p.n_seq, 2 * (int64_t)plan.units, MT * 16, D);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(plan.units / kWarps));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = kWarps * plan.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(attend_rows<T, FMT, D, MT>, kWarps * kRoom, plan.device, done);
    if (e != cudaSuccess) return e;
    e = cudaLaunchKernelEx(&cfg, attend_rows<T, FMT, D, MT>, p, parts, plan);
    if (e != cudaSuccess) return e;
    return launch_join(p, parts, type, plan.row_tiles, kTile, plan.units, s);
}

template <int FMT, int D>
cudaError_t pick(const qc_ctx *c, int type, const Attend &p, cudaStream_t s) {
    const Plan plan = plan_rows<FMT, D>(c, p.n_nodes * p.group, p.n_seq, p.max_len, p.n_nodes);
    if (type == QC_F16) return plan.mt == 1 ? run<__half, FMT, D, 1>(plan, p, type, s) : run<__half, FMT, D, 2>(plan, p, type, s);
    return plan.mt == 1 ? run<__nv_bfloat16, FMT, D, 1>(plan, p, type, s) : run<__nv_bfloat16, FMT, D, 2>(plan, p, type, s);
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
