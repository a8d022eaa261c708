// Attention over the quantised cache for few query rows per key/value head (single tokens, chains, small
// trees) or short prefixes.
//
// Each warp on an SM (CTAs of four, so that every scheduler has as many) has a run of tiles of 32 places of its
// own. It copies them from the pages, as they lie, to its ring of shared-memory stages with bulk asynchronous
// copies, two or more tiles ahead, and turns codes into tensor-core fragments in registers. Warps never wait
// for one another; what one leaves unused of the memory's bandwidth, for instance at the start of a job, the
// others on its SM take.
//
// What bounds it: in the limit the pages, read once; as measured the latency of dependent conversions and
// products, two to three warps a scheduler. 4 rows over 32 sequences of up to 32,768 places (e2m1, fp16 queries, 637 MB)
// take 186 us (3.4 TB/s, 50 % of the card's copy rate), 20 rows over 16 x 16,384 (int8, bf16 queries, 555 MB) 173
// us (3.2 TB/s). With queries as the products' 16 rows and places as their 8 columns, twice the registers for the
// outputs of up to 8 queries and eight warps on an SM, it was 226 and 195 us.
//
// Products. Places are the products' 16 rows and queries their 8 columns (S^T = K Q^T, O^T = V^T P^T): the
// conversion, which costs most, goes over places, and few queries leave few columns empty. NT column tiles
// of 8 queries share it. Codes are exact in fp16, and so are e2m1 codes times their e4m3 block scale (5
// bits), so the products q . code are exact and summed in float32; the row's scale multiplies the score
// afterwards. A bf16 query row is brought into fp16's range by a power of two: 8 bits fit 11, and elements from 2^-30
// of the row's largest on keep them all (below, fp16's step is 2^-37 of the largest). For the values,
// the weight p_t times the row's scale is the operand: w_t = p_t * (s_t / ref) * 2^12, ref a power of two, the
// running bound of the scales seen. A row's reference m moves only when a score passes it by 3 (base 2), to 3
// above that score: so p_t <= 2^3 and w_t <= 2^15, the sums are rescaled seldom (a first tile's reference
// serves until a score is 2^6 times heavier), and the maximum is only reduced over the lanes when it is. w_t
// keeps fp16's 11 bits down to 2^-14; `add_tile` says what becomes of lighter weights, and of the other bits. A query
// whose sums turn out below kLeastSum of what the unit is for (all values that it gives weight are small beside
// others of the sequence) has the segment's places taken again in float32, one after the other (`plain_rows`).
//
// Order of elements. A sum over d may take them in any order as long as both operands do: lane c of a quad
// takes elements c d / 4 .. of a key, so one 16-byte load feeds four (e2m1: eight) steps. For the values lane
// group g takes elements g d / 8 .., two per 16-row tile of the output, and pairs of places are put together
// by byte permutes; there is no transposed copy of the values. Weights go from the scores' layout to the second
// product's by an 8 x 8 transpose between lanes (movmatrix). The pages' swizzle keeps the loads free of bank
// conflicts, with places assigned to rows as `place` says.
#include <math.h>

#include "qc_attend.cuh"
#include "qc_convert.cuh"

namespace qc {
namespace {

using namespace fq::sm100;

constexpr int kTile = 32;               // places per stage
constexpr int kWarps = 4;               // of a CTA
// CTAs on an SM and shared memory of a warp: 168 registers a lane where a warp's outputs take no more than 32 of
// them, else 255.
constexpr int per_sm(int nt, int d) { return nt * d <= 128 ? 3 : 2; }
constexpr int room(int nt, int d) { return (nt * d <= 128 ? 18 : 27) * 1024; }
constexpr float kWeight = 4096.f;       // 2^12
constexpr float kLag = 3.f;             // how far (base 2) a score may pass the row's reference
constexpr float kHead = 3.f;            // how far above the largest score a new reference is put
constexpr float kLeastNormal = 6.103515625e-05f;    // 2^-14, fp16's
constexpr float kLift = 16777216.f;     // 2^24
constexpr float kHeavy = 2.44140625e-04f;   // 2^-12
constexpr float kLeastSum = 0.03125f;       // 2^-5: fp16's least step is 2^-19 of it
// Heavy places that a row must have met: so many that an element is seldom zero in all of them. Of normally distributed
// values about one in six e2m1 codes is a zero, one in fifty of int8's, one in thousands of e4m3's. (Channels that
// stand out, or blocks of zeros, make it oftener: `add_tile` says what holds then.)
template <int FMT>
constexpr int kSettled = FMT == QC_E2M1 ? 12 : FMT == QC_INT8 ? 5 : 3;

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
    // Place (0 .. 15 of a half tile) of row 8 u + n of a score tile.
    static __device__ __forceinline__ int place(int u, int n) {
        if constexpr (kRow == 128) return 8 * u + n;
        if constexpr (kRow == 64) return 4 * (n >> 1) + 2 * u + (n & 1);
        return (n >> 1) + 4 * (2 * u + (n & 1));
    }
};

// The transpose of an 8 x 8 matrix of fp16, two neighbours of row lane / 4 to a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

struct Plan {
    int device;
    int row_tiles;      // tiles of 8 NT rows per head
    int nt;             // tiles of 8 queries of a warp (1 .. 4)
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

// The scales of the lane's four places: [2 x + u] is that of place(u, g) of half tile x.
template <int FMT, int D>
__device__ __forceinline__ void load_scales(const unsigned char *p, int g, float (&s)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = reinterpret_cast<const float *>(p)[16 * (i >> 1) + Shape<FMT, D>::place(i & 1, g)];
}

// Scores of a tile before any scale: s[n][x][2 u + e] of place(u, g) of half x, query 2 c + e of column tile n.
template <int FMT, int D, int NT>
__device__ __forceinline__ void scores(const unsigned char *st, const Offsets<FMT, D> &o, const uint32_t (&q)[NT][D / 16][2], int lane,
                                       float (&s)[NT][2][4]) {
    using S = Shape<FMT, D>;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) s[n][x][0] = s[n][x][1] = s[n][x][2] = s[n][x][3] = 0.f;
    constexpr int kChunks = S::kRow == 128 ? 2 : 1, kWords = S::kRow / 16 / kChunks;     // a lane's words per place
    constexpr int kSteps = FMT == QC_E2M1 ? 2 : 1;                                       // 16-wide steps per word
#pragma unroll
    for (int h = 0; h < kChunks; ++h) {
        uint32_t w[4][kWords];
        uint32_t sb[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            load_words<kWords>(st + o.key(i >> 1, i & 1, h), w[i]);
            if constexpr (FMT == QC_E2M1) {
                const unsigned char *b = st + S::kBlockScales + (16 * (i >> 1) + S::place(i & 1, lane >> 2)) * S::kBlocks + (lane & 3) * (S::kBlocks / 4);
                if constexpr (D == 128) {
                    const uint32_t x = *reinterpret_cast<const uint16_t *>(b);
                    sb[i][0] = cvt_e4m3(__byte_perm(x, 0, 0x4400));
                    sb[i][1] = cvt_e4m3(__byte_perm(x, 0, 0x4411));
                } else {
                    sb[i][0] = both_e4m3(*b);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                uint32_t k[2][4];               // of the half's two place groups: pairs of a word, two a step
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t v = w[2 * x + u][i];
                    if constexpr (FMT == QC_E2M1) {
                        cvt_e2m1(v, k[u]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) k[u][j] = mul2(k[u][j], sb[2 * x + u][i / 2]);
                    } else if constexpr (FMT == QC_INT8) {
                        const uint32_t y = v ^ 0x80808080u;
                        k[u][0] = sub1152(__byte_perm(y, 0x64646464u, 0x4140));
                        k[u][1] = sub1152(__byte_perm(y, 0x64646464u, 0x4342));
                    } else {
                        k[u][0] = cvt_e4m3(v);
                        k[u][1] = cvt_e4m3(v >> 16);
                    }
                }
#pragma unroll
                for (int j = 0; j < kSteps; ++j) {
                    const uint32_t a[4] = {k[0][2 * j], k[1][2 * j], k[0][2 * j + 1], k[1][2 * j + 1]};
                    const int step = (h * kWords + i) * kSteps + j;
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma(s[n][x], a, q[n][step][0], q[n][step][1]);
                }
            }
        }
    }
}

// out[n][j] += the values of half tile x times weights p[0][n][x] (+ p[1][n][x]); j: elements g D / 8 + 2 j and 2 j + 1. keep: which of
// the eight places that the lane loads exist (only asked when MASK; the others' bytes may be anything, NaN
// codes included, and count as zeros).
template <int FMT, int D, int NT, int TERMS, bool MASK>
__device__ __forceinline__ void add_values(const unsigned char *st, const Offsets<FMT, D> &o, const uint32_t (&p)[TERMS][NT][2][2], int lane,
                                           uint32_t keep, float (&out)[NT][D / 16][4]) {
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
        // lo, hi: pairs of places of the first and second group, elements 2 j and 2 j + 1
        auto add = [&](int j, uint32_t lo0, uint32_t lo1, uint32_t hi0, uint32_t hi1) {
            const uint32_t a[4] = {lo0, lo1, hi0, hi1};
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int t = 0; t < TERMS; ++t) mma(out[n][j], a, p[t][n][x][0], p[t][n][x][1]);
        };
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
                for (int e = 0; e < 4; ++e)
                    add(4 * j + e, mul2(__byte_perm(h[0][e], h[1][e], 0x5410), sb[0]), mul2(__byte_perm(h[0][e], h[1][e], 0x7632), sb[0]),
                        mul2(__byte_perm(h[2][e], h[3][e], 0x5410), sb[1]), mul2(__byte_perm(h[2][e], h[3][e], 0x7632), sb[1]));
            }
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j) {
                if constexpr (FMT == QC_INT8) {
                    // bytes of two places side by side, then fp16 pairs of (place, next place)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t y = __byte_perm(w[0][j], w[1][j], e ? 0x7362 : 0x5140) ^ 0x80808080u;
                        const uint32_t z = __byte_perm(w[2][j], w[3][j], e ? 0x7362 : 0x5140) ^ 0x80808080u;
                        add(2 * j + e, sub1152(__byte_perm(y, 0x64646464u, 0x4140)), sub1152(__byte_perm(y, 0x64646464u, 0x4342)),
                            sub1152(__byte_perm(z, 0x64646464u, 0x4140)), sub1152(__byte_perm(z, 0x64646464u, 0x4342)));
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t h[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) h[i] = cvt_e4m3(e ? w[i][j] >> 16 : w[i][j]);
                        add(2 * j + e, __byte_perm(h[0], h[1], 0x5410), __byte_perm(h[0], h[1], 0x7632), __byte_perm(h[2], h[3], 0x5410),
                            __byte_perm(h[2], h[3], 0x7632));
                    }
                }
            }
        }
    }
}

// The softmax state of a warp's queries: a lane has queries 2 c and 2 c + 1 of each column tile.
template <int D, int NT>
struct State {
    float m[NT][2], l[NT][2];   // reference (base-2 units), this lane's share of the sum
    float ref;                  // power of two, bound of the values' scales; 0: none yet
    int heavy[NT];              // places of weight kHeavy or more that each query met, 16 bits each, at most 127
    bool settled;               // kSettled or more for every query of the warp
    float o[NT][D / 16][4];
    __device__ __forceinline__ void clear() {
        ref = 0.f;
        settled = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
            heavy[n] = 0;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
        }
    }
};

// Over the eight lanes that hold a query's places.
__device__ __forceinline__ float column_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
template <typename T>
__device__ __forceinline__ T column_sum(T x) {
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// What a lane's scores see: bit 4 e + 2 x + u of row[n] for query 2 c + e and place(u, g) of half x. there: the lane's
// four score places that exist; keep: the eight whose values it loads, place(u, 2 c + e) of half x at 4 x + 2 u + e.
template <int NT>
struct Seen {
    uint32_t row[NT], there, keep;
};

template <int FMT, int D, int NT, int TERMS, bool MASK>
__device__ __forceinline__ void add_tile(const unsigned char *st, const Offsets<FMT, D> &of, const uint32_t (&q)[NT][D / 16][2], float up,
                                         const float (&down)[NT][2], const Seen<NT> &seen, int lane, State<D, NT> &z) {
    using S = Shape<FMT, D>;
    float s[NT][2][4];
    scores<FMT, D, NT>(st, of, q, lane, s);
    float ks[4], vs[4], vtop = 0.f, top[NT][2];
    load_scales<FMT, D>(st + S::kScales, lane >> 2, ks);
    load_scales<FMT, D>(st + S::kScales + 4 * kTile, lane >> 2, vs);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        ks[i] *= up;
        if (MASK && !((seen.there >> i) & 1u)) vs[i] = 0.f;
        vtop = fmaxf(vtop, vs[i]);
    }
    bool grows = vtop > z.ref;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float &y = s[n][i >> 1][2 * (i & 1) + e];
                y *= ks[i];
                if (MASK && !((seen.row[n] >> (4 * e + i)) & 1u)) y = -INFINITY;
            }
            top[n][e] = fmaxf(fmax3(s[n][0][e], s[n][0][2 + e], s[n][1][e]), s[n][1][2 + e]) * down[n][e];
            grows |= top[n][e] > z.m[n][e] + kLag;
        }
    }
    if (__any_sync(0xffffffffu, grows)) {
        const float ref = fmaxf(z.ref, power_above(column_max(vtop)));
        const float shrink = ref > 0.f ? z.ref / ref : 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float x = column_max(top[n][e]);
                const float m = x > z.m[n][e] + kLag ? x + kHead : z.m[n][e];
                const float old = m == -INFINITY ? 1.f : ex2(z.m[n][e] - m);
                z.m[n][e] = m;
                z.l[n][e] *= old;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    z.o[n][i][e] *= old * shrink;
                    z.o[n][i][2 + e] *= old * shrink;
                }
            }
            z.heavy[n] = 0;
        }
        z.ref = ref;
        z.settled = false;
    }
    const float unit = z.ref > 0.f ? kWeight / z.ref : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) vs[i] *= unit;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float m = z.m[n][e] == -INFINITY ? 0.f : z.m[n][e];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float &y = s[n][i >> 1][2 * (i & 1) + e];
                y = ex2(fmaf(y, down[n][e], -m));
                z.l[n][e] += y;
                y *= vs[i];
            }
        }
    }
    // Weights below fp16's normals are off by up to 2^-25, which shows only where all heavier places hold
    // an exact zero. Until a row has met kSettled places of weight 2^-12 or more since its reference last
    // moved, what the rounding of light weights leaves is added in a pass of its own, scaled up, with the sums
    // scaled along (powers of two: exact). From then on it is dropped: where an element is not zero in one of those
    // places, which is likely but not certain, the error is below 2^-11 of it. In any case it is below 2^-25 of the
    // largest code a place, and a row's largest element sums to 2^-5 of that code or more (`plain_rows` takes the
    // others): 2^-20 of the row's largest element, 2^-34 where the heaviest place's values are not smaller than others.
    // (Following weights until places of 2^-5 were met: 192 us instead of 173, chain of five.)
    bool light = false;
    if (!z.settled) {
        bool few = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float least = kLeastNormal;
                int k = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float y = s[n][i >> 1][2 * (i & 1) + e];
                    k += y >= kHeavy;
                    least = fminf(least, y > 0.f ? y : kLeastNormal);
                }
                k = min(column_sum(k) + ((z.heavy[n] >> (16 * e)) & 0xff), 127);
                z.heavy[n] = (z.heavy[n] & ~(0xff << (16 * e))) | k << (16 * e);
                few |= k < kSettled<FMT>;
                light |= k < kSettled<FMT> && least < kLeastNormal;
            }
        }
        light = __any_sync(0xffffffffu, light);
        z.settled = !__any_sync(0xffffffffu, few);
    }
    // A weight to 11 bits, and for fp16 outputs what that leaves, to 22. With 11 an fp16 output was 1.3 to 1.7 times
    // as far from 64 bits as its own rounding is; bf16's eight bits hide it. (One token over 32 ragged sequences,
    // e2m1: 170 us with one term, 182 with two, before rows were followed to their largest sums.)
    uint32_t p[TERMS][NT][2][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float &w0 = s[n][x][2 * u], &w1 = s[n][x][2 * u + 1];
#pragma unroll
                for (int t = 0; t < TERMS; ++t) {
                    const uint32_t h = pack2(w0, w1);
                    p[t][n][x][u] = transpose8(h);
                    const float2 had = float2_of(h);
                    if (t + 1 < TERMS) w0 -= had.x, w1 -= had.y;
                }
            }
#pragma unroll 1
    for (int pass = 0;; ++pass) {
        add_values<FMT, D, NT, TERMS, MASK>(st, of, p, lane, seen.keep, z.o);
        if (!light) break;
        const float by = pass ? 1.f / kLift : kLift;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < D / 16; ++i) z.o[n][i][0] *= by, z.o[n][i][1] *= by, z.o[n][i][2] *= by, z.o[n][i][3] *= by;
        if (pass) break;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    // what the terms leave of the light ones
                    const float w0 = s[n][x][2 * u], w1 = s[n][x][2 * u + 1];
                    const bool l0 = fabsf(w0) < kLeastNormal, l1 = fabsf(w1) < kLeastNormal;
                    const float2 had = float2_of(pack2(w0, w1));
                    p[0][n][x][u] = transpose8(pack2(l0 ? (w0 - had.x) * kLift : 0.f, l1 ? (w1 - had.y) * kLift : 0.f));
                    if (TERMS == 2) p[TERMS - 1][n][x][u] = 0;
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

// The queries as fragments; down: the power of two that the scores of the lane's queries 2 c, 2 c + 1 are multiplied by.
template <typename T, int FMT, int D, int NT>
__device__ __forceinline__ void load_queries(const Attend &p, const Walk &w, int kv, int r0, int R, int lane, uint32_t (&qf)[NT][D / 16][2],
                                             float (&down)[NT][2]) {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int row = r0 + 8 * n + g;
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
            for (int j = 0; j < 8; ++j) v[8 * i + j] = finite_or_nan(f[j]);
        }
        float back = 1.f;
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < D / 4; ++i) top = fmaxf(top, fabsf(v[i]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // largest magnitude to [2^13, 2^14)
            const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -100), 127);
            const float f = __uint_as_float((uint32_t)(13 - e + 127) << 23);
            back = __uint_as_float((uint32_t)(e - 13 + 127) << 23);
#pragma unroll
            for (int i = 0; i < D / 4; ++i) v[i] *= f;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) down[n][e] = __shfl_sync(0xffffffffu, back, 4 * (2 * c + e));
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            qf[n][i][0] = pack2(v[4 * i], v[4 * i + 1]);
            qf[n][i][1] = pack2(v[4 * i + 2], v[4 * i + 3]);
        }
    }
}

template <int FMT, int D, int NT>
__device__ __forceinline__ Seen<NT> look(const Attend &p, const Walk &w, int t0, uint32_t bad, int r0, int R, int lane) {
    using S = Shape<FMT, D>;
    const int g = lane >> 2, c = lane & 3;
    const int exist = w.n.x + w.n.y - t0;
    const uint32_t good = (exist >= 32 ? 0xffffffffu : (1u << max(exist, 0)) - 1u) & ~((bad & 1u ? 0xffffu : 0u) | (bad & 2u ? 0xffff0000u : 0u));
    uint32_t win[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int row = r0 + 8 * n + 2 * c + e, node = row < R ? row / p.group : 0;
            const uint32_t *tree = p.tree ? p.tree + ((int64_t)w.b * p.n_nodes + node) * p.words : nullptr;
            win[n][e] = window(p, tree, node, w.n.y, t0 - w.n.x) & good;
            if (row >= R || node >= w.n.y) win[n][e] = 0;
        }
    }
    Seen<NT> seen;
    seen.there = seen.keep = 0;
#pragma unroll
    for (int n = 0; n < NT; ++n) seen.row[n] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = 16 * (i >> 1) + S::place(i & 1, g);
        seen.there |= ((good >> at) & 1u) << i;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) seen.row[n] |= ((win[n][e] >> at) & 1u) << (4 * e + i);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) seen.keep |= ((good >> (16 * (i >> 2) + S::place((i >> 1) & 1, 2 * c + (i & 1)))) & 1u) << i;
    return seen;
}

// Places first .. last - 1 of one query row in float32, one after the other (the whole warp; a lane holds D / 32
// elements). m, l and o as add_tile leaves them.
template <typename T, int FMT, int D>
__device__ __forceinline__ void plain_row(const Attend &p, int b, int2 n, int kv, int row, int first, int last, int lane, float &m, float &l,
                                          float (&o)[D / 32]) {
    using S = Shape<FMT, D>;
    constexpr int E = D / 32;
    const int node = row / p.group, h = kv * p.group + row % p.group;
    const T *q = static_cast<const T *>(p.q) + b * p.q_seq + node * p.q_node + h * p.q_head + lane * E;
    const uint32_t *tree = p.tree ? p.tree + ((int64_t)b * p.n_nodes + node) * p.words : nullptr;
    const int32_t *table = p.table + b * p.table_stride;
    float x[E];
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = (float)q[i], o[i] = 0.f;
    m = -INFINITY, l = 0.f;
    // the lane's E elements of place t's keys or values, scaled
    auto fetch_row = [&](const unsigned char *part, int which, int t, float (&v)[E]) {
        const int byte = t * S::kRow + lane * S::kRow / 32;
        const unsigned char *c = part + p.g.codes(which) + piece_at(byte >> 4) * 16 + (byte & 15);
        const float scale = reinterpret_cast<const float *>(part + p.g.scales(which))[t];
        float block = 0.f;
        if constexpr (FMT == QC_E2M1) block = e4m3_value(part[p.g.block_scales(which) + t * S::kBlocks + lane * E / 16]) * 16384.f;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if constexpr (FMT == QC_INT8) v[i] = (float)(signed char)c[i] * scale;
            if constexpr (FMT == QC_E4M3) v[i] = e4m3_value(c[i]) * scale;
            if constexpr (FMT == QC_E2M1) v[i] = float2_of(half2_e2m1((c[i / 2] >> (4 * (i & 1))) & 0xfu)).x * block * scale;
        }
    };
    for (int t = first; t < last; ++t) {
        if (t >= n.x && !(window(p, tree, node, n.y, t - n.x) & 1u)) continue;
        const int page = __ldg(table + (t >> p.g.shift));
        if (page < 0 || page >= p.n_pages) continue;
        const unsigned char *part = p.pages + ((int64_t)page * p.g.heads + kv) * (int64_t)p.g.part;
        float v[E], s = 0.f;
        fetch_row(part, 0, t & (p.g.page - 1), v);
#pragma unroll
        for (int i = 0; i < E; ++i) s = fmaf(x[i], v[i], s);
#pragma unroll
        for (int i = 16; i >= 1; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
        s *= p.scale * kLog2e;
        const float top = fmaxf(m, s), old = m == -INFINITY ? 0.f : exp2f(m - top), weight = exp2f(s - top);
        fetch_row(part, 1, t & (p.g.page - 1), v);
        l = fmaf(l, old, weight);
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = fmaf(v[i], weight, o[i] * old);
        m = top;
    }
}

// The rows of `faint` (bit r: row r0 + r) of a segment, anew and over what is there (the whole warp). Not inlined: it
// is hardly ever called, and the tiles' loop needs the registers and the instruction cache.
template <typename T, int FMT, int D>
__device__ __noinline__ void plain_rows(const Attend &p, const Parts &parts, int b, int2 n, int kv, int r0, uint32_t faint, int first, int last,
                                        int64_t part) {
    const int lane = threadIdx.x & 31;
    for (; faint; faint &= faint - 1) {
        const int at_row = __ffs(faint) - 1, row = r0 + at_row, node = row / p.group, h = kv * p.group + row % p.group;
        float m, l, v[D / 32];
        plain_row<T, FMT, D>(p, b, n, kv, row, first, last, lane, m, l, v);
        if (part < 0) {
            const float inv = 1.f / l;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) v[i] *= inv;
            const int64_t o = ((int64_t)b * p.n_nodes + node) * p.n_q_heads + h;
            store_row<T, D / 32>(static_cast<T *>(p.out) + o * D + lane * (D / 32), v);
            if (p.lse && lane == 0) p.lse[o] = (m + log2f(l)) * kLn2;
        } else {
            float *to = parts.row(part, at_row) + lane * (D / 32);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) to[i] = v[i];
            if (lane == 0) *parts.stat(part, at_row) = make_float2(m, l);
        }
    }
}

template <typename T, int FMT, int D, int NT>
__global__ void __launch_bounds__(32 * kWarps, per_sm(NT, D)) attend_rows(const __grid_constant__ Attend p, const __grid_constant__ Parts parts, const Plan plan) {
    using S = Shape<FMT, D>;
    constexpr int kTerms = std::is_same<T, __half>::value ? 2 : 1;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint64_t bars[kWarps][4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, unit = blockIdx.x * kWarps + warp;
    const int R = p.n_nodes * p.group, jobs = p.g.heads * plan.row_tiles;
    uint64_t *full = bars[warp];
    unsigned char *ring = smem + warp * plan.smem;
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
        const int kv = w.job / plan.row_tiles, r0 = w.job % plan.row_tiles * (8 * NT);
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
        uint32_t q[NT][D / 16][2];
        float down[NT][2];
        load_queries<T, FMT, D, NT>(p, w, kv, r0, R, lane, q, down);
        State<D, NT> z;
        z.clear();
        int tile = from;
        for (; tile < end; ++tile) {
            ok = __all_sync(0xffffffffu, mbar_wait(&full[stage], phase));
            if (!ok) break;
            const unsigned char *st = ring + stage * S::kStage;
            const int t0 = tile * kTile;
            const uint32_t b = (bad >> (2 * stage)) & 3u;
            if (t0 + kTile <= w.n.x && !b) {
                add_tile<FMT, D, NT, kTerms, false>(st, of, q, up, down, Seen<NT>{}, lane, z);
            } else {
                add_tile<FMT, D, NT, kTerms, true>(st, of, q, up, down, look<FMT, D, NT>(p, w, t0, b, r0, R, lane), lane, z);
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
        uint32_t faint = 0;         // queries whose sums are too small for the unit: bit 2 n + e
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float l = column_sum(z.l[n][e]);
                float most = 0.f;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) most = fmax3(most, fabsf(z.o[n][i][e]), fabsf(z.o[n][i][2 + e]));
                const bool enough = (__ballot_sync(0xffffffffu, most >= kLeastSum * kTop<FMT>) >> c) & 0x11111111u;
                const int at_row = 8 * n + 2 * c + e, rr = r0 + at_row;
                if (rr >= R) continue;
                if (!enough && z.ref > 0.f && l > 0.f && rr / p.group < w.n.y) {
                    faint |= 1u << (2 * n + e);
                    continue;
                }
                // the lane's elements g D / 8 ..
                float v[D / 8];
                const float unit = z.ref * (1.f / kWeight);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) v[2 * i] = z.o[n][i][e] * unit, v[2 * i + 1] = z.o[n][i][2 + e] * unit;
                if (whole) {
                    const int node = rr / p.group, h = kv * p.group + rr % p.group;
                    const bool there = node < w.n.y && l != 0.f;        // a NaN goes out
                    const float inv = there ? 1.f / l : 0.f;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) v[i] = there ? v[i] * inv : 0.f;
                    const int64_t o = ((int64_t)w.b * p.n_nodes + node) * p.n_q_heads + h;
                    store_row<T, D / 8>(static_cast<T *>(p.out) + o * D + g * (D / 8), v);
                    if (p.lse && g == 0) p.lse[o] = there ? (z.m[n][e] + log2f(l)) * kLn2 : -INFINITY;
                } else {
                    float4 *to = reinterpret_cast<float4 *>(parts.row(part, at_row) + g * (D / 8));
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) to[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    if (g == 0) *parts.stat(part, at_row) = make_float2(z.m[n][e], l);
                }
            }
        }
        // what they see is small beside other values of the sequence, of which the unit is
        if (__any_sync(0xffffffffu, faint)) {
            uint32_t rows = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t x = __shfl_sync(0xffffffffu, faint, i);
#pragma unroll
                for (int n = 0; n < NT; ++n) rows |= ((x >> (2 * n)) & 3u) << (8 * n + 2 * i);
            }
            plain_rows<T, FMT, D>(p, parts, w.b, w.n, kv, r0, rows, from * kTile, min(end * kTile, w.n.x + w.n.y), whole ? -1 : part);
        }
        ++segment;
        w.left -= end - from;
        next_job(p, w, jobs, kTile);
    }
    griddep_launch_dependents();
}

// Rows of a warp at most: 32, in eights (24 with heads of 128, whose fourth tile does not fit the registers).
template <int D>
constexpr int kMostRows = D == 64 ? 32 : 24;

inline int units_rows(const qc_ctx *c, int nt, int d, int row_tiles, int64_t n_seq, int64_t places) {
    const int units = per_sm(nt, d) * kWarps * c->num_sms;
    const int64_t most = n_seq * c->heads * row_tiles * ((places + kTile - 1) / kTile);
    return units > most ? (int)(most + kWarps - 1) / kWarps * kWarps : units;
}

template <int FMT, int D>
Plan plan_rows(const qc_ctx *c, int rows, int64_t n_seq, int64_t max_len, int n_nodes) {
    using S = Shape<FMT, D>;
    Plan p;
    p.device = c->device;
    // more rows than kMostRows are dealt evenly to several warps, each with its own conversion
    p.row_tiles = (rows + kMostRows<D> - 1) / kMostRows<D>;
    p.nt = ((rows + p.row_tiles - 1) / p.row_tiles + 7) / 8;
    p.stages = room(p.nt, D) / S::kStage;
    if (p.stages > 4) p.stages = 4;
    p.smem = p.stages * S::kStage;
    p.units = units_rows(c, p.nt, D, p.row_tiles, n_seq, max_len + n_nodes);
    return p;
}

template <typename T, int FMT, int D, int NT>
cudaError_t run(const Plan &plan, const Attend &p, int type, cudaStream_t s) {
    const Parts parts = parts_at(p.workspace, p.n_seq, 2 * (int64_t)plan.units, NT * 8, D);
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
    cudaError_t e = allow_smem(attend_rows<T, FMT, D, NT>, kWarps * room(NT, D), plan.device, done);
    if (e != cudaSuccess) return e;
    e = cudaLaunchKernelEx(&cfg, attend_rows<T, FMT, D, NT>, p, parts, plan);
    if (e != cudaSuccess) return e;
    return launch_join(p, parts, type, plan.row_tiles, kTile, plan.units, s);
}

template <typename T, int FMT, int D>
cudaError_t pick(const qc_ctx *c, int type, const Attend &p, cudaStream_t s) {
    const Plan plan = plan_rows<FMT, D>(c, p.n_nodes * p.group, p.n_seq, p.max_len, p.n_nodes);
    return plan.nt == 1   ? run<T, FMT, D, 1>(plan, p, type, s)
           : plan.nt == 2 ? run<T, FMT, D, 2>(plan, p, type, s)
           : plan.nt == 3 ? run<T, FMT, D, 3>(plan, p, type, s)
                          : run<T, FMT, D, D == 64 ? 4 : 3>(plan, p, type, s);
}

}  // namespace

// One translation unit per head dimension (QC_ROWS_D).
template <>
cudaError_t attend_rows_d<QC_ROWS_D>(const qc_ctx *c, int type, const Attend &p, cudaStream_t s) {
    constexpr int D = QC_ROWS_D;
    if (type == QC_F16)
        return c->fmt == QC_INT8   ? pick<__half, QC_INT8, D>(c, type, p, s)
               : c->fmt == QC_E4M3 ? pick<__half, QC_E4M3, D>(c, type, p, s)
                                   : pick<__half, QC_E2M1, D>(c, type, p, s);
    return c->fmt == QC_INT8   ? pick<__nv_bfloat16, QC_INT8, D>(c, type, p, s)
           : c->fmt == QC_E4M3 ? pick<__nv_bfloat16, QC_E4M3, D>(c, type, p, s)
                               : pick<__nv_bfloat16, QC_E2M1, D>(c, type, p, s);
}

// The most that any call of up to these sizes wants: over all numbers of column tiles that up to so many rows take.
template <>
int64_t rows_workspace_d<QC_ROWS_D>(const qc_ctx *c, int rows, int64_t n_seq, int n_nodes, int64_t max_len) {
    constexpr int D = QC_ROWS_D;
    int64_t most = 0;
    for (int nt = 1; nt <= kMostRows<D> / 8 && 8 * (nt - 1) < rows; ++nt) {
        const int units = units_rows(c, nt, D, (rows + kMostRows<D> - 1) / kMostRows<D>, n_seq, max_len + n_nodes);
        const int64_t bytes = workspace_bytes(n_seq, 2 * (int64_t)units, nt * 8, D);
        if (bytes > most) most = bytes;
    }
    return most;
}

}  // namespace qc
