// Attention of chunks of new tokens over the quantised cache: products on the fifth-generation tensor cores, a pair of
// SMs on one tile.
//
// A cluster of two CTAs; NM row tiles of 256 query rows (128 in each CTA), tiles of 128 places. A product takes the rows
// of both CTAs, and half of its other operand from each: so a CTA turns only half of a tile's codes into operands, 64
// places' keys and half of every value row, and its tensor cores read that half from shared memory, whose
// bandwidth would else bound both. Roles, in each CTA:
//   softmax (4 NM warps) a thread per row: scores from TMEM, weights back to TMEM as fp16;
//   converters (4 warps) turn codes into operands, exactly: values and fp16 queries' keys to fp16, bf16 queries' keys
//                        to bf16;
//   producers (2 warps)  copy codes and scales, as the pages hold them, to rings of raw stages, keys and values apart;
//   MMA (1 thread of the first CTA, for both)  S = Q K^T into TMEM, then O += P V with P read from TMEM.
// While one row tile's softmax runs, the tensor cores work for the other. Scores come a whole tile at a time (in halves of 64
// places the products alone take 1.29 ms of the long chunk's instead of 0.95: the queries are read twice as often), weights go
// back in halves of 64. A job of one row tile has both softmax groups at its rows, every second tile each, with sums of their
// own that are joined at its end.
//
// Arithmetic. Products of codes and queries are exact, sums float32. A row has a reference M: with its scores u (base 2), p =
// 2^(u - M) goes to the sum of weights, and P = p s_v, s_v a value row's scale, to the tensor cores. M follows the
// largest P, not the largest score: so fp16 holds P whatever the magnitude of the values that the row gives weight to. A new
// one puts the largest at 2^kTop, and it is moved when one nears fp16's largest: so what fp16 rounds light products off
// by, 2^-25, is 2^-29 of the row's largest product or less. P is rounded to 11 bits for bf16 outputs; for fp16's to 22, in two terms:
// with one, an output was 1.5 to 1.7 times as far from 64 bits as its own rounding is. Value rows of zeros (s_v = 0) have no
// P; their weights are summed apart, with a reference of their own.
//
// Range. In a sum of weights p is P / s_v, and float32 has room for that as long as s_v is neither too small nor too large.
// qc_write makes scales of 2^-112 to 2^121. In units of 2^-20, as here, the small ones give p of 2^107 at most; above 2^64
// weights as heavy as the heaviest would come too near to 2^-126. So from the first tile with such a scale on, a warp sums all
// of a job's weights apart, by the scores' own largest, and takes its tiles step by step; P is then made with 2^64 at
// the weight and 2^-64 at the scale. (Caches in earnest hold no values of 2^51.) Where sums of unlike references meet, as a
// reference moves, in a row's two warps, in units' parts, factors below 2^-100 are taken in two steps, so that none is lost.
// That costs the calls that have none of it up to 5 % (single tokens over windows 335 -> 343 us, short prompts 108 -> 113), for
// the code that they step over; long chunks gain one.
//
// As M moves seldom, weights are made from scores at once, without a look for the largest first, and looked over afterwards;
// where one passes the limit, or some place is not seen, that half is done again, step by step.
//
// What bounds it. Long chunks (4,096 tokens over 28,672, 32/8 heads of 128, int8, bf16: 1,810 us, 1.14 PFLOP/s, 60 % of a large
// matrix product's rate; fp16, with two terms a weight, 2,150) are bound by no pipe: over 2,048 tokens and 8,192 places the issue
// slots are 46 % busy, the tensor pipe 34, the integer pipe 30, the multiply-add pipe 26, the exponentials' 19. It is the chain
// scores, weights, products, next scores: two row tiles in turn do not hide it (products alone take 0.95 ms, with the conversion
// 1.14). Two CTAs apart, each with all of a tile's operands, are bound by shared memory instead. Single tokens (32 over windows
// of 4,096, e2m1, capped: 329 to 352 us for 24 of memory) use one row in 256 of a tile, and a tile takes 2.9 us all the same, longer than
// a full one of the long chunk (2.25): 19 % of the issue slots, warps waiting for loads; conversion and one warp's capped scores
// follow one another. Short prompts (4 of up to 2,048 over 577: 114 us for 7) are starts, masked tiles step by step, and ends;
// so are tiles of a last warp in which lanes have no row, since those count as the first token's. A job's own start and end
// take 9.7 us where nothing else of the unit hides them (4,096 single tokens of empty contexts over 8 heads: 4.14 ms).
#pragma once

#include <math.h>

#include <atomic>
#include <type_traits>

#include "qc_chunk.cuh"
#include "qc_tc.cuh"

namespace qc {
namespace chunk {

using namespace fq::sm100;

static_assert(kTile == kChunkTile, "tiles of places");

// One above this has its reference moved with the next tile. A move ahead of need costs a tile its rescaling, one in need the
// step-by-step half besides: 4,096 tokens over 28,672 (int8, bf16, 128) took 2,145 us when all moves waited for the limit, 2,080 with
// 30,000 here. With 8,192, 2,048, 512 and 128 they take 1,944, 1,845, 1,814 and 1,810; fp16's 2,294, 2,186, 2,157, 2,143; heads
// of 64 (e4m3, fp16) 2,165, 2,045, 1,980, 1,958; windows of 4,096 429, 410, 397, 390; with a bias by distance 1,884 to 1,887.
constexpr float kSoon = 512.f;
constexpr float kMostLog = 15.9f, kMostP = 61147.f;     // the largest product that is let to fp16, and its log2
constexpr float kTop = 4.f;              // a new reference puts the largest one at 2^kTop, or up to twice that
constexpr float kScaleUnit = 1048576.f;  // values' scales are held times 2^20
// Those above 2^44, 2^kHugeLog in that unit, are huge, and held times 2^-44 (up to 2^84: qc_write makes none above that).
constexpr float kHuge = 17592186044416.f, kHugeUnit = 5.684341886080802e-14f, kHugeLog = 64.f, kMostHuge = 1.9342813113834067e25f;
constexpr int kMostStages = 4;
constexpr int kConverters = 4, kProducerWarps = 2;

constexpr int NM = 2, ROWS = 256 * NM;  // row tiles, and a job's rows
// Warps of a CTA: whole groups of four, since registers are moved between those.
constexpr int kThreads = 32 * (4 * NM + 8);
// 512 threads are launched with 128 registers each; the softmax's 256 take 176, the others 80: 65,536.
#define QC_SOFT_REGS "176"
#define QC_OTHER_REGS "80"

// What a call has beside scores, in bits: a bias by distance, a cap.
enum { kPlain = 0, kBias = 1, kCap = 2 };

template <int FMT, int D>
struct Raw {                            // a stage of keys: codes of the CTA's 64 places, both scales of all 128
    static constexpr int kRow = FMT == QC_E2M1 ? D / 2 : D;
    static constexpr int kBlocks = FMT == QC_E2M1 ? D / 16 : 0;
    static constexpr int kScales = kTile / 2 * kRow, kKeyBlocks = kScales + 8 * kTile;
    static constexpr int kKeyBytes = kKeyBlocks + kTile / 2 * kBlocks;
    static constexpr int kValueBlocks = kTile * kRow, kValueBytes = kTile * (kRow + kBlocks);
};

struct Ring {
    uint64_t full[kMostStages], empty[kMostStages];
    uint32_t bad[kMostStages];          // sixteenths of a stage's tile whose page does not exist
    uint32_t issued[kMostStages];       // 1 + parity of the stage's last copy; 0: none
    __device__ __forceinline__ void init(int stages) {
        for (int i = 0; i < kMostStages; ++i) {
            issued[i] = 0;
            if (i < stages) {
                mbar_init(&full[i], 1);
                mbar_init(&empty[i], kConverters);
            }
        }
    }
    // Waits for what is still under way (one warp, after everything else): true when all has landed.
    __device__ __forceinline__ bool land(int stages, int lane) {
        const uint32_t i = lane < stages ? issued[lane] : 0;
        const bool ok = !i || mbar_wait(&full[lane < stages ? lane : 0], i - 1);
        return __all_sync(0xffffffffu, ok);
    }
};

struct Bars {
    Ring keys, values;
    // the first CTA's are waited on by the MMA thread: both CTAs arrive there
    uint64_t k_full[2], v_full[2], q_ready, p_ready[2][2];
    // arrived at in both CTAs when products are done
    uint64_t k_free[2], v_free[2], s_full[2], o_done[2], job_done, last, join;
};

struct Small {
    Bars b;
    // of a tile's places, two at a time: keys' scales, times what makes the product a score (base 2; with a cap: twice its
    // argument), and the values' scales; and log2 of those
    alignas(16) float kv[4][kTile / 2][4];
    alignas(16) float lv[4][kTile];
    // places that exist: with values of no huge scale, with values of any, and with rows of zeros for them
    alignas(16) uint32_t exist[4][4], product[4][4], zero[4][4];
    alignas(16) float4 other[128];      // of a row that two warps share: the second's references and sums
    ChunkWalk start;
    uint32_t tmem;
};

// ---- instructions of a pair of CTAs -----------------------------------------------------------

__device__ __forceinline__ void pair_alloc(uint32_t *slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_dealloc(uint32_t taddr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void pair_mma_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
        "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrives at the barrier of this place in both CTAs once the products issued so far are done.
__device__ __forceinline__ void pair_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_addr(bar)),
                 "h"((uint16_t)3)
                 : "memory");
}
// Where a place of this CTA's shared memory lies in the first CTA's.
__device__ __forceinline__ uint32_t in_first(const void *p) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_addr(p)));
    return r;
}
// One lane of a warp arrives at a barrier of the cluster. Orders within the CTA are enough: what the barrier guards is read
// by the tensor cores of the CTA that wrote it, and fenced for them.
__device__ __forceinline__ void arrive_at(uint32_t bar, int lane) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %1, 0;\n\t@p mbarrier.arrive.shared::cluster.b64 _, [%0];\n\t}" ::"r"(bar), "r"(lane) : "memory");
}
// A barrier's phase, by its number, for at most about two seconds, polled: for the chain of products and softmax, which
// sleeping (qc_tc.cuh's warp_wait) would hold up. The others sleep: polling, they would take the softmax's issue slots.
__device__ __forceinline__ bool poll(uint64_t *bar, uint32_t phase) { return mbar_wait(bar, phase & 1u); }
__device__ __forceinline__ bool warp_poll(uint64_t *bar, uint32_t phase) { return __all_sync(0xffffffffu, poll(bar, phase)); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Operand descriptor of rows (places) of 32 elements (64 bytes, 64-byte swizzle) that hold the output's dimension.
__device__ __forceinline__ uint64_t sdesc_sw64_mn(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)1u << 16;
    d |= (uint64_t)(512u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)4u << 61;
    return d;
}

// floor(log2(x)), x > 0 and normal
__device__ __forceinline__ float log2_below(float x) { return (float)((int)(__float_as_uint(x) >> 23) - 127); }
// 2^t as two factors, for t from -226 to 226
__device__ __forceinline__ float2 power_of_2(float t) {
    const float a = fminf(fmaxf(t, -100.f), 100.f);
    return make_float2(ex2(a), ex2(t - a));
}
// A sum of weights, w 2^ref. One that is a NaN stays one.
struct Sum {
    float ref, w;
};
// a + b with each at its own height first, so that neither is lost where references are far from the sums
__device__ __forceinline__ Sum joined(Sum a, Sum b) {
    if (b.w == 0.f) return a;
    if (a.w == 0.f) return b;
    auto level = [](Sum x) {
        if (!(x.w < INFINITY)) return x;
        return Sum{x.ref + log2_below(x.w), __uint_as_float((__float_as_uint(x.w) & 0x007fffffu) | 0x3f800000u)};
    };
    a = level(a), b = level(b);
    const float ref = fmaxf(a.ref, b.ref);
    return {ref, a.w * ex2(a.ref - ref) + b.w * ex2(b.ref - ref)};
}
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
        "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// tanh(a) / a for a = y ln 2 / 2, |a| <= 1/4, two at a time: the polynomial in a^2, of degree 3, through its values at the
// Chebyshev points of [0, 1/16], off by 6e-8 in float32.
constexpr float kNear = 0.5f * kLog2e;
__device__ __forceinline__ float2 tanh_over(float2 y) {
    constexpr float h = 0.5f * kLn2, u = h * h, c0 = 1.f, c1 = -0.3333320617675781f * u, c2 = 0.13323144614696503f * u * u,
                    c3 = -0.05132901296019554f * u * u * u;
    const float2 z = mul2f(y, y);
    float2 f = fma2f(make_float2(c3, c3), z, make_float2(c2, c2));
    f = fma2f(f, z, make_float2(c1, c1));
    return fma2f(f, z, make_float2(c0, c0));
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// ---- codes to bf16 ------------------------------------------------------------------------------

__device__ __forceinline__ uint32_t bsub2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t bmul2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}
// Two fp16 numbers as bf16, where bf16 holds them.
__device__ __forceinline__ uint32_t bf16_of_half2(uint32_t h) {
    const float2 f = float2_of(h);
    const __nv_bfloat162 r = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t *>(&r);
}
// int8: 0x4300 | low seven bits is 128 + them; less 128, or 256 where the sign is set.
__device__ __forceinline__ uint32_t bf16_int8(uint32_t x, uint32_t sel) {
    const uint32_t h = __byte_perm(x, 0x43434343u, sel);
    return bsub2(h & 0xff7fff7fu, h & 0xff80ff80u);
}
// e4m3 (bias 7): sign, and the rest four places down, is value * 2^-120 as bf16 (bias 127).
__device__ __forceinline__ uint32_t bf16_e4m3(uint32_t x, uint32_t sel) {
    const uint32_t h = __byte_perm(x, 0, sel);
    return bmul2((h & 0x80008000u) | ((h >> 4) & 0x07f007f0u), 0x7b807b80u);
}

// One 16-byte piece of codes to operand pieces of eight elements, in bf16 (B) or fp16: put(i, pairs) takes the i-th. sb: the
// piece's two block scales (e2m1 alone).
template <int FMT, bool B, typename Put>
__device__ __forceinline__ void convert_piece(uint4 c, uint32_t sb, Put put) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    if constexpr (FMT == QC_E2M1) {
        const uint32_t s[2] = {both_e4m3(__byte_perm(sb, 0, 0x4440)), both_e4m3(__byte_perm(sb, 0, 0x4441))};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t h[4];
            cvt_e2m1(w[i], h);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                h[e] = mul2(h[e], s[i >> 1]);
                if constexpr (B) h[e] = bf16_of_half2(h[e]);
            }
            put(i, h);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t x = w[2 * i + e];
                if constexpr (FMT == QC_INT8 && B) {
                    h[2 * e] = bf16_int8(x, 0x4140);
                    h[2 * e + 1] = bf16_int8(x, 0x4342);
                } else if constexpr (FMT == QC_INT8) {
                    const uint32_t y = x ^ 0x80808080u;
                    h[2 * e] = sub1152(__byte_perm(y, 0x64646464u, 0x4140));
                    h[2 * e + 1] = sub1152(__byte_perm(y, 0x64646464u, 0x4342));
                } else if constexpr (B) {
                    h[2 * e] = bf16_e4m3(x, 0x1404);
                    h[2 * e + 1] = bf16_e4m3(x, 0x3424);
                } else {
                    h[2 * e] = cvt_e4m3(x);
                    h[2 * e + 1] = cvt_e4m3(x >> 16);
                }
            }
            put(i, h);
        }
    }
}

// ---- the roles ----------------------------------------------------------------------------------

// Copies of a tile's keys (which = 0: the CTA's 64 places' codes, and both scales of all) or values. False if a wait
// gave up.
template <int FMT, int D, int ROWS>
__device__ __forceinline__ bool produce_tiles(const Chunk &p, ChunkWalk run, int stages, unsigned char *raw, Ring &ring, int which, int cta, int lane,
                                              PartLine *lines) {
    using R = Raw<FMT, D>;
    const int bytes = which ? R::kValueBytes : R::kKeyBytes;
    const int sub = p.g.page < kTile ? p.g.page : kTile, parts = kTile / sub;
    const int64_t page_bytes = (int64_t)p.g.heads * p.g.part;
    int stage = 0;
    uint32_t round = 0;
    PartLine line[2] = {};
    for (int segment = 0; run.left > 0; run.template next<ROWS>(p), ++segment) {
        const int end = run.end(), places = run.s.len + run.s.news;
        if (run.tile > run.first || end < run.last)
            line[segment ? 1 : 0] = {run.b, run.kv, run.run, kHolds | (run.tile == run.first ? kOpens : 0) | (end == run.last ? kCloses : 0)};
        const int32_t *row = p.table + run.b * p.table_stride;
        const unsigned char *head = p.pages + run.kv * (int64_t)p.g.part;
        // lane i: the page of the tile's i-th part
        auto entry_of = [&](int step) {
            const int t = run.place(step) * kTile + lane * sub;
            int e = -1;
            if (lane < parts && step < end && t < places)
                asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(e) : "l"(row + (t >> p.g.shift)));     // not later than here
            return e;
        };
        int entry = entry_of(run.tile);
        for (int step = run.tile; step < end; ++step) {
            const int next = entry_of(step + 1), tile = run.place(step);
            const bool here = lane < parts && tile * kTile + lane * sub < places;
            const bool good = here && entry >= 0 && entry < p.n_pages;
            const uint32_t have = __ballot_sync(0xffffffffu, good), missing = __ballot_sync(0xffffffffu, here && !good);
            uint32_t bad = 0;
            if (missing) {
                for (int i = 0; i < parts; ++i)
                    if ((missing >> i) & 1u) bad |= ((1u << (sub / 16)) - 1u) << (i * (sub / 16));
                if (lane == 0 && which == 0 && cta == 0) atomicOr(p.flags, QC_FLAG_RANGE);
            }
            if (round && !warp_wait(&ring.empty[stage], round - 1)) return false;
            unsigned char *to = raw + stage * bytes;
            // keys: the part of a page within the CTA's half of the tile
            const int at = tile * kTile & (p.g.page - 1);       // where in a page of 256 the tile begins
            const int half = kTile / 2, mine = sub < half ? sub : half;
            const uint32_t own = sub < kTile ? have & (((1u << (parts / 2)) - 1u) << (cta * (parts / 2))) : have;
            if (elect_one()) {
                ring.bad[stage] = bad;
                ring.issued[stage] = 1 + (round & 1);
                const uint32_t n = which ? __popc(have) * sub * (R::kRow + R::kBlocks)
                                         : __popc(have) * sub * 8 + __popc(own) * mine * (R::kRow + R::kBlocks);
                mbar_arrive_expect_tx(&ring.full[stage], n);
            }
            for (int i = 0; i < parts; ++i) {
                const int64_t page = __shfl_sync(0xffffffffu, entry, i);
                if (!((have >> i) & 1u)) continue;
                const unsigned char *src = head + page * page_bytes;
                const int first = i * sub;
                if (elect_one()) {
                    if (which) {
                        bulk_g2s(to + first * R::kRow, src + p.g.codes(1) + at * R::kRow, sub * R::kRow, &ring.full[stage]);
                        if constexpr (R::kBlocks != 0)
                            bulk_g2s(to + R::kValueBlocks + first * R::kBlocks, src + p.g.block_scales(1) + at * R::kBlocks, sub * R::kBlocks,
                                     &ring.full[stage]);
                    } else {
                        bulk_g2s(to + R::kScales + first * 4, src + p.g.scales(0) + at * 4, sub * 4, &ring.full[stage]);
                        bulk_g2s(to + R::kScales + (kTile + first) * 4, src + p.g.scales(1) + at * 4, sub * 4, &ring.full[stage]);
                        if ((own >> i) & 1u) {
                            const int from = sub < kTile ? at : at + cta * half, row0 = sub < kTile ? first - cta * half : 0;
                            bulk_g2s(to + row0 * R::kRow, src + p.g.codes(0) + from * R::kRow, mine * R::kRow, &ring.full[stage]);
                            if constexpr (R::kBlocks != 0)
                                bulk_g2s(to + R::kKeyBlocks + row0 * R::kBlocks, src + p.g.block_scales(0) + from * R::kBlocks,
                                         mine * R::kBlocks, &ring.full[stage]);
                        }
                    }
                }
            }
            if (++stage == stages) stage = 0, ++round;
            entry = next;
        }
    }
    if (lines && lane == 0) {
        lines[0] = line[0];
        lines[1] = line[1];
    }
    return true;
}

// Whether a job has rows for one row tile alone. The other's buffers then serve the same rows: its softmax takes every second
// tile of places, with references and sums of its own, and the two are joined at the job's end.
__device__ __forceinline__ bool solo(const Chunk &p, const ChunkWalk &run) { return run.s.news * p.group - run.run * ROWS <= 256; }

template <typename T, int FMT, int D, int X>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_tc(const Chunk p, const ChunkParts parts, const ChunkPlan plan) {
    using R = Raw<FMT, D>;
    constexpr bool kB = std::is_same<T, __nv_bfloat16>::value;
    constexpr int kTerms = kB ? 1 : 2;
    constexpr int kSoft = 4 * NM, kConv = kSoft, kProducer = kSoft + kConverters, kMma = kProducer + kProducerWarps;
    constexpr int kQ = 128 * D * 2, kK = kTile / 2 * D * 2, kV = kTile * D;         // bytes of a CTA's operand tiles
    constexpr int kVRow = D;                                                        // bytes of a value operand's row: D / 2 elements
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char *q_op = smem, *k_op = q_op + NM * kQ, *v_op = k_op + 2 * kK, *raw_k = v_op + 2 * kV, *raw_v = raw_k + plan.raw * R::kKeyBytes;
    Small &sm = *reinterpret_cast<Small *>(raw_v + plan.raw * R::kValueBytes);
    Bars &bar = sm.b;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cta = (int)cluster_ctarank(), unit = (int)(blockIdx.x >> 1);
    const uint32_t first_bars = in_first(&bar);
    auto arrive_first = [&](const uint64_t *b) { arrive_at(first_bars + (uint32_t)((const char *)b - (const char *)&bar), lane); };

    if (warp == kMma) {
        if (lane == 0) {
            bar.keys.init(plan.raw);
            bar.values.init(plan.raw);
            for (int i = 0; i < 2; ++i) {
                mbar_init(&bar.k_full[i], 2 * kConverters);
                mbar_init(&bar.v_full[i], 2 * kConverters);
                mbar_init(&bar.k_free[i], 1);
                mbar_init(&bar.v_free[i], 1);
                mbar_init(&bar.s_full[i], 1);
                mbar_init(&bar.o_done[i], 1);
                mbar_init(&bar.p_ready[i][0], 8);
                mbar_init(&bar.p_ready[i][1], 8);
            }
            mbar_init(&bar.q_ready, 2 * kSoft);
            mbar_init(&bar.job_done, 1);
            mbar_init(&bar.last, 1);
            mbar_init(&bar.join, 4);
            fence_barrier_init();
        }
        __syncwarp();
        pair_alloc(&sm.tmem, 512);
    }
    griddep_wait();
    if (warp == kProducer) {
        const ChunkWalk w = find_run<ROWS>(p, unit, plan.units, blockIdx.x == 0, lane);
        if (lane == 0) sm.start = w;
        if (lane < 2 && cta == 0) parts.lines[2 * unit + lane] = {};        // of an earlier call, or of none
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();             // the barriers of both CTAs are there
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    ChunkWalk run = sm.start;
    bool ok = true;
    int it = 0;                 // tiles so far, over all jobs of the run

    // each of the two takes what it will need of the registers, here and not before: what comes before is compiled for
    // those that the launch gives
    if (warp >= kSoft) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 " QC_OTHER_REGS ";");
        if (warp == kProducer || warp == kProducer + 1) {
            const int which = warp - kProducer;
            ok = produce_tiles<FMT, D, ROWS>(p, run, plan.raw, which ? raw_v : raw_k, which ? bar.values : bar.keys, which, cta, lane,
                                             which == 0 && cta == 0 ? parts.lines + 2 * unit : nullptr);
        } else if (warp >= kConv && warp < kConv + kConverters) {
            const int quarter = warp - kConv, t = quarter * 32 + lane;
            const bool short_runs = R::kRow == 32 && p.g.page == 16;
            const float up = X & kCap ? p.scale * (2.f * kLog2e) / p.cap : p.scale * kLog2e;
            int stage = 0;
            uint32_t phase = 0;
            // the 16-byte piece p of a run of codes, as it lies in a stage
            auto piece = [&](const unsigned char *st, int i) {
                return *reinterpret_cast<const uint4 *>(st + (i ^ ((i >> 3) & (short_runs ? 3 : 7))) * 16);
            };
            for (; ok && run.left > 0; run.template next<ROWS>(p)) {
                const int end = run.end(), places = run.s.len + run.s.news;
                for (int step = run.tile; ok && step < end; ++step, ++it) {
                    const int tile = run.place(step);
                    // keys: the operand's last reader, then the codes
                    if (it >= 2) ok = ok && warp_wait(&bar.k_free[it & 1], (it >> 1) - 1);
                    ok = ok && warp_wait(&bar.keys.full[stage], phase);
                    if (!ok) break;
                    {
                        const unsigned char *st = raw_k + stage * R::kKeyBytes;
                        const uint32_t bad = bar.keys.bad[stage];
                        auto is_there = [&](int i) { return tile * kTile + i < places && !((bad >> (i >> 4)) & 1u); };
                        const bool good = is_there(t);
                        const float *scale = reinterpret_cast<const float *>(st + R::kScales);
                        const float sv = good ? scale[kTile + t] : 0.f;
                        const bool some = sv > 0.f, huge = sv > kHuge;
                        const float vs = !some ? 0.f : huge ? fminf(sv * kHugeUnit, kMostHuge) : sv * kScaleUnit;
                        sm.kv[it & 3][t >> 1][t & 1] = good ? scale[t] * up : 0.f;
                        sm.kv[it & 3][t >> 1][2 + (t & 1)] = vs;
                        sm.lv[it & 3][t] = some ? log2f(vs) + (huge ? kHugeLog : 0.f) : 0.f;
                        const uint32_t e = __ballot_sync(0xffffffffu, some && !huge), z = __ballot_sync(0xffffffffu, good && !some),
                                       v = __ballot_sync(0xffffffffu, some);
                        if (lane == 0) {
                            sm.exist[it & 3][quarter] = e;
                            sm.zero[it & 3][quarter] = z;
                            sm.product[it & 3][quarter] = v;
                        }
                        // a place and half of its row
                        const int i = t & 63, h = t >> 6;
                        const bool have = is_there(cta * 64 + i);
                        constexpr int P = R::kRow / 16, kHalf = P >= 2 ? P / 2 : 1;
                        unsigned char *out = k_op + (it & 1) * kK;
                        uint32_t sb[2] = {0, 0};        // the half row's block scales
                        if constexpr (FMT == QC_E2M1) {
                            if constexpr (D == 128)
                                sb[0] = *reinterpret_cast<const uint32_t *>(st + R::kKeyBlocks + i * R::kBlocks + h * 4);
                            else
                                sb[0] = *reinterpret_cast<const uint16_t *>(st + R::kKeyBlocks + i * R::kBlocks + h * 2);
                        }
                        constexpr int kEights = D / 2 / 8 / kHalf;      // operand pieces per piece of codes
#pragma unroll
                        for (int j = 0; j < kHalf; ++j) {
                            uint4 c = piece(st, i * P + h * kHalf + j);
                            if (!have) c = make_uint4(0, 0, 0, 0);
                            convert_piece<FMT, kB>(c, have ? sb[0] >> (16 * j) : 0u, [&](int q, const uint32_t(&v)[4]) {
                                const int at = h * (D / 16) + j * kEights + q;          // of the row's D / 8 pieces
                                *reinterpret_cast<uint4 *>(out + (at >> 3) * (64 * 128) + i * 128 + (((at & 7) ^ (i & 7)) * 16)) =
                                    make_uint4(v[0], v[1], v[2], v[3]);
                            });
                        }
                        fence_async();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar.keys.empty[stage]);
                        arrive_first(&bar.k_full[it & 1]);
                    }
                    // values: every place, the CTA's half of the row
                    if (it >= 2) ok = ok && warp_wait(&bar.v_free[it & 1], (it >> 1) - 1);
                    ok = ok && warp_wait(&bar.values.full[stage], phase);
                    if (!ok) break;
                    {
                        const unsigned char *st = raw_v + stage * R::kValueBytes;
                        const bool good = tile * kTile + t < places && !((bar.values.bad[stage] >> (t >> 4)) & 1u);
                        constexpr int P = R::kRow / 16, kHalf = P / 2;
                        unsigned char *out = v_op + (it & 1) * kV;
                        uint32_t sb = 0;
                        if constexpr (FMT == QC_E2M1) {
                            if constexpr (D == 128)
                                sb = *reinterpret_cast<const uint32_t *>(st + R::kValueBlocks + t * R::kBlocks + cta * 4);
                            else
                                sb = *reinterpret_cast<const uint16_t *>(st + R::kValueBlocks + t * R::kBlocks + cta * 2);
                        }
                        constexpr int kEights = D / 2 / 8 / kHalf;
#pragma unroll
                        for (int j = 0; j < kHalf; ++j) {
                            uint4 c = piece(st, t * P + cta * kHalf + j);
                            if (!good) c = make_uint4(0, 0, 0, 0);
                            convert_piece<FMT, false>(c, good ? sb >> (16 * j) : 0u, [&](int q, const uint32_t(&v)[4]) {
                                const int at = j * kEights + q;
                                const int turn = D == 128 ? t & 7 : (t >> 1) & 3;
                                *reinterpret_cast<uint4 *>(out + t * kVRow + ((at ^ turn) * 16)) = make_uint4(v[0], v[1], v[2], v[3]);
                            });
                        }
                        fence_async();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar.values.empty[stage]);
                        arrive_first(&bar.v_full[it & 1]);
                    }
                    if (++stage == plan.raw) stage = 0, phase ^= 1u;
                }
            }
        } else if (warp == kMma) {
            if (cta == 0 && elect_one()) {          // one thread, from here to the end
                constexpr uint32_t kTypes = kB ? 1u << 7 | 1u << 10 : 0u;
                const uint32_t qk = idesc_f16_f32(256, kTile) | kTypes, pv = idesc_f16_f32(256, D) | 1u << 16;      // values: output dimension contiguous
                // descriptors of the operands' starts; a place further on is so many 16 bytes more. They are made anew for each
                // product: kept for all, they would take more registers than the thread has.
                const uint64_t q_desc = sdesc_sw128(smem_addr(q_op)), k_desc = sdesc_sw128(smem_addr(k_op));
                const uint64_t v_desc = D == 128 ? sdesc_sw128_mn(smem_addr(v_op), kTile * 128) : sdesc_sw64_mn(smem_addr(v_op));
                auto from_here = [](uint64_t x) {
                    asm volatile("" : "+l"(x));
                    return x;
                };
                auto scores = [&](int rt, int buf, int kb) {   // S[buf] = Q[rt] K^T
                    tc_fence_after();
                    const uint64_t q = from_here(q_desc + rt * (kQ >> 4)), kd = from_here(k_desc + kb * (kK >> 4));
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        pair_mma(tmem + buf * kTile, q + (((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4), kd + (((k >> 2) * (64 * 128) + (k & 3) * 32) >> 4), qk,
                                 k > 0);
                    pair_commit(&bar.s_full[buf]);
                };
                auto values = [&](int rt, int buf, int h, int vb, bool first) {        // O[rt] (+)= P[buf][h] V[half h]
                    tc_fence_after();
                    const uint64_t v = from_here(v_desc + vb * (kV >> 4));
#pragma unroll
                    for (int k = 0; k < 4 * kTerms; ++k) {       // 16 places at a time, the weights' terms one after the other
                        const int step = k / kTerms, term = k % kTerms;
                        pair_mma_ts(tmem + 256 + rt * D, tmem + buf * kTile + 64 * h + 32 * (step >> 1) + 16 * term + 8 * (step & 1),
                                    v + (((4 * h + step) * 16 * kVRow) >> 4), pv, !first || k > 0);
                    }
                };
                auto wait = [&](uint64_t *b, uint32_t phase) { ok = ok && poll(b, phase); };
                int n[2] = {0, 0};          // how often each of the scores' buffers has been filled
                for (int segment = 0; ok && run.left > 0; run.template next<ROWS>(p), ++segment) {
                    const int end = run.end();
                    int2 of[2];
#pragma unroll
                    for (int rt = 0; rt < NM; ++rt) of[rt] = tiles_of_rows(p, run.s, run.run * ROWS + rt * 256, 256);
                    auto has = [&](int rt, int step) { return run.place(step) >= of[rt].x && run.place(step) < of[rt].y; };
                    wait(&bar.q_ready, segment);
                    wait(&bar.k_full[it & 1], it >> 1);
                    if (!ok) break;
                    bool some[2] = {false, false};
                    if (solo(p, run)) {
                        // scores of the next tile are made while the softmax has these
                        scores(0, 0, it & 1);
                        pair_commit(&bar.k_free[it & 1]);
                        for (int step = run.tile, buf = 0; ok && step < end; ++step, ++it, buf ^= 1) {
                            if (step + 1 < end) {
                                wait(&bar.k_full[(it + 1) & 1], (it + 1) >> 1);
                                if (!ok) break;
                                scores(0, buf ^ 1, (it + 1) & 1);
                                pair_commit(&bar.k_free[(it + 1) & 1]);
                            }
                            wait(&bar.v_full[it & 1], it >> 1);
#pragma unroll 1
                            for (int h = 0; ok && h < 2; ++h) {
                                wait(&bar.p_ready[buf][h], n[buf]);
                                if (ok) values(buf, buf, h, it & 1, !some[buf]);
                                if (ok && h == 0) pair_commit(&bar.o_done[buf]);
                                some[buf] = true;
                            }
                            ++n[buf];
                            if (ok) pair_commit(&bar.v_free[it & 1]);
                        }
                        if (ok) pair_commit(&bar.job_done);
                        continue;
                    }
#pragma unroll
                    for (int rt = 0; rt < NM; ++rt)
                        if (has(rt, run.tile)) scores(rt, rt, it & 1);
                    pair_commit(&bar.k_free[it & 1]);
                    for (int step = run.tile; ok && step < end; ++step, ++it) {
                        const bool more = step + 1 < end;
                        wait(&bar.v_full[it & 1], it >> 1);
#pragma unroll
                        for (int rt = 0; rt < NM; ++rt) {
                            if (has(rt, step)) {
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    wait(&bar.p_ready[rt][h], n[rt]);
                                    if (ok) values(rt, rt, h, it & 1, !some[rt]);
                                    if (ok && h == 0) pair_commit(&bar.o_done[rt]);
                                    some[rt] = true;
                                }
                                ++n[rt];
                            }
                            if (rt == 0 && more) wait(&bar.k_full[(it + 1) & 1], (it + 1) >> 1);
                            if (ok && more && has(rt, step + 1)) scores(rt, rt, (it + 1) & 1);
                        }
                        if (ok) {
                            pair_commit(&bar.v_free[it & 1]);
                            if (more) pair_commit(&bar.k_free[(it + 1) & 1]);
                        }
                    }
                    if (ok) pair_commit(&bar.job_done);
                }
                // products under way end before the operands' shared memory and the TMEM go
                pair_commit(&bar.last);
                const bool ended = mbar_wait(&bar.last, 0);      // also where a wait gave up before
                ok = ok && ended;
            }
            ok = __all_sync(0xffffffffu, ok);
        }
    } else {
        // ---- softmax: thread = row
        asm volatile("setmaxnreg.inc.sync.aligned.u32 " QC_SOFT_REGS ";");
        const int rt = warp >> 2;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;                     // 32 lanes of TMEM per warp
        const uint32_t s_col = tmem + lanes + rt * kTile, o_col = tmem + lanes + 256 + rt * D;
        int n = 0;                              // tiles that the row tile has had
        for (int segment = 0, joins = 0; run.left > 0; run.template next<ROWS>(p), ++segment) {
            const Sequence &s = run.s;
            const bool alone = solo(p, run);
            const int part_row = (alone ? 0 : rt * 256) + cta * 128 + (threadIdx.x & 127);         // of the job's rows
            const int end = run.end(), rows = s.news * p.group, row = run.run * ROWS + part_row;
            const bool there = row < rows, active = row - lane < rows;
            const int token = there ? row / p.group : 0, h = there ? row - token * p.group : 0;
            const int64_t out_row = (int64_t)(s.first + token) * p.n_q_heads + run.kv * p.group + h;
            const int t = s.len + token;
            const int2 seen = sees(p, s, t);
            // places that all of the warp's rows see; lo is kApart once the warp sums all weights apart: then no tile is among them
            constexpr int kApart = INT32_MAX;
            int lo = __reduce_max_sync(0xffffffffu, there ? seen.x : 0);
            const int hi = __reduce_min_sync(0xffffffffu, there ? seen.y : INT32_MAX);
            const int2 of = tiles_of_rows(p, s, run.run * ROWS + rt * 256, 256);
            if (active && !(alone && rt)) {
                const T *q = static_cast<const T *>(p.q) + (s.first + token) * p.q_token + (run.kv * p.group + h) * p.q_head;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    float v[8] = {};
                    if (there) {
                        Eight<T> e;
                        e.load(q + 8 * i);
                        e.get(v);
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] = finite_or_nan(v[j]);
                    }
                    const int x = threadIdx.x & 127;
                    Eight<T>::store(reinterpret_cast<T *>(q_op + rt * kQ + (i >> 3) * (128 * 128) + x * 128 + (((i & 7) ^ (x & 7)) * 16)), v);
                }
                fence_async();
            }
            __syncwarp();
            arrive_first(&bar.q_ready);
            float slope = 0.f;
            if constexpr ((X & kBias) != 0) slope = __ldg(p.slopes + run.kv * p.group + h) * kLog2e;
            const float top_score = X & kCap ? p.cap * kLog2e : 1.f;
            float m = -INFINITY;
            float2 l = make_float2(0.f, 0.f);
            float mz = -INFINITY, lz = 0.f;     // of weights that are summed apart
            float last = 0.f;                   // the row's largest product of the last tile
            // the last of its tiles first: what a bias by distance favours, so that references seldom move
            const int from = min(run.place(run.tile), of.y - 1), to = max(run.place(end - 1), of.x);
            const int tiles = alone ? (end - run.tile + 1 - rt) >> 1 : max(from - to + 1, 0);
            if (!active) {                      // none of the warp's rows is there: its place in the barriers is
                for (int i = 0; ok && i < tiles; ++i) {
                    ok = warp_wait(&bar.s_full[rt], n + i);
                    arrive_first(&bar.p_ready[rt][0]);
                    arrive_first(&bar.p_ready[rt][1]);
                }
            }
            // the products' sums so far, in another unit
            auto rescale = [&](float by) {
#pragma unroll 1
                for (int i = 0; i < D / 32; ++i) {
                    uint32_t o[32];
                    tmem_ld32_nowait(o_col + 32 * i, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * by);
                    tmem_st32(o_col + 32 * i, o);
                }
                tmem_wait_st();                 // a tile may rescale twice, and loads are not ordered behind stores by themselves
            };
            for (int i = 0; ok && i < (active ? tiles : 0); ++i) {
                const int tile = alone ? run.place(run.tile + 2 * i + rt) : from - i, c = (it + run.place(tile) - run.tile) & 3;
                ok = warp_poll(&bar.s_full[rt], n + i);
                if (!ok) break;
                tc_fence_after();
                if (__any_sync(0xffffffffu, last > kSoon)) {
                    // a reference that will have to go up goes now: all products that were added to the sums ended before this
                    // tile's scores were made
                    const float up = last > kSoon ? log2_below(last) - kTop : 0.f;
                    m += up;
                    const float by = ex2(-up);
                    l = mul2f(l, make_float2(by, by));
                    rescale(by);
                }
                last = 0.f;
                const uint4 ex4 = *reinterpret_cast<const uint4 *>(sm.exist[c]);
                const bool odd = tile * kTile < lo || tile * kTile + kTile > hi || (ex4.x & ex4.y & ex4.z & ex4.w) != 0xffffffffu;
                const bool plain = !__any_sync(0xffffffffu, odd || m == -INFINITY);     // every row sees every place, and has a reference
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    {
                        const int place = tile * kTile + 64 * half;
                        const float4 *kv = reinterpret_cast<const float4 *>(sm.kv[c][32 * half]);
                        const float far = X & kBias ? slope * (float)(place - t) : 0.f;      // the bias at the first place
                        // scores of places 2 i and 2 i + 1 of the half, plus `more`
                        auto biased = [&](float2 x, int i) {
                            if constexpr ((X & kBias) != 0)
                                x = add2f(x, fma2f(make_float2((float)(2 * i), (float)(2 * i + 1)), make_float2(slope, slope), make_float2(far, far)));
                            return x;
                        };
                        // cap tanh(a) = cap - 2 cap / (1 + e^2a); for small a, where that would leave few of a score's digits, by a
                        // polynomial. y = log2(e^2a). small: both are, or a NaN
                        auto capped = [&](float2 y, auto small) {
                            const float2 near = mul2f(mul2f(y, make_float2(0.5f * kLn2 * top_score, 0.5f * kLn2 * top_score)), tanh_over(y));
                            if constexpr (decltype(small)::value) return near;
                            float2 e = add2f(make_float2(ex2(y.x), ex2(y.y)), make_float2(1.f, 1.f));
                            e.x = rcp(e.x), e.y = rcp(e.y);
                            e = fma2f(e, make_float2(-2.f * top_score, -2.f * top_score), make_float2(top_score, top_score));
                            return make_float2(fabsf(y.x) < kNear ? near.x : e.x, fabsf(y.y) < kNear ? near.y : e.y);
                        };
                        auto score = [&](float2 s2, int i, float2 more) {
                            const float2 k2 = *reinterpret_cast<const float2 *>(kv + i);
                            if constexpr ((X & kCap) != 0) return biased(add2f(capped(mul2f(s2, k2), std::false_type{}), more), i);
                            return biased(fma2f(s2, k2, more), i);
                        };
                        // their weights, from scores less the reference: to the sum, and packed to w[0], w[16] for the products
                        auto weigh = [&](float2 x, int i, float2 &sum, uint32_t *w) {
                            x.x = ex2(x.x), x.y = ex2(x.y);
                            sum = add2f(sum, x);
                            x = mul2f(x, *reinterpret_cast<const float2 *>(&kv[i].z));
                            w[0] = pack2(x.x, x.y);
                            if constexpr (kTerms == 2) {
                                const float2 back = float2_of(w[0]);
                                w[16] = pack2(x.x - back.x, x.y - back.y);
                            }
                        };
                        auto pair_of = [](const uint32_t *sc, int i) { return make_float2(__uint_as_float(sc[2 * i]), __uint_as_float(sc[2 * i + 1])); };
                        // weights of 32 places to TMEM, over their scores: the terms in 16 columns each
                        auto put = [&](uint32_t col, const uint32_t *w) {
                            if constexpr (kTerms == 2)
                                tmem_st32(col, w);
                            else
                                st16(col, w);
                        };
                        bool again = true;
                        if (plain) {
                            uint32_t sc[64], w[32 * kTerms], most[2] = {0, 0};
                            tmem_ld32_nowait(s_col + 64 * half, reinterpret_cast<uint32_t(&)[32]>(sc[0]));
                            tmem_ld32_nowait(s_col + 64 * half + 32, reinterpret_cast<uint32_t(&)[32]>(sc[32]));
                            const float2 neg = make_float2(-m, -m);
                            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                            tmem_wait_ld();
                            auto weigh_all = [&](auto x_of) {
#pragma unroll
                                for (int i = 0; i < 32; ++i) {
                                    uint32_t *to = w + (i >> 4) * (16 * kTerms) + (i & 15);
                                    weigh(x_of(i), i, sum[i & 1], to);
                                    most[i & 1] = max2(most[i & 1], to[0]);
                                }
                            };
                            if constexpr ((X & kCap) != 0) {
                                // where all of the warp's are small, as with a cap well above the scores, the polynomial alone (332 us
                                // instead of 346 for single tokens over windows of 4,096); each score is the same either way
                                float big = 0.f;
#pragma unroll
                                for (int i = 0; i < 32; ++i) {
                                    const float2 y = mul2f(pair_of(sc, i), *reinterpret_cast<const float2 *>(kv + i));
                                    big = fmax3(big, fabsf(y.x), fabsf(y.y));
                                    sc[2 * i] = __float_as_uint(y.x), sc[2 * i + 1] = __float_as_uint(y.y);
                                }
                                if (__any_sync(0xffffffffu, big >= kNear))
                                    weigh_all([&](int i) { return biased(add2f(capped(pair_of(sc, i), std::false_type{}), neg), i); });
                                else
                                    weigh_all([&](int i) { return biased(add2f(capped(pair_of(sc, i), std::true_type{}), neg), i); });
                            } else {
                                weigh_all([&](int i) { return score(pair_of(sc, i), i, neg); });
                            }
                            const float2 top2 = float2_of(max2(most[0], most[1]));
                            const float top = fmaxf(top2.x, top2.y);
                            again = __any_sync(0xffffffffu, top > kMostP);
                            if (!again) {
                                last = fmaxf(last, top);
                                l = add2f(l, add2f(sum[0], sum[1]));
                                put(s_col + 64 * half, w);
                                put(s_col + 64 * half + 32, w + 16 * kTerms);
                            }
                        }
                        if (again) {
                            // step by step: the largest product, the reference, the weights; 32 places at a time
                            const uint2 ex = *reinterpret_cast<const uint2 *>(&sm.product[c][2 * half]);
                            const uint2 no = *reinterpret_cast<const uint2 *>(&sm.exist[c][2 * half]);
                            uint2 ze = *reinterpret_cast<const uint2 *>(&sm.zero[c][2 * half]);
                            const bool any_huge = ex.x != no.x || ex.y != no.y;
                            if (any_huge || lo == kApart) {
                                // all weights are summed apart, and those that were not go there; what l has from here on says nothing
                                if (lo != kApart) {
                                    const Sum z = joined({m, l.x + l.y}, {mz, lz});
                                    mz = z.ref, lz = z.w;
                                    lo = kApart;
                                }
                                l = make_float2(0.f, 0.f);
                                ze.x |= ex.x, ze.y |= ex.y;
                            }
                            const float2 *lv = reinterpret_cast<const float2 *>(&sm.lv[c][64 * half]);
                            // which of places 32 j .. the row sees
                            auto sees_of = [&](int j) {
                                const int at = place + 32 * j, a = min(max(seen.x - at, 0), 32), b = min(max(seen.y - at, 0), 32);
                                return (b == 32 ? ~0u : (1u << b) - 1u) & (a == 32 ? 0u : ~0u << a);
                            };
                            float top = -INFINITY;
#pragma unroll 1
                            for (int j = 0; j < 2; ++j) {
                                uint32_t x32[32];
                                tmem_ld32_nowait(s_col + 64 * half + 32 * j, x32);
                                const uint32_t in = sees_of(j), see = in & (j ? ex.y : ex.x), zero = in & (j ? ze.y : ze.x);
                                tmem_wait_ld();
                                float zt = mz;
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    const float2 u = score(pair_of(x32, i), 16 * j + i, make_float2(0.f, 0.f)), y = add2f(u, lv[16 * j + i]);
                                    if ((see >> (2 * i)) & 1u) top = fmaxf(top, y.x);
                                    if ((see >> (2 * i)) & 2u) top = fmaxf(top, y.y);
                                    if ((zero >> (2 * i)) & 1u) zt = fmaxf(zt, u.x);
                                    if ((zero >> (2 * i)) & 2u) zt = fmaxf(zt, u.y);
                                }
                                if (j ? ze.y : ze.x) {
                                    const float ref = zt == -INFINITY ? 0.f : zt;
                                    lz *= ex2(mz - ref);
                                    mz = zt;
#pragma unroll
                                    for (int i = 0; i < 16; ++i) {
                                        const float2 u = score(pair_of(x32, i), 16 * j + i, make_float2(-ref, -ref));
                                        if ((zero >> (2 * i)) & 1u) lz += ex2(u.x);
                                        if ((zero >> (2 * i)) & 2u) lz += ex2(u.y);
                                    }
                                }
                            }
                            const bool move = top > m + kMostLog;
                            if (__any_sync(0xffffffffu, move)) {
                                const float m2 = move ? top - kTop : m;
                                const float d = m == m2 ? 0.f : m - m2, by = ex2(d);
                                const float2 f = power_of_2(d);
                                l = mul2f(mul2f(l, make_float2(f.x, f.x)), make_float2(f.y, f.y));
                                m = m2;
                                // the first half's products may still be added to the sums
                                if (half) ok = warp_poll(&bar.o_done[rt], n + i);
                                if (!ok) break;
                                tc_fence_after();
                                if (i > 0 || half) rescale(by);             // before, there are none
                            }
                            // as above, so that a row's bits do not hang on its neighbours'
                            const float neg = m == -INFINITY ? 0.f : -m;
                            uint32_t most = 0;
                            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                            auto weigh_half = [&](auto with_huge) {
#pragma unroll 1
                                for (int j = 0; j < 2; ++j) {
                                    uint32_t x32[32], w[16 * kTerms];
                                    tmem_ld32_nowait(s_col + 64 * half + 32 * j, x32);
                                    const uint32_t see = sees_of(j) & (j ? ex.y : ex.x), big = j ? ex.y ^ no.y : ex.x ^ no.x;
                                    tmem_wait_ld();
#pragma unroll
                                    for (int i = 0; i < 16; ++i) {
                                        float2 x = score(pair_of(x32, i), 16 * j + i, make_float2(neg, neg));
                                        if (!((see >> (2 * i)) & 1u)) x.x = -INFINITY;
                                        if (!((see >> (2 * i)) & 2u)) x.y = -INFINITY;
                                        if constexpr (decltype(with_huge)::value) {
                                            if ((big >> (2 * i)) & 1u) x.x += kHugeLog;
                                            if ((big >> (2 * i)) & 2u) x.y += kHugeLog;
                                        }
                                        weigh(x, 16 * j + i, sum[i & 1], w + i);
                                        most = max2(most, w[i]);
                                    }
                                    put(s_col + 64 * half + 32 * j, w);
                                }
                            };
                            if (any_huge)
                                weigh_half(std::true_type{});
                            else
                                weigh_half(std::false_type{});
                            l = add2f(l, add2f(sum[0], sum[1]));
                            const float2 top2 = float2_of(most);
                            last = fmaxf(last, fmaxf(top2.x, top2.y));
                        }
                        tmem_wait_st();
                        tc_fence_before();
                    }
                    arrive_first(&bar.p_ready[rt][half]);
                }
            }
            ok = ok && warp_poll(&bar.job_done, segment);
            if (!ok) break;
            n += tiles;
            tc_fence_after();
            float4 *other = &sm.other[threadIdx.x & 127];
            if (alone && rt) {                  // the other warp with these rows joins both
                *other = make_float4(m, lo == kApart ? 0.f : l.x + l.y, mz, lz);
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.join);
            } else if (active) {
                const bool whole = run.tile == run.first && end == run.last;
                const int64_t part = 2 * (int64_t)unit + (segment ? 1 : 0);
                // of this warp's products, and of the other's: are there any, and their factors in the larger reference's unit
                const bool product = m > -INFINITY;
                bool product1 = false;
                float up = 1.f, up1 = 0.f, most = m;
                Sum sum = {m, lo == kApart ? 0.f : l.x + l.y}, apart = {mz, lz};
                float2 unit2 = make_float2(1.f / kScaleUnit, 1.f);      // of the products, in that of the weights
                if (alone) {
                    ok = warp_poll(&bar.join, joins);
                    if (!ok) break;
                    const float4 x = *other;
                    product1 = x.x > -INFINITY;
                    most = fmaxf(m, x.x);
                    const float2 f = product ? power_of_2(m - most) : make_float2(0.f, 0.f);
                    const float2 f1 = product1 ? power_of_2(x.x - most) : make_float2(0.f, 0.f);
                    up = f.x * f.y, up1 = f1.x * f1.y;
                    // (a NaN has no reference, and goes out)
                    const Sum both = {most, (product ? sum.w * f.x * f.y : isnan(sum.w) ? sum.w : 0.f) +
                                                (product1 ? x.y * f1.x * f1.y : isnan(x.y) ? x.y : 0.f)};
                    if (__any_sync(0xffffffffu, lz != 0.f || x.w != 0.f)) {
                        apart = joined(apart, {x.z, x.w});
                        if (apart.w != 0.f) sum = joined(sum, {x.x, x.y});
                    }
                    if (apart.w == 0.f) sum = both;
                }
                if (__any_sync(0xffffffffu, apart.w != 0.f)) {
                    sum = joined(sum, apart);
                    const float2 f = power_of_2(most == sum.ref ? 0.f : most - sum.ref);
                    unit2 = make_float2(f.x * (1.f / kScaleUnit), f.y);
                }
                const float total = sum.w;
                const bool some = total != 0.f, odd = isnan(total);
                const float by = some ? 1.f / total : 0.f;
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {
                    uint32_t o[16], o1[16];
                    tmem_ld16_nowait(o_col + 16 * c, o);
                    if (alone) tmem_ld16_nowait(o_col + D + 16 * c, o1);
                    tmem_wait_ld();
                    if (there) {
                        float v[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float x = product ? __uint_as_float(o[i]) * up : 0.f;
                            if (product1) x = fmaf(__uint_as_float(o1[i]), up1, x);
                            v[i] = odd ? total : some ? x * by * unit2.x * unit2.y : 0.f;
                        }
                        if (whole) {
                            store_row<T, 16>(static_cast<T *>(p.out) + out_row * D + 16 * c, v);
                        } else {
                            float4 *out = reinterpret_cast<float4 *>(parts.row(part, part_row) + 16 * c);
#pragma unroll
                            for (int i = 0; i < 4; ++i) out[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                        }
                    }
                }
                if (there) {
                    if (!whole)
                        *parts.stat(part, part_row) = make_float2(some ? sum.ref : -INFINITY, total);
                    else if (p.lse)
                        p.lse[out_row] = some ? (sum.ref + log2f(total)) * kLn2 : -INFINITY;
                }
            }
            joins += alone;
            tc_fence_before();
            it += end - run.tile;
        }
    }
    if (!ok && lane == 0) atomicOr(p.flags, QC_FLAG_TIMEOUT);
    griddep_launch_dependents();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp >= kProducer && warp < kProducer + 2 && !(warp == kProducer ? bar.keys : bar.values).land(plan.raw, lane) && lane == 0)
        atomicOr(p.flags, QC_FLAG_TIMEOUT);
    __syncthreads();
    cluster_sync();             // neither CTA's shared memory or TMEM is used any more
    if (warp == kMma) pair_dealloc(tmem, 512);
}

template <int FMT, int D>
ChunkPlan plan_of(const qc_ctx *c, int units) {
    using R = Raw<FMT, D>;
    ChunkPlan plan;
    plan.device = c->device;
    plan.units = units;
    const int fixed = NM * 128 * D * 2 + 2 * (kTile / 2 * D * 2) + 2 * kTile * D + (int)sizeof(Small);
    plan.raw = (227 * 1024 - fixed) / (R::kKeyBytes + R::kValueBytes);
    if (plan.raw > kMostStages) plan.raw = kMostStages;
    plan.smem = fixed + plan.raw * (R::kKeyBytes + R::kValueBytes);
    return plan;
}

template <typename T, int FMT, int D, int X>
cudaError_t launch(const qc_ctx *c, int type, const Chunk &p, int units, cudaStream_t s) {
    const ChunkPlan plan = plan_of<FMT, D>(c, units);
    const ChunkParts parts = chunk_parts_at(p.workspace, units, ROWS, D);
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(chunk_tc<T, FMT, D, X>, 227 * 1024, plan.device, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (unsigned)units);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = plan.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, chunk_tc<T, FMT, D, X>, p, parts, plan);
    if (e != cudaSuccess || units == 1) return e;
    return launch_chunk_join(p, parts, type, units, s);
}

template <typename T, int FMT, int D>
cudaError_t pick(const qc_ctx *c, int type, const Chunk &p, cudaStream_t s) {
    const int units = chunk_units(c, p.n_seq, p.n_tokens, p.group, p.max_len, p.max_new);
    if (p.cap > 0.f) return p.slopes ? launch<T, FMT, D, kCap | kBias>(c, type, p, units, s) : launch<T, FMT, D, kCap>(c, type, p, units, s);
    if (p.slopes) return launch<T, FMT, D, kBias>(c, type, p, units, s);
    return launch<T, FMT, D, kPlain>(c, type, p, units, s);
}

}  // namespace chunk

// Each of the .cu files defines one format and head dimension.
#define QC_CHUNK_TC(FMT, D)                                                                                                  \
    template <>                                                                                                              \
    cudaError_t launch_chunk_tc<FMT, D>(const qc_ctx *c, int type, const Chunk &p, cudaStream_t s) {                         \
        return type == QC_F16 ? chunk::pick<__half, FMT, D>(c, type, p, s) : chunk::pick<__nv_bfloat16, FMT, D>(c, type, p, s); \
    }

}  // namespace qc
