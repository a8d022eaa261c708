// Attention over the quantised cache for many query rows per key/value head over long prefixes: products on
// the fifth-generation tensor cores.
//
// One CTA per SM; NM row tiles of 128 query rows, tiles of 128 places. Roles:
//   producer (3 warps)   copies keys' or values' codes and scales of a tile, as the pages hold them, to a
//                        ring of raw stages with bulk asynchronous copies;
//   converters (4 warps) turn a tile's codes into fp16, exactly, in the tensor cores' 128-byte swizzle: a
//                        lane takes a whole row (place), which keeps loads and stores free of bank
//                        conflicts;
//   MMA (1 thread)       S = Q K^T into TMEM, then O += P V with P read from TMEM;
//   softmax (4 NM warps) a thread per row: scores from TMEM, weights back to TMEM as fp16.
// Scores and weights of a tile are two halves of 64 places, a buffer each: while a half's softmax runs, the
// tensor cores take the other half's weights and make the next tile's scores.
//
// What bounds it: the softmax's and the conversion's issue slots and latency, with 256 rows 710 TFLOP/s of the
// two products (37 % of a large matrix product's rate; 0.387 ms for 256 bf16 rows over 8 x 32,768 int8 places, 8
// heads). A tile's half of 64 scores takes a softmax warp about 1,800 cycles, an operand's conversion a warp
// about 1,300.
//
// Arithmetic is that of qc_attend_rows.cuh: exact products of fp16 operands, float32 sums; weights relative to a
// reference that is put 2^3 above a score that passes it, times the values' row scale, in fp16 (two of them for
// fp16 outputs). The values' scales of a job are multiplied by the power of two that brings those of its first tile
// to 2^12. From there each row's products have a power of two of their own, folded into the exponent (the running
// sum l is in it too; as a rule it is 1, so that weights keep their bits). It follows the row's largest product,
// which it keeps between 2^4 and fp16's largest, whatever the values of places that the row does not see or gives no
// weight. So fp16's least step of 2^-24 is 2^-28 of the largest product or less; lighter ones are not followed further
// here, where prefixes are long. (One unit per warp, from the scales' bound alone: 0.380 ms instead of 0.387, and rows lost
// whose values were 2^-34 of the largest.)
#include <math.h>

#include "qc_attend.cuh"
#include "qc_tc.cuh"

namespace qc {
namespace {

using namespace fq::sm100;

// A score may pass the row's reference by kLag (base 2), which is what fp16 holds; one that passes it by kSoon has
// the reference moved with the next half tile, which costs the sums' rescaling but no second sweep.
constexpr float kLag = 3.9f, kSoon = 2.f;
constexpr float kHead = 3.f;            // how far above the largest score a new reference is put
// A row's unit 2^e is such that its largest product of a weight and its value's scale lies between 2^kFaint and 2^kMost.
constexpr int kTop = 12;                // a new unit brings the scales, or the largest product, up to 2^kTop
constexpr int kMostUnit = 100;          // sums of weights in the unit stay in float32
constexpr float kMostScale = 8.507059173023462e37f;     // 2^126
constexpr float kFaint = 4.f, kMost = 15.95f;

template <int D>
constexpr int kOperand = kTile * D * 2;     // bytes of one fp16 operand tile

struct Bars {
    RawRing raw;
    uint64_t k_full, k_free, v_full[2], v_free[2], s_full[4], p_ready[4], o_done[2], job_done, q_ready, last;
};

struct Small {
    Bars b;
    alignas(16) float ks[4][kTile], vs[4][kTile];       // scales of a tile's places (keys': times scale * log2 e)
    alignas(16) uint32_t exist[4][4];                   // places that exist
    alignas(16) float vtop[4][4], vleast[4][4];         // log2 of each quarter's largest and least values' scale
    float base[2];                                      // what a job's values' scales are multiplied by
    Walk start;
    uint32_t tmem;
};

__device__ __forceinline__ float lg2(float x) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

struct Plan {
    int device;
    int row_tiles;      // tiles of 128 NM rows per head
    int nm;
    int raw;            // raw stages
    int units;          // CTAs
    int smem;
};

template <typename T, int FMT, int D, int NM>
__global__ void __launch_bounds__(32 * (4 * NM + 5 + kProducers), 1) attend_tc(const Attend p, const Parts parts, const Plan plan) {
    using I = Item<FMT, D>;
    // A weight to 11 bits, and for fp16 outputs what that leaves, to 22: with 11 an fp16 output was 1.5 to 1.7 times
    // as far from 64 bits as its own rounding is, bf16's eight bits hide it. (Trees of 16, e4m3: 31.5 us with one
    // term, 35.3 with two, 36.6 with units of the rows' own.)
    constexpr int kTerms = std::is_same<T, __half>::value ? 2 : 1;
    constexpr int kOp = kOperand<D>, kSoft = 4 * NM, kConv = kSoft, kProducer = kSoft + 4, kMma = kProducer + kProducers;
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char *q_op = smem, *k_op = q_op + NM * kOp, *v_op = k_op + kOp, *raw = v_op + 2 * kOp;
    Small &sm = *reinterpret_cast<Small *>(raw + plan.raw * I::kBytes);
    Bars &bar = sm.b;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int R = p.n_nodes * p.group, jobs = p.g.heads * plan.row_tiles;

    if (warp == kMma) {
        if (lane == 0) {
            bar.raw.init(plan.raw);
            mbar_init(&bar.k_full, 4);
            mbar_init(&bar.k_free, 1);
            for (int i = 0; i < 2; ++i) {
                mbar_init(&bar.v_full[i], 4);
                mbar_init(&bar.v_free[i], 1);
                mbar_init(&bar.o_done[i], 1);
            }
            for (int i = 0; i < 4; ++i) {
                mbar_init(&bar.s_full[i], 1);
                mbar_init(&bar.p_ready[i], 4);
            }
            mbar_init(&bar.q_ready, kSoft);
            mbar_init(&bar.job_done, 1);
            mbar_init(&bar.last, 1);
            fence_barrier_init();
        }
        __syncwarp();
        tmem_alloc(&sm.tmem, 512);
    }
    griddep_wait();
    if (warp == kProducer) {
        const int64_t total = all_tiles(p, kTile, lane) * jobs, per = run_length(total, plan.units), at = per * blockIdx.x;
        if (blockIdx.x == 0) write_before(p, parts.before, jobs, kTile, lane);
        const Walk w = find(p, at, at < total ? (total - at < per ? total - at : per) : 0, jobs, kTile, lane);
        if (lane == 0) sm.start = w;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    Run run;
    run.w = sm.start;
    bool ok = true;
    int it = 0;                 // tiles so far, over all jobs of the run

    if (warp >= kProducer && warp < kProducer + kProducers) {
        ok = produce<FMT, D>(p, run, jobs, plan.row_tiles, plan.raw, raw, bar.raw, warp - kProducer, lane);
    } else if (warp >= kConv && warp < kConv + 4) {
        const int quarter = warp - kConv, t = quarter * 32 + lane;
        const bool short_runs = I::kRow == 32 && p.g.page == 16;
        const float up = p.scale * kLog2e;
        int stage = 0, segment = 0;
        uint32_t phase = 0;
        float base = 1.f;
        for (; ok && run.begin(); run.next(p, jobs, kTile), ++segment) {
            const int end = run.w.n.x + run.w.n.y;
            for (int tile = run.from; ok && tile < run.end; ++tile, ++it) {
#pragma unroll 1
                for (int which = 0; which < 2; ++which) {
                    // the operand's last reader, then the codes
                    if (which == 0) {
                        if (it >= 1) ok = ok && warp_wait(&bar.k_free, it - 1);
                    } else {
                        if (it >= 2) ok = ok && warp_wait(&bar.v_free[it & 1], (it >> 1) - 1);
                    }
                    ok = ok && warp_wait(&bar.raw.full[stage], phase);
                    if (!ok) break;
                    const unsigned char *st = raw + stage * I::kBytes;
                    auto is_there = [&](int i) { return tile * kTile + i < end && !((bar.raw.bad[stage] >> (i >> 4)) & 1u); };
                    const bool good = is_there(t);
                    if (which == 0) {
                        // the scales, the values' too: the softmax need not wait for the values
                        const float *scale = reinterpret_cast<const float *>(st + I::kScales);
                        if (tile == run.from) {     // the first tile's scales to 2^kTop, a power of two for the whole job
                            float top = 0.f;
                            for (int i = lane; i < kTile; i += 32) top = fmaxf(top, is_there(i) ? scale[kTile + i] : 0.f);
                            const int x = (int)(__float_as_uint(power_above(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top))))) >> 23);
                            base = x ? __uint_as_float((uint32_t)min(max(127 + kTop + 127 - x, 27), 227) << 23) : 1.f;
                            if (t == 0) sm.base[segment & 1] = base;
                        }
                        const float vs = good ? fminf(scale[kTile + t] * base, kMostScale) : 0.f;
                        sm.ks[it & 3][t] = good ? scale[t] * up : 0.f;
                        sm.vs[it & 3][t] = vs;
                        const uint32_t e = __ballot_sync(0xffffffffu, good), bits = __float_as_uint(vs);
                        const uint32_t most = __reduce_max_sync(0xffffffffu, bits), least = __reduce_min_sync(0xffffffffu, bits);
                        if (lane == 0) {
                            sm.exist[it & 3][quarter] = e;
                            sm.vtop[it & 3][quarter] = lg2(__uint_as_float(most));
                            sm.vleast[it & 3][quarter] = lg2(__uint_as_float(least));
                        }
                    }
                    unsigned char *out = which == 0 ? k_op : v_op + (it & 1) * kOp;
                    convert_row<FMT, D>(st, st + I::kBlockScales + t * I::kBlocks, t, short_runs, good,
                                        [&](int q, const uint32_t(&h)[4]) { put_piece(out, t, q, h); });
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&bar.raw.empty[stage]);
                        mbar_arrive(which == 0 ? &bar.k_full : &bar.v_full[it & 1]);
                    }
                    if (++stage == plan.raw) stage = 0, phase ^= 1u;
                }
            }
        }
    } else if (warp == kMma) {
        if (elect_one()) {          // one thread, from here to the end
            const uint32_t qk = idesc_f16_f32(128, 64), pv = idesc_f16_f32(128, D) | 1u << 16;      // values: output dimension contiguous
            const uint32_t qa = smem_addr(q_op), ka = smem_addr(k_op), va = smem_addr(v_op);
            auto scores = [&](int rt, int h) {          // S[rt][h] = Q[rt] K[half h]^T
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = (k >> 2) * (kTile * 128) + (k & 3) * 32;
                    mma_f16(tmem + (2 * rt + h) * 64, sdesc_sw128(qa + rt * kOp + off), sdesc_sw128(ka + h * 8192 + off), qk, k > 0);
                }
                mma_commit(&bar.s_full[2 * rt + h]);
                if (rt == NM - 1 && h == 1) mma_commit(&bar.k_free);
            };
            auto values = [&](int rt, int h, int vb, bool first) {      // O[rt] (+)= P[rt][h] V[vb][half h]
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 4 * kTerms; ++k)         // the weights' terms one after the other
                    mma_f16_ts(tmem + 256 + rt * 128, tmem + (2 * rt + h) * 64 + 8 * k,
                               sdesc_sw128_mn(va + vb * kOp + (4 * h + (k & 3)) * 2048, kTile * 128), pv, !first || k > 0);
                mma_commit(&bar.o_done[rt]);
                if (rt == NM - 1 && h == 1) mma_commit(&bar.v_free[vb]);
            };
            auto wait = [&](uint64_t *b, uint32_t parity) { ok = ok && wait_phase(b, parity); };
            int segment = 0;
            for (; ok && run.begin(); run.next(p, jobs, kTile), ++segment) {
                wait(&bar.q_ready, segment);
                wait(&bar.k_full, it);
                if (!ok) break;
                for (int i = 0; i < 2 * NM; ++i) scores(i % NM, i / NM);
                for (int tile = run.from; ok && tile < run.end; ++tile, ++it) {
                    for (int i = 0; ok && i < 2 * NM; ++i) {
                        const int rt = i % NM, h = i / NM;
                        wait(&bar.p_ready[2 * rt + h], it);
                        if (i == 0) wait(&bar.v_full[it & 1], it >> 1);
                        if (ok) values(rt, h, it & 1, tile == run.from && h == 0);
                        if (tile + 1 < run.end) {
                            if (i == 0) wait(&bar.k_full, it + 1);
                            if (ok) scores(rt, h);
                        }
                    }
                }
                // its own barrier: two of the output's phases may end here, which parity does not tell apart
                mma_commit(&bar.job_done);
            }
            // products under way end before the operands' shared memory and the TMEM go
            mma_commit(&bar.last);
            const bool ended = mbar_wait(&bar.last, 0);      // also where a wait gave up before
            ok = ok && ended;
        }
        ok = __all_sync(0xffffffffu, ok);
    } else {
        // ---- softmax: thread = row
        const int rt = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;          // 32 lanes of TMEM per warp
        int segment = 0;
        for (; run.begin(); run.next(p, jobs, kTile), ++segment) {
            const Walk &w = run.w;
            const int kv = w.job / plan.row_tiles, row = (w.job % plan.row_tiles * NM + rt) * 128 + r;
            const bool there = row < R;
            const int node = there ? row / p.group : 0, h = there ? row % p.group : 0;
            const bool active = __any_sync(0xffffffffu, there);
            const T *q = static_cast<const T *>(p.q) + w.b * p.q_seq + node * p.q_node + (kv * p.group + h) * p.q_head;
            float down = 1.f;
            if (active) {
                down = put_query<T, D>(q, there, q_op + rt * kOp, r, 128);
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.q_ready);
            const uint32_t *tree = p.tree ? p.tree + ((int64_t)w.b * p.n_nodes + node) * p.words : nullptr;
            float m = -INFINITY;
            int e = 0;                          // log2 of the weights' unit
            float big = -INFINITY;              // log2 of the row's largest product so far, or less, in the unit
            float2 l = make_float2(0.f, 0.f);
            float soon = -INFINITY;             // the row's next reference, where one waits
            for (int tile = run.from; ok && tile < run.end; ++tile, ++it) {
                for (int half = 0; half < 2; ++half) {
                    const int buf = 2 * rt + half, place = tile * kTile + 64 * half;
                    ok = ok && warp_wait(&bar.s_full[buf], it);
                    if (!ok) break;
                    if (active) {
                        tc_fence_after();
                        const float4 vt = *reinterpret_cast<const float4 *>(sm.vtop[it & 3]);
                        const uint2 ex = *reinterpret_cast<const uint2 *>(&sm.exist[it & 3][2 * half]);
                        const bool mask = place + 64 > w.n.x || (ex.x & ex.y) != 0xffffffffu;
                        const float4 vl = *reinterpret_cast<const float4 *>(sm.vleast[it & 3]);
                        const float vtop = fmaxf(fmax3(vt.x, vt.y, vt.z), vt.w), vleast = fminf(fminf(vl.x, vl.y), fminf(vl.z, vl.w));
                        const uint32_t s_at = tmem + lanes + buf * 64;
                        uint32_t pw[32 * kTerms];
                        float2 sum;
                        float top;
                        // one pass with the reference and the unit as they are; others if a score or a product is too
                        // far from them
                        auto sweep = [&](auto masked) {
                            constexpr bool kMasked = decltype(masked)::value;
                            const float mm = (m == -INFINITY ? 0.f : m) - (float)e;
                            const float2 neg = make_float2(-mm, -mm), dn = make_float2(down, down);
                            float top1 = -INFINITY;
                            float2 sum1 = make_float2(0.f, 0.f);
                            top = -INFINITY;
                            sum = make_float2(0.f, 0.f);
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                uint32_t s[32];
                                tmem_ld32_nowait(s_at + 32 * c, s);
                                uint32_t sees = 0xffffffffu;
                                if constexpr (kMasked) {
                                    sees = window(p, tree, node, w.n.y, place + 32 * c - w.n.x) & (c == 0 ? ex.x : ex.y);
                                    if (!there || node >= w.n.y) sees = 0;
                                }
                                const float *kp = &sm.ks[it & 3][64 * half + 32 * c], *vp = &sm.vs[it & 3][64 * half + 32 * c];
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 32; i += 4) {
                                    const float4 ks = *reinterpret_cast<const float4 *>(kp + i);
                                    const float4 vs = *reinterpret_cast<const float4 *>(vp + i);
                                    float2 a = mul2f(make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), make_float2(ks.x, ks.y));
                                    float2 b = mul2f(make_float2(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])), make_float2(ks.z, ks.w));
                                    if constexpr (kMasked) {
                                        if (!((sees >> i) & 1u)) a.x = -INFINITY;
                                        if (!((sees >> (i + 1)) & 1u)) a.y = -INFINITY;
                                        if (!((sees >> (i + 2)) & 1u)) b.x = -INFINITY;
                                        if (!((sees >> (i + 3)) & 1u)) b.y = -INFINITY;
                                    }
                                    top = fmax3(top, a.x, a.y);
                                    top1 = fmax3(top1, b.x, b.y);
                                    a = fma2f(a, dn, neg);
                                    b = fma2f(b, dn, neg);
                                    a.x = ex2(a.x), a.y = ex2(a.y), b.x = ex2(b.x), b.y = ex2(b.y);
                                    sum = add2f(sum, a);
                                    sum1 = add2f(sum1, b);
                                    a = mul2f(a, make_float2(vs.x, vs.y));
                                    b = mul2f(b, make_float2(vs.z, vs.w));
                                    pw[16 * c + i / 2] = pack2(a.x, a.y);
                                    pw[16 * c + i / 2 + 1] = pack2(b.x, b.y);
                                    if constexpr (kTerms == 2) {
                                        const float2 ha = float2_of(pw[16 * c + i / 2]), hb = float2_of(pw[16 * c + i / 2 + 1]);
                                        pw[32 + 16 * c + i / 2] = pack2(a.x - ha.x, a.y - ha.y);
                                        pw[32 + 16 * c + i / 2 + 1] = pack2(b.x - hb.x, b.y - hb.y);
                                    }
                                }
                            }
                            top = fmaxf(top, top1);
                            sum = add2f(sum, sum1);
                        };
                        // the sums so far, in another unit
                        auto rescale = [&](float by) {
                            ok = ok && warp_wait(&bar.o_done[rt], 2 * it + half - 1);
                            if (!ok) return;        // products may still be added to them
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) {
                                uint32_t o[32];
                                const uint32_t at = tmem + lanes + 256 + rt * 128 + 32 * c;
                                tmem_ld32_nowait(at, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * by);
                                tmem_st32(at, o);
                            }
                        };
                        const bool sums = tile > run.from || half;      // there are some
                        float by = 1.f;
                        bool moved = __any_sync(0xffffffffu, soon > m);
                        if (moved) {
                            const float m2 = fmaxf(soon, m);
                            by = m2 == m ? 1.f : ex2(m - m2);
                            big -= m2 == m ? 0.f : m2 - m;
                            m = m2;
                        }
                        // The row's largest product lies between the heaviest place's weight times the tile's least
                        // scale (where nothing is masked) and times its largest: scores within `lower` and `upper` need
                        // no more, reference and unit serve. Others have the products looked at.
                        for (int pass = 0;; ++pass) {
                            const bool none = m == -INFINITY;
                            const float at = m - (float)e, upper = fminf(m + kLag, at + kMost - vtop);
                            float lower = mask ? INFINITY : at + kFaint - vleast;
                            if (none || big >= kFaint || vtop == -INFINITY) lower = -INFINITY;
                            if (mask)
                                sweep(std::true_type{});
                            else
                                sweep(std::false_type{});
                            top *= down;
                            if (pass == 12 || !__any_sync(0xffffffffu, top > upper || top < lower)) {
                                if (!mask) big = fmaxf(big, top - at + vleast);
                                break;
                            }
                            uint32_t t[2] = {pw[0], pw[1]};
#pragma unroll
                            for (int i = 2; i < 32; ++i) t[i & 1] = max2(t[i & 1], pw[i]);
                            const float2 f2 = float2_of(max2(t[0], t[1]));
                            const bool lag = top > m + kLag;
                            float high = big;
                            bool off = false;
                            if (!lag && !none && vtop > -INFINITY) {
                                high = fmaxf(big, lg2(fmaxf(f2.x, f2.y)));
                                // nothing to be seen even in the largest unit: back, where the sums of weights are best
                                const bool blank = high == -INFINITY && pass >= 4;
                                off = high > kMost || (blank ? e != 0 : high < kFaint && e < kMostUnit && fabsf(top) < INFINITY);
                            }
                            if (high <= kMost) big = high;
                            if (!__any_sync(0xffffffffu, lag || off)) break;
                            const float m2 = lag ? top + kHead : m;
                            int e2 = e;
                            if (none && lag)
                                e2 = vtop > -INFINITY ? min(kTop - (int)ceilf(vtop), kMostUnit) : e;
                            else if (off)       // products beyond fp16's range: a step on
                                e2 = high > kMost       ? max(e - 36, min(kTop - (int)ceilf(vtop), kMostUnit))
                                     : high > -INFINITY ? min(e + min(kTop - (int)floorf(high), 100), kMostUnit)
                                     : pass < 4         ? min(e + 36, kMostUnit)
                                                        : 0;
                            moved |= __any_sync(0xffffffffu, m2 != m || e2 != e);
                            const float d = none ? -INFINITY : m - m2 + (float)(e2 - e);
                            by *= ex2(d);
                            big += d;
                            m = m2;
                            e = e2;
                        }
                        if (moved) {
                            l.x *= by;
                            l.y *= by;
                            if (sums) rescale(by);
                            if (!ok) break;
                        }
                        soon = top > m + kSoon ? top + kHead : -INFINITY;
                        l = add2f(l, sum);
                        tmem_st32(s_at, pw);
                        if constexpr (kTerms == 2) tmem_st32(s_at + 32, pw + 32);
                        tmem_wait_st();
                        tc_fence_before();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.p_ready[buf]);
                }
            }
            ok = ok && warp_wait(&bar.job_done, segment);
            if (!ok) break;
            if (active) {
                tc_fence_after();
                const bool whole = run.from == 0 && run.end == w.tiles;
                const int64_t part = 2 * (int64_t)blockIdx.x + (segment ? 1 : 0);
                const float sum = l.x + l.y;
                const bool some = sum != 0.f && node < w.n.y;        // a NaN goes out
                // out = O / (unit base) / (l / unit); a part keeps l and O free of them
                const float unit = __uint_as_float((uint32_t)(127 - e) << 23);
                const float back = 1.f / sm.base[segment & 1], by = (whole ? (some ? 1.f / sum : 0.f) : unit) * back;
                const int64_t at = ((int64_t)w.b * p.n_nodes + node) * p.n_q_heads + kv * p.group + h;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld32_nowait(tmem + lanes + 256 + rt * 128 + 32 * c, o);
                    tmem_wait_ld();
                    if (there) {
                        float v[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = whole && !some ? 0.f : __uint_as_float(o[i]) * by;
                        if (whole) {
                            store_row<T, 32>(static_cast<T *>(p.out) + at * D + 32 * c, v);
                        } else {
                            float4 *to = reinterpret_cast<float4 *>(parts.row(part, rt * 128 + r) + 32 * c);
#pragma unroll
                            for (int i = 0; i < 8; ++i) to[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                        }
                    }
                }
                if (there) {
                    if (!whole)
                        *parts.stat(part, rt * 128 + r) = make_float2(m, sum * unit);
                    else if (p.lse)
                        p.lse[at] = some ? (m + log2f(sum * unit)) * kLn2 : -INFINITY;
                }
                tc_fence_before();
            }
        }
    }
    if (!ok && lane == 0) atomicOr(p.flags, QC_FLAG_TIMEOUT);
    griddep_launch_dependents();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kProducer && !bar.raw.land(plan.raw, lane) && lane == 0) atomicOr(p.flags, QC_FLAG_TIMEOUT);
    if (warp == kMma) tmem_dealloc(tmem, 512);
}

int units_tc(const qc_ctx *c, int row_tiles, int64_t n_seq, int64_t places) {
    const int64_t most = n_seq * c->heads * row_tiles * ((places + kTile - 1) / kTile);
    return c->num_sms > most ? (int)most : c->num_sms;
}

template <int FMT, int D>
Plan plan_tc(const qc_ctx *c, int rows, int64_t n_seq, int64_t max_len, int n_nodes) {
    using I = Item<FMT, D>;
    Plan p;
    p.device = c->device;
    p.nm = rows <= 128 ? 1 : 2;
    p.row_tiles = (rows + 128 * p.nm - 1) / (128 * p.nm);
    const int fixed = (p.nm + 3) * kOperand<D> + (int)sizeof(Small);
    p.raw = (227 * 1024 - fixed) / I::kBytes;
    if (p.raw > kMostRaw) p.raw = kMostRaw;
    p.smem = fixed + p.raw * I::kBytes;
    p.units = units_tc(c, p.row_tiles, n_seq, max_len + n_nodes);
    return p;
}

template <typename T, int FMT, int D, int NM>
cudaError_t launch(const Plan &plan, const Attend &p, int type, cudaStream_t s) {
    const Parts parts = parts_at(p.workspace, p.n_seq, 2 * (int64_t)plan.units, NM * 128, D);
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(attend_tc<T, FMT, D, NM>, 227 * 1024, plan.device, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)plan.units);
    cfg.blockDim = dim3(32 * (4 * NM + 5 + kProducers));
    cfg.dynamicSmemBytes = plan.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, attend_tc<T, FMT, D, NM>, p, parts, plan);
    if (e != cudaSuccess) return e;
    return launch_join(p, parts, type, plan.row_tiles, kTile, plan.units, s);
}

template <int FMT, int D>
cudaError_t pick(const qc_ctx *c, int type, const Attend &p, cudaStream_t s) {
    const Plan plan = plan_tc<FMT, D>(c, p.n_nodes * p.group, p.n_seq, p.max_len, p.n_nodes);
    if (type == QC_F16) return plan.nm == 1 ? launch<__half, FMT, D, 1>(plan, p, type, s) : launch<__half, FMT, D, 2>(plan, p, type, s);
    return plan.nm == 1 ? launch<__nv_bfloat16, FMT, D, 1>(plan, p, type, s) : launch<__nv_bfloat16, FMT, D, 2>(plan, p, type, s);
}

}  // namespace

cudaError_t launch_attend_tc(const qc_ctx *c, int type, const Attend &p, cudaStream_t s) {
    if (c->d == 64)
        return c->fmt == QC_INT8   ? pick<QC_INT8, 64>(c, type, p, s)
               : c->fmt == QC_E4M3 ? pick<QC_E4M3, 64>(c, type, p, s)
                                   : pick<QC_E2M1, 64>(c, type, p, s);
    return c->fmt == QC_INT8   ? pick<QC_INT8, 128>(c, type, p, s)
           : c->fmt == QC_E4M3 ? pick<QC_E4M3, 128>(c, type, p, s)
                               : pick<QC_E2M1, 128>(c, type, p, s);
}

// The most that any call of up to these sizes wants: one row tile or two.
int64_t tc_workspace(const qc_ctx *c, int64_t n_seq, int n_nodes, int n_q_heads, int64_t max_len) {
    const int rows = n_nodes * (n_q_heads / c->heads);
    const int64_t one = workspace_bytes(n_seq, 2 * (int64_t)units_tc(c, 1, n_seq, max_len + n_nodes), 128, c->d);
    if (rows <= 128) return one;
    const int64_t two = workspace_bytes(n_seq, 2 * (int64_t)units_tc(c, (rows + 255) / 256, n_seq, max_len + n_nodes), 256, c->d);
    return one > two ? one : two;
}

}  // namespace qc
