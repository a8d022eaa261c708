// Attention over the quantised cache for up to 64 query rows per key/value head and long prefixes: products
// on the fifth-generation tensor cores, transposed, so that places are the 128 rows of a product and the N
// query rows its columns. The tensor cores' and the softmax's time is then proportional to N, not to 128.
//
// One CTA per SM, tiles of 128 places. Roles:
//   producer (3 warps)     copies keys' and values' codes and scales, as the pages hold them, to a ring of
//                          raw stages with bulk asynchronous copies;
//   keys (4 warps)         turn codes into fp16, exactly, a lane per place, and put them into TMEM: that is
//                          where the product takes its left operand from, so the keys cross shared memory
//                          once in and once out;
//   values (4 warps)       turn codes into fp16 in shared memory, in the 128-byte swizzle;
//   MMA (1 thread)         S^T = K Q^T, then O^T += V^T P^T;
//   softmax (4 warps)      a thread per place: N scores from TMEM, N weights to shared memory.
// Scores, keys, values and weights are double-buffered.
//
// What bounds it: the pages; then shared memory's bandwidth (a tile's codes in and out, its values in fp16
// in and out) and the issue slots of the conversion.
//
// Arithmetic is that of qc_attend_rows.cu: exact products of fp16 operands, float32 sums; weights relative
// to a reference that moves only when a score passes it by 2^3, times the values' row scale, in fp16. Their
// unit is a power of two (2^12 over the bound of the values' scales) and is folded into the exponent, so
// the running sum l is in that unit too. fp16 holds a weight to 11 bits down to 2^-29 of the heaviest. A
// reference concerns all places: the four softmax warps agree before each tile's weights on whether one has
// to move, and a thread sums l over its own places until the job ends.
#include <math.h>

#include "qc_tc.cuh"

namespace qc {
namespace {

constexpr float kLag = 3.f;
constexpr int kTop = 12;                // weights' unit: 2^12 over the scales' bound
constexpr float kNone = -1e30f;         // reference of a row that has seen nothing

constexpr int kSoft = 4, kKeys = 4, kValues = 8, kProducer = 12, kMma = kProducer + kProducers, kThreads = 32 * (kMma + 1);

struct Bars {
    RawRing raw;
    uint64_t k_full[2], k_free[2], v_full[2], v_free[2], s_full[2], p_ready[2], o_done, q_ready, last;
};

template <int N>
struct Small {
    Bars b;
    alignas(16) float ks[4][kTile], vs[2][kTile];       // scales of a tile's places (keys': times scale * log2 e)
    alignas(16) uint32_t exist[4][4];                   // places that exist
    alignas(16) float vtop[2][4];                       // largest values' scale of each quarter
    alignas(16) float mm[N], down[N], by[N];            // rows: reference less the unit's log2; power of two of the query; rescale
    float most[4][N];                       // warps' maxima
    int node[N];                            // rows' nodes; -1: no such row
    Walk start;
    uint32_t tmem;
};

struct Plan {
    int device;
    int row_tiles;      // tiles of N rows per head
    int n;
    int raw;            // raw stages
    int units;          // CTAs
    int smem;
};

// Order-preserving integers of floats, for the warp's maximum.
__device__ __forceinline__ float warp_max(float x) {
    int i = __float_as_int(x);
    i ^= (i >> 31) & 0x7fffffff;
    i = __reduce_max_sync(0xffffffffu, i);
    i ^= (i >> 31) & 0x7fffffff;
    return __int_as_float(i);
}

// 16 consecutive float columns of the thread's lane.
__device__ __forceinline__ void load16(uint32_t at, uint32_t (&r)[16]) {
    tmem_ld16_nowait(at, r);
    tmem_wait_ld();
}

template <typename T, int FMT, int D, int N>
__global__ void __launch_bounds__(kThreads, 1) attend_cols(const Attend p, const Parts parts, const Plan plan) {
    using I = Item<FMT, D>;
    constexpr int kV = kTile * D * 2, kP = N * kTile * 2, kQ = N * D * 2;
    constexpr int kTmemK = 0, kTmemS = 128, kTmemO = 128 + 2 * N;       // columns: keys 2 x 64, scores 2 x N, output N
    constexpr int kCols = kTmemO + N <= 256 ? 256 : 512;
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char *v_op = smem, *p_op = v_op + 2 * kV, *q_op = p_op + 2 * kP, *raw = q_op + kQ;
    Small<N> &sm = *reinterpret_cast<Small<N> *>(raw + plan.raw * I::kBytes);
    Bars &bar = sm.b;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int R = p.n_nodes * p.group, jobs = p.g.heads * plan.row_tiles;

    if (warp == kMma) {
        if (lane == 0) {
            bar.raw.init(plan.raw);
            for (int i = 0; i < 2; ++i) {
                mbar_init(&bar.k_full[i], 4);
                mbar_init(&bar.k_free[i], 1);
                mbar_init(&bar.v_full[i], 4);
                mbar_init(&bar.v_free[i], 1);
                mbar_init(&bar.s_full[i], 1);
                mbar_init(&bar.p_ready[i], 4);
            }
            mbar_init(&bar.o_done, 1);
            mbar_init(&bar.q_ready, 4);
            mbar_init(&bar.last, 1);
            fence_barrier_init();
        }
        __syncwarp();
        tmem_alloc(&sm.tmem, kCols);
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
    } else if (warp >= kKeys && warp < kKeys + 8) {
        // ---- converters: keys (even raw stages in order) and values (odd)
        const bool values = warp >= kValues;
        const int quarter = warp & 3, t = quarter * 32 + lane;
        const bool short_runs = I::kRow == 32 && p.g.page == 16;
        const float up = p.scale * kLog2e;
        int stage = values ? 1 % plan.raw : 0;
        uint32_t phase = values ? (1 / plan.raw) & 1 : 0;
        for (; ok && run.begin(); run.next(p, jobs, kTile)) {
            const int end = run.w.n.x + run.w.n.y;
            for (int tile = run.from; tile < run.end; ++tile, ++it) {
                const int b = it & 1;
                // the operand's last reader, then the codes
                if (it >= 2) ok = warp_wait(values ? &bar.v_free[b] : &bar.k_free[b], (it >> 1) - 1);
                ok = ok && warp_wait(&bar.raw.full[stage], phase);
                if (!ok) break;
                const unsigned char *st = raw + stage * I::kBytes;
                const bool good = tile * kTile + t < end && !((bar.raw.bad[stage] >> (t >> 4)) & 1u);
                const float s = good ? *reinterpret_cast<const float *>(st + I::kCodes + 4 * t) : 0.f;
                const unsigned char *block = st + I::kCodes + 4 * kTile + t * I::kBlocks;
                if (values) {
                    sm.vs[b][t] = s;
                    const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(s));
                    if (lane == 0) sm.vtop[b][quarter] = __uint_as_float(m);
                    unsigned char *out = v_op + b * kV;
                    convert_row<FMT, D>(st, block, t, short_runs, good, [&](int q, const uint32_t(&h)[4]) { put_piece(out, t, q, h); });
                    fence_proxy_async_smem();
                } else {
                    sm.ks[it & 3][t] = s * up;
                    const uint32_t e = __ballot_sync(0xffffffffu, good);
                    if (lane == 0) sm.exist[it & 3][quarter] = e;
                    uint32_t r[D / 2];
                    convert_row<FMT, D>(st, block, t, short_runs, good, [&](int q, const uint32_t(&h)[4]) {
                        r[4 * q] = h[0], r[4 * q + 1] = h[1], r[4 * q + 2] = h[2], r[4 * q + 3] = h[3];
                    });
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) tmem_st32(tmem + ((uint32_t)quarter << 21) + kTmemK + 64 * b + 32 * c, r + 32 * c);
                    tmem_wait_st();
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bar.raw.empty[stage]);
                    mbar_arrive(values ? &bar.v_full[b] : &bar.k_full[b]);
                }
                stage += 2;
                if (stage >= plan.raw) stage -= plan.raw, phase ^= 1u;
            }
        }
    } else if (warp == kMma) {
        if (elect_one()) {          // one thread, from here to the end
            // values: the output dimension (rows of the product) contiguous; d = 64 fills the 128 rows twice
            const uint32_t qk = idesc_f16_f32(128, N), pv = idesc_f16_f32(128, N) | 1u << 15;
            constexpr uint32_t kNext = D == 64 ? 0 : kTile * 128;
            const uint32_t qa = smem_addr(q_op), va = smem_addr(v_op), pa = smem_addr(p_op);
            auto scores = [&](int b) {          // S^T[b] = K[b] Q^T
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    mma_f16_ts(tmem + kTmemS + b * N, tmem + kTmemK + 64 * b + 8 * k, sdesc_sw128(qa + (k >> 2) * (N * 128) + (k & 3) * 32), qk, k > 0);
                mma_commit(&bar.s_full[b]);
                mma_commit(&bar.k_free[b]);
            };
            auto values = [&](int b, bool first) {      // O^T (+)= V[b]^T P[b]^T
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                    mma_f16(tmem + kTmemO, sdesc_sw128_mn(va + b * kV + k * 2048, kNext),
                            sdesc_sw128(pa + b * kP + (k >> 2) * (N * 128) + (k & 3) * 32), pv, !first || k > 0);
                mma_commit(&bar.o_done);
                mma_commit(&bar.v_free[b]);
            };
            auto wait = [&](uint64_t *b, uint32_t parity) { ok = ok && wait_phase(b, parity); };
            int segment = 0;
            for (; ok && run.begin(); run.next(p, jobs, kTile), ++segment) {
                wait(&bar.q_ready, segment);
                wait(&bar.k_full[it & 1], it >> 1);
                if (!ok) break;
                scores(it & 1);
                for (int tile = run.from; ok && tile < run.end; ++tile, ++it) {
                    if (tile + 1 < run.end) {
                        wait(&bar.k_full[(it + 1) & 1], (it + 1) >> 1);
                        if (ok) scores((it + 1) & 1);
                    }
                    wait(&bar.v_full[it & 1], it >> 1);
                    wait(&bar.p_ready[it & 1], it >> 1);
                    if (ok) values(it & 1, tile == run.from);
                }
            }
            // products under way end before the operands' shared memory and the TMEM go
            mma_commit(&bar.last);
            ok = mbar_wait(&bar.last, 0) && ok;
        }
        ok = __all_sync(0xffffffffu, ok);
    } else {
        // ---- softmax: thread = place of the tile; at the job's end, thread = output element
        const int t = threadIdx.x;
        const uint32_t lanes = (uint32_t)warp << 21;
        constexpr int kHalf = N < 32 ? N : 32;
        int segment = 0;
        for (; run.begin(); run.next(p, jobs, kTile), ++segment) {
            const Walk &w = run.w;
            const int kv = w.job / plan.row_tiles, r0 = w.job % plan.row_tiles * N;
            // queries: four threads a row would be idle most of the time; N threads take one each
            for (int r = t; r < N; r += 128) {
                const int row = r0 + r;
                const bool there = row < R;
                const int node = there ? row / p.group : 0, h = there ? row % p.group : 0;
                const T *q = static_cast<const T *>(p.q) + w.b * p.q_seq + node * p.q_node + (kv * p.group + h) * p.q_head;
                sm.down[r] = put_query<T, D>(q, there, q_op, r, N);
                sm.node[r] = there && node < w.n.y ? node : -1;
                sm.mm[r] = kNone;
            }
            fence_proxy_async_smem();
            named_sync(1, 128);
            if (lane == 0) mbar_arrive(&bar.q_ready);
            float ref = 0.f, l[N];
            int e = 0;                          // log2 of the weights' unit
#pragma unroll
            for (int i = 0; i < N; ++i) l[i] = 0.f;
            for (int tile = run.from; tile < run.end; ++tile, ++it) {
                const int b = it & 1;
                bool mine = ok && warp_wait(&bar.v_full[b], it >> 1) && warp_wait(&bar.s_full[b], it >> 1);
                tc_fence_after();
                const float ks = sm.ks[it & 3][t], vs = sm.vs[b][t];
                const float4 vt = *reinterpret_cast<const float4 *>(sm.vtop[b]);
                const uint4 ex = *reinterpret_cast<const uint4 *>(sm.exist[it & 3]);
                const float vtop = fmaxf(fmax3(vt.x, vt.y, vt.z), vt.w);
                const bool mask = tile * kTile + kTile > w.n.x || (ex.x & ex.y & ex.z & ex.w) != 0xffffffffu;
                // rows that see this place
                uint32_t sees[N / kHalf];
#pragma unroll
                for (int c = 0; c < N / kHalf; ++c) sees[c] = 0xffffffffu;
                if (mask) {
                    // a lane looks the warp's 32 places up for its rows; then each row's bits go round
                    const uint32_t exist = sm.exist[it & 3][warp];
#pragma unroll
                    for (int c = 0; c < N / kHalf; ++c) {
                        const int node = lane < kHalf ? sm.node[c * kHalf + lane] : -1;
                        const uint32_t *tree = p.tree ? p.tree + ((int64_t)w.b * p.n_nodes + max(node, 0)) * p.words : nullptr;
                        uint32_t win = window(p, tree, max(node, 0), w.n.y, tile * kTile + 32 * warp - w.n.x) & exist;
                        if (node < 0) win = 0;
                        sees[c] = 0;
#pragma unroll
                        for (int i = 0; i < kHalf; ++i) sees[c] |= ((__shfl_sync(0xffffffffu, win, i) >> lane) & 1u) << i;
                    }
                }
                const uint32_t at = tmem + lanes + kTmemS + b * N;
                // exponents of half c's weights: s * ks * down - mm
                float x[kHalf];
                auto exponents = [&](int c) {
                    uint32_t s[kHalf];
                    if constexpr (kHalf == 32) {
                        tmem_ld32_nowait(at + 32 * c, s);
                    } else {
                        tmem_ld16_nowait(at, s);
                    }
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < kHalf; i += 4) {
                        const float4 mm = *reinterpret_cast<const float4 *>(&sm.mm[c * kHalf + i]);
                        float4 dn = make_float4(1.f, 1.f, 1.f, 1.f);
                        if constexpr (std::is_same<T, __nv_bfloat16>::value) dn = *reinterpret_cast<const float4 *>(&sm.down[c * kHalf + i]);
                        x[i] = fmaf(__uint_as_float(s[i]) * ks, dn.x, -mm.x);
                        x[i + 1] = fmaf(__uint_as_float(s[i + 1]) * ks, dn.y, -mm.y);
                        x[i + 2] = fmaf(__uint_as_float(s[i + 2]) * ks, dn.z, -mm.z);
                        x[i + 3] = fmaf(__uint_as_float(s[i + 3]) * ks, dn.w, -mm.w);
                    }
                    if (mask) {
#pragma unroll
                        for (int i = 0; i < kHalf; ++i)
                            if (!((sees[c] >> i) & 1u)) x[i] = -INFINITY;
                    }
                };
                float top = -INFINITY;
#pragma unroll
                for (int c = 0; c < N / kHalf; ++c) {
                    exponents(c);
                    float a0 = -INFINITY, a1 = -INFINITY;
#pragma unroll
                    for (int i = 0; i < kHalf; i += 4) a0 = fmax3(a0, x[i], x[i + 1]), a1 = fmax3(a1, x[i + 2], x[i + 3]);
                    top = fmax3(top, a0, a1);
                }
                // all four warps: may the references stay? (one that gave up ends the others, too)
                const bool stay = named_sync_and(1, 128, mine && !(top > kLag + (float)e || vtop > ref));
                if (!stay) {
                    ok = named_sync_and(2, 128, mine);
                    if (!ok) break;
                    const float ref2 = fmaxf(ref, fmaxf(power_above(vtop), 3.2311742677852644e-27f));     // at least 2^-88
                    const int e2 = kTop + 127 - (int)(__float_as_uint(ref2) >> 23);
                    // largest scores of the tile, row by row
#pragma unroll
                    for (int c = 0; c < N / 16; ++c) {
                        uint32_t s[16];
                        load16(at + 16 * c, s);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const bool see = (sees[c * 16 / kHalf] >> ((c * 16 + i) % kHalf)) & 1u;
                            const float y = warp_max(see ? __uint_as_float(s[i]) * ks * sm.down[16 * c + i] : -INFINITY);
                            if (lane == 0) sm.most[warp][16 * c + i] = y;
                        }
                    }
                    named_sync(1, 128);
                    if (t < N) {
                        const float y = fmaxf(fmax3(sm.most[0][t], sm.most[1][t], sm.most[2][t]), sm.most[3][t]);
                        const float old = sm.mm[t];
                        const bool seen = old > 0.5f * kNone;
                        const float m = seen ? old + (float)e : -INFINITY;
                        const float m2 = y > m + kLag ? y + kLag : m;
                        sm.by[t] = seen ? ex2(m - m2 + (float)(e2 - e)) : 0.f;
                        sm.mm[t] = m2 == -INFINITY ? kNone : m2 - (float)e2;
                    }
                    named_sync(1, 128);
#pragma unroll
                    for (int i = 0; i < N; ++i) l[i] *= sm.by[i];
                    if (tile > run.from) {
                        mine = warp_wait(&bar.o_done, it - 1);
                        tc_fence_after();
#pragma unroll
                        for (int c = 0; c < N / 16; ++c) {
                            uint32_t o[16];
                            load16(tmem + lanes + kTmemO + 16 * c, o);
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * sm.by[16 * c + i]);
                            tmem_st16(tmem + lanes + kTmemO + 16 * c, o);
                        }
                        tmem_wait_st();
                        ok = named_sync_and(2, 128, mine);
                        if (!ok) break;
                    }
                    ref = ref2;
                    e = e2;
                }
                unsigned char *to = p_op + b * kP + (t >> 6) * (N * 128) + (t & 7) * 2;
                const int piece = (t & 63) >> 3;
#pragma unroll
                for (int c = 0; c < N / kHalf; ++c) {
                    if (N > kHalf || !stay) exponents(c);
#pragma unroll
                    for (int i = 0; i < kHalf; i += 2) {
                        const float p0 = ex2(x[i]), p1 = ex2(x[i + 1]);
                        l[c * kHalf + i] += p0;
                        l[c * kHalf + i + 1] += p1;
                        const uint32_t h = pack2(p0 * vs, p1 * vs);
                        const int r = c * kHalf + i;
                        *reinterpret_cast<uint16_t *>(to + r * 128 + ((piece ^ (r & 7)) * 16)) = (uint16_t)h;
                        *reinterpret_cast<uint16_t *>(to + (r + 1) * 128 + ((piece ^ ((r + 1) & 7)) * 16)) = (uint16_t)(h >> 16);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.p_ready[b]);
            }
            if (ok) ok = warp_wait(&bar.o_done, it - 1);
            ok = named_sync_and(2, 128, ok);
            if (!ok) break;
            tc_fence_after();
            // sums over the places: the warp's, then all four
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float s = l[i];
#pragma unroll
                for (int x = 16; x >= 1; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
                if (lane == 0) sm.most[warp][i] = s;
            }
            named_sync(1, 128);
            const bool whole = run.from == 0 && run.end == w.tiles;
            const int64_t part = 2 * (int64_t)blockIdx.x + (segment ? 1 : 0);
            const float unit = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll 1
            for (int c = 0; c < N / 16; ++c) {
                uint32_t o[16];
                load16(tmem + lanes + kTmemO + 16 * c, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int r = 16 * c + i, row = r0 + r;
                    if (row >= R) break;
                    const float sum = (sm.most[0][r] + sm.most[1][r]) + (sm.most[2][r] + sm.most[3][r]);
                    const bool some = sum > 0.f && sm.node[r] >= 0;
                    const float v = __uint_as_float(o[i]);
                    if (whole) {
                        const int node = row / p.group, h = row % p.group;
                        const int64_t to = ((int64_t)w.b * p.n_nodes + node) * p.n_q_heads + kv * p.group + h;
                        if (t < D) put_one(static_cast<T *>(p.out) + to * D + t, some ? v / sum : 0.f);
                        if (t == 0 && p.lse) p.lse[to] = some ? (sm.mm[r] + log2f(sum)) * kLn2 : -INFINITY;
                    } else {
                        if (t < D) parts.row(part, r)[t] = v * unit;
                        if (t == 0) *parts.stat(part, r) = some ? make_float2(sm.mm[r] + (float)e, sum * unit) : make_float2(-INFINITY, 0.f);
                    }
                }
            }
            tc_fence_before();
            named_sync(1, 128);         // the rows' arrays are free again
        }
    }
    if (!ok && lane == 0) atomicOr(p.flags, QC_FLAG_TIMEOUT);
    griddep_launch_dependents();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kProducer && !bar.raw.land(plan.raw, lane) && lane == 0) atomicOr(p.flags, QC_FLAG_TIMEOUT);
    if (warp == kMma) tmem_dealloc(tmem, kCols);
}

template <int FMT, int D, int N>
int fixed_smem() {
    return 2 * kTile * D * 2 + 2 * N * kTile * 2 + N * D * 2 + (int)sizeof(Small<N>);
}

template <int FMT, int D>
Plan plan_cols(const qc_ctx *c, int rows, int64_t n_seq, int64_t max_len, int n_nodes) {
    using I = Item<FMT, D>;
    Plan p;
    p.device = c->device;
    p.n = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    p.row_tiles = (rows + p.n - 1) / p.n;
    const int fixed = p.n == 16 ? fixed_smem<FMT, D, 16>() : p.n == 32 ? fixed_smem<FMT, D, 32>() : fixed_smem<FMT, D, 64>();
    p.raw = (227 * 1024 - fixed) / I::kBytes;
    if (p.raw > kMostRaw) p.raw = kMostRaw;
    p.smem = fixed + p.raw * I::kBytes;
    p.units = c->num_sms;
    const int64_t most = n_seq * c->heads * p.row_tiles * ((max_len + n_nodes + kTile - 1) / kTile);
    if (p.units > most) p.units = (int)most;
    return p;
}

template <int FMT, int D>
int64_t workspace(const qc_ctx *c, int rows, int64_t n_seq, int64_t max_len, int n_nodes) {
    const Plan p = plan_cols<FMT, D>(c, rows, n_seq, max_len, n_nodes);
    return workspace_bytes(n_seq, 2 * (int64_t)p.units, p.n, D);
}

template <typename T, int FMT, int D, int N>
cudaError_t launch(const Plan &plan, const Attend &p, int type, cudaStream_t s) {
    const Parts parts = parts_at(p.workspace, p.n_seq, 2 * (int64_t)plan.units, N, D);
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(attend_cols<T, FMT, D, N>, 227 * 1024, plan.device, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)plan.units);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = plan.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, attend_cols<T, FMT, D, N>, p, parts, plan);
    if (e != cudaSuccess) return e;
    return launch_join(p, parts, type, plan.row_tiles, kTile, plan.units, s);
}

template <typename T, int FMT, int D>
cudaError_t pick_n(const qc_ctx *c, int type, const Attend &p, cudaStream_t s) {
    const Plan plan = plan_cols<FMT, D>(c, p.n_nodes * p.group, p.n_seq, p.max_len, p.n_nodes);
    return plan.n == 16   ? launch<T, FMT, D, 16>(plan, p, type, s)
           : plan.n == 32 ? launch<T, FMT, D, 32>(plan, p, type, s)
                          : launch<T, FMT, D, 64>(plan, p, type, s);
}

template <typename T>
cudaError_t pick(const qc_ctx *c, int type, const Attend &p, cudaStream_t s) {
    if (c->d == 64)
        return c->fmt == QC_INT8   ? pick_n<T, QC_INT8, 64>(c, type, p, s)
               : c->fmt == QC_E4M3 ? pick_n<T, QC_E4M3, 64>(c, type, p, s)
                                   : pick_n<T, QC_E2M1, 64>(c, type, p, s);
    return c->fmt == QC_INT8   ? pick_n<T, QC_INT8, 128>(c, type, p, s)
           : c->fmt == QC_E4M3 ? pick_n<T, QC_E4M3, 128>(c, type, p, s)
                               : pick_n<T, QC_E2M1, 128>(c, type, p, s);
}

}  // namespace

cudaError_t launch_attend_cols(const qc_ctx *c, int type, const Attend &p, cudaStream_t s) {
    return type == QC_F16 ? pick<__half>(c, type, p, s) : pick<__nv_bfloat16>(c, type, p, s);
}

int64_t cols_workspace(const qc_ctx *c, int64_t n_seq, int n_nodes, int n_q_heads, int64_t max_len) {
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
