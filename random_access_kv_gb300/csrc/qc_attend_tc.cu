// Attention over the quantised cache for many query rows per key/value head or long prefixes: products
// on the fifth-generation tensor cores.
//
// One CTA per SM; NM row tiles of 128 query rows, tiles of 128 places. Roles:
//   producer (1 warp)    copies keys' or values' codes and scales of a tile, as the pages hold them, to a
//                        ring of raw stages with bulk asynchronous copies;
//   converters (4 warps) turn a tile's codes into fp16, exactly, in the tensor cores' 128-byte swizzle: a
//                        lane takes a whole row (place), which keeps loads and stores free of bank
//                        conflicts;
//   MMA (1 thread)       S = Q K^T into TMEM, then O += P V with P read from TMEM;
//   softmax (4 NM warps) a thread per row: scores from TMEM, weights back to TMEM as fp16.
// With NM = 1 the scores are double-buffered, so that the next product runs under the softmax; with NM = 2
// the two row tiles take turns.
//
// What bounds it: few rows, the pages (bytes); 128 rows, the issue slots of conversion and softmax; 256
// rows and more, tensor cores and issue slots alike.
//
// Arithmetic is that of qc_attend_rows.cu: exact products of fp16 operands, float32 sums; weights relative
// to a reference that moves only when a score passes it by 2^3, times the values' row scale, in fp16. Their
// unit is a power of two (2^12 over the bound of the values' scales) and is folded into the exponent, so
// the running sum l is in that unit too. fp16 holds a weight to 11 bits down to 2^-29 of the heaviest.
#include <math.h>

#include "qc_attend.cuh"
#include "qc_convert.cuh"

namespace qc {
namespace {

using namespace fq::sm100;

constexpr int kTile = 128;
constexpr float kLag = 3.f;
constexpr int kTop = 12;                // weights' unit: 2^12 over the scales' bound
constexpr int kMostRaw = 8;

template <int FMT, int D>
struct Item {           // a raw stage: keys or values of a tile
    static constexpr int kRow = FMT == QC_E2M1 ? D / 2 : D;
    static constexpr int kBlocks = FMT == QC_E2M1 ? D / 16 : 0;
    static constexpr int kCodes = kTile * kRow;
    static constexpr int kBytes = kTile * (kRow + 4 + kBlocks);     // codes, scales, block scales
};

template <int D>
constexpr int kOperand = kTile * D * 2;     // bytes of one fp16 operand tile

struct Bars {
    uint64_t raw_full[kMostRaw], raw_empty[kMostRaw];
    uint64_t k_full, k_free, v_full[2], v_free[2], s_full[2], p_ready[2], o_done[2], q_ready, last;
};

struct Small {
    Bars b;
    float ks[4][kTile], vs[2][kTile];       // scales of a tile's places (keys': times scale * log2 e)
    uint32_t exist[4][4];                   // places that exist
    float vtop[2][4];                       // largest values' scale of each quarter
    uint32_t raw_bad[kMostRaw];             // sixteenths of a raw stage whose page does not exist
    Walk start;
    uint32_t tmem;
};

struct Plan {
    int row_tiles;      // tiles of 128 NM rows per head
    int nm;
    int raw;            // raw stages
    int units;          // CTAs
    int smem;
};

// A place in a unit's run: what every role steps through alike.
struct Run {
    Walk w;
    int from, end;
    __device__ __forceinline__ bool begin() {
        if (w.left <= 0) return false;
        from = w.tile;
        end = (int)(w.left < w.tiles - from ? from + w.left : w.tiles);
        return true;
    }
    __device__ __forceinline__ void next(const Attend &p, int jobs) {
        w.left -= end - from;
        next_job(p, w, jobs, kTile);
    }
};

// Matrix descriptor of an operand whose rows (places) of 64 elements hold the output's dimension: groups of 8
// rows 1024 bytes apart, the next 64 elements kTile rows on.
__device__ __forceinline__ uint64_t sdesc_sw128_mn(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)((kTile * 128) >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}

__device__ __forceinline__ void mma_f16_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
        "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
        "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
        "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two float32 operations at once.
__device__ __forceinline__ float2 mul2f(float2 a, float2 b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
    return *reinterpret_cast<float2 *>(&r);
}
__device__ __forceinline__ float2 add2f(float2 a, float2 b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
    return *reinterpret_cast<float2 *>(&r);
}
__device__ __forceinline__ float2 fma2f(float2 a, float2 b, float2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(r)
        : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)), "l"(*reinterpret_cast<uint64_t *>(&c)));
    return *reinterpret_cast<float2 *>(&r);
}

// One lane's place: its raw row to fp16 at row t of an operand tile. good: the place exists (else zeros).
template <int FMT, int D>
__device__ __forceinline__ void convert_row(const unsigned char *raw, const unsigned char *block, unsigned char *out, int t, bool short_runs,
                                            bool good) {
    using I = Item<FMT, D>;
    constexpr int P = I::kRow / 16;
    const int p0 = t * P;
    uint32_t sb[2] = {0, 0};
    if constexpr (FMT == QC_E2M1) {
        if constexpr (D == 128) {
            const uint2 x = *reinterpret_cast<const uint2 *>(block);
            sb[0] = x.x, sb[1] = x.y;
        } else {
            sb[0] = *reinterpret_cast<const uint32_t *>(block);
        }
        if (!good) sb[0] = sb[1] = 0;
    }
#pragma unroll
    for (int j = 0; j < P; ++j) {
        const int p = p0 + j, phase = (p >> 3) & (short_runs ? 3 : 7);
        uint4 c = *reinterpret_cast<const uint4 *>(raw + (p ^ phase) * 16);
        if (!good) c = make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
        if constexpr (FMT == QC_E2M1) {
            // 32 codes: two blocks, four 16-byte pieces
            uint32_t s[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int b = 2 * j + i;
                s[i] = both_e4m3(__byte_perm(sb[b >> 2], 0, 0x4440 + (b & 3)));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t h[4];
                cvt_e2m1(w[i], h);
#pragma unroll
                for (int e = 0; e < 4; ++e) h[e] = mul2(h[e], s[i >> 1]);
                const int q = 4 * j + i;        // piece of the fp16 row
                *reinterpret_cast<uint4 *>(out + (q >> 3) * (kTile * 128) + t * 128 + (((q & 7) ^ (t & 7)) * 16)) =
                    make_uint4(h[0], h[1], h[2], h[3]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t h[4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t x = w[2 * i + e];
                    if constexpr (FMT == QC_INT8) {
                        const uint32_t y = x ^ 0x80808080u;
                        h[2 * e] = sub1152(__byte_perm(y, 0x64646464u, 0x4140));
                        h[2 * e + 1] = sub1152(__byte_perm(y, 0x64646464u, 0x4342));
                    } else {
                        h[2 * e] = cvt_e4m3(x);
                        h[2 * e + 1] = cvt_e4m3(x >> 16);
                    }
                }
                const int q = 2 * j + i;
                *reinterpret_cast<uint4 *>(out + (q >> 3) * (kTile * 128) + t * 128 + (((q & 7) ^ (t & 7)) * 16)) =
                    make_uint4(h[0], h[1], h[2], h[3]);
            }
        }
    }
}

// A row's query, in fp16 and brought to its range, at row r of the operand tile. Returns the power of two that
// the row's scores are multiplied by.
template <typename T, int D>
__device__ __forceinline__ float put_query(const T *q, bool there, unsigned char *out, int r) {
    float down = 1.f, f = 1.f;
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        float top = 0.f;
        if (there) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                Eight<T> e;
                float v[8];
                e.load(q + 8 * i);
                e.get(v);
#pragma unroll
                for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(v[j]));
            }
        }
        // largest magnitude to [2^13, 2^14)
        const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -100), 127);
        f = __uint_as_float((uint32_t)(13 - e + 127) << 23);
        down = __uint_as_float((uint32_t)(e - 13 + 127) << 23);
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
        float v[8] = {};
        if (there) {
            Eight<T> e;
            e.load(q + 8 * i);
            e.get(v);
        }
        *reinterpret_cast<uint4 *>(out + (i >> 3) * (kTile * 128) + r * 128 + (((i & 7) ^ (r & 7)) * 16)) =
            make_uint4(pack2(v[0] * f, v[1] * f), pack2(v[2] * f, v[3] * f), pack2(v[4] * f, v[5] * f), pack2(v[6] * f, v[7] * f));
    }
    return down;
}

template <typename T, int FMT, int D, int NM>
__global__ void __launch_bounds__(32 * (4 * NM + 6), 1) attend_tc(const Attend p, const Parts parts, const Plan plan) {
    using I = Item<FMT, D>;
    constexpr int kOp = kOperand<D>, kSoft = 4 * NM, kConv = kSoft, kProducer = kSoft + 4, kMma = kSoft + 5;
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char *q_op = smem, *k_op = q_op + NM * kOp, *v_op = k_op + kOp, *raw = v_op + 2 * kOp;
    Small &sm = *reinterpret_cast<Small *>(raw + plan.raw * I::kBytes);
    Bars &bar = sm.b;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int R = p.n_nodes * p.group, jobs = p.g.heads * plan.row_tiles;

    if (warp == kMma) {
        if (lane == 0) {
            for (int i = 0; i < plan.raw; ++i) {
                mbar_init(&bar.raw_full[i], 1);
                mbar_init(&bar.raw_empty[i], 4);
            }
            mbar_init(&bar.k_full, 4);
            mbar_init(&bar.k_free, 1);
            for (int i = 0; i < 2; ++i) {
                mbar_init(&bar.v_full[i], 4);
                mbar_init(&bar.v_free[i], 1);
                mbar_init(&bar.s_full[i], 1);
                mbar_init(&bar.p_ready[i], 4);
                mbar_init(&bar.o_done[i], 1);
            }
            mbar_init(&bar.q_ready, kSoft);
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

    if (warp == kProducer) {
        int stage = 0, used = 0;
        uint32_t phase = 0;
        const int sub = p.g.page < kTile ? p.g.page : kTile, sub_shift = p.g.shift < 7 ? p.g.shift : 7;
        const int part = lane & 7, kind = lane >> 3;
        for (; ok && run.begin(); run.next(p, jobs)) {
            const int kv = run.w.job / plan.row_tiles, end = run.w.n.x + run.w.n.y;
            const int32_t *row = p.table + run.w.b * p.table_stride;
            auto entry_of = [&](int tile) {
                const int t = tile * kTile + (part << sub_shift);
                return part < kTile / sub && kind < 3 && tile < run.end && t < end ? __ldg(row + (t >> p.g.shift)) : -1;
            };
            int entry = entry_of(run.from);
            for (int tile = run.from; ok && tile < run.end; ++tile) {
                const int next = entry_of(tile + 1);
                const int t = tile * kTile + (part << sub_shift);
                const bool mine = part < kTile / sub && kind < (I::kBlocks ? 3 : 2) && t < end;
                const bool good = mine && entry >= 0 && entry < p.n_pages;
                const uint32_t have = __ballot_sync(0xffffffffu, good) & 0xffu, missing = __ballot_sync(0xffffffffu, mine && !good) & 0xffu;
                uint32_t bad = 0;
                for (int i = 0; i < kTile / sub; ++i)
                    if ((missing >> i) & 1u) bad |= ((1u << (sub / 16)) - 1u) << (i * (sub / 16));
                if (missing && lane == 0) atomicOr(p.flags, QC_FLAG_RANGE);
                for (int which = 0; which < 2; ++which) {
                    if (used >= plan.raw) {
                        ok = __all_sync(0xffffffffu, mbar_wait(&bar.raw_empty[stage], phase ^ 1u));
                        if (!ok) break;
                    }
                    if (lane == 0) {
                        sm.raw_bad[stage] = bad;
                        mbar_arrive_expect_tx(&bar.raw_full[stage], __popc(have) * sub * (I::kBytes / kTile));
                    }
                    __syncwarp();
                    if (good) {
                        const unsigned char *src = p.pages + ((int64_t)entry * p.g.heads + kv) * (int64_t)p.g.part;
                        const int at = t & (p.g.page - 1);
                        int dst, bytes;
                        if (kind == 0) {
                            src += p.g.codes(which) + at * I::kRow;
                            dst = 0;
                            bytes = I::kRow;
                        } else if (kind == 1) {
                            src += p.g.scales(which) + at * 4;
                            dst = I::kCodes;
                            bytes = 4;
                        } else {
                            src += p.g.block_scales(which) + at * I::kBlocks;
                            dst = I::kCodes + 4 * kTile;
                            bytes = I::kBlocks;
                        }
                        bulk_g2s(raw + stage * I::kBytes + dst + (part << sub_shift) * bytes, src, sub * bytes, &bar.raw_full[stage]);
                    }
                    ++used;
                    if (++stage == plan.raw) stage = 0, phase ^= 1u;
                }
                entry = next;
            }
        }
        // the copies still under way land before the CTA's shared memory goes
        for (int i = 0; i < plan.raw && i < used; ++i) {
            if (stage == 0) phase ^= 1u;
            stage = (stage ? stage : plan.raw) - 1;
            ok = mbar_wait(&bar.raw_full[stage], phase) && ok;
        }
        ok = __all_sync(0xffffffffu, ok);
    } else if (warp >= kConv && warp < kConv + 4) {
        const int quarter = warp - kConv, t = quarter * 32 + lane;
        const bool short_runs = I::kRow == 32 && p.g.page == 16;
        const float up = p.scale * kLog2e;
        int stage = 0;
        uint32_t phase = 0;
        for (; ok && run.begin(); run.next(p, jobs)) {
            const int end = run.w.n.x + run.w.n.y;
            for (int tile = run.from; ok && tile < run.end; ++tile, ++it) {
#pragma unroll 1
                for (int which = 0; which < 2; ++which) {
                    // the operand's last reader, then the codes
                    if (which == 0) {
                        if (it >= 1) ok = mbar_wait(&bar.k_free, (it - 1) & 1);
                    } else {
                        if (it >= 2) ok = mbar_wait(&bar.v_free[it & 1], ((it >> 1) - 1) & 1);
                    }
                    ok = ok && mbar_wait(&bar.raw_full[stage], phase);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const unsigned char *st = raw + stage * I::kBytes;
                    const bool good = tile * kTile + t < end && !((sm.raw_bad[stage] >> (t >> 4)) & 1u);
                    const float s = good ? *reinterpret_cast<const float *>(st + I::kCodes + 4 * t) : 0.f;
                    if (which == 0) {
                        sm.ks[it & 3][t] = s * up;
                        const uint32_t e = __ballot_sync(0xffffffffu, good);
                        if (lane == 0) sm.exist[it & 3][quarter] = e;
                    } else {
                        sm.vs[it & 1][t] = s;
                        const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(s));
                        if (lane == 0) sm.vtop[it & 1][quarter] = __uint_as_float(m);
                    }
                    convert_row<FMT, D>(st, st + I::kCodes + 4 * kTile + t * I::kBlocks, which == 0 ? k_op : v_op + (it & 1) * kOp, t, short_runs,
                                        good);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&bar.raw_empty[stage]);
                        mbar_arrive(which == 0 ? &bar.k_full : &bar.v_full[it & 1]);
                    }
                    if (++stage == plan.raw) stage = 0, phase ^= 1u;
                }
            }
        }
    } else if (warp == kMma) {
        const uint32_t qk = idesc_f16_f32(128, kTile), pv = idesc_f16_f32(128, D) | 1u << 16;      // values: output dimension contiguous
        const uint32_t qa = smem_addr(q_op), ka = smem_addr(k_op), va = smem_addr(v_op);
        auto scores = [&](int rt, int buf) {        // S[buf] = Q[rt] K^T
            if (lane == 0) {
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = (k >> 2) * (kTile * 128) + (k & 3) * 32;
                    mma_f16(tmem + buf * 128, sdesc_sw128(qa + rt * kOp + off), sdesc_sw128(ka + off), qk, k > 0);
                }
                mma_commit(&bar.s_full[buf]);
                if (rt == NM - 1) mma_commit(&bar.k_free);
            }
            __syncwarp();
        };
        auto values = [&](int rt, int buf, int vb, bool first) {      // O[rt] (+)= P[buf] V[vb]
            if (lane == 0) {
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                    mma_f16_ts(tmem + 256 + rt * 128, tmem + buf * 128 + 8 * k, sdesc_sw128_mn(va + vb * kOp + k * 2048), pv, !first || k > 0);
                mma_commit(&bar.o_done[rt]);
                if (rt == NM - 1) mma_commit(&bar.v_free[vb]);
            }
            __syncwarp();
        };
        auto wait = [&](uint64_t *b, uint32_t parity) { ok = ok && __all_sync(0xffffffffu, mbar_wait(b, parity & 1)); };
        int segment = 0;
        for (; ok && run.begin(); run.next(p, jobs), ++segment) {
            wait(&bar.q_ready, segment);
            wait(&bar.k_full, it);
            if (!ok) break;
            for (int rt = 0; rt < NM; ++rt) scores(rt, NM == 1 ? it & 1 : rt);
            for (int tile = run.from; ok && tile < run.end; ++tile, ++it) {
                const bool more = tile + 1 < run.end, first = tile == run.from;
                if constexpr (NM == 1) {
                    if (more) {
                        wait(&bar.k_full, it + 1);
                        if (ok) scores(0, (it + 1) & 1);
                    }
                    wait(&bar.p_ready[it & 1], it >> 1);
                    wait(&bar.v_full[it & 1], it >> 1);
                    if (ok) values(0, it & 1, it & 1, first);
                } else {
                    for (int rt = 0; ok && rt < NM; ++rt) {
                        wait(&bar.p_ready[rt], it);
                        if (rt == 0) wait(&bar.v_full[it & 1], it >> 1);
                        if (ok) values(rt, rt, it & 1, first);
                        if (more) {
                            if (rt == 0) wait(&bar.k_full, it + 1);
                            if (ok) scores(rt, rt);
                        }
                    }
                }
            }
        }
        // products under way end before the operands' shared memory and the TMEM go
        if (lane == 0) mma_commit(&bar.last);
        __syncwarp();
        ok = __all_sync(0xffffffffu, mbar_wait(&bar.last, 0)) && ok;
    } else {
        // ---- softmax: thread = row
        const int rt = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;          // 32 lanes of TMEM per warp
        int segment = 0;
        for (; run.begin(); run.next(p, jobs), ++segment) {
            const Walk &w = run.w;
            const int kv = w.job / plan.row_tiles, row = (w.job % plan.row_tiles * NM + rt) * 128 + r;
            const bool there = row < R;
            const int node = there ? row / p.group : 0, h = there ? row % p.group : 0;
            const bool active = __any_sync(0xffffffffu, there);
            const T *q = static_cast<const T *>(p.q) + w.b * p.q_seq + node * p.q_node + (kv * p.group + h) * p.q_head;
            float down = 1.f;
            if (active) {
                down = put_query<T, D>(q, there, q_op + rt * kOp, r);
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.q_ready);
            const uint32_t *tree = p.tree ? p.tree + ((int64_t)w.b * p.n_nodes + node) * p.words : nullptr;
            float m = -INFINITY, ref = 0.f;
            int e = 0;                          // log2 of the weights' unit
            float2 l = make_float2(0.f, 0.f);
            for (int tile = run.from; ok && tile < run.end; ++tile, ++it) {
                const int buf = NM == 1 ? it & 1 : rt;
                ok = mbar_wait(&bar.s_full[buf], NM == 1 ? (it >> 1) & 1 : it & 1);
                // the values' scales of the tile
                ok = ok && mbar_wait(&bar.v_full[it & 1], (it >> 1) & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (active) {
                    tc_fence_after();
                    const float4 vt = *reinterpret_cast<const float4 *>(sm.vtop[it & 1]);
                    const uint4 ex = *reinterpret_cast<const uint4 *>(sm.exist[it & 3]);
                    const bool mask = tile * kTile + kTile > w.n.x || (ex.x & ex.y & ex.z & ex.w) != 0xffffffffu;
                    const float vtop = fmaxf(fmax3(vt.x, vt.y, vt.z), vt.w);
                    const uint32_t s_at = tmem + lanes + buf * 128;
                    uint32_t pw[kTile / 2];
                    float2 sum;
                    float top;
                    // one pass with the reference as it is; a second if a score or a scale has passed it
                    for (int pass = 0;; ++pass) {
                        const float mm = (m == -INFINITY ? 0.f : m) - (float)e;
                        const float2 neg = make_float2(-mm, -mm), dn = make_float2(down, down);
                        top = -INFINITY;
                        sum = make_float2(0.f, 0.f);
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            uint32_t s[32];
                            tmem_ld32_nowait(s_at + 32 * c, s);
                            tmem_wait_ld();
                            uint32_t sees = 0xffffffffu;
                            if (mask) {
                                sees = window(p, tree, node, w.n.y, tile * kTile + 32 * c - w.n.x) & (c == 0 ? ex.x : c == 1 ? ex.y : c == 2 ? ex.z : ex.w);
                                if (!there || node >= w.n.y) sees = 0;
                            }
#pragma unroll
                            for (int i = 0; i < 32; i += 4) {
                                const float4 ks = *reinterpret_cast<const float4 *>(&sm.ks[it & 3][32 * c + i]);
                                const float4 vs = *reinterpret_cast<const float4 *>(&sm.vs[it & 1][32 * c + i]);
                                float2 a = mul2f(make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), make_float2(ks.x, ks.y));
                                float2 b = mul2f(make_float2(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])), make_float2(ks.z, ks.w));
                                if (mask) {
                                    if (!((sees >> i) & 1u)) a.x = -INFINITY;
                                    if (!((sees >> (i + 1)) & 1u)) a.y = -INFINITY;
                                    if (!((sees >> (i + 2)) & 1u)) b.x = -INFINITY;
                                    if (!((sees >> (i + 3)) & 1u)) b.y = -INFINITY;
                                }
                                top = fmax3(fmax3(top, a.x, a.y), b.x, b.y);
                                a = fma2f(a, dn, neg);
                                b = fma2f(b, dn, neg);
                                a.x = ex2(a.x), a.y = ex2(a.y), b.x = ex2(b.x), b.y = ex2(b.y);
                                sum = add2f(sum, a);
                                sum = add2f(sum, b);
                                a = mul2f(a, make_float2(vs.x, vs.y));
                                b = mul2f(b, make_float2(vs.z, vs.w));
                                pw[16 * c + i / 2] = pack2(a.x, a.y);
                                pw[16 * c + i / 2 + 1] = pack2(b.x, b.y);
                            }
                        }
                        if (pass) break;
                        top *= down;
                        if (!__any_sync(0xffffffffu, top > m + kLag || vtop > ref)) break;
                        const float m2 = top > m + kLag ? top + kLag : m;
                        const float ref2 = fmaxf(ref, fmaxf(power_above(vtop), 3.2311742677852644e-27f));     // at least 2^-88
                        const int e2 = kTop + 127 - (int)(__float_as_uint(ref2) >> 23);
                        // sums so far in the new unit
                        const float by = m == -INFINITY ? 0.f : ex2(m - m2 + (float)(e2 - e));
                        l.x *= by;
                        l.y *= by;
                        if (tile > run.from) {
                            ok = __all_sync(0xffffffffu, mbar_wait(&bar.o_done[rt], (it - 1) & 1));
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
                        }
                        m = m2;
                        ref = ref2;
                        e = e2;
                    }
                    l = add2f(l, sum);
                    tmem_st32(s_at, pw);
                    tmem_st32(s_at + 32, pw + 32);
                    tmem_wait_st();
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.p_ready[buf]);
            }
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&bar.o_done[rt], (it - 1) & 1));
            if (!ok) break;
            if (active) {
                tc_fence_after();
                const bool whole = run.from == 0 && run.end == w.tiles;
                const int64_t part = 2 * (int64_t)blockIdx.x + (segment ? 1 : 0);
                const float sum = l.x + l.y;
                const bool some = sum > 0.f && node < w.n.y;
                // out = O / (unit) / (l / unit); a part keeps l and O free of the unit
                const float unit = __uint_as_float((uint32_t)(127 - e) << 23);
                const float by = whole ? (some ? 1.f / sum : 0.f) : unit;
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
                        p.lse[at] = some ? (m + log2f(sum) - (float)e) * kLn2 : -INFINITY;
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
    if (warp == kMma) tmem_dealloc(tmem, 512);
}

template <int FMT, int D>
Plan plan_tc(const qc_ctx *c, int rows, int64_t n_seq, int64_t max_len, int n_nodes) {
    using I = Item<FMT, D>;
    Plan p;
    p.nm = rows <= 128 ? 1 : 2;
    p.row_tiles = (rows + 128 * p.nm - 1) / (128 * p.nm);
    const int fixed = (p.nm + 3) * kOperand<D> + (int)sizeof(Small);
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
    const Plan p = plan_tc<FMT, D>(c, rows, n_seq, max_len, n_nodes);
    return workspace_bytes(n_seq, 2 * (int64_t)p.units, p.nm * 128, D);
}

template <typename T, int FMT, int D, int NM>
cudaError_t launch(const Plan &plan, const Attend &p, int type, cudaStream_t s) {
    const Parts parts = parts_at(p.workspace, p.n_seq, 2 * (int64_t)plan.units, NM * 128, D);
    cudaError_t e = cudaFuncSetAttribute(attend_tc<T, FMT, D, NM>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)plan.units);
    cfg.blockDim = dim3(32 * (4 * NM + 6));
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

int64_t tc_workspace(const qc_ctx *c, int64_t n_seq, int n_nodes, int n_q_heads, int64_t max_len) {
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
