// The parts of the tensor-core attention kernel (qc_attend_tc.cu): tiles of 128 places, the producer warps that
// copy them from the pages, the conversion of rows to fp16 operands, and the instructions for them.
#pragma once

#include "qc_convert.cuh"

namespace qc {

using namespace fq::sm100;

constexpr int kTile = 128;              // places
constexpr int kMostRaw = 8;             // raw stages at most

template <int FMT, int D>
struct Item {           // a raw stage: codes and block scales of a tile's keys or values; with the keys both scales
    static constexpr int kRow = FMT == QC_E2M1 ? D / 2 : D;
    static constexpr int kBlocks = FMT == QC_E2M1 ? D / 16 : 0;
    static constexpr int kCodes = kTile * kRow;
    static constexpr int kScales = kCodes, kBlockScales = kCodes + 8 * kTile;
    static constexpr int kBytes = kTile * (kRow + 8 + kBlocks);
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
    __device__ __forceinline__ void next(const Attend &p, int jobs, int tile) {
        w.left -= end - from;
        next_job(p, w, jobs, tile);
    }
};

// Matrix descriptor of an operand whose rows (places) of 64 elements hold the output's dimension: groups of 8
// rows 1024 bytes apart, the next 64 elements `next` bytes on.
__device__ __forceinline__ uint64_t sdesc_sw128_mn(uint32_t saddr, uint32_t next) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)(next >> 4) << 16;
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

// 16-byte piece q of row t of an operand tile (chunks of 64 elements, 128-byte swizzle).
__device__ __forceinline__ void put_piece(unsigned char *out, int t, int q, const uint32_t (&h)[4]) {
    *reinterpret_cast<uint4 *>(out + (q >> 3) * (kTile * 128) + t * 128 + (((q & 7) ^ (t & 7)) * 16)) = make_uint4(h[0], h[1], h[2], h[3]);
}

// One lane's place: its raw row, row t of a stage, to fp16, eight elements at a time: put(q, pairs) takes
// elements 8 q .. 8 q + 7. good: the place exists (else zeros).
template <int FMT, int D, typename Put>
__device__ __forceinline__ void convert_row(const unsigned char *raw, const unsigned char *block, int t, bool short_runs, bool good,
                                            Put put) {
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
                put(4 * j + i, h);
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
                put(2 * j + i, h);
            }
        }
    }
}

// A row's query, in fp16 and brought to its range, at row r of the operand tile. Returns the power of two that
// the row's scores are multiplied by.
template <typename T, int D>
__device__ __forceinline__ float put_query(const T *q, bool there, unsigned char *out, int r, int chunk_rows) {
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
        // largest magnitude to [2^13, 2^14): from 2^-17 on, 2^-30 of it, fp16 holds all 8 bits
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
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = finite_or_nan(v[j]);
        }
        *reinterpret_cast<uint4 *>(out + (i >> 3) * (chunk_rows * 128) + r * 128 + (((i & 7) ^ (r & 7)) * 16)) =
            make_uint4(pack2(v[0] * f, v[1] * f), pack2(v[2] * f, v[3] * f), pack2(v[4] * f, v[5] * f), pack2(v[6] * f, v[7] * f));
    }
    return down;
}

// A barrier's phase, by its number, for at most about two seconds. The thread sleeps in the barrier unit (10 us
// at a time at most): some fifteen warps that polled would take the working ones' issue slots.
__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t phase) {
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t i = 0;; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_addr(bar)), "r"(phase & 1u), "r"(10000u)
            : "memory");
        if (ok) return true;
        if ((i & 255u) == 255u) {
            const uint64_t now = global_timer_ns();
            if (!t0) t0 = now;
            if (now - t0 > 2000000000ull) return false;
        }
    }
}
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t phase) {
    return __all_sync(0xffffffffu, wait_phase(bar, phase));
}

// Issuing a tile's copies takes one warp longer than a tile may take the SM, so that several warps take turns.
constexpr int kProducers = 3;

struct RawRing {
    uint64_t full[kMostRaw], empty[kMostRaw];
    uint32_t bad[kMostRaw];         // sixteenths of a stage's tile whose page does not exist
    uint32_t issued[kMostRaw];      // 1 + parity of the stage's last copy; 0: none
    __device__ __forceinline__ void init(int stages) {
        for (int i = 0; i < kMostRaw; ++i) {
            issued[i] = 0;
            if (i < stages) {
                mbar_init(&full[i], 1);
                mbar_init(&empty[i], 4);
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

// Producer warp `mine`: for every so manieth tile of the unit's run, its keys and its values, as the pages hold
// them, to two of `stages` (at least 2) raw stages (item 2 i: the keys of tile i; 2 i + 1: its values). A wait
// on a stage names its phase by parity, so a warp must never come to a stage two rounds ahead: as the
// converters free the items of each kind in order, that holds as long as the warps' tiles fit the ring
// together, and no more than stages / 2 of them work.
// False if a wait gave up.
template <int FMT, int D>
__device__ __forceinline__ bool produce(const Attend &p, Run &run, int jobs, int row_tiles, int stages, unsigned char *raw, RawRing &ring,
                                        int mine, int lane) {
    using I = Item<FMT, D>;
    int it = 0, item = 0;               // tiles so far; the next item's place in the ring
    uint32_t round = 0;
    auto forward = [&](int n) {
        for (item += n; item >= stages; item -= stages) ++round;
    };
    const int warps = stages / 2 < kProducers ? stages / 2 : kProducers;
    if (mine >= warps) return true;
    forward(2 * mine);
    const int sub = p.g.page < kTile ? p.g.page : kTile, sub_shift = p.g.shift < 7 ? p.g.shift : 7;
    const int parts = kTile / sub;
    for (; run.begin(); it += run.end - run.from, run.next(p, jobs, kTile)) {
        const int kv = run.w.job / row_tiles, end = run.w.n.x + run.w.n.y;
        const int32_t *row = p.table + run.w.b * p.table_stride;
        const unsigned char *head = p.pages + kv * (int64_t)p.g.part;
        const int64_t page_bytes = (int64_t)p.g.heads * p.g.part;
        // lane i: the page of the tile's i-th part
        auto entry_of = [&](int tile) {
            const int t = tile * kTile + (lane << sub_shift);
            int e = -1;
            if (lane < parts && tile < run.end && t < end)
                asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(e) : "l"(row + (t >> p.g.shift)));     // not later than here
            return e;
        };
        int tile = run.from + (mine + warps - it % warps) % warps;
        int entry = entry_of(tile);
        for (; tile < run.end; tile += warps) {
            const int next = entry_of(tile + warps);
            const bool here = lane < parts && tile * kTile + (lane << sub_shift) < end;
            const bool good = here && entry >= 0 && entry < p.n_pages;
            const uint32_t have = __ballot_sync(0xffffffffu, good), missing = __ballot_sync(0xffffffffu, here && !good);
            uint32_t bad = 0;
            if (missing) {
                for (int i = 0; i < parts; ++i)
                    if ((missing >> i) & 1u) bad |= ((1u << (sub / 16)) - 1u) << (i * (sub / 16));
                if (lane == 0) atomicOr(p.flags, QC_FLAG_RANGE);
            }
            const int at = tile * kTile & (p.g.page - 1);       // where in a page of 256 the tile begins
            const int k = item;
            const uint32_t k_round = round;
            forward(1);
            const int v = item;
            const uint32_t v_round = round;
            forward(2 * warps - 1);
            bool ok = true;
            if (k_round) ok = ok && warp_wait(&ring.empty[k], k_round - 1);
            if (v_round) ok = ok && warp_wait(&ring.empty[v], v_round - 1);
            if (!ok) return false;
            unsigned char *kt = raw + k * I::kBytes, *vt = raw + v * I::kBytes;
            if (elect_one()) {
                ring.bad[k] = ring.bad[v] = bad;
                ring.issued[k] = 1 + (k_round & 1);
                ring.issued[v] = 1 + (v_round & 1);
                const uint32_t places = __popc(have) * sub;
                mbar_arrive_expect_tx(&ring.full[k], places * (I::kRow + 8 + I::kBlocks));
                mbar_arrive_expect_tx(&ring.full[v], places * (I::kRow + I::kBlocks));
            }
            for (int i = 0; i < parts; ++i) {
                const int64_t page = __shfl_sync(0xffffffffu, entry, i);
                if ((have >> i) & 1u) {
                    const unsigned char *src = head + page * page_bytes;
                    const int first = i << sub_shift;
                    if (elect_one()) {
                        bulk_g2s(kt + first * I::kRow, src + at * I::kRow, sub * I::kRow, &ring.full[k]);
                        bulk_g2s(kt + I::kScales + first * 4, src + p.g.scales(0) + at * 4, sub * 4, &ring.full[k]);
                        bulk_g2s(kt + I::kScales + (kTile + first) * 4, src + p.g.scales(1) + at * 4, sub * 4, &ring.full[k]);
                        bulk_g2s(vt + first * I::kRow, src + p.g.codes(1) + at * I::kRow, sub * I::kRow, &ring.full[v]);
                        if constexpr (I::kBlocks != 0) {
                            bulk_g2s(kt + I::kBlockScales + first * I::kBlocks, src + p.g.block_scales(0) + at * I::kBlocks,
                                     sub * I::kBlocks, &ring.full[k]);
                            bulk_g2s(vt + I::kBlockScales + first * I::kBlocks, src + p.g.block_scales(1) + at * I::kBlocks,
                                     sub * I::kBlocks, &ring.full[v]);
                        }
                    }
                }
            }
            entry = next;
        }
    }
    return true;
}

}  // namespace qc
