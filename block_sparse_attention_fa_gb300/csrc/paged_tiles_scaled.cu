// paged_tiles_scaled.cu -- paged_tiles.cu's attention for many rows, over a cache
// held in 8 bits (e4m3 codes, a scale for each page and kv head).
//
// Units, the line of tiles, TMEM, the pipeline of 64-key halves and the joining
// are paged_tiles.cu's.  What differs:
//
// S = Q K^T takes K's codes as they are: its operands are 8-bit.  Q, which is
// bf16, becomes the sum of two e4m3 numbers: a row is scaled by a power of two
// to a largest element in (224, 448], hi = e4m3(q), lo = e4m3(q - hi), and
// S = hi K^T + lo K^T into one accumulator.  A bf16 number has 8 significant
// bits, hi and lo 4 each, and lo's last one is at least 2^-9: this is exact for
// elements of 1/4 and more, 2^-9.8 of the row's largest, and off by at most 2^-10,
// 2^-17.8 of that, below.  Two 8-bit products
// cost what a bf16 one does (a product takes twice the columns at once), and K
// is neither converted nor moved again.  The softmax warps split their rows of Q
// in place, in shared memory.
//
// P V keeps P at 11 bits, in f16.  V's codes become f16, which holds them exactly:
// four more warps (12-15) convert 64-key halves from a ring of codes to one of
// operands.  v's scales cannot stay out of P, for a product adds up keys of many
// pages: with x the score in base 2, lv = log2(v's scale) and M a reference below the
// largest x + lv (kPHead, or with fp32 output kPTop),
//     P = 2^(x + lv - M),   l = sum of P / (v's scale),
// so that P is at most 2^kPTop, its roundings are relative to the largest share that
// any key has in O, and one exponential serves both sums; O / l and M + log2 l are
// what they are without scales.  The scale is the same for 16 columns (of one page).
// A scale below 2^-80 of the largest so far in the unit, or below 2^-82, counts as
// that: what such a page adds to O is nothing beside the others, and l keeps all of
// its keys.  k's scale and the row's stay with S.
//
// What bounds it is the chain of a 64-key half, 1500 to 1700 cycles of softmax
// alone: 4 chunks of up to 1024 tokens on up to 8192 keys, 32 heads on 8 of 128
// columns, take 221 us (187 over bf16, 116 at the bf16 rate); without V's
// conversion 215, with half of S's products 210, without either, the exponentials
// and most of P V 197.  A shared prefix of 16384 keys for 64 tokens takes 28: its
// first products start after 8, the partials' stores take 4.
//
// 512 threads: softmax 0-3, 4-7; loader 8; MMA 9, 10; none 11; convert 12-15.
#include <algorithm>

#include "paged_tile_parts.cuh"

namespace fa {
namespace {

constexpr int kThreads8 = 512;
// Registers per thread: launched with 128; 128 x (2 x 184 + 88 + 56) = 512 x 128.
// build.py checks the launch count.
constexpr uint32_t kRegsSoftmax8 = 184, kRegsOther8 = 88, kRegsConvert8 = 56;
static_assert(2 * kRegsSoftmax8 + kRegsOther8 + kRegsConvert8 == 4 * 128, "register split must match the launch");
constexpr int kMaxRing8 = 4;
// Tiles whose scales are kept.  K(g) is loaded once S of tile g - stages is done,
// which came after P of the tile before that: the loader is at most five tiles
// ahead of the softmax warps.
constexpr int kScaleRing = 8;

enum TBar8 {
    T_Q_FULL = 0,                                // two: the 4 softmax warps of the tile
    T_K_FULL = 2, T_K_EMPTY = T_K_FULL + kMaxRing8,
    T_RAW_FULL = T_K_EMPTY + kMaxRing8, T_RAW_EMPTY = T_RAW_FULL + kMaxRing8,   // V's codes, tile by tile
    T_V_FULL = T_RAW_EMPTY + kMaxRing8, T_V_EMPTY = T_V_FULL + kMaxRing8,       // V in f16, half by half
    T_SCALES = T_V_EMPTY + kMaxRing8,            // [kScaleRing]
    T_S_FULL = T_SCALES + kScaleRing,            // four (2 t + h)
    T_P_FULL = T_S_FULL + 4,                     // four (2 t + h)
    T_O_DONE = T_P_FULL + 4,                     // two
    T_O_UPD = T_O_DONE + 2,                      // two
    T_DRAIN = T_O_UPD + 2,                       // two
    T_SEG_FULL = T_DRAIN + 2,                    // two slots
    T_SEG_EMPTY = T_SEG_FULL + 2,
    T_Q_HERE = T_SEG_EMPTY + 2,                  // the first unit's rows of tile 0, before they are split
    T_COUNT = T_Q_HERE + 1
};
static_assert(T_COUNT <= kThreads8, "a thread to a barrier");
constexpr uint32_t kSegReaders = 14;             // the MMA, softmax and converting warps
enum TSite8 : uint32_t { S_T_Q = 128, S_T_K_FULL, S_T_K_EMPTY, S_T_RAW_FULL, S_T_RAW_EMPTY, S_T_V_FULL, S_T_V_EMPTY,
                         S_T_SCALES, S_T_S, S_T_P, S_T_O, S_T_UPD, S_T_DRAIN, S_T_SEG, S_T_SEG_EMPTY };

// Q of a row tile: first bf16 (two boxes of 64 columns, or one), then 128 columns:
// the box of hi and the box of lo; 64: a row is hi, then lo.  Tiles of codes: a
// key to a row of D bytes, in that width's swizzle.
template <int D>
struct TileLayout8 {
    static constexpr int kKStages = D == 64 ? 4 : 3, kRaw = D == 64 ? 4 : 2, kHalves = D == 64 ? 4 : 3;
    static constexpr uint32_t kTile = 128u * D * 2u, kCodes = 128u * D, kHalf = 64u * D * 2u, kBoxHalf = 8192u;
    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kK = kQ + 2 * kTile;
    static constexpr uint32_t kRawAt = kK + kKStages * kCodes;
    static constexpr uint32_t kV = kRawAt + kRaw * kCodes;
    static constexpr uint32_t kBars = kV + kHalves * kHalf;
    static constexpr uint32_t kTmemSlot = kBars + 8 * T_COUNT;
    static constexpr uint32_t kAbort = kTmemSlot + 4;
    static constexpr uint32_t kMinMax = kAbort + 4;          // positions of the batch (shared prefix)
    static constexpr uint32_t kScales = (kMinMax + 8 + 15) & ~15u;   // [tile][k's scale, log2 of v's, 1 / v's][8 x 16 keys]
    static constexpr uint32_t kSeg = kScales + 96 * kScaleRing;    // two units
    static constexpr uint32_t kScan = kSeg + 2 * sizeof(TileSeg);
    static constexpr uint32_t kPre = kScan + 4 * (kThreads8 / 32);   // TileLine's arrays
    static constexpr uint32_t bytes(int B) { return kPre + 4u * (3u * B + 2u) + 1024u; }
    static_assert(kKStages <= kMaxRing8 && kRaw <= kMaxRing8 && kHalves <= kMaxRing8, "rings");
    static_assert(kPre + 4 * (3 * kPagedMaxSeqs + 2) + 1024 <= 227u * 1024u, "shared memory budget");
};

// Instruction descriptors: fp32 accumulators, A and B e4m3 (kind::f8f6f4) or f16
// (kind::f16, B with its N columns contiguous).
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__host__ __device__ constexpr uint32_t idesc_f16_mn(int M, int N) {
    return (1u << 4) | (1u << 16) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// As sdesc_sw128, for rows of 64 bytes with 64-byte swizzle (layout 4).
__device__ __forceinline__ uint64_t sdesc_sw64(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return (sdesc_sw128(saddr, lbo, sbo) & ~(7ull << 61)) | (4ull << 61);
}
// D[tmem] (+)= A[smem] B[smem], 32 columns of e4m3; a whole warp, one elected lane issues.
__device__ __forceinline__ void mma_codes_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ float bf_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Four e4m3 codes as two pairs of f16: exact.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
// Two f16 numbers to e4m3 (16 bits), and what is left of them (exact).
__device__ __forceinline__ uint32_t split_pair(uint32_t& w) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(w));
    uint32_t x;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(x) : "h"(r));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(w) : "r"(w), "r"(x));
    return r;
}
__device__ __forceinline__ uint32_t to_e4m3(uint32_t w) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(w));
    return r;
}

// A warp's 32 rows of Q, bf16 in their row tile at `tile` from row `first` on, into
// hi and lo in their place.  Returns what S of row first + lane is to be multiplied
// by.  A row is its lanes' (16 columns each), some rows at a time: a thread to a row
// would take six times the instructions, which a CTA's first unit has to wait for.
template <int D>
__device__ __forceinline__ float split_rows(uint8_t* tile, int first, int lane) {
    constexpr int kLanes = D / 16, kAtOnce = 32 / kLanes;
    const int c = lane % kLanes;
    float mine = 1.f;
#pragma unroll 1
    for (int r0 = 0; r0 < 32; r0 += kAtOnce) {
        const int row = first + r0 + lane / kLanes;
        auto at = [&](int k) { return tile + (k >> 3) * 16384 + row * 128 + (((k & 7) ^ (row & 7)) << 4); };
        const uint4 v0 = *reinterpret_cast<const uint4*>(at(2 * c)), v1 = *reinterpret_cast<const uint4*>(at(2 * c + 1));
        const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmax3(top, fabsf(bf_low(w[e])), fabsf(bf_high(w[e])));
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        // top = 1.f 2^x: times 2^(8 - x), or 2^(7 - x) where 1.f is past 7/4
        const int bits = __float_as_int(top), x = max((bits >> 23) + ((bits & 0x7fffff) > 0x600000 ? 1 : 0), 10);
        const float up = __int_as_float((262 - x) << 23);
        // (an infinity would become 448: it makes all of the row's scores NaN instead)
        const float down = top < CUDART_INF_F ? __int_as_float((x - 8) << 23) : CUDART_NAN_F;
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t p = w[2 * e], q = w[2 * e + 1];
            uint32_t a = pack_f16x2(bf_low(p) * up, bf_high(p) * up), b = pack_f16x2(bf_low(q) * up, bf_high(q) * up);
            const uint32_t ha = split_pair(a), hb = split_pair(b);
            hi[e] = __byte_perm(ha, hb, 0x5410);
            lo[e] = __byte_perm(to_e4m3(a), to_e4m3(b), 0x5410);
        }
        // (the shuffles above: all of the rows' pieces have been read)
        *reinterpret_cast<uint4*>(at(c)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(at(kLanes + c)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        const float theirs = __shfl_sync(0xffffffffu, down, kLanes * (lane % kAtOnce));
        if (lane / kAtOnce == r0 / kAtOnce) mine = theirs;
    }
    return mine;
}

// A converting warp's 16 keys (of 64, from 16 w on) of a half of V: codes at
// `raw` to f16 at `to`; keys that are not `live` become zeros.  Eight lanes read
// 128 bytes that lie on distinct banks, and write so: two keys, of 128 columns
// the other half of each in turn.
template <int D, class F>
__device__ __forceinline__ void convert_half(const uint8_t* raw, uint8_t* to, int w, int lane, F live) {
    constexpr int kTimes = 16 * (D / 16) / 32;
#pragma unroll
    for (int e = 0; e < kTimes; ++e) {
        const int key = 16 * w + 8 * (D == 128 ? e >> 1 : e) + 2 * (lane >> 3) + ((lane >> 2) & 1);
        const int c = (lane & 3) + (D == 128 ? 4 * (((lane >> 2) ^ e) & 1) : 0);
        const uint32_t from = D == 128 ? key * 128 + ((c ^ (key & 7)) << 4) : key * 64 + ((c ^ ((key >> 1) & 3)) << 4);
        uint4 codes = *reinterpret_cast<const uint4*>(raw + from);
        if (!live(key)) codes = make_uint4(0u, 0u, 0u, 0u);
        uint4 a, b;
        codes_to_f16(codes.x, a.x, a.y);
        codes_to_f16(codes.y, a.z, a.w);
        codes_to_f16(codes.z, b.x, b.y);
        codes_to_f16(codes.w, b.z, b.w);
        uint8_t* const row = to + (c >> 2) * 8192 + key * 128;
        *reinterpret_cast<uint4*>(row + (((2 * (c & 3)) ^ (key & 7)) << 4)) = a;
        *reinterpret_cast<uint4*>(row + (((2 * (c & 3) + 1) ^ (key & 7)) << 4)) = b;
    }
}

template <int D, int SCORE>
__global__ void __launch_bounds__(kThreads8, 1)
paged_tiles_scaled_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                          const PagedScaledParams p) {
    using L = TileLayout8<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_addr(smem);
    auto bar = [&](int k) { return sbase + L::kBars + 8u * k; };
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + L::kTmemSlot);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kAbort);
    int* const minmax = reinterpret_cast<int*>(smem + L::kMinMax);
    int* const pre = reinterpret_cast<int*>(smem + L::kPre);
    int* const q0_s = pre + p.c.B + 1;
    int* const len_s = q0_s + p.c.B + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;

    if (threadIdx.x < T_COUNT) {
        const int k = threadIdx.x;
        uint32_t cnt = 1;
        if (k < T_K_FULL) cnt = 4;
        if (k >= T_P_FULL && k < T_P_FULL + 4) cnt = 4;
        if (k == T_Q_HERE) cnt = 4;
        if (k >= T_RAW_EMPTY && k < T_RAW_EMPTY + kMaxRing8) cnt = 4;         // the converting warps
        if (k >= T_V_FULL && k < T_V_FULL + kMaxRing8) cnt = 4;
        if (k >= T_K_EMPTY && k < T_K_EMPTY + kMaxRing8) cnt = 2;             // both MMA warps
        if (k >= T_V_EMPTY && k < T_V_EMPTY + kMaxRing8) cnt = 2;
        if (k >= T_SEG_EMPTY && k < T_SEG_EMPTY + 2) cnt = kSegReaders;
        mbar_init(bar(k), cnt);
        if (k == 0) {
            *abort_flag = 0;
            minmax[0] = INT_MAX;
            minmax[1] = INT_MIN;
        }
        mbar_fence_init();
    }
    if (warp == 9) {
        tmem_alloc(smem_addr(const_cast<uint32_t*>(tmem_slot)), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const WaitCtl wc{abort_flag, p.ws, p.timeout_ns};

    // (a shared prefix's kernel is no input of the sequences' own: that one
    // waits for it at the end)
    if (p.join_rows && !p.prefix)
        wait_before_prefix(p);
    else
        pdl_wait_previous();
    if (threadIdx.x == 0) {
        if (p.prefix && cta == 0) mark_prefix(p);
        pdl_launch_next();
    }
    // the line of tiles, as in paged_tiles.cu
    TileLine line{};
    line.pre = pre;
    line.kv = len_s;
    line.q0 = q0_s;
    int total;
    if (p.prefix) {
        for (int b = threadIdx.x; b < p.c.B; b += kThreads8) {
            const SeqInfo s = seq_info(p.c, b, p.max_q, p.shared, cta == 0 ? p.ws : nullptr);
            len_s[b] = s.kv;
            q0_s[b + 1] = load_i32(p.c.q_start + b + 1);
            if (s.n > 0) {
                atomicMin(minmax, s.kv - s.n);
                atomicMax(minmax + 1, s.kv - 1);
            }
        }
        __syncthreads();
        line.imin = minmax[0];
        line.imax = minmax[1];
        total = prefix_line(p, line, load_i32(p.c.q_start + p.c.B));
    } else {
        const bool few = p.c.B <= kThreads8 / 32;
        bool ordered = true;
        for (int b = few ? warp : threadIdx.x; b < p.c.B; b += few ? kThreads8 / 32 : kThreads8) {
            const bool first = !few || lane == 0;
            const SeqInfo s = seq_info(p.c, b, p.max_q, p.shared, cta == 0 && first ? p.ws : nullptr);
            int sum = 0;
            for (int rt = few ? lane : 0; rt * kPagedTileRows < s.n * p.group; rt += few ? 32 : 1)
                sum += unit_length(p, s.n, s.kv, rt);
            if (few) sum = __reduce_add_sync(0xffffffffu, sum);
            ordered = ordered && s.ordered;
            if (first) {
                pre[b] = sum;
                len_s[b] = s.kv;
                q0_s[b] = s.q0;
                if (b == p.c.B - 1) q0_s[p.c.B] = s.q0 + s.n;
            }
        }
        ordered = __syncthreads_and(ordered);
        block_prefix<kThreads8>(p.c.B, pre, reinterpret_cast<int*>(smem + L::kScan),
                                [&](int b) { return ordered ? pre[b] : 0; });
        total = p.c.Hkv * pre[p.c.B];
    }
    line_share(total, p.ctas, cta, line.per, line.t, line.t1);
    if (p.prefix) {
        if (cta == 0 && threadIdx.x == 0) {
            p.hdr[0] = line.prefix_tiles;
            p.hdr[1] = line.per;
        }
    } else if (line.t < line.t1) {
        line.b = line_find(pre, p.c.B, p.c.Hkv, line.t);
        line.start = p.c.Hkv * pre[line.b];
    }

    // Only the loader walks the line; it passes each unit through a two-slot
    // queue (rows = 0: none left).  take(): the warp's next unit.
    TileSeg* const seg_s = reinterpret_cast<TileSeg*>(smem + L::kSeg);
    uint32_t nu = 0;
    auto take = [&](TileSeg& s) -> bool {
        const uint32_t slot = nu & 1;
        if (!mbar_wait_warp(bar(T_SEG_FULL + slot), (nu >> 1) & 1, wc, S_T_SEG)) return false;
        s = seg_s[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(T_SEG_EMPTY + slot));
        ++nu;
        return s.rows > 0;
    };

    // Barrier phases run on counters that every role keeps alike: g counts tiles,
    // j halves of V, uq units in which row tile t has rows, n the steps of tile t.
    if (warp >= 12) {
        // ----------------------------------------------------------- convert V
        regs_decrease<kRegsConvert8>();
        uint32_t g = 0, j = 0;
        bool ok = true;
        TileSeg s;
        while (ok && take(s)) {
            for (int k = s.k0; ok && k < s.k1; ++k, ++g) {
                const uint32_t raw = g % L::kRaw;
                if (!mbar_wait_warp(bar(T_RAW_FULL + raw), (g / L::kRaw) & 1, wc, S_T_RAW_FULL)) { ok = false; break; }
#pragma unroll 1
                for (int h = 0; h < 2; ++h, ++j) {
                    const uint32_t slot = j % L::kHalves;
                    if (j >= L::kHalves && !mbar_wait_warp(bar(T_V_EMPTY + slot), (j / L::kHalves - 1) & 1, wc, S_T_V_EMPTY)) {
                        ok = false;
                        break;
                    }
                    const int c0 = s.hull.tile(k) * kBlock + 64 * h;
                    const uint8_t* const from = smem + L::kRawAt + raw * L::kCodes + h * (L::kCodes / 2);
                    uint8_t* const to = smem + L::kV + slot * L::kHalf;
                    if (s.hull.all(c0, c0 + 64))
                        convert_half<D>(from, to, warp - 12, lane, [](int) { return true; });
                    else
                        convert_half<D>(from, to, warp - 12, lane, [&](int key) { return s.hull.live(c0 + key); });
                    fence_async_shared();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bar(T_V_FULL + slot));
                        if (h == 1) mbar_arrive(bar(T_RAW_EMPTY + raw));
                    }
                }
            }
        }
    } else if (warp >= 8) {
    regs_decrease<kRegsOther8>();
    if (warp == 8) {
        // ------------------------------------------------------------ loader
        if (lane == 0) {
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmV);
        }
        const int span = min(p.c.page_size, kBlock);
        const uint32_t page_bytes = static_cast<uint32_t>(span) * D;
        uint32_t g = 0;
        int last_k = -1, last_v = -1;
        bool ok = true;
        TileSeg s{};
        if (!p.prefix && line.t < line.t1) seek(p, line, lane);
        // the copies of one tile of K or V: `id` the lane's page, `row` its first
        // row within the page
        auto load = [&](const CUtensorMap* tm, uint32_t base, int stages, int full, int empty, uint32_t gg, int id, int row,
                        uint32_t site) -> bool {
            const uint32_t st = gg % stages;
            if (gg >= static_cast<uint32_t>(stages) && !mbar_wait_warp(bar(empty + st), (gg / stages - 1) & 1, wc, site)) return false;
            const uint32_t pages = __popc(__ballot_sync(0xffffffffu, id >= 0));
            if (lane == 0) mbar_arrive_expect_tx(bar(full + st), pages * page_bytes);
            __syncwarp();
            if (id >= 0)
                tma_load_3d(sbase + base + st * L::kCodes + static_cast<uint32_t>(lane * span) * D, tm, bar(full + st), 0, row,
                            id * p.c.Hkv + s.h);
            return true;
        };
        auto load_v = [&](uint32_t gg, int id, int row) -> bool {
            if (!load(&tmV, L::kRawAt, L::kRaw, T_RAW_FULL, T_RAW_EMPTY, gg, id, row, S_T_RAW_EMPTY)) return false;
            last_v = static_cast<int>(gg);
            return true;
        };
        while (ok) {
            if (nu >= 2 && !mbar_wait_warp(bar(T_SEG_EMPTY + (nu & 1)), ((nu >> 1) - 1) & 1, wc, S_T_SEG_EMPTY)) break;
            const bool more = next_seg(p, line, s);
            if (lane == 0) {
                if (!more) s.rows = 0;
                seg_s[nu & 1] = s;
                mbar_arrive(bar(T_SEG_FULL + (nu & 1)));
            }
            ++nu;
            if (!more) break;
            const int32_t* table = p.c.page_table + (size_t)s.b * p.c.max_pages;
            // page ids come two tiles ahead, the scales, which need them, one
            auto page_of = [&](int k) {
                return k < s.k1 ? tile_page<kBlock>(p.c, table, s.hull, s.hull.tile(k), lane, s.b, p.ws) : -1;
            };
            auto scale_of = [&](const float* scales, int id) {
                return id >= 0 ? scales[(size_t)id * p.c.Hkv + s.h] : 0.f;
            };
            int page = page_of(s.k0), page2 = page_of(s.k0 + 1), id_v = -1, row_v = 0;
            float ks = scale_of(p.k_scale, page), vs = scale_of(p.v_scale, page), largest = 0.f;
            for (int k = s.k0; k < s.k1; ++k) {
                const int id = page, row = (s.hull.tile(k) * kBlock + lane * span) & (p.c.page_size - 1);
                const float ks_now = ks, vs_now = vs;
                page = page2;
                ks = scale_of(p.k_scale, page);
                vs = scale_of(p.v_scale, page);
                page2 = page_of(k + 2);
                if (!load(&tmK, L::kK, L::kKStages, T_K_FULL, T_K_EMPTY, g, id, row, S_T_K_EMPTY)) { ok = false; break; }
                last_k = static_cast<int>(g);
                // (bits of numbers that are not negative are in their order)
                largest = fmaxf(largest, __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(vs_now, 0.f)))));
                float v_scale = fmaxf(fmaxf(vs_now, largest * kLeastRatio), kLeastScale);
                if (vs_now != vs_now) v_scale = vs_now;
                const float lv = log2f(v_scale), iv = 1.f / v_scale;
                float* const sc = reinterpret_cast<float*>(smem + L::kScales + 96 * (g % kScaleRing));
                const int from = (16 * lane / span) & 31;      // the page of 16 keys
                const float ks_at = __shfl_sync(0xffffffffu, ks_now, from), lv_at = __shfl_sync(0xffffffffu, lv, from),
                            iv_at = __shfl_sync(0xffffffffu, iv, from);
                if (lane < 8) {
                    sc[lane] = ks_at;
                    sc[8 + lane] = lv_at;
                    sc[16 + lane] = iv_at;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(T_SCALES + g % kScaleRing));
                // the first unit's rows of Q come before the rest of the ring:
                // behind it they would wait for all of it to arrive
                if (g == 0 && !mbar_wait_warp(bar(T_Q_HERE), 0, wc, S_T_Q)) { ok = false; break; }
                if (k > s.k0 && !load_v(g - 1, id_v, row_v)) { ok = false; break; }
                id_v = id;
                row_v = row;
                ++g;
            }
            if (ok) ok = load_v(g - 1, id_v, row_v);
        }
        // every issued copy lands before the CTA may exit
        if (lane == 0) {
            auto drain = [&](int last, int stages, int full) {
                for (int st = 0; st < stages; ++st) {
                    const int x = last - (((last - st) % stages + stages) % stages);
                    if (x >= 0) paged_drain_wait(bar(full + st), (x / stages) & 1, wc, S_T_DRAIN);
                }
            };
            drain(last_k, L::kKStages, T_K_FULL);
            drain(last_v, L::kRaw, T_RAW_FULL);
        }
        __syncwarp();
    } else if (warp < 11) {
        // --------------------------------------------------------------- MMA
        const int t = warp - 9;
        constexpr uint32_t idesc_qk = idesc_e4m3(128, 64), idesc_pv = idesc_f16_mn(128, D);
        const uint64_t q_desc = sdesc_sw128(sbase + L::kQ + t * L::kTile, 16, 1024);
        const uint64_t k_desc0 = D == 128 ? sdesc_sw128(sbase + L::kK, 16, 1024) : sdesc_sw64(sbase + L::kK, 16, 512);
        const uint64_t v_desc0 = sdesc_sw128(sbase + L::kV, L::kBoxHalf, 1024);
        const uint32_t tSt = tmem + 128u * t, tOt = tmem + 256u + D * t;
        // where lo lies: in the box behind hi's, or behind hi in the same row
        constexpr uint32_t kLo = (D == 128 ? 16384u : 64u) >> 4;
        uint32_t g = 0, j = 0, uq = 0, np = 0;
        bool ok = true;
        TileSeg s;
        while (ok && take(s)) {
            const bool active = s.rows > 128 * t;
            const int steps = s.k1 - s.k0;
            // pass k: O += P V(k - 1), then S = Q K(k) into the buffer which
            // that product has released, half by half.  A tile without rows
            // only releases the stages.
            for (int k = 0; ok && k <= steps; ++k) {
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    if (k > 0) {
                        const uint32_t slot = j % L::kHalves;
                        if (!mbar_wait_warp(bar(T_V_FULL + slot), (j / L::kHalves) & 1, wc, S_T_V_FULL)) { ok = false; break; }
                        if (active) {
                            if (!mbar_wait_warp(bar(T_P_FULL + 2 * t + h), np & 1, wc, S_T_P)) { ok = false; break; }
                            tc_fence_after();
                            const uint64_t vd = v_desc0 + ((slot * L::kHalf) >> 4);
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma_ts_elect(tOt, tSt + 64u * h + kk * 8u, vd + kk * 128u, idesc_pv,
                                             (k > 1 || h > 0 || kk > 0) ? 1u : 0u);
                            mma_commit_elect(bar(T_O_UPD + t));
                            if (k == steps && h == 1) mma_commit_elect(bar(T_O_DONE + t));
                        }
                        mma_commit_elect(bar(T_V_EMPTY + slot));
                        ++j;
                    }
                    if (k < steps) {
                        const uint32_t st = g % L::kKStages;
                        if (h == 0 && !mbar_wait_warp(bar(T_K_FULL + st), (g / L::kKStages) & 1, wc, S_T_K_FULL)) { ok = false; break; }
                        if (active) {
                            if (k == 0 && h == 0 && !mbar_wait_warp(bar(T_Q_FULL + t), uq & 1, wc, S_T_Q)) { ok = false; break; }
                            tc_fence_after();
                            const uint64_t kd = k_desc0 + ((st * L::kCodes + h * (L::kCodes / 2)) >> 4);
#pragma unroll
                            for (int kk = 0; kk < D / 32; ++kk)
                                mma_codes_elect(tSt + 64u * h, q_desc + 2u * kk, kd + 2u * kk, idesc_qk, kk > 0);
#pragma unroll
                            for (int kk = 0; kk < D / 32; ++kk)
                                mma_codes_elect(tSt + 64u * h, q_desc + kLo + 2u * kk, kd + 2u * kk, idesc_qk, 1u);
                            mma_commit_elect(bar(T_S_FULL + 2 * t + h));
                        }
                    }
                }
                if (!ok) break;
                if (k > 0 && active) ++np;
                if (k < steps) {
                    mma_commit_elect(bar(T_K_EMPTY + g % L::kKStages));
                    ++g;
                }
            }
            if (active) ++uq;
        }
        mma_commit_elect(bar(T_DRAIN + t));
        paged_drain_wait(bar(T_DRAIN + t), 0, wc, S_T_DRAIN);
        __syncwarp();
    }
    } else {
        // ----------------------------------------------------------- softmax
        regs_increase<kRegsSoftmax8>();
        const int t = warp >> 2, wq = warp & 3, r = wq * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
        const uint32_t tS = tmem + 128u * t + lane_off, tO = tmem + 256u + D * t + lane_off;
        const float sl2 = p.scale * kPagedLog2e;
        const SoftCap cap = soft_cap(p.score.softcap, SCORE == FA_SCORE_SOFTCAP ? p.scale : 1.f);
        const bool out32 = (p.flags & FA_OUT_FP32) != 0;
        const float head = out32 ? kPTop : kPHead;
        uint32_t n = 0, uq = 0, g = 0;                 // g: tiles of all units
        bool ok = true;
        PagedMeta meta{};
        // The warp's 32 rows of a unit's Q, as in paged_tiles.cu, and their split
        // (the copies of all lanes are waited for first).
        float down_next = 1.f;
        bool q_here = false;
        auto bring = [&](const TileSeg& u) {
            if (u.rows > 128 * t) load_rows<D>(p, u, 128 * t + 32 * wq, sbase + L::kQ + t * L::kTile, lane);
        };
        auto announce = [&](const TileSeg& u) {
            if (u.rows <= 128 * t) return;
            copies_wait();
            __syncwarp();
            if (t == 0 && !q_here && lane == 0) mbar_arrive(bar(T_Q_HERE));
            q_here = true;
            down_next = split_rows<D>(smem + L::kQ + t * L::kTile, 32 * wq, lane);
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(T_Q_FULL + t));
        };
        // One pass: the next unit's Q sets out, the current unit's O is written
        // out, the next unit's tiles.
        TileSeg s{}, next{};
        bool have = take(next), done = false;      // done: s has an O to write out
        bool valid = false;
        int ur = 0, hq = 0, trow = 0;
        float m = -CUDART_INF_F, l = 0.f;          // M, l
        for (;;) {
            if (have) bring(next);
            // (the next unit's first products may come while O is read: they go to S)
            if (have) announce(next);
            if (done) {
                if (!mbar_wait_warp(bar(T_O_DONE + t), uq & 1, wc, S_T_O)) { ok = false; break; }
                tc_fence_after();
                ++uq;
                // the unit's end in this CTA: O / l and lse, or a partial
                const bool whole = s.begins() && s.ends(), last = whole && !p.join_rows;
                const long long row = (long long)trow * p.Hq + hq;
                const long long at = whole ? row : (2LL * cta + (s.begins() ? 1 : 0)) * kPagedTileRows + ur;
                const bool f32 = !last || out32;
                uint8_t* const dst = static_cast<uint8_t*>(last ? p.o : static_cast<void*>(whole ? p.parts.row_o : p.parts.slot_o)) +
                                     at * (D * (f32 ? 4 : 2));
                const bool wide = (reinterpret_cast<uintptr_t>(dst) & 31u) == 0;
                const float inv = !last ? even_out(m, l) : l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld32(tO + 32u * c, o);
                    if (!valid) {
                    } else if (f32) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * inv);
#pragma unroll
                        for (int e = 0; e < 32; e += 8) store8(dst + 128 * c + 4 * e, o + e, wide);
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            o[e] = pack_bf16x2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
#pragma unroll
                        for (int e = 0; e < 16; e += 8) store8(dst + 64 * c + 4 * e, o + e, wide);
                    }
                    __syncwarp();                      // together again for the next load
                }
                if (valid) {
                    if (last) {
                        p.lse[row] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * kPagedLn2;
                    } else {
                        (whole ? p.parts.row_ml : p.parts.slot_ml)[at] = make_float2(m, l);
                        if (p.join_rows && !p.prefix && s.begins())
                            p.rowdesc[row] = whole ? make_int2(-1, 1) : make_int2(static_cast<int>(at), s.count(line.per));
                    }
                }
                tc_fence_before();
            }
            if (!have) break;
            s = next;
            const float down = down_next;
            if (s.begins() && !s.ends()) {
                meta.count = s.count(line.per);
                meta.q0 = s.q0;
                meta.row0 = s.row0;
                meta.rows = s.rows;
                meta.h = s.h;
            }
            done = s.rows > 128 * t;
            if (done) {
                // this thread's row: token, query head, position
                ur = 128 * t + r;
                valid = ur < s.rows;
                const int R = s.row0 + min(ur, s.rows - 1), tok = quotient(R, p.by_group);
                hq = s.h * p.group + R - tok * p.group;
                trow = s.q0 + tok;
                int i = s.kv - s.n + tok;
                if (p.prefix) {
                    int lo = 0, hi = p.c.B - 1;        // the first sequence that ends behind the row
                    while (lo < hi) {
                        const int mid = (lo + hi) >> 1;
                        if (q0_s[mid + 1] <= trow) lo = mid + 1; else hi = mid;
                    }
                    i = max(len_s[lo] - q0_s[lo + 1] + trow, -1);
                }
                float slope = 0.f;
                if (SCORE == FA_SCORE_ALIBI) slope = p.score.slopes[hq] * kPagedLog2e;
                if (SCORE == FA_SCORE_ALIBI_SOFTCAP) slope = p.score.slopes[hq];
                const float* rb = nullptr;
                if (SCORE == FA_SCORE_REL_BIAS) rb = p.score.rel_bias + (size_t)hq * (2 * p.score.rel_max + 1);
                // the row's keys: [vlo, vhi] and the sinks from jlo on
                const int vhi = p.mask.causal ? min(s.jhi - 1, i) : s.jhi - 1;
                const int vlo = p.mask.window >= 0 ? max(s.jlo, i - p.mask.window) : s.jlo;

                m = -CUDART_INF_F;
                l = 0.f;
                const float row_scale = SCORE == FA_SCORE_NONE ? down * sl2 : down;
                for (int k = s.k0; ok && k < s.k1; ++k, ++n) {
                    const int kb = s.hull.tile(k);
                    const bool open = tile_open(p.mask, kb, s.i0, s.i1, s.jlo, s.jhi, 7);
                    const uint32_t gt = g + (k - s.k0);
                    const float* const scales = reinterpret_cast<const float*>(smem + L::kScales + 96 * (gt % kScaleRing));
                    if (!mbar_wait_warp(bar(T_SCALES + gt % kScaleRing), (gt / kScaleRing) & 1, wc, S_T_SCALES)) { ok = false; break; }
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t tSh = tS + 64u * h;
                        const int ch = kb * kBlock + 64 * h;
                        // of 16 columns each: what S is to be multiplied by (k's scale
                        // and the row's), v's scale
                        const float4 ks4 = *reinterpret_cast<const float4*>(scales + 4 * h);
                        const float4 lv4 = *reinterpret_cast<const float4*>(scales + 8 + 4 * h);
                        const float4 iv4 = *reinterpret_cast<const float4*>(scales + 16 + 4 * h);
                        const float lv[4] = {lv4.x, lv4.y, lv4.z, lv4.w}, iv[4] = {iv4.x, iv4.y, iv4.z, iv4.w};
                        float sc[4] = {row_scale * ks4.x, row_scale * ks4.y, row_scale * ks4.z, row_scale * ks4.w};
                        if (!mbar_wait_warp(bar(T_S_FULL + 2 * t + h), n & 1, wc, S_T_S)) { ok = false; break; }
                        tc_fence_after();
                        float x[64];
                        {
                            uint32_t raw[64];
                            tmem_ld64(tSh, raw);
#pragma unroll
                            for (int e = 0; e < 64; ++e) x[e] = __uint_as_float(raw[e]);
                        }
                        // with a score_mod x becomes q.k here and the modified score
                        // in base 2 below; without one it stays as it is, to be
                        // multiplied by sc (which is no 0, so that -inf stays what it
                        // is)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const float f = sc[c];
                            if (SCORE == FA_SCORE_NONE) {
                                asm("max.NaN.f32 %0, %1, %2;" : "=f"(sc[c]) : "f"(f), "f"(FLT_MIN));
                            } else {
#pragma unroll
                                for (int e = 16 * c; e < 16 * c + 16; e += 2)
                                    ffma2(x[e], x[e + 1], x[e], x[e + 1], f, f, -0.f, -0.f);
                                sc[c] = 1.f;
                            }
                        }
                        if (SCORE == FA_SCORE_SOFTCAP) softcap_all<true>(x, cap);
                        if (SCORE == FA_SCORE_ALIBI || SCORE == FA_SCORE_ALIBI_SOFTCAP) {
                            const float di = static_cast<float>(i - ch), mul = SCORE == FA_SCORE_ALIBI ? sl2 : p.scale;
                            if (__all_sync(0xffffffffu, di >= 63.f)) {     // i - j >= 0: affine in the column
                                const float c0 = -slope * di;
#pragma unroll
                                for (int e = 0; e < 64; e += 2) {
                                    float b0, b1;
                                    ffma2(b0, b1, slope, slope, static_cast<float>(e), static_cast<float>(e + 1), c0, c0);
                                    ffma2(x[e], x[e + 1], x[e], x[e + 1], mul, mul, b0, b1);
                                }
                            } else {
#pragma unroll
                                for (int e = 0; e < 64; ++e)
                                    x[e] = fmaf(-slope, fabsf(di - static_cast<float>(e)), x[e] * mul);
                            }
                        }
                        if (SCORE == FA_SCORE_ALIBI_SOFTCAP) softcap_all<false>(x, cap);
                        if (SCORE == FA_SCORE_REL_BIAS) {
#pragma unroll
                            for (int e = 0; e < 64; ++e) {
                                const int rr = min(max(i - ch - e, -p.score.rel_max), p.score.rel_max);
                                x[e] = fmaf(rb[rr + p.score.rel_max], kPagedLog2e, x[e] * sl2);
                            }
                        }
                        if (!open) {
                            // the row's visible columns as bits: [jlo, vhi] within
                            // the window or the sinks
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const int c0 = ch + 32 * c;
                                const uint32_t see = bits_from(s.jlo - c0) & bits_to(vhi - c0) &
                                                     (bits_from(vlo - c0) | bits_to(p.mask.sinks - 1 - c0));
#pragma unroll
                                for (int e = 0; e < 32; ++e) x[32 * c + e] = (see >> e) & 1u ? x[32 * c + e] : -CUDART_INF_F;
                            }
                        }
                        float top = -CUDART_INF_F;
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const float* const y = x + 16 * c;
                            float a = fmax3(y[0], y[1], y[2]), b = fmax3(y[3], y[4], y[5]);
                            a = fmax3(a, y[6], y[7]);
                            b = fmax3(b, y[8], y[9]);
                            a = fmax3(a, y[10], y[11]);
                            b = fmax3(b, y[12], y[13]);
                            top = fmaxf(top, fmaf(fmax3(fmaxf(a, b), y[14], y[15]), sc[c], lv[c]));
                        }
                        const bool unset = m == -CUDART_INF_F;
                        const bool need = !unset && top > m + kPTop;
                        const bool raise = __any_sync(0xffffffffu, need);
                        const float to = top - head;
                        float alpha = 1.f;
                        if (raise) {
                            // (in two steps: see times_2_to)
                            const float half = need ? ex2_approx(0.5f * (m - to)) : 1.f;
                            alpha = half * half;
                            l = l * half * half;
                        }
                        if (unset || need) m = to;
                        const float m0 = m == -CUDART_INF_F ? 0.f : m;
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            uint32_t pk[16];
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const int q = 2 * c + u;
                                const float nm = lv[q] - m0;
                                float rs[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    float p0, p1;
                                    exp2_pair(p0, p1, x[16 * q + 2 * e], x[16 * q + 2 * e + 1], sc[q], nm);
                                    const int a2 = (e & 1) * 2;
                                    fadd2(rs[a2], rs[a2 + 1], rs[a2], rs[a2 + 1], p0, p1);
                                    pk[8 * u + e] = pack_p(p0, p1);
                                }
                                l = fmaf((rs[0] + rs[1]) + (rs[2] + rs[3]), iv[q], l);
                            }
                            tmem_st16_nowait(tSh + 16u * c, pk);
                        }
                        // O holds the products of the unit's earlier halves; wait
                        // for the last of them and scale
                        if (raise) {
                            const uint32_t prev = 2 * n + h - 1;
                            if (!mbar_wait_warp(bar(T_O_UPD + t), prev & 1, wc, S_T_UPD)) { ok = false; break; }
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) {
                                uint32_t o[32];
                                tmem_ld32(tO + 32u * c, o);
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                tmem_st32_nowait(tO + 32u * c, o);
                            }
                        }
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(T_P_FULL + 2 * t + h));
                    }
                }
                if (!ok) break;
            }
            g += s.k1 - s.k0;
            have = take(next);
        }
        if (!ok) copies_wait();
        if (!p.join_rows && threadIdx.x == 0) p.meta[cta] = ok ? meta : PagedMeta{};
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (!p.prefix && p.join_rows) pdl_wait_previous();
}

template <int D, int SCORE>
cudaError_t launch_tiles(const PagedScaledParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
    auto kern = paged_tiles_scaled_kernel<D, SCORE>;
    using L = TileLayout8<D>;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::bytes(kPagedMaxSeqs));
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    return paged_launch(kern, dim3(p.ctas), kThreads8, L::bytes(p.c.B), true, s, tk, tv, p);
}

template <int D>
cudaError_t launch_tiles_d(const PagedScaledParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
    switch (p.score.kind) {
        case FA_SCORE_SOFTCAP: return launch_tiles<D, FA_SCORE_SOFTCAP>(p, tk, tv, s);
        case FA_SCORE_ALIBI: return launch_tiles<D, FA_SCORE_ALIBI>(p, tk, tv, s);
        case FA_SCORE_REL_BIAS: return launch_tiles<D, FA_SCORE_REL_BIAS>(p, tk, tv, s);
        case FA_SCORE_ALIBI_SOFTCAP: return launch_tiles<D, FA_SCORE_ALIBI_SOFTCAP>(p, tk, tv, s);
        default: return launch_tiles<D, FA_SCORE_NONE>(p, tk, tv, s);
    }
}

}  // namespace

cudaError_t launch_paged_tiles_scaled(const PagedScaledParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                                      cudaStream_t s) {
    return p.D == 64 ? launch_tiles_d<64>(p, tk, tv, s) : launch_tiles_d<128>(p, tk, tv, s);
}

}  // namespace fa
