// paged_small.cuh -- the attention kernel for a few rows per (sequence, kv
// head), over a cache of bf16 (paged_small.cu, which explains it) or of 8 bits
// (paged_small_scaled.cu: what differs there).
#pragma once

#include <algorithm>
#include <cuda_bf16.h>
#include <math_constants.h>
#include <type_traits>

#include "paged_line.cuh"

namespace fa {
namespace {

constexpr int kWarps = 8;                        // consumers; warp 8 loads
constexpr int kThreadsS = 32 * (kWarps + 1);
constexpr int kRows = kPagedSmallRows;
constexpr int kTileOpen = 1, kTileClear = 2;    // every row sees every key; some key is seen by no row
enum PagedSite : uint32_t { S_PG_FULL = 64, S_PG_EMPTY, S_PG_DRAIN, S_PG_Q, S_PG_Q_EMPTY };

// F8: the cache is held in 8 bits.
template <bool F8>
using SmallParams = std::conditional_t<F8, PagedScaledParams, PagedParams>;
template <int D, bool F8>
struct SmallLayout {
    static constexpr int kKeys = F8 || D == 64 ? 128 : 64;       // = paged_small_keys(D), kPagedSmallScaledKeys
    static constexpr int kShift = kKeys == 128 ? 7 : 6;
    static constexpr uint32_t kBox = kKeys * 64u * 2u;           // bf16: the tile's keys x 64 columns
    static constexpr uint32_t kTile = kKeys * static_cast<uint32_t>(D) * (F8 ? 1u : 2u);
    static constexpr uint32_t kStage = 2u * kTile;               // K then V
    static constexpr int kStages = 98304 / kStage;               // 96 KB
    static constexpr uint32_t kPRow = 2u * kKeys + 16u;          // 16 bytes of padding: rows on distinct banks
    static constexpr uint32_t kP = kStages * kStage;
    static constexpr uint32_t kMax = kP + kRows * kPRow;         // [16 rows][8 warps] fp32
    static constexpr uint32_t kSum = kMax + kRows * kWarps * 4u;
    static constexpr uint32_t kQRow = 2u * D + 16u;
    static constexpr uint32_t kQ = kSum + kRows * kWarps * 4u;   // two units' rows of Q
    static constexpr uint32_t kSeg = kQ + 2u * kRows * kQRow;    // two units, the last one flagged by b < 0
    static constexpr uint32_t kInfo = kSeg + 2u * sizeof(SmallSeg);   // [stage]: 4 x tile + kTileOpen, kTileClear
    static constexpr uint32_t kScale = kInfo + 4u * kStages;     // F8: [stage]: k's scale of each of the tile's pages, v's
    static constexpr uint32_t kScaleStage = F8 ? 8u * (kKeys / 16) : 0u;
    static constexpr uint32_t kBars = (kScale + kScaleStage * kStages + 7u) & ~7u;  // FULL, EMPTY [stage], Q_FULL, Q_EMPTY [2]
    static constexpr uint32_t kAbort = kBars + 16u * kStages + 32u;
    static constexpr uint32_t kScan = kAbort + 16u;              // warp sums
    static constexpr uint32_t kPre = kScan + 64u;                // first tile of each group of sequences
    // two CTAs fit on an SM (228 KB less 1 KB for each); F8's P is wider, and
    // leaves room for fewer entries of the line's index
    static constexpr int kEntries = F8 && D == 128 ? 400 : kLineEntries;
    static constexpr uint32_t bytes(int B) { return kPre + 4u * (groups_of(B, kEntries) + 1u) + 1024u; }
    static_assert(2u * (kPre + 4u * (kEntries + 1u) + 1024u) <= 226u * 1024u, "shared memory budget");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// c += a b, one m16n8k16 tile: a 16x16 bf16 (row), b 16x8 bf16 (col), c fp32
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Byte offset of 16-byte chunk `chunk` of row `row` in a box of 128-byte rows
// written with 128-byte swizzle.
__device__ __forceinline__ uint32_t swz(int row, int chunk) {
    return static_cast<uint32_t>(row * 128 + ((chunk ^ (row & 7)) << 4));
}
// d = a b, one m16n8k16 tile of f16, fp32 sums from 0
__device__ __forceinline__ void mma_f16_from_0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// c += a b, the same
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two e4m3 codes (the lower 16 bits of w, its upper ones) as f16: exact.
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Byte offset of 16-byte chunk `chunk` of key `key` in a tile of codes: a row of
// 128 bytes holds a key of 128 columns, or two of 64.
template <int D>
__device__ __forceinline__ uint32_t swz8(int key, int chunk) {
    return D == 128 ? swz(key, chunk) : swz(key >> 1, 4 * (key & 1) + chunk);
}
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
// The same barrier with a vote: whether `ok` holds in every thread.
__device__ __forceinline__ bool consumers_all(bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(ok))
        : "memory");
    return r != 0;
}

__device__ __forceinline__ float bf_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// F8: a thread's columns of row e of O (times inv), as fp32, and to the output.
template <int D>
__device__ __forceinline__ void store_columns(float* dst, int warp, int tq, const float (&o)[D / 64][4], int e, float inv) {
    if constexpr (D == 128) {
        *reinterpret_cast<float4*>(dst + 16 * warp + 4 * tq) =
            make_float4(o[0][2 * e] * inv, o[1][2 * e] * inv, o[0][2 * e + 1] * inv, o[1][2 * e + 1] * inv);
    } else {
        dst += 16 * (warp >> 1) + 4 * tq + (warp & 1);
        dst[0] = o[0][2 * e] * inv;
        dst[2] = o[0][2 * e + 1] * inv;
    }
}
template <int D>
__device__ __forceinline__ void put_columns(const PagedParams& p, long long at, int warp, int tq,
                                            const float (&o)[D / 64][4], int e, float inv) {
    if (p.flags & FA_OUT_FP32) {
        store_columns<D>(static_cast<float*>(p.o) + at, warp, tq, o, e, inv);
        return;
    }
    if constexpr (D == 128) {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + at + 16 * warp + 4 * tq) =
            make_uint2(pack_bf16x2(o[0][2 * e] * inv, o[1][2 * e] * inv),
                       pack_bf16x2(o[0][2 * e + 1] * inv, o[1][2 * e + 1] * inv));
    } else {
        uint16_t* const dst = static_cast<uint16_t*>(p.o) + at + 16 * (warp >> 1) + 4 * tq + (warp & 1);
        const uint32_t w = pack_bf16x2(o[0][2 * e] * inv, o[0][2 * e + 1] * inv);
        dst[0] = static_cast<uint16_t>(w);
        dst[2] = static_cast<uint16_t>(w >> 16);
    }
}

template <int D, int SCORE, bool F8>
__global__ void __launch_bounds__(kThreadsS, 2)
paged_small_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const SmallParams<F8> p) {
    using L = SmallLayout<D, F8>;
    constexpr int ST = L::kStages, KT = L::kKeys, SH = L::kShift;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_addr(smem);
    auto full_bar = [&](int st) { return sbase + L::kBars + 8u * st; };
    auto empty_bar = [&](int st) { return sbase + L::kBars + 8u * (ST + st); };
    auto q_full = [&](int u) { return sbase + L::kBars + 8u * (2 * ST + (u & 1)); };
    auto q_empty = [&](int u) { return sbase + L::kBars + 8u * (2 * ST + 2 + (u & 1)); };
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kAbort);
    int* const pre = reinterpret_cast<int*>(smem + L::kPre);
    SmallSeg* const seg_s = reinterpret_cast<SmallSeg*>(smem + L::kSeg);
    volatile int* const info_s = reinterpret_cast<volatile int*>(smem + L::kInfo);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;

    if (threadIdx.x == 0) {
        for (int st = 0; st < ST; ++st) {
            mbar_init(full_bar(st), 1);
            mbar_init(empty_bar(st), kWarps);
        }
        for (int u = 0; u < 2; ++u) {
            mbar_init(q_full(u), 1);
            mbar_init(q_empty(u), kWarps);
        }
        *abort_flag = 0;
        mbar_fence_init();
    }
    // (a shared prefix's kernel is no input of this one: it is waited for at the end)
    if (p.join_rows)
        wait_before_prefix(p);
    else
        pdl_wait_previous();
    pdl_launch_next();
    // the line of tiles
    Line line{};
    line.pre = pre;
    line.shift = group_shift(p.c.B, L::kEntries);
    const int groups = groups_of(p.c.B, L::kEntries);
    int* const scan = reinterpret_cast<int*>(smem + L::kScan);
    block_prefix<kThreadsS>(groups, pre, scan, [&](int g) {
        return group_length<SH>(p, line.shift, g, cta == 0 ? p.ws : nullptr);
    });
    line.front = p.c.Hkv * pre[groups] >= kManyTiles * p.ctas;
    if (line.front) {
        block_prefix<kThreadsS>(groups, pre, scan, [&](int g) {
            return group_length_front<SH>(p, line.shift, g, pre[g + 1] - pre[g]);
        });
    }
    const int total = p.c.Hkv * pre[groups];
    line_share(total, p.ctas, cta, line.per, line.t, line.t1);
    if (line.t < line.t1) {
        line.g = line_find(pre, groups, p.c.Hkv, line.t);
        if (warp == kWarps) open_group<SH>(p, line);
    }
    const WaitCtl wc{abort_flag, p.ws, p.timeout_ns};

    if (warp == kWarps) {
        // ------------------------------------------------------------ loader
        if (lane == 0) {
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmV);
        }
        const int span = min(p.c.page_size, KT);
        const uint32_t page_bytes = static_cast<uint32_t>(span) * D * (F8 ? 2u : 4u);    // K and V
        int last[ST];
#pragma unroll
        for (int st = 0; st < ST; ++st) last[st] = -1;
        int g = 0, nu = 0;
        bool ok = true, marked = false;
        SmallSeg s;
        for (; ok; ++nu) {
            const bool more = next_seg<SH>(p, line, s);
            if (nu >= 2 && !mbar_wait_warp(q_empty(nu), ((nu >> 1) - 1) & 1, wc, S_PG_Q_EMPTY)) break;
            if (!more) {
                if (lane == 0) {
                    seg_s[nu & 1].b = -1;
                    mbar_arrive(q_full(nu));
                }
                marked = true;
                break;
            }
            const int32_t* table = p.c.page_table + (size_t)s.b * p.c.max_pages;
            int page = tile_page<KT>(p.c, table, s.hull, s.hull.tile(s.k0), lane, s.b, p.ws);
            // (F8: the page ids come two tiles ahead, the scales, which need them, one)
            int page2 = -1;
            float ks = 0.f, vs = 0.f;
            auto scales_of = [&](int id) {
                if constexpr (F8) {
                    ks = id >= 0 ? p.k_scale[(size_t)id * p.c.Hkv + s.h] : 0.f;
                    vs = id >= 0 ? p.v_scale[(size_t)id * p.c.Hkv + s.h] : 0.f;
                }
            };
            if constexpr (F8) {
                if (s.k0 + 1 < s.k1) page2 = tile_page<KT>(p.c, table, s.hull, s.hull.tile(s.k0 + 1), lane, s.b, p.ws);
                scales_of(page);
            }
            // the unit and its rows of Q, a lane to each, into the slots that
            // the unit before the last has left
            const int rows = s.n * p.group, i0 = s.kv - s.n, i1 = s.kv - 1;
            if (lane == 0) {
                seg_s[nu & 1] = s;
                mbar_arrive_expect_tx(q_full(nu), static_cast<uint32_t>(rows) * 2u * D);
            }
            __syncwarp();
            if (lane < rows) {
                const int tok = quotient(lane, p.by_group);
                bulk_load(sbase + L::kQ + ((nu & 1) * kRows + lane) * L::kQRow,
                          p.q + (long long)(s.q0 + tok) * p.qs[0] +
                              (long long)(s.h * p.group + lane - tok * p.group) * p.qs[1],
                          2u * D, q_full(nu));
            }
            for (int k = s.k0; k < s.k1; ++k, ++g) {
                const int kb = s.hull.tile(k), st = g % ST;
                const int id = page;
                const float ks_now = ks, vs_now = vs;
                if constexpr (F8) {
                    page = page2;
                    if (k + 1 < s.k1) scales_of(page);
                    if (k + 2 < s.k1) page2 = tile_page<KT>(p.c, table, s.hull, s.hull.tile(k + 2), lane, s.b, p.ws);
                } else if (k + 1 < s.k1) {
                    page = tile_page<KT>(p.c, table, s.hull, s.hull.tile(k + 1), lane, s.b, p.ws);
                }
                if (g >= ST && !mbar_wait_warp(empty_bar(st), (g / ST - 1) & 1, wc, S_PG_EMPTY)) { ok = false; break; }
                const uint32_t pages = __popc(__ballot_sync(0xffffffffu, id >= 0));
                if (lane == 0) {
                    info_s[st] = 4 * kb + (tile_open(p.mask, kb, i0, i1, p.shared, s.kv, SH) ? kTileOpen : 0) +
                                 (s.hull.all(kb * KT, kb * KT + KT) ? 0 : kTileClear);
                    if constexpr (F8)
                        mbar_expect_tx(full_bar(st), pages * page_bytes);
                    else
                        mbar_arrive_expect_tx(full_bar(st), pages * page_bytes);
                }
                __syncwarp();
                if (F8 && id >= 0) {
                    const uint32_t dst = sbase + st * L::kStage + static_cast<uint32_t>(lane * span) * D;
                    const int row = ((kb * KT + lane * span) & (p.c.page_size - 1)) / (128 / D);
                    const int block = id * p.c.Hkv + s.h;
                    tma_load_3d(dst, &tmK, full_bar(st), 0, row, block);
                    tma_load_3d(dst + L::kTile, &tmV, full_bar(st), 0, row, block);
                }
                if constexpr (F8) {
                    // the scales, and only then the loader's arrival
                    float* const sc = reinterpret_cast<float*>(smem + L::kScale + st * L::kScaleStage);
                    if (lane < KT / 16) {
                        sc[lane] = ks_now;
                        sc[KT / 16 + lane] = vs_now;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(full_bar(st));
                }
                if (!F8 && id >= 0) {
                    const uint32_t dst = sbase + st * L::kStage + static_cast<uint32_t>(lane * span) * 128u;
                    const int row = (kb * KT + lane * span) & (p.c.page_size - 1);
                    const int block = id * p.c.Hkv + s.h;
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        tma_load_3d(dst + c * L::kBox, &tmK, full_bar(st), c * 64, row, block);
                        tma_load_3d(dst + (D / 64 + c) * L::kBox, &tmV, full_bar(st), c * 64, row, block);
                    }
                }
                last[st] = g;
            }
        }
        // every issued copy lands before the CTA exits
        if (lane == 0) {
#pragma unroll
            for (int st = 0; st < ST; ++st)
                if (last[st] >= 0) paged_drain_wait(full_bar(st), (last[st] / ST) & 1, wc, S_PG_DRAIN);
            // (behind the end mark only the last unit's rows can be on their
            // way: the mark's slot had been read)
            for (int u = max(nu - (marked ? 1 : 2), 0); u < nu; ++u)
                paged_drain_wait(q_full(u), (u >> 1) & 1, wc, S_PG_DRAIN);
        }
        __syncwarp();
        if (p.join_rows) pdl_wait_previous();
        return;
    }

    // --------------------------------------------------------------- consumers
    const int gr = lane >> 2, tq = lane & 3, mi = lane >> 3, l8 = lane & 7;
    float* const smax = reinterpret_cast<float*>(smem + L::kMax);
    float* const ssum = reinterpret_cast<float*>(smem + L::kSum);
    const uint32_t sP = sbase + L::kP;
    // score_mod, to base 2
    const float sl2 = p.scale * kPagedLog2e;
    const SoftCap cap = soft_cap(p.score.softcap, SCORE == FA_SCORE_SOFTCAP ? p.scale : 1.f);
    constexpr int kNT = D / 64;                    // n8 tiles of O per warp
    // F8: columns of O by thread: 16 (warp's chunk) + 4 tq + {0, 2} of tile 0,
    // {1, 3} of tile 1; with 64 columns two warps share a chunk, a tile each
    const int chunk8 = D == 128 ? warp : warp >> 1;
    const uint32_t pick8 = D == 128 ? 0x3120u : (warp & 1) ? 0x0031u : 0x0020u;
    const int by_page = min(p.c.page_shift, SH);   // F8: 2^by_page keys of a tile share a page
    constexpr int kKW = KT / 8, kNK = kKW / 8;     // keys per warp, n8 tiles of S
    const int col0 = warp * (D / 8);               // the warp's first column of O
    int g = 0;
    bool ok = true;
    PagedMeta meta{};
    for (int nu = 0;; ++nu) {
        const bool q_here = mbar_wait_warp(q_full(nu), (nu >> 1) & 1, wc, S_PG_Q);
        // (the vote keeps the warps together where a wait has run out)
        if (!consumers_all(q_here)) { ok = false; break; }
        const SmallSeg s = seg_s[nu & 1];
        if (s.b < 0) break;
        const int rows = s.n * p.group, i0 = s.kv - s.n;
        int tok[2], hq[2];
        float slope[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = min(gr + 8 * e, rows - 1);
            tok[e] = quotient(r, p.by_group);
            hq[e] = s.h * p.group + r - tok[e] * p.group;
            if (SCORE == FA_SCORE_ALIBI) slope[e] = p.score.slopes[hq[e]] * kPagedLog2e;
            if (SCORE == FA_SCORE_ALIBI_SOFTCAP) slope[e] = p.score.slopes[hq[e]];
        }
        // Q's fragments (what the rows past the unit's hold stays in those rows)
        uint32_t qa[D / 16][4];
        float unscale[2] = {1.f, 1.f};
        if constexpr (F8) {
            // In f16, which holds a code exactly and a bf16 number too, within
            // f16's exponents: each row is scaled by a power of two to a largest
            // element of 2^14 .. 2^15, so that those below f16's normal numbers
            // are 2^28 times smaller than it.  (A code's row of 16 columns takes
            // its columns 4 tq .. 4 tq + 3 where the matrix product has 2 tq,
            // 2 tq + 1, 2 tq + 8 and 2 tq + 9.)
            uint2 raw[2][D / 16];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float top = 0.f;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    raw[e][ks] = *reinterpret_cast<const uint2*>(smem + L::kQ + ((nu & 1) * kRows + gr + 8 * e) * L::kQRow +
                                                                 2 * (16 * ks + 4 * tq));
                    top = fmaxf(top, fmaxf(fmaxf(fabsf(bf_low(raw[e][ks].x)), fabsf(bf_high(raw[e][ks].x))),
                                           fmaxf(fabsf(bf_low(raw[e][ks].y)), fabsf(bf_high(raw[e][ks].y)))));
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int at = max(__float_as_int(top) >> 23, 15);
                const float up = __int_as_float((268 - at) << 23);
                unscale[e] = __int_as_float((at - 14) << 23);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    qa[ks][e] = pack_f16x2(bf_low(raw[e][ks].x) * up, bf_high(raw[e][ks].x) * up);
                    qa[ks][2 + e] = pack_f16x2(bf_low(raw[e][ks].y) * up, bf_high(raw[e][ks].y) * up);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(q_empty(nu));
        } else {
            const uint32_t q_row = sbase + L::kQ + ((nu & 1) * kRows + l8 + 8 * (mi & 1)) * L::kQRow + 16 * (mi >> 1);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) ldsm4(q_row + 32 * ks, qa[ks]);
            __syncwarp();
            if (lane == 0) mbar_arrive(q_empty(nu));
        }
        float m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f};
        float o[kNT][4];
#pragma unroll
        for (int n = 0; n < kNT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;

        for (int k = s.k0; k < s.k1; ++k, ++g) {
            const int st = g % ST;
            const uint32_t kbase = sbase + st * L::kStage, vbase = kbase + L::kTile;
            const bool here = mbar_wait_warp(full_bar(st), (g / ST) & 1, wc, S_PG_FULL);
            const int info = info_s[st], c0 = (info >> 2) * KT;
            float x[kNK][4];
#pragma unroll
            for (int nt = 0; nt < kNK; ++nt) x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.f;
            float mx[2] = {-CUDART_INF_F, -CUDART_INF_F};
            bool cleared = false;
            if (here) {
                if constexpr (F8) {
                    const int key = 16 * warp + 8 * (mi >> 1) + l8;
#pragma unroll
                    for (int ks = 0; ks < D / 16; ks += 2) {
                        uint32_t kf[4];
                        ldsm4(kbase + swz8<D>(key, ks + (mi & 1)), kf);
                        mma_f16(x[0], qa[ks], codes_lo(kf[0]), codes_hi(kf[0]));
                        mma_f16(x[1], qa[ks], codes_lo(kf[2]), codes_hi(kf[2]));
                        mma_f16(x[0], qa[ks + 1], codes_lo(kf[1]), codes_hi(kf[1]));
                        mma_f16(x[1], qa[ks + 1], codes_lo(kf[3]), codes_hi(kf[3]));
                    }
                    const float* const sc = reinterpret_cast<const float*>(smem + L::kScale + st * L::kScaleStage);
                    const float k_scale = sc[16 * warp >> by_page];
#pragma unroll
                    for (int nt = 0; nt < kNK; ++nt) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) x[nt][c] = x[nt][c] * unscale[c >> 1] * k_scale;
                    }
                } else if constexpr (kNK == 2) {
                    const int key = 16 * warp + 8 * (mi >> 1) + l8;
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        uint32_t kf[4];
                        ldsm4(kbase + (ks >> 2) * L::kBox + swz(key, 2 * (ks & 3) + (mi & 1)), kf);
                        mma_16816(x[0], qa[ks], kf[0], kf[1]);
                        mma_16816(x[1], qa[ks], kf[2], kf[3]);
                    }
                } else {
                    // 8 keys: two K steps per load; two sums, so that the products do not all wait in one chain
                    float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int ks = 0; ks < D / 16; ks += 2) {
                        uint32_t kf[4];
                        ldsm4(kbase + (ks >> 2) * L::kBox + swz(8 * warp + l8, 2 * (ks & 3) + mi), kf);
                        mma_16816(x[0], qa[ks], kf[0], kf[1]);
                        mma_16816(y, qa[ks + 1], kf[2], kf[3]);
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) x[0][c] += y[c];
                }
                const bool open = (info & kTileOpen) != 0;
#pragma unroll
                for (int nt = 0; nt < kNK; ++nt) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int e = c >> 1, j = c0 + kKW * warp + 8 * nt + 2 * tq + (c & 1);
                        float v = x[nt][c];
                        const float far = fabsf(static_cast<float>(i0 + tok[e] - j));
                        if (SCORE == FA_SCORE_NONE || SCORE == FA_SCORE_REL_BIAS) v *= sl2;
                        if (SCORE == FA_SCORE_SOFTCAP) v = softcap_one(v, cap);
                        if (SCORE == FA_SCORE_ALIBI) v = fmaf(-slope[e], far, v * sl2);
                        if (SCORE == FA_SCORE_ALIBI_SOFTCAP) v = softcap_one(fmaf(-slope[e], far, v * p.scale), cap);
                        if (SCORE == FA_SCORE_REL_BIAS) {
                            const int R = p.score.rel_max, d = min(max(i0 + tok[e] - j, -R), R);
                            v = fmaf(p.score.rel_bias[(size_t)hq[e] * (2 * R + 1) + d + R], kPagedLog2e, v);
                        }
                        if (!open && !paged_visible(p.mask, i0 + tok[e], j, p.shared, s.kv)) v = -CUDART_INF_F;
                        x[nt][c] = v;
                        mx[e] = fmaxf(mx[e], v);
                    }
                }
                // V rows that no row of the unit sees
                const int a = c0 + kKW * warp;
                if (info & kTileClear) {
                    cleared = true;
                    for (int r = 0; r < kKW; ++r) {
                        if (s.hull.live(a + r)) continue;
                        if (F8 && lane < D / 16)
                            *reinterpret_cast<uint4*>(smem + st * L::kStage + L::kTile + swz8<D>(kKW * warp + r, lane)) =
                                make_uint4(0u, 0u, 0u, 0u);
                        if (!F8 && lane < D / 8)
                            *reinterpret_cast<uint4*>(smem + st * L::kStage + (D / 64 + (lane >> 3)) * L::kBox +
                                                      swz(kKW * warp + r, lane & 7)) = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
                    mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
                    if (tq == 0) smax[(gr + 8 * e) * kWarps + warp] = mx[e];
                }
            }
            // (a warp whose wait ran out still comes here, so that all leave together)
            if (!consumers_all(here)) { ok = false; break; }
            float alpha[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float4 a = *reinterpret_cast<const float4*>(smax + (gr + 8 * e) * kWarps);
                const float4 b = *reinterpret_cast<const float4*>(smax + (gr + 8 * e) * kWarps + 4);
                const float m_new = fmaxf(fmaxf(fmaxf(fmaxf(a.x, a.y), fmaxf(a.z, a.w)),
                                                fmaxf(fmaxf(b.x, b.y), fmaxf(b.z, b.w))), m[e]);
                alpha[e] = m_new == m[e] ? 1.f : ex2_approx(m[e] - m_new);
                const float nm = m_new == -CUDART_INF_F ? 0.f : -m_new;
                m[e] = m_new;
                l[e] *= alpha[e];
#pragma unroll
                for (int nt = 0; nt < kNK; ++nt) {
                    const float p0 = ex2_approx(x[nt][2 * e] + nm), p1 = ex2_approx(x[nt][2 * e + 1] + nm);
                    l[e] += p0 + p1;
                    *reinterpret_cast<uint32_t*>(smem + L::kP + (gr + 8 * e) * L::kPRow +
                                                 2 * (kKW * warp + 8 * nt + 2 * tq)) =
                        F8 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
                }
            }
#pragma unroll
            for (int n = 0; n < kNT; ++n) {
                o[n][0] *= alpha[0];
                o[n][1] *= alpha[0];
                o[n][2] *= alpha[1];
                o[n][3] *= alpha[1];
            }
            consumers_sync();
            // O[:, col0 ..] += P V over the tile's keys
            const uint32_t p_row = sP + (l8 + 8 * (mi & 1)) * L::kPRow + 16 * (mi >> 1);
            if constexpr (F8) {
                // 16 keys at a time, which are of one page, and its scale on their sum
                const float* const sc = reinterpret_cast<const float*>(smem + L::kScale + st * L::kScaleStage) + KT / 16;
#pragma unroll
                for (int ks = 0; ks < KT / 16; ks += 2) {
                    uint32_t vf[4];
                    ldsm4_t(vbase + swz8<D>(16 * ks + 8 * mi + l8, chunk8), vf);
#pragma unroll
                    for (int e = 0; e < 4; ++e) vf[e] = __byte_perm(vf[e], 0u, pick8);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t pa[4];
                        ldsm4(p_row + 32 * (ks + e), pa);
                        const float v_scale = sc[16 * (ks + e) >> by_page];
                        float y[4];
                        mma_f16_from_0(y, pa, codes_lo(vf[2 * e]), codes_lo(vf[2 * e + 1]));
#pragma unroll
                        for (int c = 0; c < 4; ++c) o[0][c] = fmaf(y[c], v_scale, o[0][c]);
                        if constexpr (kNT == 2) {
                            mma_f16_from_0(y, pa, codes_hi(vf[2 * e]), codes_hi(vf[2 * e + 1]));
#pragma unroll
                            for (int c = 0; c < 4; ++c) o[1][c] = fmaf(y[c], v_scale, o[1][c]);
                        }
                    }
                }
            } else
#pragma unroll
            for (int ks = 0; ks < KT / 16; ks += 2) {
                uint32_t pa[4], pb[4], vf[4];
                ldsm4(p_row + 32 * ks, pa);
                ldsm4(p_row + 32 * (ks + 1), pb);
                if constexpr (kNT == 2) {
                    const int dt = 2 * warp + (mi >> 1);
                    const uint32_t v0 = vbase + (dt >> 3) * L::kBox;
                    uint32_t vg[4];
                    ldsm4_t(v0 + swz(16 * ks + 8 * (mi & 1) + l8, dt & 7), vf);
                    ldsm4_t(v0 + swz(16 * (ks + 1) + 8 * (mi & 1) + l8, dt & 7), vg);
                    mma_16816(o[0], pa, vf[0], vf[1]);
                    mma_16816(o[1], pa, vf[2], vf[3]);
                    mma_16816(o[0], pb, vg[0], vg[1]);
                    mma_16816(o[1], pb, vg[2], vg[3]);
                } else {
                    ldsm4_t(vbase + swz(16 * ks + 8 * mi + l8, warp), vf);
                    mma_16816(o[0], pa, vf[0], vf[1]);
                    mma_16816(o[0], pb, vf[2], vf[3]);
                }
            }
            if (cleared) fence_async_shared();     // the next copy into this stage comes after the clearing
            __syncwarp();
            if (lane == 0) mbar_arrive(empty_bar(st));
        }
        if (!ok) break;

        // the unit's end in this CTA: row sums over the lanes and warps
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
            if (tq == 0) ssum[(gr + 8 * e) * kWarps + warp] = l[e];
        }
        consumers_sync();
        const bool whole = s.begins() && s.ends();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = gr + 8 * e;
            if (r >= rows) continue;
            const float4 a = *reinterpret_cast<const float4*>(ssum + r * kWarps);
            const float4 b = *reinterpret_cast<const float4*>(ssum + r * kWarps + 4);
            const float sum = ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w));
            const long long row = (long long)(s.q0 + tok[e]) * p.Hq + hq[e];
            if (whole && !p.join_rows) {
                const float inv = sum == 0.f ? 0.f : 1.f / sum;      // a NaN stays one
                if constexpr (F8) {
                    put_columns<D>(p, row * D, warp, tq, o, e, inv);
                } else
#pragma unroll
                for (int n = 0; n < kNT; ++n) {
                    const long long at = row * D + col0 + 8 * n + 2 * tq;
                    const float y0 = o[n][2 * e] * inv, y1 = o[n][2 * e + 1] * inv;
                    if (p.flags & FA_OUT_FP32)
                        *reinterpret_cast<float2*>(static_cast<float*>(p.o) + at) = make_float2(y0, y1);
                    else
                        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + at) = pack_bf16x2(y0, y1);
                }
                if (warp == 0 && tq == 0) p.lse[row] = sum == 0.f ? -CUDART_INF_F : (m[e] + log2f(sum)) * kPagedLn2;
            } else {
                const long long slot = whole ? row : (2LL * cta + (s.begins() ? 1 : 0)) * kRows + r;
                float* dst = (whole ? p.parts.row_o : p.parts.slot_o) + slot * D + col0 + 2 * tq;
                if constexpr (F8) {
                    store_columns<D>((whole ? p.parts.row_o : p.parts.slot_o) + slot * D, warp, tq, o, e, 1.f);
                } else
#pragma unroll
                for (int n = 0; n < kNT; ++n)
                    *reinterpret_cast<float2*>(dst + 8 * n) = make_float2(o[n][2 * e], o[n][2 * e + 1]);
                if (warp == 0 && tq == 0) {
                    (whole ? p.parts.row_ml : p.parts.slot_ml)[slot] = make_float2(m[e], sum);
                    if (p.join_rows && s.begins())
                        p.rowdesc[row] = whole ? make_int2(-1, 1)
                                               : make_int2((2 * cta + 1) * kRows + r, s.count);
                }
            }
        }
        if (s.begins() && !s.ends()) {
            meta.count = s.count;
            meta.q0 = s.q0;
            meta.rows = rows;
            meta.h = s.h;
        }
    }
    if (!p.join_rows && threadIdx.x == 0) p.meta[cta] = ok ? meta : PagedMeta{};
    if (p.join_rows) pdl_wait_previous();
}

template <int D, int SCORE, bool F8>
cudaError_t launch_small(const SmallParams<F8>& p, const CUtensorMap& tk, const CUtensorMap& tv,
                         cudaStream_t s) {
    auto kern = paged_small_kernel<D, SCORE, F8>;
    using L = SmallLayout<D, F8>;
    constexpr size_t most = L::bytes(L::kEntries);
    static bool attr_set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    return paged_launch(kern, dim3(p.ctas), kThreadsS, L::bytes(p.c.B), true, s, tk, tv, p);
}

template <int D, bool F8>
cudaError_t launch_small_d(const SmallParams<F8>& p, const CUtensorMap& tk, const CUtensorMap& tv,
                           cudaStream_t s) {
    switch (p.score.kind) {
        case FA_SCORE_SOFTCAP: return launch_small<D, FA_SCORE_SOFTCAP, F8>(p, tk, tv, s);
        case FA_SCORE_ALIBI: return launch_small<D, FA_SCORE_ALIBI, F8>(p, tk, tv, s);
        case FA_SCORE_REL_BIAS: return launch_small<D, FA_SCORE_REL_BIAS, F8>(p, tk, tv, s);
        case FA_SCORE_ALIBI_SOFTCAP: return launch_small<D, FA_SCORE_ALIBI_SOFTCAP, F8>(p, tk, tv, s);
        default: return launch_small<D, FA_SCORE_NONE, F8>(p, tk, tv, s);
    }
}

}  // namespace
}  // namespace fa
