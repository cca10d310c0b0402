// paged_codes.cuh -- what the two kernels for a few rows over a cache held in 8
// bits share (paged_eight_scaled.cu, paged_small_scaled.cu): codes in registers,
// where they lie in shared memory, the line of tiles and the loader.
#pragma once

#include <algorithm>
#include <math_constants.h>

#include "paged_line.cuh"

namespace fa {
namespace {

constexpr int kKeys = kPagedSmallScaledKeys, kShift = 7;
constexpr int kTileOpen = 1, kTileClear = 2;    // every row sees every key; some key is seen by no row
static_assert(kKeys == 1 << kShift, "keys of a tile");
// Units that the consumers read where the loader puts them.  It writes unit nu once
// all of them have begun unit nu - 2, and so are done with nu - 3.
constexpr int kSegs = 4;
// Entries of the line's index: what two CTAs on an SM leave room for (the assertion
// below; 16 rows of 128 columns have 268 bytes to spare).
constexpr int kCodeEntries = 300;
enum CodeSite : uint32_t { S_PC_FULL = 112, S_PC_EMPTY, S_PC_DRAIN, S_PC_Q, S_PC_Q_EMPTY };

// Shared memory of such a kernel: the ring of tiles, `EXTRA` bytes of the
// kernel's own, two units' rows of Q, units, scales, barriers, the line's index.
template <int D, int WARPS, int LOADERS, int ROWS, uint32_t EXTRA>
struct CodeLayout {
    static constexpr int kD = D, kWarps = WARPS, kThreads = 32 * (WARPS + LOADERS), kRows = ROWS;
    static constexpr uint32_t kTile = kKeys * static_cast<uint32_t>(D);
    static constexpr uint32_t kStage = 2u * kTile;               // K then V
    static constexpr int kStages = 98304 / kStage;               // 96 KB
    static constexpr uint32_t kExtra = kStages * kStage;
    static constexpr uint32_t kQRow = 2u * D + 16u;              // rows on distinct banks
    static constexpr uint32_t kQ = (kExtra + EXTRA + 15u) & ~15u;
    static constexpr uint32_t kSeg = kQ + 2u * kRows * kQRow;    // [kSegs], the one behind the last flagged by b < 0
    // [stage][k's scale, v's, its log2, 1 / it][the tile's pages]
    static constexpr uint32_t kScale = kSeg + kSegs * sizeof(SmallSeg);
    static constexpr uint32_t kScaleStage = 16u * (kKeys / 16);
    static constexpr uint32_t kInfo = kScale + kScaleStage * kStages;     // [stage]: 4 x tile + kTileOpen, kTileClear
    static constexpr uint32_t kBars = (kInfo + 4u * kStages + 7u) & ~7u;  // FULL, EMPTY [stage], Q_FULL, Q_EMPTY [2]
    static constexpr uint32_t kAbort = kBars + 16u * kStages + 32u;
    static constexpr uint32_t kScan = kAbort + 16u;              // warp sums
    static constexpr uint32_t kPre = kScan + 64u;                // first tile of each group of sequences
    static constexpr uint32_t bytes(int B) { return kPre + 4u * (groups_of(B, kCodeEntries) + 1u) + 1024u; }
    // two CTAs fit on an SM (228 KB less 1 KB for each)
    static_assert(2u * (kPre + 4u * (kCodeEntries + 1u) + 1024u) <= 226u * 1024u, "shared memory budget");
    static __device__ __forceinline__ uint32_t full(uint32_t sbase, int st) { return sbase + kBars + 8u * st; }
    static __device__ __forceinline__ uint32_t empty(uint32_t sbase, int st) { return sbase + kBars + 8u * (kStages + st); }
    static __device__ __forceinline__ uint32_t q_full(uint32_t sbase, int u) { return sbase + kBars + 8u * (2 * kStages + (u & 1)); }
    static __device__ __forceinline__ uint32_t q_empty(uint32_t sbase, int u) {
        return sbase + kBars + 8u * (2 * kStages + 2 + (u & 1));
    }
    static __device__ __forceinline__ void init(uint32_t sbase) {
        for (int st = 0; st < kStages; ++st) {
            mbar_init(full(sbase, st), LOADERS);
            mbar_init(empty(sbase, st), kWarps);
        }
        for (int u = 0; u < 2; ++u) {
            mbar_init(q_full(sbase, u), 1);
            mbar_init(q_empty(sbase, u), kWarps);
        }
    }
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
// Four e4m3 codes as two pairs of f16: exact.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float bf_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// Byte offset of 16-byte chunk `chunk` of key `key` in a tile of codes, rows of
// 128 bytes written with 128-byte swizzle: a key of 128 columns, or two of 64.
template <int D>
__device__ __forceinline__ uint32_t swz8(int key, int chunk) {
    const int row = D == 128 ? key : key >> 1, at = D == 128 ? chunk : 4 * (key & 1) + chunk;
    return static_cast<uint32_t>(row * 128 + ((at ^ (row & 7)) << 4));
}

// The CTA's stretch of the line of tiles (the whole block).
template <class L>
__device__ __forceinline__ Line code_line(const PagedParams& p, uint8_t* smem, int cta, bool loads) {
    int* const pre = reinterpret_cast<int*>(smem + L::kPre);
    Line line{};
    line.pre = pre;
    line.shift = group_shift(p.c.B, kCodeEntries);
    const int groups = groups_of(p.c.B, kCodeEntries);
    int* const scan = reinterpret_cast<int*>(smem + L::kScan);
    block_prefix<L::kThreads>(groups, pre, scan, [&](int g) {
        return group_length<kShift>(p, line.shift, g, cta == 0 ? p.ws : nullptr);
    });
    line.front = p.c.Hkv * pre[groups] >= kManyTiles * p.ctas;
    if (line.front) {
        block_prefix<L::kThreads>(groups, pre, scan, [&](int g) {
            return group_length_front<kShift>(p, line.shift, g, pre[g + 1] - pre[g]);
        });
    }
    const int total = p.c.Hkv * pre[groups];
    line_share(total, p.ctas, cta, line.per, line.t, line.t1);
    if (line.t < line.t1) {
        line.g = line_find(pre, groups, p.c.Hkv, line.t);
        if (loads) open_group<kShift>(p, line);
    }
    return line;
}

// The loader warp: walks the stretch, hands each unit and its rows of Q to the
// consumers, and brings the tiles of codes, their scales and what else there is
// to know of them.
//
// Up to 32 pages, a lane to each, are a batch of a unit's tiles.  Three batches
// are on their way: the copies of one are issued, the next one's scales come, and
// the page ids, which those need, of the one behind (128 ragged chats of 64
// columns: a quarter less time than with ids and scales a tile or two ahead
// within a unit).
//
// Pages of 16 keys are 16 copies a tile, which a warp issues one lane after the
// other.  Two warps may share them, one for K and all else, one for V: 76.6 us for
// those chats instead of 83.4, 9.9 for a single one instead of 9.1.  Copies of 16
// bytes by every lane, which a page of 1 KB is still small enough for: 88.8.
enum LoadPart { kLoadBoth, kLoadK, kLoadV };
template <class L, int PART>
__device__ __forceinline__ void load_codes(const PagedScaledParams& p, const CUtensorMap& tmK, const CUtensorMap& tmV, Line line,
                                           uint8_t* smem, uint32_t sbase, const WaitCtl& wc, int lane) {
    constexpr int D = L::kD, ST = L::kStages;
    SmallSeg* const seg_s = reinterpret_cast<SmallSeg*>(smem + L::kSeg);
    volatile int* const info_s = reinterpret_cast<volatile int*>(smem + L::kInfo);
    auto full_bar = [&](int st) { return L::full(sbase, st); };
    auto empty_bar = [&](int st) { return L::empty(sbase, st); };
    auto q_full = [&](int u) { return L::q_full(sbase, u); };
    auto q_empty = [&](int u) { return L::q_empty(sbase, u); };
    if (lane == 0) {
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    const int span = min(p.c.page_size, kKeys), pages = kKeys / span;    // 1, 2, 4 or 8
    const int most = 32 / pages, mine = lane / pages, at = lane & (pages - 1);
    const uint32_t page_bytes = static_cast<uint32_t>(span) * D * (PART == kLoadBoth ? 2u : 1u);
    int last[ST];
#pragma unroll
    for (int st = 0; st < ST; ++st) last[st] = -1;
    struct Batch {
        SmallSeg s;
        int k, tiles, id;
    };
    int at_k = 0;
    bool in_unit = false;
    // (b holds the batch before this one, and its unit if that goes on)
    auto next_batch = [&](Batch& b) {
        b.tiles = 0;
        b.id = -1;
        if (!in_unit) {
            if (!next_seg<kShift>(p, line, b.s)) return;
            at_k = b.s.k0;
        }
        b.k = at_k;
        b.tiles = min(most, b.s.k1 - at_k);
        at_k += b.tiles;
        in_unit = at_k < b.s.k1;
        if (mine < b.tiles)
            b.id = tile_page<kKeys>(p.c, p.c.page_table + (size_t)b.s.b * p.c.max_pages, b.s.hull, b.s.hull.tile(b.k + mine), at,
                                    b.s.b, p.ws);
    };
    auto scales_of = [&](const Batch& b) {
        const size_t x = (size_t)max(b.id, 0) * p.c.Hkv + b.s.h;
        return PART != kLoadV && b.id >= 0 ? make_float2(p.k_scale[x], p.v_scale[x]) : make_float2(0.f, 0.f);
    };
    int g = 0, nu = 0;
    bool ok = true, marked = false, first = true;
    Batch now, next{};
    float2 scales, scales_next{};
    float largest = 0.f;                           // of v's scales in the unit
    next_batch(next);
    for (;; first = false) {
        now = next;
        scales = scales_next;
        next_batch(next);
        const bool fresh = now.tiles == 0 || now.k == now.s.k0;
        if (PART == kLoadV) {
            if (now.tiles == 0) break;
        } else if (fresh) {
            if (nu >= 2 && !mbar_wait_warp(q_empty(nu), ((nu >> 1) - 1) & 1, wc, S_PC_Q_EMPTY)) break;
            if (now.tiles == 0) {
                if (lane == 0) {
                    seg_s[nu % kSegs].b = -1;
                    mbar_arrive(q_full(nu));
                }
                marked = true;
                break;
            }
            // the unit and its rows of Q, a lane to each, into the slots that
            // the unit before the last has left
            largest = 0.f;
            const SmallSeg& s = now.s;
            const int rows = s.n * p.group;
            if (lane == 0) {
                seg_s[nu % kSegs] = s;
                mbar_arrive_expect_tx(q_full(nu), static_cast<uint32_t>(rows) * 2u * D);
            }
            __syncwarp();
            if (lane < rows) {
                const int tok = quotient(lane, p.by_group);
                bulk_load(sbase + L::kQ + ((nu & 1) * L::kRows + lane) * L::kQRow,
                          p.q + (long long)(s.q0 + tok) * p.qs[0] +
                              (long long)(s.h * p.group + lane - tok * p.group) * p.qs[1],
                          2u * D, q_full(nu));
            }
            ++nu;
        }
        // (the first batch's scales need its page ids, which Q does not wait for)
        if (first) scales = scales_of(now);
        scales_next = scales_of(next);
        float lv = 0.f, iv = 0.f;
        for (int e = 0; e < now.tiles; ++e, ++g) {
            const int kb = now.s.hull.tile(now.k + e), st = g % ST;
            const bool here = mine == e;
            if (g >= ST && !mbar_wait_warp(empty_bar(st), (g / ST - 1) & 1, wc, S_PC_EMPTY)) { ok = false; break; }
            const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, here && now.id >= 0)) * page_bytes;
            if (lane == 0) {
                if (PART == kLoadV)
                    mbar_arrive_expect_tx(full_bar(st), bytes);
                else
                    mbar_expect_tx(full_bar(st), bytes);
            }
            __syncwarp();
            if (here && now.id >= 0) {
                const uint32_t dst = sbase + st * L::kStage + static_cast<uint32_t>(at * span) * D;
                const int row = ((kb * kKeys + at * span) & (p.c.page_size - 1)) / (128 / D);
                const int block = now.id * p.c.Hkv + now.s.h;
                if (PART != kLoadV) tma_load_3d(dst, &tmK, full_bar(st), 0, row, block);
                if (PART != kLoadK) tma_load_3d(dst + L::kTile, &tmV, full_bar(st), 0, row, block);
            }
            last[st] = g;
            if (PART == kLoadV) continue;
            // what else the consumers need of the tile, and only then the loader's
            // arrival; the first copies do not wait for the scales
            if (e == 0) {
                // (bits of numbers that are not negative are in their order)
                largest = fmaxf(largest, __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(scales.y, 0.f)))));
                float least = fmaxf(fmaxf(scales.y, largest * kLeastRatio), kLeastScale);
                if (scales.y != scales.y) least = scales.y;
                lv = log2f(least);
                iv = 1.f / least;
            }
            float* const sc = reinterpret_cast<float*>(smem + L::kScale + st * L::kScaleStage);
            if (here) {
                sc[at] = scales.x;
                sc[kKeys / 16 + at] = scales.y;
                sc[2 * (kKeys / 16) + at] = lv;
                sc[3 * (kKeys / 16) + at] = iv;
            }
            if (lane == 0)
                info_s[st] = 4 * kb +
                             (tile_open(p.mask, kb, now.s.kv - now.s.n, now.s.kv - 1, p.shared, now.s.kv, kShift) ? kTileOpen : 0) +
                             (now.s.hull.all(kb * kKeys, kb * kKeys + kKeys) ? 0 : kTileClear);
            __syncwarp();
            if (lane == 0) mbar_arrive(full_bar(st));
        }
        if (!ok) break;
    }
    // every issued copy lands before the CTA exits
    if (lane == 0) {
#pragma unroll
        for (int st = 0; st < ST; ++st)
            if (last[st] >= 0) paged_drain_wait(full_bar(st), (last[st] / ST) & 1, wc, S_PC_DRAIN);
        // (behind the end mark only the last unit's rows can be on their
        // way: the mark's slot had been read)
        for (int u = max(nu - (marked ? 1 : 2), 0); u < nu; ++u)         // (kLoadV has none)
            paged_drain_wait(q_full(u), (u >> 1) & 1, wc, S_PC_DRAIN);
    }
    __syncwarp();
}

}  // namespace
}  // namespace fa
