// paged_small.cu -- attention over the paged cache for a few rows per
// (sequence, kv head), and the kernels that join split units.
//
// The definition is fa_fwd's, for rows at position i of their sequence and
// keys on pages.  A unit of work is a (sequence, kv head): its n x Hq / Hkv
// rows (at most 16) against the keys that some row sees.  With one row per
// query head there is nothing to reuse: every K and V byte is read once and
// HBM bounds the kernel.
//
// Split.  The tiles of all units stand in one line, unit after unit; CTA c of
// the grid (two per SM) takes an equal stretch of it, whatever the sequences'
// lengths.  Only the first and the last unit of a stretch can
// be shared with a neighbour; those leave partials (unnormalised O, running
// max and sum) in two slots per CTA, and a second kernel joins them in the
// order of the keys, so that results do not depend on timing.  The loader runs
// over the whole stretch without a stop at unit boundaries.  Every CTA finds
// its stretch by itself: the lengths are on the device, and a prefix sum over
// the sequences costs about a microsecond.
//
// A tile is 32 KB of K and V (128 keys of 64 columns, 64 of 128), three of them
// are in flight per CTA, and two CTAs share an SM: what one CTA waits for (the
// start, the barriers of a tile, the change from one unit to the next) the
// other's work covers.  One CTA of three 64 KB stages per SM read as much at
// once, but its tiles of 64 columns took 1.05 us instead of the 0.73 us that
// HBM needs: 121 us instead of 89 for 64 sequences of 4096 keys, 8 kv heads of
// 64 columns (537 MB; at 128 columns the two are even).
//
// CTA: 8 consumer warps and a loader warp.  The loader's lanes stand for the
// tile's pages: each reads its page's id ahead of time and issues the page's
// TMA boxes into a ring of stages.  Pages without a visible key are neither
// looked up nor read.  Consumer warp w computes S for an eighth of the tile's
// keys (mma.sync m16n8k16; 16 rows are too few for a tcgen05 tile, and
// the tensor pipe is not the bound), the warps exchange their row maxima and
// then P (bf16) through shared memory, and warp w accumulates columns
// w D / 8 .. of O over all the tile's keys: no warp holds a second copy of O, so a
// unit's end needs no merge and costs one barrier.
//
// V rows of keys that no row of the unit sees (past the end of the sequence,
// before the window, on pages that were not read) are cleared in shared
// memory before the product: their P is 0, but 0 x NaN is not.
#include <algorithm>
#include <cuda_bf16.h>
#include <math_constants.h>

#include "paged_line.cuh"

namespace fa {
namespace {

constexpr int kWarps = 8;                        // consumers; warp 8 loads
constexpr int kThreadsS = 32 * (kWarps + 1);
constexpr int kRows = kPagedSmallRows;
constexpr int kTileOpen = 1, kTileClear = 2;    // every row sees every key; some key is seen by no row
enum PagedSite : uint32_t { S_PG_FULL = 64, S_PG_EMPTY, S_PG_DRAIN, S_PG_Q, S_PG_Q_EMPTY };

template <int D>
struct SmallLayout {
    static constexpr int kStages = 3;
    static constexpr int kKeys = D == 64 ? 128 : 64;             // = paged_small_keys(D)
    static constexpr int kShift = D == 64 ? 7 : 6;
    static constexpr uint32_t kBox = kKeys * 64u * 2u;           // the tile's keys x 64 columns
    static constexpr uint32_t kStage = 2u * (D / 64) * kBox;     // K then V
    static constexpr uint32_t kPRow = 2u * kKeys + 16u;          // 16 bytes of padding: rows on distinct banks
    static constexpr uint32_t kP = kStages * kStage;
    static constexpr uint32_t kMax = kP + kRows * kPRow;         // [16 rows][8 warps] fp32
    static constexpr uint32_t kSum = kMax + kRows * kWarps * 4u;
    static constexpr uint32_t kQRow = 2u * D + 16u;
    static constexpr uint32_t kQ = kSum + kRows * kWarps * 4u;   // two units' rows of Q
    static constexpr uint32_t kSeg = kQ + 2u * kRows * kQRow;    // two units, the last one flagged by b < 0
    static constexpr uint32_t kInfo = kSeg + 2u * sizeof(SmallSeg);   // [stage]: 4 x tile + kTileOpen, kTileClear
    static constexpr uint32_t kBars = (kInfo + 4u * kStages + 7u) & ~7u;  // FULL, EMPTY [stage], Q_FULL, Q_EMPTY [2]
    static constexpr uint32_t kAbort = kBars + 16u * kStages + 32u;
    static constexpr uint32_t kScan = kAbort + 16u;              // warp sums
    static constexpr uint32_t kPre = kScan + 64u;                // first tile of each group of sequences
    static constexpr uint32_t bytes(int B) { return kPre + 4u * (groups_of(B) + 1u) + 1024u; }
    // two CTAs fit on an SM (228 KB less 1 KB for each)
    static_assert(2u * (kPre + 4u * 1001u + 1024u) <= 226u * 1024u, "shared memory budget");
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

template <int D, int SCORE>
__global__ void __launch_bounds__(kThreadsS, 2)
paged_small_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const PagedParams p) {
    using L = SmallLayout<D>;
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
    line.shift = group_shift(p.c.B);
    const int groups = groups_of(p.c.B);
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
        const uint32_t page_bytes = static_cast<uint32_t>(span) * D * 4u;    // K and V
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
                if (k + 1 < s.k1) page = tile_page<KT>(p.c, table, s.hull, s.hull.tile(k + 1), lane, s.b, p.ws);
                if (g >= ST && !mbar_wait_warp(empty_bar(st), (g / ST - 1) & 1, wc, S_PG_EMPTY)) { ok = false; break; }
                const uint32_t pages = __popc(__ballot_sync(0xffffffffu, id >= 0));
                if (lane == 0) {
                    info_s[st] = 4 * kb + (tile_open(p.mask, kb, i0, i1, p.shared, s.kv, SH) ? kTileOpen : 0) +
                                 (s.hull.all(kb * KT, kb * KT + KT) ? 0 : kTileClear);
                    mbar_arrive_expect_tx(full_bar(st), pages * page_bytes);
                }
                __syncwarp();
                if (id >= 0) {
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
        {
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
            const uint32_t kbase = sbase + st * L::kStage, vbase = kbase + (D / 64) * L::kBox;
            const bool here = mbar_wait_warp(full_bar(st), (g / ST) & 1, wc, S_PG_FULL);
            const int info = info_s[st], c0 = (info >> 2) * KT;
            float x[kNK][4];
#pragma unroll
            for (int nt = 0; nt < kNK; ++nt) x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.f;
            float mx[2] = {-CUDART_INF_F, -CUDART_INF_F};
            bool cleared = false;
            if (here) {
                if constexpr (kNK == 2) {
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
                        if (lane < D / 8)
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
                                                 2 * (kKW * warp + 8 * nt + 2 * tq)) = pack_bf16x2(p0, p1);
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

// Joins the partials of rows, the parts of `a` and then those of `b`:
//   M = max m_k, L = sum 2^(m_k - M) l_k, O = sum 2^(m_k - M) O_k / L.
// Eight lanes to a row, four rows to a warp.  What it costs is the loads'
// latency, so many are in flight at once: a lane holds the (m, l) of every
// eighth part for the weights, and reads its 4 x D / 32 columns of several
// parts at a time.  SHARE warps, the block, take the parts of the same four
// rows in turn and add up through shared memory (single tokens and shared
// prefixes, where a row has tens of parts); 1: each of four warps has rows of
// its own.  With few rows eight warps share (one token, 520 keys, 8 blocks:
// the call 8.6 us, with four 9.4; 64 rows after a prefix of 5024 keys, 188
// blocks: 17.5 and 18.9); with many, four that need fewer registers together,
// for then all blocks run at once (64 chats after a prefix of 16384 keys, 512
// blocks: 55.5 us, with eight 58.5).  Summing is in a
// fixed order either way.
template <int SHARE>
constexpr int kJoinWarps = SHARE == 1 ? 4 : SHARE;
template <int D, int SHARE>
__device__ __forceinline__ void join_rows(const PagedParams& p, const RowParts& a, const RowParts& b, long long row,
                                          bool valid, float4* sums) {
    constexpr int kC = D / 32;                     // float4 columns per lane, 32 apart
    constexpr bool SPLIT = SHARE > 1;
    constexpr int kHold = SPLIT ? SHARE / 2 : 1;   // weights per lane: 8 kHold parts per pass
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane & 7;
    const int n = valid ? a.count + b.count : 0;
    auto ml_of = [&](int k) {
        if (k >= n) return make_float2(-CUDART_INF_F, 0.f);
        return k < a.count ? __ldcg(a.ml + a.at(k)) : __ldcg(b.ml + b.at(k - a.count));
    };
    const int longest = __reduce_max_sync(0xffffffffu, n);
    float2 ml[kHold];
#pragma unroll
    for (int t = 0; t < kHold; ++t) ml[t] = ml_of(8 * t + sub);
    float m = ml[0].x;
#pragma unroll
    for (int t = 1; t < kHold; ++t) m = fmaxf(m, ml[t].x);
    for (int k0 = 8 * kHold; k0 < longest; k0 += 8) m = fmaxf(m, ml_of(k0 + sub).x);
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float ref = m == -CUDART_INF_F ? 0.f : m;
    float l = 0.f;
    float4 o[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < longest; k0 += 8 * kHold) {
        float w[kHold];
#pragma unroll
        for (int t = 0; t < kHold; ++t) {
            if (k0) ml[t] = ml_of(k0 + 8 * t + sub);
            w[t] = ml[t].y == 0.f ? 0.f : ex2_approx(ml[t].x - ref);   // 0: the part has no visible key for this row
            l += ml[t].y * w[t];
        }
        // this warp's parts of the pass
#pragma unroll
        for (int e = 0; e < 8 * kHold; e += SHARE) {
            const int k = k0 + e + (SPLIT ? warp : 0);
            const float we = __shfl_sync(0xffffffffu, w[e >> 3], (lane & 24) + (e & 7) + (SPLIT ? warp : 0));
            if (k >= n) continue;
            const float4* src = reinterpret_cast<const float4*>(
                k < a.count ? a.o + a.at(k) * D : b.o + b.at(k - a.count) * D) + sub;
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                const float4 v = __ldcg(src + 8 * c);
                o[c].x = fmaf(we, v.x, o[c].x);
                o[c].y = fmaf(we, v.y, o[c].y);
                o[c].z = fmaf(we, v.z, o[c].z);
                o[c].w = fmaf(we, v.w, o[c].w);
            }
        }
    }
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    if (SPLIT) {
        if (warp > 0) {
#pragma unroll
            for (int c = 0; c < kC; ++c) sums[((warp - 1) * kC + c) * 32 + lane] = o[c];
        }
        __syncthreads();
        if (warp > 0) return;
#pragma unroll
        for (int w = 0; w < SHARE - 1; ++w) {
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                const float4 v = sums[(w * kC + c) * 32 + lane];
                o[c].x += v.x;
                o[c].y += v.y;
                o[c].z += v.z;
                o[c].w += v.w;
            }
        }
    }
    if (!valid) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int c = 0; c < kC; ++c) {
        const long long at = row * D + 32 * c + 4 * sub;
        if (p.flags & FA_OUT_FP32)
            *reinterpret_cast<float4*>(static_cast<float*>(p.o) + at) =
                make_float4(o[c].x * inv, o[c].y * inv, o[c].z * inv, o[c].w * inv);
        else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + at) =
                make_uint2(pack_bf16x2(o[c].x * inv, o[c].y * inv), pack_bf16x2(o[c].z * inv, o[c].w * inv));
    }
    if (sub == 0) p.lse[row] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * kPagedLn2;
}

// Without a shared prefix: block (c, y) joins rows of the unit that starts in
// CTA c of the attention kernel and runs on into the next ones.
template <int D, int SHARE>
__global__ void __launch_bounds__(32 * kJoinWarps<SHARE>) paged_join_units_kernel(const PagedParams p, int rows_per_unit) {
    __shared__ float4 sums[SHARE > 1 ? (SHARE - 1) * (D / 32) * 32 : 1];
    pdl_launch_next();
    pdl_wait_previous();
    const PagedMeta t = p.meta[blockIdx.x];
    const int r = (SHARE > 1 ? blockIdx.y : blockIdx.y * kJoinWarps<SHARE> + (threadIdx.x >> 5)) * 4 + ((threadIdx.x & 31) >> 3);
    if (t.count == 0 || (r & ~3) >= t.rows) return;        // (uniform: four rows to a warp, and to a block that shares them)
    const bool valid = r < t.rows;
    const RowParts a = unit_parts(p.parts, blockIdx.x, t.count, rows_per_unit, r);
    const RowParts none{nullptr, nullptr, 0, 0, 0};
    if (!a.within(2LL * gridDim.x * rows_per_unit)) return;     // (the same for all rows of a unit)
    const int R = t.row0 + r, tok = quotient(R, p.by_group);
    join_rows<D, SHARE>(p, a, none, (long long)(t.q0 + tok) * p.Hq + t.h * p.group + R - tok * p.group, valid, sums);
}

// With a shared prefix: block (t, h, y) joins four rows of token t and kv head
// h, the prefix's partials first, then those of the sequence's own keys.
template <int D, int SHARE>
__global__ void __launch_bounds__(32 * SHARE) paged_join_rows_kernel(const PagedJoin j) {
    constexpr int kThreads = 32 * SHARE;
    __shared__ float4 sums[(SHARE - 1) * (D / 32) * 32];
    const PagedParams& p = j.own;
    pdl_launch_next();
    pdl_wait_previous();
    const int t = blockIdx.x, h = blockIdx.y;
    const int2 pre = *reinterpret_cast<const int2*>(p.hdr);
    if ((blockIdx.x | blockIdx.y | blockIdx.z | threadIdx.x) == 0) *prefix_mark(p) = 0;
    const int gq = blockIdx.z * 4 + ((threadIdx.x & 31) >> 3);
    const bool valid = gq < p.group;
    const long long row = (long long)t * p.Hq + h * p.group + min(gq, p.group - 1);
    const int2 d = __ldcg(p.rowdesc + row);        // (what it says of a row without a unit is not used)
    int b = 0;
    for (int b0 = 0; b0 < p.c.B; b0 += kThreads) {
        const int x = b0 + threadIdx.x;
        b += __syncthreads_count(x < p.c.B && __ldg(p.c.q_start + min(x, p.c.B - 1) + 1) <= t);
    }
    if (b >= p.c.B) return;
    const SeqInfo s = seq_info(p.c, b, p.max_q, p.shared, nullptr);
    if (s.n == 0 || t < s.q0 || t >= s.q0 + s.n) return;
    RowParts a = prefix_parts(j.pre, pre.x, pre.y, p.c.Hkv, t * p.group + min(gq, p.group - 1), h, row);
    RowParts own{p.parts.slot_o, p.parts.slot_ml, d.x, d.y, j.own_rows};
    if (d.x < 0) own = RowParts{p.parts.row_o, p.parts.row_ml, row, 1, 0};
    // (a q_start that decreases can name rows past the prefix's line)
    if (a.stride > 0 && !a.within(2LL * j.pre_ctas * kPagedTileRows)) a.count = 0;
    // (a CTA whose wait ran out leaves its rows' places as the scratch held them)
    if (d.x >= 0 && !own.within(2LL * p.ctas * j.own_rows)) own.count = 0;
    join_rows<D, SHARE>(p, a, own, row, valid, sums);
}

template <int D, int SCORE>
cudaError_t launch_small(const PagedParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                         cudaStream_t s) {
    auto kern = paged_small_kernel<D, SCORE>;
    using L = SmallLayout<D>;
    constexpr size_t most = L::bytes(kLineEntries);
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

template <int D>
cudaError_t launch_small_d(const PagedParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                           cudaStream_t s) {
    switch (p.score.kind) {
        case FA_SCORE_SOFTCAP: return launch_small<D, FA_SCORE_SOFTCAP>(p, tk, tv, s);
        case FA_SCORE_ALIBI: return launch_small<D, FA_SCORE_ALIBI>(p, tk, tv, s);
        case FA_SCORE_REL_BIAS: return launch_small<D, FA_SCORE_REL_BIAS>(p, tk, tv, s);
        case FA_SCORE_ALIBI_SOFTCAP: return launch_small<D, FA_SCORE_ALIBI_SOFTCAP>(p, tk, tv, s);
        default: return launch_small<D, FA_SCORE_NONE>(p, tk, tv, s);
    }
}

}  // namespace

cudaError_t launch_paged_small(const PagedParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                               cudaStream_t s) {
    return p.D == 64 ? launch_small_d<64>(p, tk, tv, s) : launch_small_d<128>(p, tk, tv, s);
}

namespace {

// Eight warps to four rows while that is at most one block per SM and a half.
bool few_joins(long long blocks) { return 2 * blocks <= 3 * device_sm_count(); }

template <int D>
cudaError_t launch_join_units(const PagedParams& p, int rows_per_unit, cudaStream_t s) {
    // the blocks that find something to join: at most the units', or one per CTA
    const long long rows = std::min((long long)p.max_q * p.group, (long long)rows_per_unit);
    const long long units = ((long long)p.c.B + (long long)p.c.total_q * p.group / rows_per_unit) * p.c.Hkv;
    const dim3 grid(p.ctas, (unsigned)((rows + 3) / 4));
    if (few_joins(std::min<long long>(units, p.ctas) * grid.y))
        return paged_launch(paged_join_units_kernel<D, 8>, grid, 32 * 8, 0, true, s, p, rows_per_unit);
    if (rows_per_unit == kPagedSmallRows)
        return paged_launch(paged_join_units_kernel<D, 4>, grid, 32 * 4, 0, true, s, p, rows_per_unit);
    return paged_launch(paged_join_units_kernel<D, 1>, dim3(p.ctas, (grid.y + kJoinWarps<1> - 1) / kJoinWarps<1>),
                        32 * kJoinWarps<1>, 0, true, s, p, rows_per_unit);
}

template <int D>
cudaError_t launch_join_rows(const PagedJoin& j, cudaStream_t s) {
    const dim3 grid(j.own.c.total_q, j.own.c.Hkv, (j.own.group + 3) / 4);
    return few_joins((long long)grid.x * grid.y * grid.z)
               ? paged_launch(paged_join_rows_kernel<D, 8>, grid, 32 * 8, 0, true, s, j)
               : paged_launch(paged_join_rows_kernel<D, 4>, grid, 32 * 4, 0, true, s, j);
}

}  // namespace

cudaError_t launch_paged_join_units(const PagedParams& p, int rows_per_unit, cudaStream_t s) {
    return p.D == 64 ? launch_join_units<64>(p, rows_per_unit, s) : launch_join_units<128>(p, rows_per_unit, s);
}

cudaError_t launch_paged_join_rows(const PagedJoin& p, cudaStream_t s) {
    return p.own.D == 64 ? launch_join_rows<64>(p, s) : launch_join_rows<128>(p, s);
}

}  // namespace fa
