// paged_tiles.cu -- attention over the paged cache for many rows: chunks of
// prompts, and the shared prefix of a whole batch (tcgen05 + TMEM + TMA).
//
// The definition is fa_fwd's, for rows at position i of their sequence and
// keys on pages.  The rows of a kv head are the (token, query head of the
// group) pairs of one sequence, or for a shared prefix of all sequences at
// once: that is what lets a prefix's K and V be read once for the batch.  A
// unit is 256 consecutive rows of a kv head (two tiles of 128, which share
// every K and V tile) against the keys that some row of them sees.  As in
// paged_small.cu the 128-key tiles of all units stand in one line, every CTA
// (one per SM) takes an equal stretch of it, and the units that two CTAs share
// are joined by a second kernel.  Chunks of 4 x up to 1024 tokens up to 8192
// keys (32 heads on 8, 128 columns) take 186 us with the join, a prompt of
// 4096 tokens 123, one of 16384 1500 (1.47 PFLOP/s).
//
// 384 threads:
//   warps 0-3, 4-7  softmax of row tile 0, 1: thread r owns row r (TMEM lane
//                   r).  A warp brings its 32 rows of Q into shared memory
//                   (asynchronous copies, while the unit before ends), then
//                   for each 64-key half reads S, applies score_mod and mask,
//                   keeps the running max and sum (base 2), writes P (bf16)
//                   over S.
//   warp 8          loader: walks the line and hands each unit to the other
//                   warps; its lanes stand for the pages of a tile: each reads
//                   its page's id ahead of time and issues the page's TMA
//                   boxes (K one step ahead of V).
//   warps 9, 10     MMA of row tile 0, 1: O += P V(k), then S = Q K(k + 1).
//   warp 11         clears the V rows of keys that no row sees (their P is 0,
//                   but 0 x NaN is not) before the product may read the tile.
// TMEM (512 columns): S_t,h at 128 t + 64 h, O_t at 256 + D t, P_t,h in the
// first 32 columns of S_t,h.
//
// Bound: with 256 rows per K/V tile the tensor pipe and HBM are about even
// (4 x 256 x 128 x D flops against 512 D bytes); with fewer rows HBM.
//
// Every wait is bounded; on a timeout the CTA records the site, the roles
// leave their loops, copies and products in flight are waited for, TMEM is
// freed and the kernel returns.
#include <algorithm>
#include <cuda_bf16.h>
#include <math_constants.h>

#include "paged_line.cuh"

namespace fa {
namespace {

constexpr int kThreadsT = 384;
// Registers per thread: launched with 168 (65536 / 384, rounded down to 8); the
// loader, MMA and clearing warps hand theirs to the two softmax warpgroups:
// 128 x (2 x 184 + 136) = 384 x 168.  build.py checks the launch count.
constexpr uint32_t kRegsSoftmaxT = 184, kRegsOtherT = 136;
static_assert(2 * kRegsSoftmaxT + kRegsOtherT == 3 * 168, "register split must match the launch");
constexpr uint32_t kTmemColsT = 512;
constexpr int kMaxRing = 4;
// With bf16 output the running max is raised (and O, l rescaled) only when it
// grows by more than 2^8; with fp32 output it follows every increase, so that
// the largest P is 1 and rounds exactly.
constexpr float kLazyMaxT = 8.f;

enum TBar {
    T_Q_FULL = 0,                                // two: the 4 softmax warps of the tile
    T_K_FULL = 2, T_K_EMPTY = T_K_FULL + kMaxRing,
    T_V_FULL = T_K_EMPTY + kMaxRing, T_V_EMPTY = T_V_FULL + kMaxRing,
    T_V_OK = T_V_EMPTY + kMaxRing,               // V's unseen rows are cleared
    T_S_FULL = T_V_OK + kMaxRing,                // four (2 t + h)
    T_P_FULL = T_S_FULL + 4,                     // four (2 t + h)
    T_O_DONE = T_P_FULL + 4,                     // two
    T_O_UPD = T_O_DONE + 2,                      // two
    T_DRAIN = T_O_UPD + 2,                       // two
    T_SEG_FULL = T_DRAIN + 2,                    // two slots
    T_SEG_EMPTY = T_SEG_FULL + 2,
    T_COUNT = T_SEG_EMPTY + 2
};
constexpr uint32_t kSegReaders = 11;             // the MMA, clearing and softmax warps
enum TSite : uint32_t { S_T_Q = 80, S_T_K_FULL, S_T_K_EMPTY, S_T_V_FULL, S_T_V_EMPTY, S_T_V_OK, S_T_S, S_T_P, S_T_O,
                        S_T_UPD, S_T_DRAIN, S_T_SEG, S_T_SEG_EMPTY };

template <int D>
struct TileLayout {
    static constexpr int kStages = D == 64 ? 4 : 2;
    static constexpr uint32_t kTile = 128u * D * 2u;
    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kK = kQ + 2 * kTile;
    static constexpr uint32_t kV = kK + kStages * kTile;
    static constexpr uint32_t kBars = kV + kStages * kTile;
    static constexpr uint32_t kTmemSlot = kBars + 8 * T_COUNT;
    static constexpr uint32_t kAbort = kTmemSlot + 4;
    static constexpr uint32_t kMinMax = kAbort + 4;          // positions of the batch (shared prefix)
    static constexpr uint32_t kSeg = kMinMax + 8;            // two units
    static constexpr uint32_t kScan = kSeg + 2 * sizeof(TileSeg);
    static constexpr uint32_t kPre = kScan + 4 * (kThreadsT / 32);   // TileLine's arrays
    static constexpr uint32_t bytes(int B) { return kPre + 4u * (3u * B + 2u) + 1024u; }
    static_assert(kStages <= kMaxRing, "ring");
    static_assert(kPre + 4 * (3 * kPagedMaxSeqs + 2) + 1024 <= 227u * 1024u, "shared memory budget");
};

// x <- the soft-capped score, base 2.  TRY: where no element of the warp is past
// the polynomial's range, two elements to an instruction (4 x 1024 new tokens
// at 8192 keys, cap 30: 529 us).  Otherwise, and always without TRY, the
// exponential form, at two MUFU operations per element (cap 2: 747).  A cap far
// above the scores takes the polynomial where it holds, with or without TRY;
// a warp that needs both forms evaluates both (ALiBi then a cap of 100: 1134 us,
// 1e5, where the polynomial alone does: 771; 30, exponential: 792).
template <bool TRY>
__device__ __forceinline__ void softcap_all(float (&x)[64], const SoftCap& c) {
    bool inner = false;
    if (TRY || c.fine) {
        float am = 0.f;
#pragma unroll
        for (int e = 0; e < 64; e += 2) am = fmax3(am, fabsf(x[e]), fabsf(x[e + 1]));
        inner = !__any_sync(0xffffffffu, !(am * c.in <= kTanhFineRange));
    }
    const float q0 = c.mul * kTanhFineC0, q1 = c.mul * kTanhFineC1, q2 = c.mul * kTanhFineC2, q3 = c.mul * kTanhFineC3,
                q4 = c.mul * kTanhFineC4;
    // u = x in and x mul q(u^2) of a pair
    auto pair = [&](int e, float& u0, float& u1, float& y0, float& y1) {
        float w0, w1;
        ffma2(u0, u1, x[e], x[e + 1], c.in, c.in, -0.f, -0.f);
        ffma2(w0, w1, u0, u1, u0, u1, -0.f, -0.f);
        ffma2(y0, y1, w0, w1, q4, q4, q3, q3);
        ffma2(y0, y1, y0, y1, w0, w1, q2, q2);
        ffma2(y0, y1, y0, y1, w0, w1, q1, q1);
        ffma2(y0, y1, y0, y1, w0, w1, q0, q0);
        ffma2(y0, y1, x[e], x[e + 1], y0, y1, -0.f, -0.f);
    };
    if (inner) {
#pragma unroll
        for (int e = 0; e < 64; e += 2) {
            float u0, u1, y0, y1;
            pair(e, u0, u1, y0, y1);
            x[e] = y0;
            x[e + 1] = y1;
        }
    } else if (c.fine) {
#pragma unroll
        for (int e = 0; e < 64; e += 2) {
            float u0, u1, y0, y1;
            pair(e, u0, u1, y0, y1);
            x[e] = softcap_pick(y0, u0, c);
            x[e + 1] = softcap_pick(y1, u1, c);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 64; ++e) x[e] = softcap_outer(x[e] * c.in, c);
    }
}

__device__ __forceinline__ void exp2_pair(float& p0, float& p1, float x0, float x1, float sc, float nm) {
    float a0, a1;
    ffma2(a0, a1, x0, x1, sc, sc, nm, nm);
    p0 = ex2_approx(a0);
    p1 = ex2_approx(a1);
}

// 16 bytes from global into shared memory, without passing registers; zeros
// where `there` does not hold.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16u : 0u) : "memory");
}
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// Eight words; `wide`: to a 32-byte boundary (16 otherwise).
__device__ __forceinline__ void store8(void* dst, const uint32_t* w, bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        static_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// Bits a .. 31, and bits 0 .. a, of a word (any a).
__device__ __forceinline__ uint32_t bits_from(int a) { return a <= 0 ? 0xffffffffu : a > 31 ? 0u : 0xffffffffu << a; }
__device__ __forceinline__ uint32_t bits_to(int a) { return a < 0 ? 0u : a >= 31 ? 0xffffffffu : 0xffffffffu >> (31 - a); }

// Finds the unit group of ln.b in which the stretch begins: a lane to a group
// of the next 32.
__device__ __forceinline__ void seek(const PagedParams& p, TileLine& ln, int lane) {
    const int q0 = ln.q0[ln.b], n = ln.q0[ln.b + 1] - q0, kv = ln.kv[ln.b];
    for (; ln.rt * kPagedTileRows < n * p.group; ln.rt += 32) {
        int len = 0;
        if ((ln.rt + lane) * kPagedTileRows < n * p.group) len = p.c.Hkv * unit_length(p, n, kv, ln.rt + lane);
        int upto = len;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += y;
        }
        const uint32_t behind = __ballot_sync(0xffffffffu, ln.start + upto > ln.t);
        const int at = behind ? __ffs(behind) - 1 : 31;
        ln.start += __shfl_sync(0xffffffffu, behind ? upto - len : upto, at);
        if (behind) {
            ln.rt += at;
            return;
        }
    }
}

// Rows r0 .. r0 + 31 of a unit's Q into their row tile at `tile` (128-byte
// swizzled, zeros past the unit's rows), D / 8 lanes to a row, so that whole
// lines are read.
template <int D>
__device__ __forceinline__ void load_rows(const PagedParams& p, const TileSeg& s, int r0, uint32_t tile, int lane) {
    constexpr int kLanes = D / 8, kPer = 32 / kLanes;      // lanes per row, rows per copy
    const int ur = r0 + lane, R = s.row0 + min(ur, s.rows - 1), tok = quotient(R, p.by_group);
    const long long mine = ur < s.rows ? (long long)(s.q0 + tok) * p.qs[0] +
                                             (long long)(s.h * p.group + R - tok * p.group) * p.qs[1]
                                       : -1;
    const int c = lane % kLanes;
    tile += (c >> 3) * 16384u;
#pragma unroll 4
    for (int e = 0; e < kLanes; ++e) {
        const long long at = __shfl_sync(0xffffffffu, mine, e * kPer + lane / kLanes);
        const int rr = (r0 & 127) + e * kPer + lane / kLanes;
        copy16(tile + rr * 128 + (((c & 7) ^ (rr & 7)) << 4), p.q + (at >= 0 ? at + 8 * c : 0), at >= 0);
    }
}

template <int D, int SCORE>
__global__ void __launch_bounds__(kThreadsT, 1)
paged_tiles_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const PagedParams p) {
    using L = TileLayout<D>;
    constexpr int ST = L::kStages;
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

    if (threadIdx.x == 0) {
        for (int k = 0; k < T_COUNT; ++k) {
            uint32_t cnt = 1;
            if (k < T_K_FULL) cnt = 4;
            if (k >= T_P_FULL && k < T_P_FULL + 4) cnt = 4;
            if (k >= T_K_EMPTY && k < T_K_EMPTY + kMaxRing) cnt = 2;      // both MMA warps
            if (k >= T_V_EMPTY && k < T_V_EMPTY + kMaxRing) cnt = 2;
            if (k >= T_SEG_EMPTY && k < T_SEG_EMPTY + 2) cnt = kSegReaders;
            mbar_init(bar(k), cnt);
        }
        *abort_flag = 0;
        minmax[0] = INT_MAX;
        minmax[1] = INT_MIN;
        mbar_fence_init();
    }
    if (warp == 9) {
        tmem_alloc(smem_addr(const_cast<uint32_t*>(tmem_slot)), kTmemColsT);
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
    // the line of tiles
    TileLine line{};
    line.pre = pre;
    line.kv = len_s;
    line.q0 = q0_s;
    int total;
    if (p.prefix) {
        for (int b = threadIdx.x; b < p.c.B; b += kThreadsT) {
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
        // the sequences' lengths: a warp to each of a few sequences (long
        // prompts have hundreds of units), a thread to each of many
        const bool few = p.c.B <= kThreadsT / 32;
        bool ordered = true;
        for (int b = few ? warp : threadIdx.x; b < p.c.B; b += few ? kThreadsT / 32 : kThreadsT) {
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
        // Offsets that decrease (0, T, 0, T, ..) can make of T rows any number, more
        // than 32 bits count and than the slots hold: such a batch is no work.
        ordered = __syncthreads_and(ordered);
        block_prefix<kThreadsT>(p.c.B, pre, reinterpret_cast<int*>(smem + L::kScan),
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

    // Barrier phases run on counters that every role keeps alike: g counts
    // steps (ring stage g % ST), uq units in which row tile t has rows, n the
    // steps of tile t.
    if (warp >= 8) {
    regs_decrease<kRegsOtherT>();
    if (warp == 8) {
        // ------------------------------------------------------------ loader
        if (lane == 0) {
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmV);
        }
        const int span = min(p.c.page_size, kBlock);
        const uint32_t page_bytes = static_cast<uint32_t>(span) * D * 2u;
        uint32_t g = 0;
        int last_k = -1, last_v = -1;
        bool ok = true;
        TileSeg s{};
        if (!p.prefix && line.t < line.t1) seek(p, line, lane);
        // the copies of one tile of K or V: `id` the lane's page, `row` its
        // first row within the page
        auto load = [&](const CUtensorMap* tm, uint32_t base, int full, int empty, uint32_t gg, int id, int row,
                        uint32_t site) -> bool {
            const uint32_t st = gg % ST;
            if (gg >= ST && !mbar_wait_warp(bar(empty + st), (gg / ST - 1) & 1, wc, site)) return false;
            const uint32_t pages = __popc(__ballot_sync(0xffffffffu, id >= 0));
            if (lane == 0) mbar_arrive_expect_tx(bar(full + st), pages * page_bytes);
            __syncwarp();
            if (id >= 0) {
                const uint32_t dst = sbase + base + st * L::kTile + static_cast<uint32_t>(lane * span) * 128u;
                const int block = id * p.c.Hkv + s.h;
#pragma unroll
                for (int c = 0; c < D / 64; ++c) tma_load_3d(dst + c * 16384u, tm, bar(full + st), c * 64, row, block);
            }
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
            int page = tile_page<kBlock>(p.c, table, s.hull, s.hull.tile(s.k0), lane, s.b, p.ws);
            int id_v = -1, row_v = 0;
            for (int k = s.k0; k < s.k1; ++k) {
                const int id = page, row = (s.hull.tile(k) * kBlock + lane * span) & (p.c.page_size - 1);
                if (k + 1 < s.k1) page = tile_page<kBlock>(p.c, table, s.hull, s.hull.tile(k + 1), lane, s.b, p.ws);
                if (!load(&tmK, L::kK, T_K_FULL, T_K_EMPTY, g, id, row, S_T_K_EMPTY)) { ok = false; break; }
                last_k = static_cast<int>(g);
                // the first unit's rows of Q come before the rest of the ring:
                // behind it they would wait for all of it to arrive
                if (g == 0 && !mbar_wait_warp(bar(T_Q_FULL), 0, wc, S_T_Q)) { ok = false; break; }
                if (k > s.k0) {
                    if (!load(&tmV, L::kV, T_V_FULL, T_V_EMPTY, g - 1, id_v, row_v, S_T_V_EMPTY)) { ok = false; break; }
                    last_v = static_cast<int>(g - 1);
                }
                id_v = id;
                row_v = row;
                ++g;
            }
            if (ok) {
                ok = load(&tmV, L::kV, T_V_FULL, T_V_EMPTY, g - 1, id_v, row_v, S_T_V_EMPTY);
                if (ok) last_v = static_cast<int>(g - 1);
            }
        }
        // every issued copy lands before the CTA may exit
        if (lane == 0) {
            for (int st = 0; st < ST; ++st) {
                const int lk = last_k - (((last_k - st) % ST + ST) % ST);
                if (lk >= 0) paged_drain_wait(bar(T_K_FULL + st), (lk / ST) & 1, wc, S_T_DRAIN);
                const int lv = last_v - (((last_v - st) % ST + ST) % ST);
                if (lv >= 0) paged_drain_wait(bar(T_V_FULL + st), (lv / ST) & 1, wc, S_T_DRAIN);
            }
        }
        __syncwarp();
    } else if (warp == 11) {
        // -------------------------------------------------- V's unseen rows
        uint32_t g = 0;
        bool ok = true;
        TileSeg s;
        while (ok && take(s)) {
            for (int k = s.k0; k < s.k1; ++k, ++g) {
                const uint32_t st = g % ST;
                const int c0 = s.hull.tile(k) * kBlock;
                if (!mbar_wait_warp(bar(T_V_FULL + st), (g / ST) & 1, wc, S_T_V_FULL)) { ok = false; break; }
                if (!s.hull.all(c0, c0 + kBlock)) {
                    uint8_t* v = smem + L::kV + st * L::kTile;
                    for (int r = lane; r < kBlock; r += 32) {
                        if (s.hull.live(c0 + r)) continue;
#pragma unroll
                        for (int c = 0; c < D / 8; ++c)
                            *reinterpret_cast<uint4*>(v + (c >> 3) * 16384 + r * 128 + (c & 7) * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_async_shared();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(T_V_OK + st));
            }
        }
    } else {
        // --------------------------------------------------------------- MMA
        const int t = warp - 9;
        constexpr uint32_t idesc_qk = idesc_bf16_f32(128, 64, false);
        constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, true);
        const uint64_t q_desc = sdesc_sw128(sbase + L::kQ + t * L::kTile, 16, 1024);
        const uint64_t k_desc0 = sdesc_sw128(sbase + L::kK, 16, 1024);
        const uint64_t v_desc0 = sdesc_sw128(sbase + L::kV, 16384, 1024);
        const uint32_t tSt = tmem + 128u * t, tOt = tmem + 256u + D * t;
        auto issue_qk = [&](int h, uint32_t gg) {
            const uint64_t kd = k_desc0 + (((gg % ST) * L::kTile + 8192u * h) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = ((kk >> 2) * 16384u + (kk & 3) * 32u) >> 4;
                mma_ss_elect(tSt + 64u * h, q_desc + off, kd + off, idesc_qk, kk > 0);
            }
            mma_commit_elect(bar(T_S_FULL + 2 * t + h));
        };
        auto issue_pv = [&](int h, uint32_t gg, bool accumulate) {
            const uint64_t vd = v_desc0 + (((gg % ST) * L::kTile + 8192u * h) >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                mma_ts_elect(tOt, tSt + 64u * h + kk * 8u, vd + kk * 128u, idesc_pv, (accumulate || kk > 0) ? 1u : 0u);
            mma_commit_elect(bar(T_O_UPD + t));
        };
        uint32_t g = 0, uq = 0, np = 0;
        bool ok = true;
        TileSeg s;
        while (ok && take(s)) {
            const bool active = s.rows > 128 * t;
            const int steps = s.k1 - s.k0;
            // pass k: O += P V(k - 1), then S = Q K(k) into the buffer which
            // that product has released.  A tile without rows only releases
            // the stages.
            for (int k = 0; ok && k <= steps; ++k) {
                const uint32_t gp = g - 1;
                if (k > 0) {
                    if (!mbar_wait_warp(bar(T_V_FULL + gp % ST), (gp / ST) & 1, wc, S_T_V_FULL) ||
                        !mbar_wait_warp(bar(T_V_OK + gp % ST), (gp / ST) & 1, wc, S_T_V_OK)) { ok = false; break; }
                }
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    if (k > 0 && active) {
                        if (!mbar_wait_warp(bar(T_P_FULL + 2 * t + h), np & 1, wc, S_T_P)) { ok = false; break; }
                        tc_fence_after();
                        issue_pv(h, gp, k > 1 || h > 0);
                    }
                    if (k < steps) {
                        if (h == 0 && !mbar_wait_warp(bar(T_K_FULL + g % ST), (g / ST) & 1, wc, S_T_K_FULL)) { ok = false; break; }
                        if (active) {
                            if (k == 0 && h == 0 && !mbar_wait_warp(bar(T_Q_FULL + t), uq & 1, wc, S_T_Q)) { ok = false; break; }
                            tc_fence_after();
                            issue_qk(h, g);
                        }
                    }
                }
                if (!ok) break;
                if (k > 0) {
                    if (active) {
                        ++np;
                        if (k == steps) mma_commit_elect(bar(T_O_DONE + t));
                    }
                    mma_commit_elect(bar(T_V_EMPTY + gp % ST));
                }
                if (k < steps) {
                    mma_commit_elect(bar(T_K_EMPTY + g % ST));
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
        regs_increase<kRegsSoftmaxT>();
        const int t = warp >> 2, wq = warp & 3, r = wq * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
        const uint32_t tS = tmem + 128u * t + lane_off, tO = tmem + 256u + D * t + lane_off;
        const float sl2 = p.scale * kPagedLog2e;
        const SoftCap cap = soft_cap(p.score.softcap, SCORE == FA_SCORE_SOFTCAP ? p.scale : 1.f);
        const bool out32 = (p.flags & FA_OUT_FP32) != 0;
        const float lazy = out32 ? 0.f : kLazyMaxT;
        uint32_t n = 0, uq = 0;
        bool ok = true;
        PagedMeta meta{};
        // The warp's 32 rows of a unit's Q.  The unit before has no use for
        // that buffer any more once its last S is there, so that the copies of
        // the next unit run while this one's O is written out (4 x 1024 new
        // tokens up to 8192 keys: 196 us; brought at the unit's start, 203).
        auto bring = [&](const TileSeg& u) {
            if (u.rows > 128 * t) load_rows<D>(p, u, 128 * t + 32 * wq, sbase + L::kQ + t * L::kTile, lane);
        };
        auto announce = [&](const TileSeg& u) {
            if (u.rows <= 128 * t) return;
            copies_wait();
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
        float m_use = -CUDART_INF_F, l = 0.f;
        for (;;) {
            if (have) bring(next);
            if (done) {
                if (!mbar_wait_warp(bar(T_O_DONE + t), uq & 1, wc, S_T_O)) { ok = false; break; }
                tc_fence_after();
                ++uq;
            }
            // (the next unit's first products may come while O is read: they go to S)
            if (have) announce(next);
            if (done) {
                // the unit's end in this CTA: O / l and lse, or a partial
                const bool whole = s.begins() && s.ends(), last = whole && !p.join_rows;
                const long long row = (long long)trow * p.Hq + hq;
                const long long at = whole ? row : (2LL * cta + (s.begins() ? 1 : 0)) * kPagedTileRows + ur;
                const bool f32 = !last || out32;
                uint8_t* const dst = static_cast<uint8_t*>(last ? p.o : static_cast<void*>(whole ? p.parts.row_o : p.parts.slot_o)) +
                                     at * (D * (f32 ? 4 : 2));
                const bool wide = (reinterpret_cast<uintptr_t>(dst) & 31u) == 0;
                const float inv = !last ? 1.f : l == 0.f ? 0.f : 1.f / l;
                // Straight from the registers, 32 bytes (a sector) per store: a
                // partial is 128 KB of fp32 per CTA at 128 columns, and their
                // writing (3 us when all CTAs end together) is what the end of
                // the kernel waits for.
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
                        p.lse[row] = l == 0.f ? -CUDART_INF_F : (m_use + log2f(l)) * kPagedLn2;
                    } else {
                        (whole ? p.parts.row_ml : p.parts.slot_ml)[at] = make_float2(m_use, l);
                        if (p.join_rows && !p.prefix && s.begins())
                            p.rowdesc[row] = whole ? make_int2(-1, 1) : make_int2(static_cast<int>(at), s.count(line.per));
                    }
                }
                tc_fence_before();
            }
            if (!have) break;
            s = next;
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

                m_use = -CUDART_INF_F;
                l = 0.f;
                for (int k = s.k0; ok && k < s.k1; ++k, ++n) {
                    const int kb = s.hull.tile(k);
                    const bool open = tile_open(p.mask, kb, s.i0, s.i1, s.jlo, s.jhi, 7);
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t tSh = tS + 64u * h;
                        const int ch = kb * kBlock + 64 * h;
                        if (!mbar_wait_warp(bar(T_S_FULL + 2 * t + h), n & 1, wc, S_T_S)) { ok = false; break; }
                        tc_fence_after();
                        float x[64];
                        {
                            uint32_t raw[64];
                            tmem_ld64(tSh, raw);
#pragma unroll
                            for (int e = 0; e < 64; ++e) x[e] = __uint_as_float(raw[e]);
                        }
                        // score_mod: x stays the raw q.k without one, and is the
                        // modified score in base 2 otherwise
                        float sc = 1.f;
                        if (SCORE == FA_SCORE_NONE) sc = sl2;
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
                        // (small caps: most distances take the score past the polynomial's range)
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
                        float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                        for (int e = 4; e < 60; e += 8) {
#pragma unroll
                            for (int q = 0; q < 4; ++q) m4[q] = fmax3(m4[q], x[e + q], x[e + 4 + q]);
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q) m4[q] = fmaxf(m4[q], x[60 + q]);
                        const float mx = fmax3(fmaxf(m4[0], m4[1]), m4[2], m4[3]) * sc;
                        const float m_new = fmaxf(m_use, mx);
                        const bool unset = m_use == -CUDART_INF_F;
                        const bool need = !unset && m_new > m_use + lazy;
                        const float alpha = need ? ex2_approx(m_use - m_new) : 1.f;
                        if (need) l *= alpha;
                        if (unset || need) m_use = m_new;
                        const float nm = m_use == -CUDART_INF_F ? 0.f : -m_use;
                        float rs[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            uint32_t pk[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float p0, p1;
                                exp2_pair(p0, p1, x[32 * c + 2 * e], x[32 * c + 2 * e + 1], sc, nm);
                                const int a2 = (e & 1) * 2;
                                fadd2(rs[a2], rs[a2 + 1], rs[a2], rs[a2 + 1], p0, p1);
                                pk[e] = pack_bf16x2(p0, p1);
                            }
                            tmem_st16_nowait(tSh + 16u * c, pk);
                        }
                        l += (rs[0] + rs[1]) + (rs[2] + rs[3]);
                        // O holds the products of the unit's earlier halves; wait
                        // for the last of them and scale
                        if (__any_sync(0xffffffffu, need)) {
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
            have = take(next);
        }
        if (!ok) copies_wait();
        if (!p.join_rows && threadIdx.x == 0) p.meta[cta] = ok ? meta : PagedMeta{};
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemColsT);
    }
    if (!p.prefix && p.join_rows) pdl_wait_previous();
}

template <int D, int SCORE>
cudaError_t launch_tiles(const PagedParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                         cudaStream_t s) {
    auto kern = paged_tiles_kernel<D, SCORE>;
    using L = TileLayout<D>;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)L::bytes(kPagedMaxSeqs));
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    return paged_launch(kern, dim3(p.ctas), kThreadsT, L::bytes(p.c.B), true, s, tk, tv, p);
}

template <int D>
cudaError_t launch_tiles_d(const PagedParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                           cudaStream_t s) {
    switch (p.score.kind) {
        case FA_SCORE_SOFTCAP: return launch_tiles<D, FA_SCORE_SOFTCAP>(p, tk, tv, s);
        case FA_SCORE_ALIBI: return launch_tiles<D, FA_SCORE_ALIBI>(p, tk, tv, s);
        case FA_SCORE_REL_BIAS: return launch_tiles<D, FA_SCORE_REL_BIAS>(p, tk, tv, s);
        case FA_SCORE_ALIBI_SOFTCAP: return launch_tiles<D, FA_SCORE_ALIBI_SOFTCAP>(p, tk, tv, s);
        default: return launch_tiles<D, FA_SCORE_NONE>(p, tk, tv, s);
    }
}

}  // namespace

cudaError_t launch_paged_tiles(const PagedParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                               cudaStream_t s) {
    return p.D == 64 ? launch_tiles_d<64>(p, tk, tv, s) : launch_tiles_d<128>(p, tk, tv, s);
}

}  // namespace fa
