// paged.cuh -- what the paged-cache kernels share: the batch as they read and
// check it, the keys a unit of work can see, and the split of the work.
#pragma once

#include <cfloat>
#include <climits>

#include "paged_internal.h"
#include "ptx.cuh"
#include "tanh_fine_poly.h"

namespace fa {

constexpr float kPagedLog2e = 1.4426950408889634f, kPagedLn2 = 0.6931471805599453f;

__host__ __device__ __forceinline__ int imin(int a, int b) { return a < b ? a : b; }
__host__ __device__ __forceinline__ int imax(int a, int b) { return a > b ? a : b; }

__host__ __device__ __forceinline__ int quotient(int n, const FastDiv& f) {
    const uint32_t u = static_cast<uint32_t>(n);
#ifdef __CUDA_ARCH__
    return static_cast<int>((__umulhi(f.m, u) + u) >> f.s);
#else
    return static_cast<int>((static_cast<uint32_t>((static_cast<uint64_t>(f.m) * u) >> 32) + u) >> f.s);
#endif
}

// A number of the step's arrays.  A plain load: the non-coherent one takes no
// part in the order that wait_before_prefix() below gives.
__host__ __device__ __forceinline__ int load_i32(const int32_t* p) { return *p; }

// A sequence of the step: its rows of the step's tensors and its length.
// n = 0: nothing to do (no new tokens, or numbers that contradict each other).
// ordered: q_start does not decrease here, and starts at 0; where that holds
// for every sequence, their rows are disjoint and no more than total_q.
struct SeqInfo {
    int q0, n, kv;
    bool ordered;
};

__device__ __forceinline__ void report_sequence(uint32_t* ws, int b) {
    atomicCAS(ws + WS_PAGED_DETAIL, 0u, static_cast<uint32_t>(b) + 1u);
    atomicOr(ws + WS_FLAGS, WS_FLAG_PAGED);
}

// Checks sequence b's numbers: s.n > 0 only if its rows lie in the step's
// tensors and its keys in its row of the page table.  `max_q`: INT_MAX where
// any number of new tokens will do; `shared`: the length that kv must reach.
// Returns false for numbers that contradict each other.
__host__ __device__ __forceinline__ bool check_sequence(const PagedView& c, int b, int q0, int q1, int kv, int max_q,
                                                        int shared, SeqInfo& s) {
    s.q0 = q0;
    s.n = 0;
    s.kv = kv;
    s.ordered = q0 <= q1 && (b > 0 || q0 == 0);
    const bool placed = s.ordered && q0 >= 0 && q1 <= c.total_q;
    if (placed && q0 == q1) return true;
    // (q1 - q0 cannot overflow once placed)
    if (!placed || q1 - q0 > max_q || kv < q1 - q0 || kv < shared ||
        kv > static_cast<long long>(c.max_pages) * c.page_size)
        return false;
    s.n = q1 - q0;
    return true;
}

// Reads and checks sequence b; every kernel takes its numbers from here, so
// that none of them indexes with numbers that were not checked.
__host__ __device__ __forceinline__ SeqInfo seq_info(const PagedView& c, int b, int max_q, int shared, uint32_t* ws) {
    SeqInfo s;
    const bool fits = check_sequence(c, b, load_i32(c.q_start + b), load_i32(c.q_start + b + 1), load_i32(c.kv_len + b),
                                     max_q, shared, s);
#ifdef __CUDA_ARCH__
    if (!fits && ws) report_sequence(ws, b);
#else
    (void)fits, (void)ws;
#endif
    return s;
}

// The keys that rows at positions i0 .. i1 (any of them) can see among the
// keys jlo .. jhi - 1: [s0, s1), the sinks, and [lo, hi), in tiles of 2^shift
// keys.
struct Hull {
    int lo, hi, s0, s1;
    int st0, ns, wt0;      // first sink tile, sink tiles, first tile of [lo, hi)
    int tiles;             // all of them (at least 1: a unit that sees nothing has one masked tile)
    __host__ __device__ __forceinline__ bool live(int j) const { return (j >= lo && j < hi) || (j >= s0 && j < s1); }
    // whether any / every key of [a, b) is live
    __host__ __device__ __forceinline__ bool any(int a, int b) const {
        return (a < hi && b > lo && hi > lo) || (a < s1 && b > s0 && s1 > s0);
    }
    __host__ __device__ __forceinline__ bool all(int a, int b) const {
        return (a >= lo && b <= hi) || (a >= s0 && b <= s1) || (a >= s0 && s1 == lo && b <= hi);
    }
    __host__ __device__ __forceinline__ int tile(int k) const { return k < ns ? st0 + k : wt0 + (k - ns); }
};

__host__ __device__ __forceinline__ Hull make_hull(const PagedMask& m, int i0, int i1, int jlo, int jhi, int shift) {
    const int up = (1 << shift) - 1;
    Hull u;
    int lo = jlo, hi = jhi;
    if (m.causal) hi = imin(hi, i1 + 1);
    if (m.window >= 0) lo = imax(lo, i0 - m.window);
    const int s1 = imin(imin(m.sinks, hi), lo);      // sinks beyond the window's reach
    u.s0 = jlo;
    u.s1 = imax(s1, jlo);
    u.lo = lo;
    u.hi = imax(hi, lo);
    const bool win = hi > lo;
    u.wt0 = lo >> shift;
    const int wt1 = win ? (hi + up) >> shift : u.wt0;
    u.st0 = u.s0 >> shift;
    int st1 = u.s1 > u.s0 ? (u.s1 + up) >> shift : u.st0;
    if (win) st1 = imin(st1, u.wt0);
    u.ns = imax(st1 - u.st0, 0);
    u.tiles = imax(u.ns + wt1 - u.wt0, 1);
    if (u.ns + wt1 - u.wt0 == 0) u.wt0 = u.st0;    // nothing seen: any tile, no page of it is read
    return u;
}

// Whether the row at position i sees key j (jlo <= j < jhi is the part's range).
__host__ __device__ __forceinline__ bool paged_visible(const PagedMask& m, int i, int j, int jlo, int jhi) {
    return j >= jlo && j < jhi && (!m.causal || j <= i) && (m.window < 0 || i - j <= m.window || j < m.sinks);
}

// Whether every row at positions i0 .. i1 sees every key of tile kb.
__host__ __device__ __forceinline__ bool tile_open(const PagedMask& m, int kb, int i0, int i1, int jlo, int jhi,
                                                   int shift) {
    const int c0 = kb << shift, c1 = c0 + (1 << shift) - 1;
    return c0 >= jlo && c1 < jhi && (!m.causal || c1 <= i0) && (m.window < 0 || i1 - c0 <= m.window || c1 < m.sinks);
}

// A soft-cap: the score x mul (base 2) becomes out tanh(x in).  Two forms: with
// u = x in, x mul q(u^2) where the polynomial q ~ tanh(u) / u holds, off by 8e-7
// of the score; and out (1 - 2 / (e^(2 |u|) + 1)), off by 3e-7 of the cap at any
// u.  Up to a cap of 64 that is 2e-5 in the exponent and the second form does
// alone; far above the scores it would be all of them, so that beyond 64 (fine)
// it is taken past the polynomial's range only.
constexpr float kSoftCapCoarse = 64.f;
struct SoftCap {
    float in, out, mul;
    bool fine;
};
__device__ __forceinline__ SoftCap soft_cap(float softcap, float scale) {
    // (finite for the smallest and the largest caps too, so that 0 stays 0)
    return {fminf(scale / softcap, FLT_MAX), fminf(softcap * kPagedLog2e, FLT_MAX), scale * kPagedLog2e,
            softcap > kSoftCapCoarse};
}
__device__ __forceinline__ float softcap_inner(float x, float u, const SoftCap& c) {
    const float w = u * u;
    float q = fmaf(kTanhFineC4, w, kTanhFineC3);
    q = fmaf(q, w, kTanhFineC2);
    q = fmaf(q, w, kTanhFineC1);
    q = fmaf(q, w, kTanhFineC0);
    return x * c.mul * q;
}
__device__ __forceinline__ float softcap_outer(float u, const SoftCap& c) {
    const float e = ex2_approx(2.f * kPagedLog2e * fabsf(u));
    return copysignf(c.out * (1.f - __fdividef(2.f, e + 1.f)), u);
}
// One form or the other (a selection: a branch costs three times as much).
__device__ __forceinline__ float softcap_pick(float inner, float u, const SoftCap& c) {
    float y;
    asm("{\n\t.reg .pred p;\n\tsetp.le.f32 p, %3, %4;\n\tselp.f32 %0, %1, %2, p;\n\t}"
        : "=f"(y)
        : "f"(inner), "f"(softcap_outer(u, c)), "f"(fabsf(u)), "f"(kTanhFineRange));
    return y;
}
__device__ __forceinline__ float softcap_one(float x, const SoftCap& c) {
    const float u = x * c.in;
    return c.fine ? softcap_pick(softcap_inner(x, u, c), u, c) : softcap_outer(u, c);
}

// The loader's share of one tile of KT keys: lane l of the warp stands for the
// tile's page l.  Reads the page's id ahead of the copy (-1: no live key, not
// read).
template <int KT>
__device__ __forceinline__ int tile_page(const PagedView& c, const int32_t* table, const Hull& u, int kb, int lane,
                                         int b, uint32_t* ws) {
    const int span = min(c.page_size, KT), a = kb * KT + lane * span;
    if (lane * span >= KT || !u.any(a, a + span)) return -1;
    const int id = load_i32(table + (a >> c.page_shift));
    if (id < 0 || id >= c.num_pages) {
        report_sequence(ws, b);
        return 0;                                  // reported; read something that exists
    }
    return id;
}

// Expect `bytes` more in the barrier's current phase, without an arrival.
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// 3-d tiled load into shared memory (as tma_load_4d).
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

// With v's scales in M (a cache held in 8 bits) l may be 2^80 before a scale of 2^100
// comes, so that 2^d, by which M's step multiplies l, is less than an fp32 number while
// l 2^d counts: l times it in two steps.
__device__ __forceinline__ float times_2_to(float l, float d) {
    const float half = ex2_approx(0.5f * d);
    return l * half * half;
}
// Nor may such an M weigh parts of a row that are to be joined, where their l are more
// than 2^90 apart: outside of 2^-16 .. 2^75 l and M times powers of two (and O by what is
// returned), so that l is 2^-17 to 2^-16 and M says what the part is worth.  (O is then
// 2^-16 of a value at most, so that no sum of parts overflows.  Inside, M stays as it
// is, for the sum may be rounded where M is past 2^20.)
__device__ __forceinline__ float even_out(float& m, float& l) {
    const int k = min(((__float_as_int(l) >> 23) & 255) - 127, 109);
    if (l == 0.f || (k >= -16 && k < 75)) return 1.f;
    const float f = __int_as_float((110 - k) << 23);
    m += static_cast<float>(k + 17);
    l *= f;
    return f;
}

// P, two f16 numbers: 65504 beyond that (2^kPTop is half of it, but a reference that far
// below scores past 2^24 is rounded, and an infinity would be no weight), NaN stays.
__device__ __forceinline__ uint32_t pack_p(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Where a row's partials lie: `count` rows of a kernel's slots, from `first`
// on: slots 2 c + 1, 2 (c + 1), 2 (c + 2), .. of `stride` rows each (or the
// one partial that is kept by row).
struct RowParts {
    const float* o;
    const float2* ml;
    long long first;
    int count, stride;
    __host__ __device__ __forceinline__ long long at(int k) const {
        return first + (k ? (2LL * k - 1) * stride : 0);
    }
    // whether all of them lie in `rows` rows
    __host__ __device__ __forceinline__ bool within(long long rows) const {
        return first >= 0 && count >= 1 && first < rows && at(count - 1) < rows;
    }
};

// Orders this thread's earlier shared-memory writes before later accesses by
// the async proxy (TMA copies, tcgen05 operands).
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Programmatic dependent launch: let the next kernel's blocks start, and wait
// until the kernel before this one is complete and its writes are visible.
__device__ __forceinline__ void pdl_launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The sequences' own kernel beside a shared prefix's.  It is launched once all
// of the prefix's CTAs have signalled, reads nothing of theirs, and would lose
// their overlap by waiting for their end (64 chats after a prefix of 16384
// keys: 55 us, 62 with the wait; 16 x 4 rows after 5024: 19.4 and 24.5).  What
// both read was written before the prefix's kernel, which has waited for that;
// but a launch that was signalled early orders no memory by itself.  So the
// prefix's kernel, behind its wait, writes a mark (release), and the own kernel
// reads it (acquire): seeing it, it also sees what the wait made visible.  Not
// seeing it, it waits after all.  The join clears the mark for the next call.
constexpr unsigned long long kPrefixMark = 0x9d3ac1f05b7e2468ull;
__device__ __forceinline__ unsigned long long* prefix_mark(const PagedParams& p) {
    return reinterpret_cast<unsigned long long*>(p.hdr) + 1;
}
__device__ __forceinline__ void mark_prefix(const PagedParams& p) {
    asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(prefix_mark(p)), "l"(kPrefixMark) : "memory");
}
// The whole block; the copies that it starts afterwards see the same memory.
__device__ __forceinline__ void wait_before_prefix(const PagedParams& p) {
    if (threadIdx.x == 0) {
        unsigned long long seen;
        asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(seen) : "l"(prefix_mark(p)) : "memory");
        if (seen != kPrefixMark) pdl_wait_previous();
    }
    __syncthreads();
    asm volatile("fence.proxy.async;" ::: "memory");
}

// A wait that only time ends (it guards copies and products still writing).
__device__ __forceinline__ bool paged_drain_wait(uint32_t bar, uint32_t parity, const WaitCtl& c, uint32_t site) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 15u) == 0u && globaltimer_ns() - t0 > c.timeout_ns) {
            record_timeout(c, site);
            return false;
        }
    }
}

// Exclusive prefix sums of value(b), b < n, into pre[0 .. n] by the whole
// block (THREADS threads, a multiple of 32); `warp_sums` holds THREADS / 32.
template <int THREADS, class F>
__device__ __forceinline__ void block_prefix(int n, int* pre, int* warp_sums, F value) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int base = 0;
    for (int b0 = 0; b0 < n; b0 += THREADS) {
        const int b = b0 + tid;
        const int v = b < n ? value(b) : 0;
        int x = v;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        if (lane == 31) warp_sums[warp] = x;
        __syncthreads();
        int before = 0, total = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp) before += warp_sums[w];
            total += warp_sums[w];
        }
        if (b < n) pre[b] = base + before + x - v;
        base += total;
        __syncthreads();
    }
    if (tid == 0) pre[n] = base;
    __syncthreads();
}

// A launch; `overlap`: as a programmatic dependent of the kernel before it.  Such
// a kernel starts (barriers, TMEM) while that one ends, and touches no memory
// that others write before pdl_wait_previous() or, beside a shared prefix,
// wait_before_prefix().  Every kernel has waited for the one before it by its
// own end, so that whoever waits for it has waited for all of them.
template <class K, class... A>
cudaError_t paged_launch(K kern, dim3 grid, int threads, size_t smem, bool overlap, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = overlap ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace fa
