// paged_append_scaled.cu -- a step's keys and values into a cache held in 8
// bits with a scale for each page and kv head (fa_kv_append_scaled).
//
// For a page's new tokens of one kv head, x the rotated keys (fp32) or the
// values:
//     amax = max |x| over the finite ones, scale = 2^e, e least with amax <= 448 2^e,
//     scale = max(scale, the page's scale before) where it holds earlier tokens,
//     code = e4m3(x / scale), and earlier codes e4m3(code scale_before / scale).
// With a = m 2^x, 1/2 <= m < 1, and 448 = 7/8 2^9, e = x - 9 if m <= 7/8, else x - 8.
// Powers of two lose nothing (e4m3 has exponents to spare), so that a code is
// rounded once, however often the page's scale grows.
//
// A token's code needs the largest of all the step's tokens on its page, so a
// unit of work is a page's share of the step, for some kv heads: a CTA takes
// kAppendThreads / G heads, G threads (whole warps) to each.  A thread holds the
// first of its 16-element items of k and of v in registers between the maximum
// and the rounding (k as it came, and rotated for both); items beyond that are
// read again, from L2.  What a unit costs is latency (its sequence, its page,
// its rows, the barrier), so warps count more than items held: 26418 tokens of
// 32 + 16 heads take 124 us with four CTAs per SM and one item, 135 with two,
// 149 and 163 with three and two CTAs and two items, 177 with k in fp32 as well.
// The loads set out before the page's id is known.  The queries are no part of
// this: the first CTAs of the launch rotate them token by token, as in
// paged_append.cu.
//
// Memory bounds it: a token is read as bf16 and written as bytes.
#include <algorithm>
#include <math_constants.h>

#include "paged_append.cuh"

namespace fa {
namespace {

constexpr int kHeld = 1;

// Which page's share of the step is unit u: the sequence, and the page's place
// in its row of the table.  Uniform over the block; false: there is none.
__device__ __forceinline__ bool find_unit(const AppendScaledParams& p, int u, bool report, SeqInfo& s, int& b, int& entry) {
    __shared__ int warp_sums[kAppendThreads / 32], found[4];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, shift = p.c.page_shift;
    int at = 0;                                  // units of the sequences before b0
    for (int b0 = 0; b0 < p.c.B; b0 += kAppendThreads) {
        SeqInfo mine{0, 0, 0, true};
        if (b0 + tid < p.c.B) mine = seq_info(p.c, b0 + tid, INT_MAX, 0, report ? p.ws : nullptr);
        const int first = (mine.kv - mine.n) >> shift, count = mine.n ? ((mine.kv - 1) >> shift) - first + 1 : 0;
        int upto = count;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += y;
        }
        if (lane == 31) warp_sums[warp] = upto;
        __syncthreads();
        int before = at, total = 0;
#pragma unroll
        for (int w = 0; w < kAppendThreads / 32; ++w) {
            if (w < warp) before += warp_sums[w];
            total += warp_sums[w];
        }
        upto += before;
        const bool here = u < at + total;
        if (u >= upto - count && u < upto) {
            found[0] = b0 + tid;
            found[1] = first + u - (upto - count);
            found[2] = mine.q0;
            found[3] = mine.n;
        }
        __syncthreads();
        if (here) {
            b = found[0];
            entry = found[1];
            s.q0 = found[2];
            s.n = found[3];
            s.kv = load_i32(p.c.kv_len + b);
            return true;
        }
        at += total;
    }
    return false;
}

__device__ __forceinline__ float needed_scale(float amax) {
    const int bits = __float_as_int(amax);
    // amax = m 2^x: a normal number's x is its exponent field - 126; smaller ones need the least scale anyway
    const int x = (bits >> 23) - 126, e = x - ((bits & 0x7fffff) <= 0x600000 ? 9 : 8);
    return __int_as_float((min(max(amax > 0.f ? e : -100, -100), 119) + 127) << 23);
}

__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// Four codes of x inv (infinities become NaN, as the conversion makes them 448).
__device__ __forceinline__ uint32_t e4m3_four(const float* x, float inv) {
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = fmaf(x[e], 0.f, x[e] * inv);
    return e4m3_pair(y[0], y[1]) | e4m3_pair(y[2], y[3]) << 16;
}
// Four codes of codes x ratio.
__device__ __forceinline__ uint32_t e4m3_again(uint32_t w, float ratio) {
    uint32_t r = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w >> (16 * e))));
        float lo, hi;
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
            : "=f"(lo), "=f"(hi)
            : "r"(h));
        r |= e4m3_pair(lo * ratio, hi * ratio) << (16 * e);
    }
    return r;
}

// A page's share of the step, heads h0 .. of k and v.
template <int D>
__device__ __forceinline__ void append_page(const AppendScaledParams& p, int u, int h0, int threads_per_head, bool report) {
    constexpr int kItems = D / 16;
    __shared__ unsigned amax_s[2][kAppendThreads / 32];
    const int tid = threadIdx.x, G = threads_per_head, slot = tid / G, g = tid - slot * G, h = h0 + slot;
    SeqInfo s;
    int b, entry;
    if (tid < 2 * (kAppendThreads / 32)) amax_s[tid & 1][tid >> 1] = 0;
    if (!find_unit(p, u, report, s, b, entry)) return;
    const int first = entry << p.c.page_shift, start = s.kv - s.n;
    const int lo = max(first, start), hi = min(first + p.c.page_size, s.kv);     // positions of the unit
    const bool active = h < p.c.Hkv;
    const int items = active ? (hi - lo) * kItems : 0, row0 = s.q0 + lo - start;
    const uint16_t* const src_k = p.k + static_cast<long long>(h) * p.ks[1];
    const uint16_t* const src_v = p.v + static_cast<long long>(h) * p.vs[1];

    // an item's two pieces of 8 (as in append_tokens), its first elements within the head
    auto pieces = [&](int x, int rot, int& ea, int& eb) {
        const int k = x % kItems;
        const bool halves = k < rot / 16 && !p.interleaved;
        ea = halves ? 8 * k : 16 * k;
        eb = halves ? 8 * k + rot / 2 : 16 * k + 8;
    };
    auto fetch = [&](int x, const uint16_t* src, long long step, int rot, Piece16& w) {
        int ea, eb;
        pieces(x, rot, ea, eb);
        const uint16_t* const from = src + static_cast<long long>(row0 + x / kItems) * step;
        load_now(from + ea, w.a);
        load_now(from + eb, w.b);
    };
    // the token's row of the tables; -1: it has no place
    auto place = [&](int x) {
        if (!p.rot) return 0;
        const int at = p.positions ? load_now(p.positions + row0 + x / kItems) : lo + x / kItems;
        if (at >= 0 && at < p.rope_len) return at;
        report_sequence(p.ws, b);
        return -1;
    };
    auto widen = [](const Piece16& w, float (&y)[16]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y[2 * e] = bf_lo(w.a[e]);
            y[2 * e + 1] = bf_hi(w.a[e]);
            y[8 + 2 * e] = bf_lo(w.b[e]);
            y[9 + 2 * e] = bf_hi(w.b[e]);
        }
    };
    auto rotate = [&](int x, int at, float (&y)[16]) {
        const int k = x % kItems;
        if (k >= p.rot / 16) return;
        float cs[8], sn[8];
        const size_t row = static_cast<size_t>(at) * (p.rot / 2) + 8 * k;
        *reinterpret_cast<float4*>(cs) = __ldg(reinterpret_cast<const float4*>(p.cos + row));
        *reinterpret_cast<float4*>(cs + 4) = __ldg(reinterpret_cast<const float4*>(p.cos + row + 4));
        *reinterpret_cast<float4*>(sn) = __ldg(reinterpret_cast<const float4*>(p.sin + row));
        *reinterpret_cast<float4*>(sn + 4) = __ldg(reinterpret_cast<const float4*>(p.sin + row + 4));
        // pairs (2 e, 2 e + 1), or (e, 8 + e) where halves are paired
        auto turn = [&](float& x0, float& x1, int e) {
            const float u0 = x0, u1 = x1;
            x0 = u0 * cs[e] - u1 * sn[e];
            x1 = u0 * sn[e] + u1 * cs[e];
        };
        if (p.interleaved) {
#pragma unroll
            for (int e = 0; e < 8; ++e) turn(y[2 * e], y[2 * e + 1], e);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) turn(y[e], y[8 + e], e);
        }
    };
    auto largest = [](const float (&y)[16], float m) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const float a = fabsf(y[e]);
            m = fmaxf(m, a < CUDART_INF_F ? a : 0.f);
        }
        return m;
    };

    Piece16 raw_k[kHeld], raw_v[kHeld];
#pragma unroll
    for (int e = 0; e < kHeld; ++e) {
        const int x = g + e * G;
        if (x >= items) continue;
        fetch(x, src_k, p.ks[0], p.rot, raw_k[e]);
        fetch(x, src_v, p.vs[0], 0, raw_v[e]);
    }
    const int page = load_i32(p.c.page_table + static_cast<size_t>(b) * p.c.max_pages + entry);
    const bool placed = page >= 0 && page < p.c.num_pages;         // (uniform)
    if (!placed) {
        if (tid == 0) report_sequence(p.ws, b);
        return;
    }
    const size_t head = static_cast<size_t>(page) * p.c.Hkv + h;
    const bool earlier = lo > first;
    const float before[2] = {active && earlier ? p.k_scale[head] : 0.f, active && earlier ? p.v_scale[head] : 0.f};
    float m[2] = {0.f, 0.f};
    int at[kHeld];
#pragma unroll
    for (int e = 0; e < kHeld; ++e) {
        const int x = g + e * G;
        at[e] = x < items ? place(x) : -1;
        if (at[e] < 0) continue;
        float y[16];
        widen(raw_v[e], y);
        m[1] = largest(y, m[1]);
        widen(raw_k[e], y);
        rotate(x, at[e], y);
        m[0] = largest(y, m[0]);
    }
    for (int x = g + kHeld * G; x < items; x += G) {
        const int at = place(x);
        if (at < 0) continue;
        Piece16 w;
        float y[16];
        fetch(x, src_v, p.vs[0], 0, w);
        widen(w, y);
        m[1] = largest(y, m[1]);
        fetch(x, src_k, p.ks[0], p.rot, w);
        widen(w, y);
        rotate(x, at, y);
        m[0] = largest(y, m[0]);
    }
    // (the bits of numbers that are not negative are in their order)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const unsigned top = __reduce_max_sync(0xffffffffu, __float_as_uint(m[q]));
        if ((tid & 31) == 0) atomicMax(&amax_s[q][slot], top);
    }
    __syncthreads();
    if (!active) return;
    float inv[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const float scale = fmaxf(needed_scale(__uint_as_float(amax_s[q][slot])), before[q]);
        inv[q] = 1.f / scale;
        if (g == 0) (q ? p.v_scale : p.k_scale)[head] = scale;
        if (!earlier || scale == before[q]) continue;
        // the earlier tokens' codes, to the new scale
        const float ratio = before[q] / scale;
        uint4* const old = reinterpret_cast<uint4*>((q ? p.v8 : p.k8) + head * p.c.page_size * D);
        for (int x = g; x < (lo - first) * kItems; x += G) {
            uint4 w = old[x];
            w.x = e4m3_again(w.x, ratio);
            w.y = e4m3_again(w.y, ratio);
            w.z = e4m3_again(w.z, ratio);
            w.w = e4m3_again(w.w, ratio);
            old[x] = w;
        }
    }
    auto put = [&](int x, int q, const float (&y)[16]) {
        int ea, eb;
        pieces(x, q ? 0 : p.rot, ea, eb);
        uint8_t* const dst = (q ? p.v8 : p.k8) + head * p.c.page_size * D + static_cast<size_t>(lo - first + x / kItems) * D;
        *reinterpret_cast<uint2*>(dst + ea) = make_uint2(e4m3_four(y, inv[q]), e4m3_four(y + 4, inv[q]));
        *reinterpret_cast<uint2*>(dst + eb) = make_uint2(e4m3_four(y + 8, inv[q]), e4m3_four(y + 12, inv[q]));
    };
#pragma unroll
    for (int e = 0; e < kHeld; ++e) {
        if (at[e] < 0) continue;
        const int x = g + e * G;
        float y[16];
        widen(raw_v[e], y);
        put(x, 1, y);
        widen(raw_k[e], y);
        rotate(x, at[e], y);
        put(x, 0, y);
    }
    for (int x = g + kHeld * G; x < items; x += G) {
        const int at = place(x);
        if (at < 0) continue;
        Piece16 w;
        float y[16];
        fetch(x, src_k, p.ks[0], p.rot, w);
        widen(w, y);
        rotate(x, at, y);
        put(x, 0, y);
        fetch(x, src_v, p.vs[0], 0, w);
        widen(w, y);
        put(x, 1, y);
    }
}

// CTAs 0 .. q_ctas - 1: the queries of per_cta tokens each; the others: page by
// page, some kv heads each.
template <int D>
__global__ void __launch_bounds__(kAppendThreads, 4)
kv_append_scaled_kernel(const AppendParams q, const AppendScaledParams p, int q_ctas, int per_cta, int threads_per_head) {
    if (static_cast<int>(blockIdx.x) < q_ctas) {
        append_tokens<D>(q, blockIdx.x, per_cta);
        return;
    }
    pdl_wait_previous();
    pdl_launch_next();
    const int at = blockIdx.x - q_ctas, heads = kAppendThreads / threads_per_head;
    const int parts = (p.c.Hkv + heads - 1) / heads;
    const int u = at / parts;
    append_page<D>(p, u, (at - u * parts) * heads, threads_per_head, at == 0);
    // the first of these CTAs reports: its unit was found among the first sequences, the
    // others have not been looked at (after the unit: 2048 sequences are eight loads more)
    if (at == 0) {
        for (int b = kAppendThreads + threadIdx.x; b < p.c.B; b += kAppendThreads) seq_info(p.c, b, INT_MAX, 0, p.ws);
    }
}

}  // namespace

cudaError_t launch_kv_append_scaled(const AppendScaledParams& p, cudaStream_t s) {
    if (p.c.total_q == 0) return cudaSuccess;
    // a warp to a head where sequences bring a few tokens each, and else as many
    // threads as hold a page's share in registers
    const long long each = (p.c.total_q + p.c.B - 1LL) / p.c.B;
    const int tokens = static_cast<int>(std::min<long long>(each, p.c.page_size));
    int G = 32;
    while (G < kAppendThreads && G * kHeld < tokens * (p.D / 16)) G *= 2;
    // pages that the step can touch: one more than it fills, twice, per sequence, and one per token at most
    const long long units = std::min<long long>(p.c.total_q, p.c.total_q / p.c.page_size + 2LL * p.c.B);
    const int heads = kAppendThreads / G;
    const long long kv_ctas = units * ((p.c.Hkv + heads - 1) / heads);
    const int per_cta = p.c.total_q >= kAppendTokens * 4 * device_sm_count() ? kAppendTokens : 1;
    const long long q_ctas = p.Hq ? (p.c.total_q + per_cta - 1LL) / per_cta : 0;
    if (q_ctas + kv_ctas > 2147483647LL) return cudaErrorInvalidConfiguration;
    AppendParams q = p;
    q.c.Hkv = 0;
    auto kern = p.D == 64 ? kv_append_scaled_kernel<64> : kv_append_scaled_kernel<128>;
    return paged_launch(kern, dim3(static_cast<unsigned>(q_ctas + kv_ctas)), kAppendThreads, 0, true, s, q, p,
                        static_cast<int>(q_ctas), per_cta, G);
}

}  // namespace fa
