// paged_append.cu -- a step's keys and values into the paged cache, the rotary
// position embedding applied on the way (fa_kv_append).
//
// For each new token (row t, sequence b, position i) and each pair (x0, x1) of
// the rotated part of a head of q or k,
//     (y0, y1) = (x0 cos - x1 sin, x0 sin + x1 cos),
// cos and sin from the token's row of the caller's fp32 tables; products and
// sums in fp32, rounded once to bf16.  k and v go to slot
// [page_table[b][i / page]][h][i % page], q to its own output.
//
// Every byte is read and written once, so memory bounds it.  A thread takes 16
// elements of one head as two 16-byte pieces: the two halves of 8 pairs
// ((d, d + rot / 2): pieces half a rotation apart; (2 d, 2 d + 1): adjacent
// pieces), for which it needs 8 cosines and 8 sines.
//
// Finding a token's slot takes three loads that wait for one another (q_start,
// the sequence's numbers, its page).  A CTA takes up to four tokens, one warp
// to a token for that part, and then moves the data of two tokens at a time,
// so that enough loads are in flight: 107 to 112 us for 26418 tokens of 32 + 16 heads
// of 128 columns (656 MB, 0.86 to 0.90 of the copy rate), 128 us with a CTA per token;
// eight tokens took 109 us, sixteen 117.  A step of few tokens gives each a CTA
// of its own.
#include <cuda_bf16.h>

#include "paged.cuh"

namespace fa {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendTokens = 4;

struct Piece16 {
    uint32_t a[4], b[4];     // two pieces of 8 bf16
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 8 pairs (a's element e, b's element e).
__device__ __forceinline__ void rotate_halves(Piece16& x, const float (&c)[8], const float (&s)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float a0 = bf_lo(x.a[e]), a1 = bf_hi(x.a[e]), b0 = bf_lo(x.b[e]), b1 = bf_hi(x.b[e]);
        x.a[e] = pack_bf16x2(a0 * c[2 * e] - b0 * s[2 * e], a1 * c[2 * e + 1] - b1 * s[2 * e + 1]);
        x.b[e] = pack_bf16x2(a0 * s[2 * e] + b0 * c[2 * e], a1 * s[2 * e + 1] + b1 * c[2 * e + 1]);
    }
}

// 8 pairs (elements 2 e, 2 e + 1 of the 16).
__device__ __forceinline__ void rotate_pairs(Piece16& x, const float (&c)[8], const float (&s)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float a0 = bf_lo(x.a[e]), a1 = bf_hi(x.a[e]), b0 = bf_lo(x.b[e]), b1 = bf_hi(x.b[e]);
        x.a[e] = pack_bf16x2(a0 * c[e] - a1 * s[e], a0 * s[e] + a1 * c[e]);
        x.b[e] = pack_bf16x2(b0 * c[4 + e] - b1 * s[4 + e], b0 * s[4 + e] + b1 * c[4 + e]);
    }
}

// Where a token goes: the row of the tables (-1: nowhere), and its slot's first
// element in the cache.
struct Place {
    int at;
    size_t kv_row;
};

// One warp finds the place of row t.
__device__ __forceinline__ Place place_of(const AppendParams& p, int t, int lane) {
    Place none{-1, 0};
    // the sequence of row t: how many of q_start[1 ..] are <= t
    int b = 0;
    for (int b0 = 0; b0 < p.c.B; b0 += 128) {
        int ends[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) ends[k] = __ldg(p.c.q_start + min(b0 + 32 * k + lane, p.c.B - 1) + 1);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            b += __popc(__ballot_sync(0xffffffffu, b0 + 32 * k + lane < p.c.B && ends[k] <= t));
    }
    if (b >= p.c.B) return none;                 // behind the last sequence
    const SeqInfo s = seq_info(p.c, b, INT_MAX, 0, lane == 0 ? p.ws : nullptr);
    if (s.n == 0) return none;
    const bool placed = t >= s.q0 && t < s.q0 + s.n;         // (not where q_start decreases)
    const int i = placed ? s.kv - s.n + (t - s.q0) : 0;
    const int at = p.positions ? __ldg(p.positions + t) : i;
    const int page = __ldg(p.c.page_table + (size_t)b * p.c.max_pages + (i >> p.c.page_shift));
    if (!placed || page < 0 || page >= p.c.num_pages || (p.rot && (at < 0 || at >= p.rope_len))) {
        if (lane == 0) report_sequence(p.ws, b);
        return none;
    }
    // (without a rotation the position is not looked at, and may be anything)
    return Place{p.rot ? at : 0, ((size_t)page * p.c.Hkv * p.c.page_size + (i & (p.c.page_size - 1))) * p.D};
}

template <int D>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendParams p, int per_cta) {
    constexpr int kItems = D / 16;               // 16-element items per head
    constexpr int kAtOnce = 2;
    __shared__ Place places[kAppendTokens];
    const int t0 = blockIdx.x * per_cta, tid = threadIdx.x, threads = blockDim.x;
    const int tokens = min(per_cta, p.c.total_q - t0);
    const int items = (p.Hq + 2 * p.c.Hkv) * kItems;
    pdl_wait_previous();
    pdl_launch_next();
    // an item's place in a head and in the cache, and its source
    struct Item {
        int head, k, h, ea, eb;
        bool is_q, is_k, turn;
        const uint16_t* src;
        long long step;
    };
    auto item_of = [&](int x) {
        Item it;
        it.head = x / kItems;
        it.k = x % kItems;
        it.is_q = it.head < p.Hq;
        it.is_k = !it.is_q && it.head < p.Hq + p.c.Hkv;
        it.h = it.is_q ? it.head : it.is_k ? it.head - p.Hq : it.head - p.Hq - p.c.Hkv;
        it.src = it.is_q ? p.q + (long long)it.h * p.qs[1]
                 : it.is_k ? p.k + (long long)it.h * p.ks[1] : p.v + (long long)it.h * p.vs[1];
        it.step = it.is_q ? p.qs[0] : it.is_k ? p.ks[0] : p.vs[0];
        // the item's two pieces of 8: half a rotation apart where halves are
        // paired, adjacent otherwise (the items past the rotation pair up the
        // pieces that are left)
        const bool rotated = it.k < p.rot / 16, halves = rotated && !p.interleaved;
        it.turn = rotated && (it.is_q || it.is_k);
        it.ea = halves ? 8 * it.k : 16 * it.k;
        it.eb = halves ? 8 * it.k + p.rot / 2 : 16 * it.k + 8;
        return it;
    };
    Piece16 v[kAtOnce];
    auto load = [&](const Item& it, int g) {
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e) {
            if (g + e >= tokens) continue;
            const uint16_t* from = it.src + (long long)(t0 + g + e) * it.step;
            *reinterpret_cast<uint4*>(v[e].a) = __ldcs(reinterpret_cast<const uint4*>(from + it.ea));
            *reinterpret_cast<uint4*>(v[e].b) = __ldcs(reinterpret_cast<const uint4*>(from + it.eb));
        }
    };
    // the thread's first data sets out before the places are known
    Item it = item_of(min(tid, items - 1));
    load(it, 0);
    for (int w = tid >> 5; w < tokens; w += threads >> 5) {
        const Place x = place_of(p, t0 + w, tid & 31);
        if ((tid & 31) == 0) places[w] = x;
    }
    __syncthreads();
    const size_t kv_head = (size_t)p.c.page_size * D;
    for (int x = tid; x < items; x += threads) {
        if (x != tid) it = item_of(x);
        uint16_t* const cache = (it.is_k ? p.kc : p.vc) + it.h * kv_head;
        for (int g = 0; g < tokens; g += kAtOnce) {
            if (x != tid || g > 0) load(it, g);
#pragma unroll
            for (int e = 0; e < kAtOnce; ++e) {
                if (g + e >= tokens) continue;
                const Place at = places[g + e];
                if (at.at < 0) continue;
                if (it.turn) {
                    float c[8], sn[8];
                    const size_t row = (size_t)at.at * (p.rot / 2) + 8 * it.k;
                    *reinterpret_cast<float4*>(c) = __ldg(reinterpret_cast<const float4*>(p.cos + row));
                    *reinterpret_cast<float4*>(c + 4) = __ldg(reinterpret_cast<const float4*>(p.cos + row + 4));
                    *reinterpret_cast<float4*>(sn) = __ldg(reinterpret_cast<const float4*>(p.sin + row));
                    *reinterpret_cast<float4*>(sn + 4) = __ldg(reinterpret_cast<const float4*>(p.sin + row + 4));
                    if (p.interleaved)
                        rotate_pairs(v[e], c, sn);
                    else
                        rotate_halves(v[e], c, sn);
                }
                uint16_t* dst = it.is_q ? p.q_out + (long long)(t0 + g + e) * p.os[0] + (long long)it.h * p.os[1]
                                        : cache + at.kv_row;
                *reinterpret_cast<uint4*>(dst + it.ea) = *reinterpret_cast<const uint4*>(v[e].a);
                *reinterpret_cast<uint4*>(dst + it.eb) = *reinterpret_cast<const uint4*>(v[e].b);
            }
        }
    }
}

}  // namespace

cudaError_t launch_kv_append(const AppendParams& p, cudaStream_t s) {
    if (p.c.total_q == 0) return cudaSuccess;
    // the items shared evenly by the threads; several tokens to a CTA once
    // every SM has some CTAs even so
    const int items = (p.Hq + 2 * p.c.Hkv) * (p.D / 16), rounds = (items + kAppendThreads - 1) / kAppendThreads;
    const int threads = ((items + rounds - 1) / rounds + 31) / 32 * 32;
    const int per_cta = p.c.total_q >= kAppendTokens * 4 * device_sm_count() ? kAppendTokens : 1;
    const dim3 grid((p.c.total_q + per_cta - 1) / per_cta);
    return p.D == 64 ? paged_launch(kv_append_kernel<64>, grid, threads, 0, true, s, p, per_cta)
                     : paged_launch(kv_append_kernel<128>, grid, threads, 0, true, s, p, per_cta);
}

}  // namespace fa
