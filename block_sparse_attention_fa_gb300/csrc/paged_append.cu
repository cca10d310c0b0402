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
// pieces), for which it needs 8 cosines and 8 sines.  One CTA per token: its
// threads find the token's sequence together (each tests a part of q_start,
// one block-wide count adds them up).
#include <cuda_bf16.h>

#include "paged.cuh"

namespace fa {
namespace {

constexpr int kAppendThreads = 256;

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

template <int D>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendParams p) {
    constexpr int kItems = D / 16;               // 16-element items per head
    const int t = blockIdx.x, tid = threadIdx.x;
    pdl_wait_previous();
    pdl_launch_next();
    // the sequence of row t: how many of q_start[1 ..] are <= t
    int b = 0;
    for (int b0 = 0; b0 < p.c.B; b0 += kAppendThreads)
        b += __syncthreads_count(b0 + tid < p.c.B && __ldg(p.c.q_start + min(b0 + tid, p.c.B - 1) + 1) <= t);
    if (b >= p.c.B) return;                      // behind the last sequence
    const SeqInfo s = seq_info(p.c, b, INT_MAX, 0, tid == 0 ? p.ws : nullptr);
    if (s.n == 0) return;
    if (t < s.q0 || t >= s.q0 + s.n) {           // q_start is not in order
        if (tid == 0) report_sequence(p.ws, b);
        return;
    }
    const int i = s.kv - s.n + (t - s.q0);
    const int at = p.positions ? __ldg(p.positions + t) : i;
    const int page = __ldg(p.c.page_table + (size_t)b * p.c.max_pages + (i >> p.c.page_shift));
    if (page < 0 || page >= p.c.num_pages || (p.rot && (at < 0 || at >= p.rope_len))) {
        if (tid == 0) report_sequence(p.ws, b);
        return;
    }
    const int slot = i & (p.c.page_size - 1);
    const size_t kv_row = ((size_t)page * p.c.Hkv * p.c.page_size + slot) * D;
    const size_t kv_head = (size_t)p.c.page_size * D;
    const int heads = p.Hq + 2 * p.c.Hkv, rot_items = p.rot / 16;
    for (int x = tid; x < heads * kItems; x += kAppendThreads) {
        const int head = x / kItems, k = x % kItems;
        const uint16_t* src;
        uint16_t* dst;
        bool turn = k < rot_items;
        if (head < p.Hq) {
            src = p.q + (long long)t * p.qs[0] + (long long)head * p.qs[1];
            dst = p.q_out + (long long)t * p.os[0] + (long long)head * p.os[1];
        } else if (head < p.Hq + p.c.Hkv) {
            const int h = head - p.Hq;
            src = p.k + (long long)t * p.ks[0] + (long long)h * p.ks[1];
            dst = p.kc + kv_row + h * kv_head;
        } else {
            const int h = head - p.Hq - p.c.Hkv;
            src = p.v + (long long)t * p.vs[0] + (long long)h * p.vs[1];
            dst = p.vc + kv_row + h * kv_head;
            turn = false;
        }
        // the item's two pieces of 8: half a rotation apart where halves are
        // paired, adjacent otherwise (the items past the rotation pair up the
        // pieces that are left)
        const bool halves = k < rot_items && !p.interleaved;
        const int ea = halves ? 8 * k : 16 * k, eb = halves ? 8 * k + p.rot / 2 : 16 * k + 8;
        Piece16 v;
        *reinterpret_cast<uint4*>(v.a) = *reinterpret_cast<const uint4*>(src + ea);
        *reinterpret_cast<uint4*>(v.b) = *reinterpret_cast<const uint4*>(src + eb);
        if (turn) {
            float c[8], sn[8];
            const size_t row = (size_t)at * (p.rot / 2) + 8 * k;
            *reinterpret_cast<float4*>(c) = __ldg(reinterpret_cast<const float4*>(p.cos + row));
            *reinterpret_cast<float4*>(c + 4) = __ldg(reinterpret_cast<const float4*>(p.cos + row + 4));
            *reinterpret_cast<float4*>(sn) = __ldg(reinterpret_cast<const float4*>(p.sin + row));
            *reinterpret_cast<float4*>(sn + 4) = __ldg(reinterpret_cast<const float4*>(p.sin + row + 4));
            if (p.interleaved)
                rotate_pairs(v, c, sn);
            else
                rotate_halves(v, c, sn);
        }
        *reinterpret_cast<uint4*>(dst + ea) = *reinterpret_cast<const uint4*>(v.a);
        *reinterpret_cast<uint4*>(dst + eb) = *reinterpret_cast<const uint4*>(v.b);
    }
}

}  // namespace

cudaError_t launch_kv_append(const AppendParams& p, cudaStream_t s) {
    if (p.c.total_q == 0) return cudaSuccess;
    return p.D == 64 ? paged_launch(kv_append_kernel<64>, dim3(p.c.total_q), kAppendThreads, 0, true, s, p)
                     : paged_launch(kv_append_kernel<128>, dim3(p.c.total_q), kAppendThreads, 0, true, s, p);
}

}  // namespace fa
