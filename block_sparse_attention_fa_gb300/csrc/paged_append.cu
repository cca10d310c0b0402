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
#include "paged_append.cuh"

namespace fa {
namespace {

template <int D>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendParams p, int per_cta) {
    append_tokens<D>(p, blockIdx.x, per_cta);
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
