// paged_small_scaled.cu -- paged_small.cu's kernel over a cache held in 8 bits
// (e4m3 codes, a scale for each page and kv head).
//
// What differs.  The codes come into shared memory as they are and are converted
// in registers, each once per CTA, to f16, which holds them exactly; so does it a
// row of Q scaled by a power of two, and P, at most 1, is rounded to f16's 11 bits
// instead of bf16's 8.  Products and sums are fp32's, k's scale is applied to S
// and v's to the sum of a page's 16 keys, in fp32 too: any scales will do.
//
// A thread's 32 bits of a row of codes are four adjacent columns where a matrix
// product's operand has two and two: K's columns go to the product in another
// order, and Q's with them; V's 16-byte chunks come transposed as pairs of
// columns, whose even and odd ones go to two products.
//
// A tile is 128 keys, 32 KB or 16 KB (64 columns), and 96 KB of them are in
// flight per CTA.  The loader reads page ids two tiles ahead and scales one.
#include "paged_small.cuh"

namespace fa {

cudaError_t launch_paged_small_scaled(const PagedScaledParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                                      cudaStream_t s) {
    return p.D == 64 ? launch_small_d<64, true>(p, tk, tv, s) : launch_small_d<128, true>(p, tk, tv, s);
}

}  // namespace fa
