// paged_tiles_scaled.cu -- paged_tiles.cu's kernel over a cache held in 8 bits
// (e4m3 codes, a scale for each page and kv head).
//
// What differs.  The tensor cores take both operands in one type, and P in 8
// bits would lose half of its bits, so the codes become bf16, which holds them
// exactly, in shared memory: four more warps (12-15) convert 64-key halves of K
// and V from a ring of codes, as TMA brings them, to one of bf16 operands, in
// the same 128-byte swizzle.  That is 256 rows' work per key converted once.
// The scales stay out of the operands and may be any: k's multiplies S as it
// leaves TMEM, v's multiplies P before it is rounded, 16 columns (of one page)
// at a time.  V's unseen rows are cleared as they are converted (no warp 11).
#include "paged_tiles.cuh"

namespace fa {

cudaError_t launch_paged_tiles_scaled(const PagedScaledParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                                      cudaStream_t s) {
    return p.D == 64 ? launch_tiles_d<64, true>(p, tk, tv, s) : launch_tiles_d<128, true>(p, tk, tv, s);
}

}  // namespace fa
