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
#include "paged_tiles.cuh"

namespace fa {

cudaError_t launch_paged_tiles(const PagedParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                               cudaStream_t s) {
    return p.D == 64 ? launch_tiles_d<64, false>(p, tk, tv, s) : launch_tiles_d<128, false>(p, tk, tv, s);
}

}  // namespace fa
