// paged_internal.h -- parameter blocks and launchers of the cache held in 8
// bits and of the step's pages (paged_api.cu and the kernels), beside those of
// the bf16 cache in fa_internal.h.
#pragma once

#include "fa_internal.h"

namespace fa {

// The paged forward over a cache held in 8 bits.
struct PagedScaledParams : PagedParams {
    const float *k_scale, *v_scale;   // [num_pages][Hkv]
};

// The append to one (kc and vc are not used).
struct AppendScaledParams : AppendParams {
    uint8_t *k8, *v8;
    float *k_scale, *v_scale;
};

// fa_paged_step's arguments as its kernels see them.
struct StepParams {
    int B, num_pages, page_size, page_shift, max_pages, shared_pages, total_q;
    const int32_t *new_len, *keep_len, *kv_len;
    int32_t *page_table, *free_pages;
    const int32_t* free_count;
    int32_t *kv_len_out, *free_count_out, *q_start;
    int64_t* slots;
    int32_t* positions;
    uint32_t* ws;
};

// Keys of a tile of the small kernel over codes: 32 KB of K and V (16 KB for 64
// columns, where 32 would be 256 keys).
constexpr int kPagedSmallScaledKeys = 128;

// P over codes is an f16 operand, whose numbers end at 2^16, lose bits below 2^-14 and
// are 0 below 2^-25.  So P is 2^(x - M) with a reference M that lies below the largest
// x: by kPHead when M is set, and M is raised once an x is past it by kPTop.  A key down
// to 2^-(kPHead + 14) of the largest keeps 11 bits, and 2^-(kPHead + 25) of it is what
// is lost below.  (l and M leave out nothing: O / l and M + log2 l are the same
// with any M.)  A larger head means more rescales: 4 chunks of up to 1024 tokens on up
// to 8192 keys 219.4 us with 7, 220.3 with 8 (as with a reference at the maximum that
// is raised by 2^8), 221.9 with 9 and 226.4 with 11; single tokens the same with all.
constexpr float kPTop = 15.f, kPHead = 8.f;
// v's scales as exponents (log2 and reciprocal): one below 2^-80 of the largest so
// far in the unit, or below 2^-82, counts as that (l, a sum of P / scale with P up to
// 2^kPTop, holds 2^30 keys of it).
constexpr float kLeastRatio = 8.271806125530277e-25f, kLeastScale = 2.0679515313825692e-25f;

cudaError_t launch_kv_append_scaled(const AppendScaledParams& p, cudaStream_t s);
cudaError_t launch_paged_step(const StepParams& p, cudaStream_t s);
cudaError_t launch_paged_small_scaled(const PagedScaledParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                                      cudaStream_t s);
cudaError_t launch_paged_eight_scaled(const PagedScaledParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                                      cudaStream_t s);
cudaError_t launch_paged_tiles_scaled(const PagedScaledParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                                      cudaStream_t s);
// Pages of codes, boxes of min(page_size, tile_keys) keys: as rows of 128 bytes
// with 128-byte swizzle (a key of 128 columns, or two of 64), or with `by_key` a
// row to each key, in the swizzle of its width.
fa_status page_tensor_map_scaled(CUtensorMap* map, const void* base, long long blocks, int page_size, int D,
                                 int tile_keys, bool by_key);

}  // namespace fa
