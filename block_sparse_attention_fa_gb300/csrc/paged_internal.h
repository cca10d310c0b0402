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
