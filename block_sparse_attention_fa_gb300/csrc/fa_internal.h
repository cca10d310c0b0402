// fa_internal.h -- parameter blocks and launchers shared by the host layer
// (fa_api.cu) and the kernels (block_mask.cu, fwd_fp32.cu, fwd_bf16.cu).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/fa.h"

namespace fa {

constexpr int kBlock = 128;       // BlockMask tile edge (q and kv)

// The BlockMask as the kernels see it.
struct BlockMaskView {
    int B, H;                     // mask extents (1 = broadcast)
    int nq, nkv;
    const int32_t* kv_num_blocks;
    const int32_t* kv_indices;
    const int32_t* full_kv_num_blocks;
    const int32_t* full_kv_indices;
};

// The transposed BlockMask (the q-blocks that visit each kv block), as the
// backward's dK/dV kernel walks it.
struct BlockMaskColsView {
    const int32_t* q_num_blocks;       // [B][H][nkv]
    const int32_t* q_indices;          // [B][H][nkv][nq]
    const int32_t* full_q_num_blocks;
    const int32_t* full_q_indices;
};

// A built-in mask_mod as the kernels see it.
struct MaskParams {
    int kind;                     // fa_mask_kind
    int window;
    int prefix_len;
    int seg_batch;
    const int32_t* seg;           // [seg_batch, seg_len]
    int seg_len;
    const uint32_t* table;        // [table_batch, q_len, table_words] attend bits
    int table_batch;
    int table_words;              // ceil(kv_len / 32)
};

struct ScoreParams {
    int kind;                     // fa_score_kind
    float softcap;
    const float* slopes;
    const float* rel_bias;
    int rel_max;
};

struct FwdParams {
    int B, Hq, Hkv, q_len, kv_len, D, group;
    int num_units;                // B * Hq * nq work units
    float scale;                  // 1/sqrt(D) unless overridden
    BlockMaskView bm;
    MaskParams mask;
    ScoreParams score;
    const void* q;
    const void* k;
    const void* v;
    void* o;
    float* lse;
    uint32_t* ws;
    uint64_t timeout_ns;
    uint32_t flags;
    uint32_t debug_flags;
};

// The split-KV decoding forward (decode_bf16.cu).
struct DecodeParams {
    int B, Hq, Hkv, q_len, kv_len, D, group;
    int rows;                     // query rows per row group (<= 16)
    int grouped;                  // 1: a row group is (b, kv head), all its query heads; 0: (b, query head)
    int num_groups;               // B * Hkv or B * Hq
    int splits;                   // kv splits per row group
    float scale;
    BlockMaskView bm;
    MaskParams mask;
    ScoreParams score;
    const void* q;
    void* o;
    float* lse;
    float* partials;              // [B][Hq][q_len][splits][D + 2]: O, m, l of each split
    uint32_t* ws;
    uint64_t timeout_ns;
    uint32_t flags;
};

// The backward (bwd_bf16.cu).
struct BwdParams {
    int B, Hq, Hkv, q_len, kv_len, D, group;
    float scale;
    BlockMaskView bm;
    MaskParams mask;
    ScoreParams score;
    const void* q;
    const void* k;
    const void* v;
    const void* o;                // the forward's output (bf16)
    const void* dout;             // upstream gradient of O (bf16)
    const float* lse;             // the forward's logsumexp
    float* rowstats;              // scratch [2][B][Hq][nq * 128]: rowsum(dO * O), then -lse log2(e)
    float* dq;
    float* dk;
    float* dv;
    BlockMaskColsView cols;
    // Window masks with sinks: the dK/dV visits of the first sink_blocks kv
    // blocks are split into sink_parts units each (0, 1: not split).
    int sink_blocks, sink_parts;
    uint32_t* ws;
    uint64_t timeout_ns;
};

struct BuildParams {
    int B, H, q_len, kv_len, nq, nkv;
    MaskParams mask;
    int32_t* kv_num_blocks;
    int32_t* kv_indices;
    int32_t* full_kv_num_blocks;
    int32_t* full_kv_indices;
    uint32_t* ws;
    int fast_rows;                // set by the launcher: rows built in shared memory, stored as int4
};

// The paged cache and the step's batch as the kernels see them (fa_paged_kv).
struct PagedView {
    int B, Hkv, num_pages, page_size, page_shift, max_pages, total_q;
    const int32_t* page_table;
    const int32_t* kv_len;
    const int32_t* q_start;
};

// The mask of a paged call: causal or not, window (-1: none), sinks.
struct PagedMask {
    int causal, window, sinks;
};

struct AppendParams {
    PagedView c;
    int Hq, D, rot, rope_len, interleaved;
    const uint16_t *q, *k, *v;
    uint16_t *q_out, *kc, *vc;
    long long qs[2], ks[2], vs[2], os[2];   // token and head strides, elements
    const float *cos, *sin;
    const int32_t* positions;
    uint32_t* ws;
};

// What a unit of work that was split over several CTAs needs to be joined:
// CTA c's last unit starts there and runs on over `count` CTAs (0: it does not).
struct PagedMeta {
    int count, q0, row0, rows, h, pad[3];
};

// The partial results of one kernel (the sequences' own keys, or the shared
// prefix).  A partial is an unnormalised row of O with its running max and
// sum (base 2).  Slot 2 c holds the partial of the unit that CTA c continues
// from the CTA before, slot 2 c + 1 that of the unit that starts in CTA c and
// continues in the next one.
struct PagedParts {
    float* slot_o;        // [2 ctas][rows_per_unit][D]
    float2* slot_ml;
    float* row_o;         // [total_q][Hq][D]: units that one CTA finishes, with a shared prefix
    float2* row_ml;
};

// n / d for 0 <= n < 2^31 by a multiplication: with 2^s >= d and
// m = floor(2^32 (2^s - d) / d) + 1, n / d = (mulhi(m, n) + n) >> s
// (Granlund and Montgomery).
struct FastDiv {
    uint32_t d, m, s;
};
inline FastDiv fast_div(uint32_t d) {
    FastDiv f{d, 0, 0};
    while ((1ull << f.s) < d) ++f.s;
    f.m = static_cast<uint32_t>((((1ull << f.s) - d) << 32) / d + 1);
    return f;
}

struct PagedParams {
    PagedView c;
    PagedMask mask;
    int Hq, group, D;
    FastDiv by_group;
    int max_q;
    int shared;           // length of the shared prefix
    int prefix;           // 1: this kernel attends to the shared prefix, 0: to the sequences' own keys
    int join_rows;        // 1: every unit leaves partials, joined row by row with the prefix's
    int ctas;             // CTAs that share the work
    float scale;
    ScoreParams score;
    const uint16_t* q;
    long long qs[2];
    void* o;
    float* lse;
    PagedParts parts;
    PagedMeta* meta;      // [ctas] (join_rows = 0)
    int2* rowdesc;        // [total_q][Hq] {first slot row or -1, count} (join_rows = 1, own keys)
    int* hdr;             // {tiles of a prefix unit, tiles per CTA} of the prefix kernel, its mark (8 bytes)
    uint32_t* ws;
    uint64_t timeout_ns;
    uint32_t flags;
};

// The joining kernel with a shared prefix: both kernels' partials.
struct PagedJoin {
    PagedParams own;
    PagedParts pre;
    int own_rows;             // rows per unit of the sequences' own kernel
    int pre_ctas;             // CTAs of the prefix's
};

// Sets this thread's fa_last_error() message and returns `st`.
fa_status report(fa_status st, const char* msg);

// Every synchronous check fa_fwd makes on its arguments, without launching
// anything (FA_OK or the status fa_fwd would return, with its message).
fa_status fwd_validate(const fa_fwd_args* a, const fa_block_mask* bm, const fa_score_desc* sc, void* workspace);

// Launchers (return the launch's cudaError_t).
cudaError_t launch_block_mask_build(const BuildParams& p, cudaStream_t s);
cudaError_t launch_fwd_fp32(const FwdParams& p, cudaStream_t s);
cudaError_t launch_fwd_bf16(const FwdParams& p, const CUtensorMap& tq, const CUtensorMap& tk,
                            const CUtensorMap& tv, cudaStream_t s);
cudaError_t launch_decode_bf16(const DecodeParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                               cudaStream_t s);
cudaError_t launch_block_mask_build_cols(const BuildParams& p, cudaStream_t s);
cudaError_t launch_bwd_tc(const BwdParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                          const CUtensorMap& tg, cudaStream_t s);
cudaError_t launch_kv_append(const AppendParams& p, cudaStream_t s);
// Rows of a unit of the two attention kernels over pages.
constexpr int kPagedSmallRows = 16;
constexpr int kPagedTileRows = 256;
constexpr int kPagedMaxSeqs = 2048;
// Keys of a tile: 32 KB of K and V for the small kernel (three such stages and
// two CTAs per SM), 128 keys for the other.
inline int paged_small_keys(int D) { return D == 64 ? 128 : 64; }
constexpr int kPagedTileKeys = 128;
constexpr int kPagedSmallCtasPerSm = 2;
cudaError_t launch_paged_small(const PagedParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s);
cudaError_t launch_paged_tiles(const PagedParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s);
cudaError_t launch_paged_join_units(const PagedParams& p, int rows_per_unit, cudaStream_t s);
cudaError_t launch_paged_join_rows(const PagedJoin& p, cudaStream_t s);
// Validates a score_mod (NULL becomes FA_SCORE_NONE in *out).
fa_status check_score_desc(const fa_score_desc* sc, fa_score_desc* out);
int device_sm_count();
// [blocks][page_size][D] bf16, boxes of min(page_size, tile_keys) rows x 64
// columns with 128-byte swizzle.
fa_status page_tensor_map(CUtensorMap* map, const void* base, long long blocks, int page_size, int D, int tile_keys);
int decode_max_splits();
int decode_max_rows();

}  // namespace fa
