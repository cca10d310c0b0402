/*
 * fa_paged.h -- C ABI of the paged key/value cache: appending rotated keys and
 * values, and attention that reads them (decoding steps, chunks of prompts,
 * and batches whose sequences share a long prefix).
 *
 * The operations are those of fa.h on keys and values that live in pages:
 * the conventions there (caller-owned device memory, streams, synchronous
 * argument checks, device-side findings reported by fa_workspace_check) hold
 * here too.  The pages of FlexAttention's source name a paged cache among its
 * uses without giving one; the layout below is this library's own.
 *
 * A step of a serving loop:
 *   1. the caller gives every sequence the pages its new tokens need and sets
 *      kv_len and q_start for the step;
 *   2. fa_kv_append rotates the step's queries and keys and writes the keys
 *      and values to their slots;
 *   3. fa_fwd_paged attends from the step's queries to the cache.
 */
#ifndef FA_GB300_PAGED_H
#define FA_GB300_PAGED_H

#include "fa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A paged cache and the batch of sequences of one step.
 *   k, v        device bf16 [num_pages][Hkv][page_size][D], contiguous,
 *               16-byte aligned.
 *   page_size   16, 32, 64, 128 or 256 tokens.  D is 64 or 128.
 *   page_table  device int32 [B][max_pages]: page_table[b][p] holds the keys
 *               p * page_size .. of sequence b.  Only entries of pages that
 *               hold a key some query of the step can see (or, in
 *               fa_kv_append, a new token) are read: others may hold anything.
 *   kv_len      device int32 [B]: the sequence's length in the cache, this
 *               step's new tokens included.
 *   q_start     device int32 [B + 1], non-decreasing, q_start[0] = 0:
 *               sequence b's new tokens are the rows q_start[b] ..
 *               q_start[b + 1] - 1 of the step's tensors (none where the two
 *               are equal).  The last one stands at position kv_len[b] - 1.
 *   total_q     rows of the step's tensors, at least q_start[B].  Rows from
 *               q_start[B] on belong to no sequence and are left as they were.
 * kv_len, q_start and page_table are read on the device, so that a captured
 * graph follows them.  A sequence whose numbers contradict each other (a
 * decreasing q_start, one past total_q, more new tokens than kv_len, kv_len
 * past max_pages x page_size, a needed page that is not in 0 .. num_pages - 1)
 * is reported by fa_workspace_check as FA_ERR_DEVICE_CHECK; its rows are
 * undefined and those of the others are not affected (unless q_start
 * decreases somewhere or does not start at 0: then all rows are undefined).
 * Nothing outside the given arrays is touched.
 * Keys and values past kv_len, outside every query's mask, or on pages that
 * no query sees may hold anything, NaN included.  A NaN or infinity among the
 * keys that some query of the sequence's step does see spreads as it does in
 * the products of the definition: 0 x NaN is NaN (in a shared prefix: that
 * some query of the step's batch sees).                                      */
typedef struct fa_paged_kv {
    int32_t B;
    int32_t Hkv;
    int32_t D;
    int32_t num_pages;
    int32_t page_size;
    int32_t max_pages;
    int32_t total_q;
    void *k;
    void *v;
    const int32_t *page_table;
    const int32_t *kv_len;
    const int32_t *q_start;
} fa_paged_kv;

/* Appending a step's keys and values, with the rotary position embedding
 * applied on the way: element pairs (x0, x1) of the first rot_dim of each
 * head of q and k become
 *     (x0 cos - x1 sin, x0 sin + x1 cos),
 * cos and sin from row `position` of the caller's tables; the rest of the
 * head, and v, are copied.  Products and sums in fp32, one rounding to bf16.
 *   q, k, v     device bf16 rows [total_q][H][D] with D contiguous and the
 *               other two strides given in elements (multiples of 8); 16-byte
 *               aligned.  Slices of one fused projection are the usual case.
 *   q_out       device bf16, as q with its own strides; may be q itself (the
 *               same pointer and strides), but must not overlap it otherwise, nor
 *               k or v.
 *               Its rows must not overlap: heads lie within the token stride,
 *               or tokens within the head stride.
 *               Hq = 0: no queries (q and q_out are ignored).
 *   rot_dim     0 (no rotation: cos and sin are ignored) or a multiple of 16
 *               up to D.
 *   interleaved 0: pairs are (d, d + rot_dim / 2); 1: pairs are (2 d, 2 d + 1).
 *   cos, sin    device fp32 [rope_len][rot_dim / 2], 16-byte aligned.
 *   positions   device int32 [total_q], or NULL for each token's place in its
 *               sequence.  Outside 0 .. rope_len - 1 the token is not written
 *               and the call is reported as above.
 * The cache's k and v must not overlap, and two tokens must not have the same
 * slot.  One kernel launch.                                                  */
typedef struct fa_kv_append_args {
    int32_t Hq;
    int32_t rot_dim;
    int32_t rope_len;
    int32_t interleaved;
    const void *q;
    const void *k;
    const void *v;
    void *q_out;
    int64_t q_stride[2];       /* between tokens, between heads */
    int64_t k_stride[2];
    int64_t v_stride[2];
    int64_t q_out_stride[2];
    const float *cos;
    const float *sin;
    const int32_t *positions;
} fa_kv_append_args;

fa_status fa_kv_append(const fa_paged_kv *c, const fa_kv_append_args *a, void *workspace, void *stream);

/* Attention from the step's queries to the cache: for row t of sequence b at
 * position i = kv_len[b] - (q_start[b + 1] - q_start[b]) + (t - q_start[b])
 * and query head hq, the softmax over the keys j < kv_len[b] that the mask
 * shows, exactly as fa_fwd defines it with i and j as positions.
 *   q           device bf16 [total_q][Hq][D] with D contiguous, the other
 *               strides in elements (multiples of 8); 16-byte aligned.
 *   o           device [total_q][Hq][D] contiguous, 16-byte aligned, bf16 (or
 *               fp32 with FA_OUT_FP32); lse device fp32 [total_q][Hq].  o may be
 *               q itself where that is contiguous; the two must not overlap
 *               otherwise.
 *   max_q_len   at least the new tokens of every sequence: a longer sequence
 *               is reported like the contradictions above.
 *   shared_len  0, or the length of a prefix that all sequences have in
 *               common: its keys are read once for the whole batch, through
 *               the page table's first row, instead of once per sequence.
 *               Every sequence with new tokens has kv_len >= shared_len.
 *   mask        FULL, CAUSAL, SLIDING_WINDOW or SINK_WINDOW, by position.
 *   scratch     caller-owned device bytes, at least fa_paged_scratch_bytes(),
 *               16-byte aligned; overwritten by every call, so calls that may
 *               overlap need their own.
 *   timeout_ms, flags, scale: as fa_fwd_args.
 * B <= 2048.  Two kernel launches, or three with a shared prefix.           */
typedef struct fa_paged_fwd_args {
    int32_t Hq;
    int32_t max_q_len;
    int32_t shared_len;
    float scale;
    const void *q;
    int64_t q_stride[2];       /* between tokens, between heads */
    void *o;
    float *lse;
    uint32_t timeout_ms;
    uint32_t flags;
} fa_paged_fwd_args;

/* Bytes of fa_fwd_paged's scratch on the current device (0 if the arguments
 * cannot be valid).                                                         */
size_t fa_paged_scratch_bytes(const fa_paged_kv *c, const fa_paged_fwd_args *a);

fa_status fa_fwd_paged(const fa_paged_kv *c, const fa_paged_fwd_args *a, const fa_mask_desc *mask,
                       const fa_score_desc *sc, void *scratch, size_t scratch_bytes, void *workspace, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* FA_GB300_PAGED_H */
