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
 *   1. every sequence gets the pages its new tokens need, and kv_len and
 *      q_start are set for the step: by the caller, or by fa_paged_step from
 *      the sequences' lengths;
 *   2. fa_kv_append rotates the step's queries and keys and writes the keys
 *      and values to their slots;
 *   3. fa_fwd_paged attends from the step's queries to the cache.
 * fa_kv_append_scaled and fa_fwd_paged_scaled do 2 and 3 on a cache held in 8
 * bits, half the memory and half the bytes that attention reads.
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

/* The scales of a cache held in 8 bits.  The cache's k and v (fa_paged_kv) are
 * then e4m3 codes, one byte each, laid out as the bf16 elements are; the value
 * of a code is
 *     code x scale[page][head],
 * one scale for the tokens of a page and a kv head, k's and v's apart.
 *   k_scale, v_scale   device fp32 [num_pages][Hkv], 4-byte aligned.  Any
 *               finite numbers that are not negative; those of pages that are
 *               not read may be anything.
 * A page that receives a token in a step belongs to one sequence of the step
 * (its earlier codes change with its scale): no other sequence's table names
 * it, except behind what that sequence reads.                                */
typedef struct fa_paged_scales {
    float *k_scale;
    float *v_scale;
} fa_paged_scales;

/* fa_kv_append into a cache held in 8 bits.  q's part is the same.  For every
 * page that receives tokens, and every kv head, of k (rotated, in fp32) and of
 * v each:
 *     amax   the largest finite magnitude among the page's new tokens,
 *     need   2^e with the smallest e for which amax <= 448 2^e, e within
 *            -100 .. 119,
 *     scale  need, or where the page holds earlier tokens of the sequence
 *            max(need, its scale before), in which case their codes are
 *            rounded again to the new scale;
 *     code   x / scale rounded to e4m3 (to the nearest, ties to even); beyond
 *            448 it is +-448, and infinities and NaN become NaN.
 * A scale grows by factors of two, so that rounding again changes nothing but
 * codes that run out of exponents (below 2^-6 of their unit).  For scales before
 * that are no powers of two, x / scale is x (1 / scale) in fp32.
 * Tokens whose position is outside 0 .. rope_len - 1 are reported, not written,
 * and do not count in amax.  One kernel launch.                             */
fa_status fa_kv_append_scaled(const fa_paged_kv *c, const fa_paged_scales *scales, const fa_kv_append_args *a,
                              void *workspace, void *stream);

/* fa_fwd_paged over a cache held in 8 bits: the same softmax over the values
 * that the codes stand for.  Scales, sums and products are fp32's (a k scale
 * times an element of q stays below 2^120).  By rows per sequence and kv head
 * (max_q_len x Hq / Hkv), and for the keys of a shared prefix as for more than 16:
 *   more than 16   a query's elements keep their 8 bits from 2^-9.8 of the row's
 *                  largest on, and are off by up to 2^-17.8 of that below; exact
 *                  for fewer rows.
 *   not 9 to 16    P is rounded to 11 significant bits where a key's share in o
 *                  (its probability times its page's v scale) is at least 2^-22 of
 *                  the row's largest, and by up to 2^-33 of that largest below.  A
 *                  v scale below 2^-80 of the largest one that the rows have seen,
 *                  or below 2^-82, counts as that.
 *   9 to 16        P is rounded so by the probability alone, from 2^-29 of the
 *                  largest on, and by up to 2^-40 of it below; any v scales.
 * scratch: fa_paged_scratch_bytes().                                        */
fa_status fa_fwd_paged_scaled(const fa_paged_kv *c, const fa_paged_scales *scales, const fa_paged_fwd_args *a,
                              const fa_mask_desc *mask, const fa_score_desc *sc, void *scratch, size_t scratch_bytes,
                              void *workspace, void *stream);

/* A step's pages, offsets and slots from its sequences' lengths, on the device:
 * what fa_kv_append and fa_fwd_paged need for the step, without a copy to the
 * host.  Sequence b had kv_len[b] tokens in the cache; the step keeps the first
 * keep_len[b] of them (fewer where drafts were rejected; 0, with new_len 0,
 * where it has ended) and brings new_len[b] new ones.  With P = page_size and
 * S = shared_pages:
 *     kv_len_out[b] = keep_len[b] + new_len[b]
 *     before = max(ceil(kv_len[b] / P), S), after = max(ceil(kv_len_out[b] / P), S)
 * Entries after .. before - 1 of its row of the page table are given back,
 * entries before .. after - 1 are filled.  The free pages are a stack: those
 * given back go on top, the last sequence's last entry first, and then the
 * entries to fill take their pages from the top, the first sequence's first
 * entry first.  (So a step that gives pages back undoes the one that took
 * them.)  The first S entries of every row are a prefix's that all sequences
 * share and stay as they are; keep_len may reach up to S x P there.
 *   new_len, keep_len, kv_len   device int32 [B]; keep_len may be NULL, or
 *               kv_len itself: all are kept.
 *   page_table  device int32 [B][max_pages], in and out.  Entries that are
 *               given back stay there, and mean nothing.
 *   free_pages  device int32 [num_pages], in and out: the stack, its bottom first.
 *   free_count  device int32 [1]: pages on the stack.
 *   kv_len_out, free_count_out   device int32 [B], [1]; may be kv_len and
 *               free_count.  Where they are not, the call may be repeated: it
 *               writes the same again.
 *   q_start     device int32 [B + 1], out: sums of new_len.
 *   slots       device int64 [total_q], out, or NULL: for each row of the step
 *               page x P + place within the page, -1 behind the last sequence.
 *   positions   device int32 [total_q], out, or NULL: the row's place in its
 *               sequence (fa_kv_append's positions), 0 behind the last one.
 *   total_q     rows of the step's tensors, at least the sum of new_len.
 * A step that cannot be made changes nothing but its outputs, which are those
 * of an empty step (kv_len_out = kv_len, free_count_out = free_count, q_start
 * all 0), and is reported by fa_workspace_check as FA_ERR_DEVICE_CHECK, with the
 * sequence at which it fails: numbers that contradict each other (a negative
 * length, keep_len past kv_len and the shared pages, more than max_pages x P
 * tokens, new_len adding up to more than total_q, a free_count outside 0 ..
 * num_pages, more pages given back than the stack holds), or too few free pages.
 * A page outside 0 .. num_pages - 1 that the step moves, or that holds one of its
 * rows, is reported too; it moves all the same, and its rows have slot -1.
 * B <= 2048; page_size as for fa_paged_kv.  No two arrays overlap, apart from
 * kv_len_out and free_count_out as said.  One kernel launch.                */
typedef struct fa_paged_step_args {
    int32_t B;
    int32_t num_pages;
    int32_t page_size;
    int32_t max_pages;
    int32_t shared_pages;
    int32_t total_q;
    const int32_t *new_len;
    const int32_t *keep_len;
    const int32_t *kv_len;
    int32_t *page_table;
    int32_t *free_pages;
    const int32_t *free_count;
    int32_t *kv_len_out;
    int32_t *free_count_out;
    int32_t *q_start;
    int64_t *slots;
    int32_t *positions;
} fa_paged_step_args;

fa_status fa_paged_step(const fa_paged_step_args *a, void *workspace, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* FA_GB300_PAGED_H */
