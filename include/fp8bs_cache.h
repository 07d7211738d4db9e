/*
 * fp8bs_cache.h -- the paged FP8 key/value cache of libfp8bs: quantized
 * append, attention over the cache, the attention weight its tokens received,
 * and eviction by that weight.  Part of the library that fp8bs.h declares; its
 * conventions (device pointers, streams, argument checks and their order,
 * status codes, nothing allocated or kept) hold here too.
 *
 * The cache.  Keys and values are E4M3 codes in pages of P tokens, one FP32
 * scale per page and head:
 *   k, v   : E4M3 [pages][heads][P][D]
 *   ks, vs : FP32 [pages][heads]         a value is code * scale
 *   table  : INT32 [batch][table_width]  page of sequence b's tokens
 *                                        [j P, (j + 1) P) is table[b][j]
 *   kv_lens: INT32 [batch]               cached tokens of each sequence, the
 *                                        rows of the current call included
 * P is 16, 32, 64 or 128 and D 64 or 128.  A token's place in its sequence is
 * its slot: slot t lies in page table[b][t / P] at row t % P.  Table entries
 * past the last cached token, and rows of a page past it, may hold anything
 * (some are read, inside the table and the pools, and not used).  A cached
 * token whose table entry lies outside [0, pages) counts as absent (nothing is
 * read or written for it).
 *
 * Packed rows.  The rows of all sequences are concatenated; sequence b owns
 * rows [q_offsets[b], q_offsets[b + 1]) (INT32 [batch + 1], device), and they
 * are its last tokens: row i of n is slot kv_lens[b] - n + i.  max_new is a
 * host-side upper bound of the rows of one sequence, max_kv of kv_lens; they
 * size the launch.  A sequence's rows past max_new and cached tokens past
 * max_kv or past its table_width * P slots are left out, as if they were not
 * there: nothing is read or written for them, and the others keep their slots.
 *
 * Checks.  Sizes (FP8BS_ERR_SHAPE): batch, rows, max_new, max_kv >= 0; pages,
 * table_width, heads >= 1; rows, table_width * P and max_new * q_heads at most
 * 2^30, rows * q_heads at most 2^40, and no more work per sequence than one
 * launch holds (2^32 work-items: of the smallest pages 2^27 / heads new tokens
 * appended or kept, 2^32 / heads slots of sums); P and D as above; the rules of
 * each call.  Flags, dtypes and scalars (FP8BS_ERR_FLAGS).  Alignment: 16 bytes
 * for codes, BF16 data, out and workspace, 4 for scales, sums, lse and the INT32
 * arrays.
 */
#ifndef FP8BS_CACHE_H
#define FP8BS_CACHE_H

#include "fp8bs.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  uint8_t* k;
  float* ks;
  uint8_t* v;
  float* vs;
  const int32_t* table;
  const int32_t* kv_lens;
  int64_t pages;       /* pages of the pools                  */
  int32_t batch;       /* sequences of this call              */
  int32_t table_width; /* entries per sequence in table       */
  int32_t heads;       /* key/value heads                     */
  int32_t page;        /* P                                   */
  int32_t dim;         /* D                                   */
} fp8bs_cache;

/* Flag of the attention calls: every row sees all cached tokens of its
 * sequence.  Without it row i of n sees slots 0 .. kv_lens[b] - n + i. */
enum { FP8BS_MASK_FULL = 2u };

/*
 * Quantize the new tokens' keys and values into the cache.
 *   k_new, v_new : BF16 [rows][heads][D], rows ld_new elements apart
 *                  (ld_new >= heads * D, a multiple of 8: slices of a joint
 *                  projection need no copy)
 * A page's scale after the call is the larger of
 *   - its scale before, where it holds older tokens of the sequence, and
 *   - max(RN(amax / 448), 2^-149), amax over the new tokens' |x| in the page
 *     and head (FP8BS_SCALE_POW2: rounded up to a power of two); 0 if amax
 *     is 0, so that an all-zero page constrains no later token.
 * New codes are E4M3(RN(x / scale)).  If the scale grew, the older tokens of
 * the page are encoded again as E4M3(RN(RN(code * old) / new)); otherwise
 * their codes stay.  Codes are 0 where the scale is 0.  Inputs must be finite.
 * No two sequences of a call may append to the same page.
 */
fp8bs_status fp8bs_cache_append(const fp8bs_cache* cache, const void* k_new, const void* v_new,
                                int64_t ld_new, const int32_t* q_offsets, int64_t rows, int32_t max_new,
                                uint32_t flags, fp8bs_stream_t stream);

/*
 * Attention over the cache: for row i of sequence b and query head hq,
 *   x_j = scale * (q . k_j)     over the visible slots j of head
 *                               hq / (q_heads / heads)
 *   x_j = softcap * tanh(x_j / softcap)                    if softcap > 0
 *   out = sum_j exp(x_j) v_j / sum_j exp(x_j),  lse = log sum_j exp(x_j)
 * A row that sees no slot gets out = 0 and lse = -inf.
 *   q   : BF16 [rows][q_heads][D], rows ld_q elements apart (>= q_heads * D, a
 *         multiple of 8)
 *   out : BF16 or FP32 [rows][q_heads][D]
 *   lse : FP32 [rows][q_heads], or NULL
 *   workspace : fp8bs_cache_attention_workspace bytes (NULL if 0)
 * Requires q_heads % heads == 0, scale finite, softcap 0 or 2^-126 .. 2^126.
 * Scores and softmax sums are FP32.  The weights enter the product with the
 * values as two BF16 parts (2^-17 of a weight is lost) where out is FP32, and in
 * calls of few rows: by max_new and the call's sizes, so that a row's sequence
 * alone does not decide it.  Elsewhere they are rounded to BF16 once (2^-9),
 * about the size of the rounding of a BF16 out.  Sums of weight * value are FP32
 * before they are divided by the sum of the weights: 2^8 times the values'
 * sizes, added up over a row, has to stay below 2^128.
 */
fp8bs_status fp8bs_cache_attention(const fp8bs_cache* cache, const void* q, int64_t ld_q, int32_t q_heads,
                                   const int32_t* q_offsets, int64_t rows, int32_t max_new, int32_t max_kv,
                                   float scale, float softcap, void* out, int32_t out_dtype, float* lse,
                                   uint32_t flags, void* workspace, int64_t workspace_bytes,
                                   fp8bs_stream_t stream);

/* Workspace bytes of fp8bs_cache_attention (bytes: HOST pointer); reads only
 * the sizes of *cache. */
fp8bs_status fp8bs_cache_attention_workspace(const fp8bs_cache* cache, int32_t q_heads, int64_t rows,
                                             int32_t max_new, int32_t max_kv, int64_t* bytes);

/* Rows per workgroup of the kernel that a fp8bs_cache_attention call of these
 * sizes would run on: 16 (few rows), 128 or 256; 0 for sizes that the call
 * refuses.  Host-side query for tests and tuning; reads only the sizes of
 * *cache. */
int32_t fp8bs_cache_attention_tile(const fp8bs_cache* cache, int32_t q_heads, int64_t rows, int32_t max_new,
                                   int32_t max_kv);

/*
 * The attention weight each cached token received from this call's rows,
 * added to a running sum:
 *   acc_out[b][h][j] = old + sum over rows and the query heads of h of
 *                      exp(x_j - lse), where the row sees slot j
 *   old = acc_in[b][h][j] for slots before this call's rows, else 0
 * x_j, q as in fp8bs_cache_attention; lse is its output (a row with
 * lse = -inf adds nothing).
 *   acc_in, acc_out : FP32 [batch][heads][acc_slots], acc_slots >= max_kv;
 *                     they may be the same array, and acc_in NULL (old = 0)
 *   workspace : fp8bs_cache_attention_weights_workspace bytes (NULL if 0)
 * Slots from kv_lens[b] on, and those left out, are set to 0.  Reads k and ks
 * of *cache only.
 */
fp8bs_status fp8bs_cache_attention_weights(const fp8bs_cache* cache, const void* q, int64_t ld_q,
                                           int32_t q_heads, const int32_t* q_offsets, int64_t rows,
                                           int32_t max_new, int32_t max_kv, float scale, float softcap,
                                           const float* lse, const float* acc_in, float* acc_out,
                                           int64_t acc_slots, uint32_t flags, void* workspace,
                                           int64_t workspace_bytes, fp8bs_stream_t stream);

/* Workspace bytes of fp8bs_cache_attention_weights (bytes: HOST pointer);
 * reads only the sizes of *cache. */
fp8bs_status fp8bs_cache_attention_weights_workspace(const fp8bs_cache* cache, int32_t q_heads,
                                                     int32_t max_new, int64_t acc_slots, int64_t* bytes);

/*
 * Evict: keep count = min(kv_lens[b], budget) tokens (of those within the
 * bounds) of each sequence and head: the last min(recent, count) ones, and of
 * the others those with the largest acc (ties: the lowest slot; NaN ranks below
 * every number).  Kept tokens keep their order and move to slots 0 .. count - 1
 * of pages dst_table[b]; heads of one sequence may keep different tokens.
 *   acc       : FP32 [batch][heads][acc_slots]
 *   dst_table : INT32 [batch][dst_width], dst_width * P >= min(budget,
 *               max_kv); pages of the same pools that no source sequence of the call holds and
 *               that appear once
 *   kept      : INT32 [batch][heads][budget], the source slots, then -1
 *   new_lens  : INT32 [batch]; may be the cache's kv_lens (in place)
 *   acc_out   : FP32 [batch][heads][acc_slots] (not acc), the kept tokens'
 *               sums, then 0
 * A destination page's scale is the largest scale of the pages its tokens come
 * from; codes of tokens from pages of that scale stay, the others are
 * E4M3(RN(RN(code * old) / new)).  Rows of the last page past the count are
 * zeroed.  Requires acc_slots >= max_kv, recent >= 0,
 * budget > 0.
 */
fp8bs_status fp8bs_cache_evict(const fp8bs_cache* cache, const float* acc, int64_t acc_slots,
                               const int32_t* dst_table, int32_t dst_width, int32_t max_kv, int32_t budget,
                               int32_t recent, int32_t* kept, int32_t* new_lens, float* acc_out,
                               fp8bs_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8BS_CACHE_H */
