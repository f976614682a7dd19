/*
 * spec_kv.h -- the paged 8-bit key/value cache of the target model's
 * verification pass: append and attention (libspecverify.so, CUDA kernels for
 * sm_103a).
 *
 * A round of speculative sampling scores K + 1 new positions of every sequence
 * in one pass of the target, keeps some of the drafted tokens and drops the
 * rest.  These entry points are that pass's work on the cache:
 *
 *   spec_kv_append     rotates the new tokens' queries and keys by position and
 *                      stores their keys and values in the sequences' pages;
 *   spec_kv_append_norm  the same, of heads that are normalised first;
 *   spec_kv_attention  attends from the new tokens' queries to every token
 *                      stored for their sequence up to their own position;
 *   spec_kv_attention_sinks  to the last ones and the first ones of them.
 *
 * Dropping rejected tokens is a smaller length at the next call: the next
 * append writes over them.
 *
 * Conventions: those of spec_verify.h.  The caller owns every buffer, which is on
 * the current device like the stream; calls are asynchronous on params->stream,
 * host-side argument errors are returned before anything is launched, and
 * device-side errors never trap (see each entry).
 *
 * The cache.  A pool of pages of page_size token slots each, shared by all
 * sequences.  Token position p of sequence b lies in page
 * page_table[b * table_stride + p / page_size], slot p % page_size.  Keys and
 * values are e4m3 codes; the value a code stands for is code * scale, with one
 * float scale for each (page, key/value head), for keys and values apart.
 * Appending chooses powers of two for the scales; attention takes any from 2^-100
 * to 2^100.  Smaller ones may count as 2^-100, and a value scale as 2^-80 times the
 * largest one of the sequence and head where it is below that.
 */
#ifndef SPEC_KV_H
#define SPEC_KV_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int32_t num_pages;         /* pages of the pool, >= 1 */
  int32_t page_size;         /* token slots a page: 16, 32, 64 or 128 */
  int32_t Hkv;               /* key/value heads, >= 1 */
  int32_t D;                 /* channels a head: a multiple of 16, 16 to 256 */
  uint8_t* k_codes;          /* device, e4m3, 16-byte aligned; channels contiguous, the other strides below */
  uint8_t* v_codes;
  float* k_scale;            /* device, [num_pages, Hkv] by the strides below */
  float* v_scale;
  /* strides in elements, the same for keys and values; positive where there is more than one, and
   * multiples of 16 for the codes */
  int64_t page_stride, head_stride, token_stride;
  int64_t scale_page_stride, scale_head_stride;
} spec_kv_cache;

typedef struct {
  int32_t B;                 /* sequences, >= 0 */
  int32_t T;                 /* new-token slots of a sequence, >= 1 (K + 1 in verification) */
  int32_t Hq;                /* query heads, a multiple of Hkv; query head h reads key/value head h / (Hq / Hkv) */
  int32_t dtype;             /* spec_dtype of q, k, v and the outputs */
  int32_t max_pages;         /* columns of the page table, >= 1 */
  int32_t window;            /* attention: tokens a query sees, its own included; 0 = all before it */
  float scale;               /* attention: factor of the scores, finite (1 / sqrt(D) as a rule) */
  int32_t rot_dim;           /* append: leading channels of a head that are rotated, even, 0 to D */
  int32_t rot_len;           /* append: rows (positions) of cos_sin */
  int32_t interleaved;       /* append: pairs are channels (2i, 2i+1), else (i, i + rot_dim / 2) */
  const int32_t* page_table; /* device [B, max_pages], rows table_stride apart */
  const int32_t* seq_lens;   /* device [B]: tokens stored before this round's new ones, >= 0 */
  const int32_t* new_lens;   /* device [B]: new tokens, 0 to T; NULL = T each */
  int64_t table_stride;
  /* strides in elements of [B, T, heads, D] tensors, channels contiguous; >= 0 for inputs (0 repeats),
   * > 0 for outputs where there is more than one */
  int64_t q_seq_stride, q_tok_stride, q_head_stride;
  int64_t k_seq_stride, k_tok_stride, k_head_stride;   /* append */
  int64_t v_seq_stride, v_tok_stride, v_head_stride;   /* append */
  int64_t o_seq_stride, o_tok_stride, o_head_stride;   /* append: q_out; attention: out */
  void* stream;              /* cudaStream_t */
  int32_t* status;           /* optional device int32[1]: first device-detected error */
  void* workspace;           /* attention: device, 256-byte aligned, zero-filled before first use */
  size_t workspace_bytes;
} spec_kv_params;

/* Rotate and store the new tokens.
 *   q        device [B, T, Hq, D], or NULL (then q_out is NULL too)
 *   k, v     device [B, T, Hkv, D]
 *   cos_sin  device float [rot_len, rot_dim], rows contiguous, 16-byte aligned:
 *            the cosines of a position's rot_dim / 2 angles, then their sines;
 *            NULL when rot_dim is 0
 *   q_out    device [B, T, Hq, D]: the rotated queries; zero in slots past
 *            new_lens[b].  May be q itself, with q's strides.
 * New token t < new_lens[b] has position seq_lens[b] + t.  Keys and queries are
 * rotated in float (each product and sum rounded), values are not.  The scale of
 * a page and head becomes 2^e, e the least integer >= -100 that brings the
 * finite values this call writes there within 448 * 2^e, or stays as it was
 * where the page holds earlier tokens of the sequence and its scale is at least
 * that; where it grows, the earlier codes are rounded again at the new scale.
 * A code is the e4m3 value nearest to x / scale, ties to even; NaN and the
 * infinities become NaN codes.  Pages written by two sequences of one call, or
 * by calls that overlap in time, race.
 * Device errors: a sequence whose lengths are out of range (negative, more than
 * T new tokens, beyond max_pages pages or beyond rot_len positions) is left out
 * and its q_out is NaN; a page number outside [0, num_pages) skips what would be
 * written to that page.  Either stores SPEC_ERR_CACHE_RANGE in *status. */
spec_status spec_kv_append(const void* q, const void* k, const void* v, const float* cos_sin,
                           const spec_kv_cache* cache, const spec_kv_params* params, void* q_out);

/* Norms of queries and keys for each head, as models have them that normalise both
 * before the rotation. */
typedef struct {
  const float* q_weight;     /* device: D weights of a head, contiguous; NULL: queries are not normalised */
  const float* k_weight;     /* likewise for the keys */
  int64_t q_head_stride;     /* elements from a head's weights to the next one's, >= 0 (0: all heads have the same) */
  int64_t k_head_stride;
  float eps;                 /* 2^-80 to 2^40 */
} spec_kv_norms;

/* spec_kv_append with norms (NULL: without): a head x of a query or key of a new token
 * becomes (x r) w before it is rotated, with r = 1 / sqrt(mean of x_i^2 + eps) as the
 * nearest float (once in about a hundred thousand heads the next one), w its weights, and each
 * product rounded to float.  A head with an infinity has r = 0, one with a NaN is NaN.
 * Everything else is as for spec_kv_append. */
spec_status spec_kv_append_norm(const void* q, const void* k, const void* v, const float* cos_sin,
                                const spec_kv_norms* norms, const spec_kv_cache* cache, const spec_kv_params* params,
                                void* q_out);

/* Workspace bytes spec_kv_attention needs (0 if the parameters are invalid);
 * a function of B, T, Hq, Hkv, D and dtype alone.  A workspace is zero-filled once
 * before its first use.  Its first 64 KB hold counters that every call leaves at
 * zero again, so it is reused across calls of any shape without clearing (but not
 * with spec_verify's; and after a SPEC_ERR_TIMEOUT it is cleared).  Calls that
 * share one must not overlap in time on the GPU. */
size_t spec_kv_attention_workspace_size(const spec_kv_cache* cache, const spec_kv_params* params);

/* The capture (the graph being recorded) that calls on the stream go to; 0: none,
 * they run.  For callers that keep workspaces: a graph may be replayed on any
 * stream, so it needs one of its own, cleared in the graph. */
uint64_t spec_kv_capture_id(void* stream);

/* Attention of the new tokens' queries over the cache.  The new tokens' keys and
 * values are in the cache already (spec_kv_append), and lengths and page table
 * are the same as for that call.
 *   q    device [B, T, Hq, D] (rotated)
 *   out  device [B, T, Hq, D], dtype: the query at position p = seq_lens[b] + t
 *        gets sum_j w_j v_j / sum_j w_j with w_j = exp(scale * q . k_j) over the
 *        positions j <= p (and j > p - window when window > 0); zero for slots
 *        t >= new_lens[b]
 *   lse  device float [B, T, Hq], contiguous, or NULL: log sum_j w_j (natural
 *        logarithm), -inf for slots t >= new_lens[b]
 * Sums and softmax statistics are float.  float32 calls, and bfloat16 ones whose
 * head size is not 64 or 128 or whose pool is laid out as no tensor map can be, hold
 * queries and weights in float too.  The other bfloat16 calls run on 8-bit matrix
 * products and hold them in 8-bit pieces: a query channel to 2^-17 of the largest of
 * its row (2^-13, where rows of one sequence and head are within 16 times of each
 * other); a weight (times its page's value scale) to 2^-9 of itself, or to 2^-32 of
 * the largest of its row where that is more.  Their running sums lose up to 2^-24 of
 * themselves for each 32 tokens.
 * Tokens a query does not see have no influence on its output, whatever their slots
 * hold; a NaN key or value that it sees makes its output NaN (a value: in the
 * affected channels at least).
 * Device errors: a sequence whose lengths are out of range gets NaN, and so does a
 * row that sees a token of a page outside [0, num_pages); both store
 * SPEC_ERR_CACHE_RANGE in *status.  Entries of the table for pages that lie wholly
 * before what any query of the sequence sees through its window may hold anything.
 * A bounded wait that runs out (about two seconds) gives NaN and SPEC_ERR_TIMEOUT. */
spec_status spec_kv_attention(const void* q, const spec_kv_cache* cache, const spec_kv_params* params, void* out,
                              float* lse);

/* The same with first tokens that stay visible: beside its window, a query sees the
 * positions j < sinks (those up to its own).  They keep the positions that they were
 * appended (and rotated) at: none is counted anew inside the cache, so a stream's positions
 * go on growing; and a sink that has a learned logit and no token is not one of these (its
 * weight can be added to the sum that lse is the logarithm of).  sinks >= 0; without a
 * window (0) every position is seen anyway.  A token of both counts once.  Entries of the
 * table for pages that lie wholly behind the sinks and before what any query of the
 * sequence sees through its window may hold anything.  Everything else, the workspace's
 * size among it, is as for spec_kv_attention, which is this with no sinks. */
spec_status spec_kv_attention_sinks(const void* q, const spec_kv_cache* cache, const spec_kv_params* params,
                                    int32_t sinks, void* out, float* lse);

#ifdef __cplusplus
}
#endif

#endif
