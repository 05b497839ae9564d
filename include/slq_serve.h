/*
 * slq_serve.h -- the part of a decode step that stands beside the weight-only
 * products of slq.h: an 8-bit key/value cache in pages (write, read back,
 * attention over it) and the choice of the next token from the logits.
 *
 * Sources (page title -> section):
 *   wispaper.ai, "SLQ": Limits (the KV cache as the next thing to quantize,
 *     named in the paper's appendix and not defined by the pages).
 *   gist.science summary, Methodology 2: the next-token distribution at a
 *     temperature, restricted to its top tokens.
 *
 * The conventions of slq.h hold: device pointers owned by the caller, work
 * enqueued on `stream` only, arguments validated on the host before any HIP
 * call, SLQ_OK with nothing enqueued where a size is zero, nothing allocated
 * or kept.  The current device must be the one that owns the pointers.
 * Lengths, page tables and sampling settings live on the device and are read
 * there; entries out of range are defined below and never lead to an access
 * outside the arrays the call was given.
 */
#ifndef SLQ_SERVE_H
#define SLQ_SERVE_H

#include "slq.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SLQ_KV_INT8 = 0,  /* two's complement -127..127                           */
  SLQ_KV_E4M3 = 1   /* 8-bit float, 4 exponent and 3 mantissa bits, max 448 */
} slq_kv_format;

typedef enum { SLQ_F32 = 0, SLQ_BF16 = 1, SLQ_F16 = 2 } slq_dtype;

/*
 * A cache of `pages` pages, each holding `page_size` tokens of every kv head:
 *   codes: byte (page, head, slot, i) at page * page_stride + head *
 *     head_stride + slot * token_stride + i, i < head_dim, for K and V alike;
 *   scales: fp32 [pages][heads], one per page and head; value = code * scale.
 * head_dim is 64, 128 or 256 (else SLQ_ENOTSUP), page_size a power of two in
 * 16..256 (else SLQ_ENOTSUP), heads in 1..1024.  Strides are in bytes,
 * multiples of 16, and must not make two (page, head, slot) rows overlap:
 * either heads outside slots or slots outside heads within a page, which
 * spans less than 2^31 bytes.
 * Alignment: codes 16 bytes, scales 4 bytes.
 */
typedef struct {
  int32_t format;       /* slq_kv_format */
  int32_t heads;
  int32_t head_dim;
  int32_t page_size;
  int64_t pages;
  int64_t page_stride, head_stride, token_stride;
  uint8_t *k_codes, *v_codes;
  float *k_scales, *v_scales;
} slq_kv_cache;

/*
 * A ragged batch of sequences in the cache.  Token t of sequence b lies in
 * page table[b * table_stride + t / page_size], slot t % page_size.  lens[b]
 * counts its tokens after this step; the rows cu[b] .. cu[b+1]-1 of the
 * caller's arrays (cu[0] = 0, ascending) are its LAST n_b = cu[b+1] - cu[b]
 * tokens: row cu[b] + i is the token at position lens[b] - n_b + i.  A write
 * and the attention after it take the same batch.
 * A token at a negative position, at or behind max_pages * page_size, or on
 * a page number outside 0..pages-1 does not exist: it is not written, reads
 * as 0, and is masked in attention.  cu is clamped to 0..rows.
 * Alignment: 4 bytes.  1 <= max_pages, max_pages * page_size <= 2^30, batch <= 65535,
 * rows * heads (of the cache or of q) < 2^30.
 */
typedef struct {
  int32_t batch;
  int32_t max_pages;        /* columns of table */
  int64_t table_stride;     /* in entries, >= max_pages */
  const int32_t *table;     /* [batch][table_stride] */
  const int32_t *lens;      /* [batch] */
  const int32_t *cu;        /* [batch + 1] */
} slq_kv_seqs;

/*
 * Quantizes new keys and values into the cache.  k, v: [rows][heads][head_dim]
 * of `dtype`, row and head strides in elements (multiples of 16 bytes), the
 * last dimension contiguous, 16-byte aligned.  Per touched (page, head), with
 * NaN taken as 0 and infinities as the largest finite fp32 value, and r =
 * fl32(1 / 127) (INT8) or fl32(1 / 448) (E4M3):
 *   c = fl32(max |x| * r) over the page's new rows;
 *   the page's first new slot is 0:  s = c;  else s = max(s_old, c), and where
 *   s > s_old the page's older codes become enc(fl32(fl32(code * s_old) / s));
 *   new code = enc(fl32(x / s));  s = 0 gives code 0;
 *   enc: round half to even and clamp to +-127, or the nearest E4M3 value
 *   (ties to even) of the argument clamped to +-448.
 * Every operation is IEEE fp32, so codes and scales are reproducible bit for
 * bit.  Slots other than the new ones (and the older ones of such a page)
 * keep their bytes.  Two sequences must not write to one page in one call
 * (pages they only share for reading are fine).
 * max_new: the largest n_b the caller expects; it only sizes the grid (any
 * value >= 1 gives the same results).
 */
slq_status slq_kv_write(const slq_kv_cache *cache, const slq_kv_seqs *seqs, const void *k,
                        const void *v, slq_dtype dtype, int64_t rows, int64_t k_row_stride,
                        int64_t k_head_stride, int64_t v_row_stride, int64_t v_head_stride,
                        int64_t max_new, slq_stream stream);

/*
 * Reads cached tokens back: row cu[b] + i of k_out and v_out
 * ([rows][heads][head_dim] of `dtype`, contiguous, 16-byte aligned) becomes
 * fl32(code * scale) rounded to dtype, for the last n_b tokens of each
 * sequence (n_b = lens[b] reads all of it).  Rows at or behind cu[batch] keep
 * their contents.  max_rows sizes the grid as max_new does.
 */
slq_status slq_kv_read(const slq_kv_cache *cache, const slq_kv_seqs *seqs, void *k_out, void *v_out,
                       slq_dtype dtype, int64_t rows, int64_t max_rows, slq_stream stream);

/* Workspace bytes slq_kv_attention needs for these arguments; may be 0 (and
 * is 0 on invalid arguments). */
size_t slq_kv_attention_workspace_bytes(const slq_kv_cache *cache, const slq_kv_seqs *seqs,
                                        int64_t rows, int32_t heads_q, int32_t window,
                                        int64_t max_q, int64_t max_len);

/*
 * Causal attention of ragged queries over the cache.  q: [rows][heads_q]
 * [head_dim] of `dtype` (SLQ_BF16 or SLQ_F16; SLQ_F32: SLQ_ENOTSUP), strides
 * in elements (multiples of 16 bytes), 16-byte aligned; heads_q a multiple of
 * the cache's heads, query head g reading kv head g / (heads_q / heads).
 * The query at position p sees the existing tokens j with j <= p, j <
 * lens[b], and j > p - window where window > 0 (0: no window):
 *   s_j = scale * q . k_j,  out = sum_j softmax(s)_j v_j,  lse = log sum_j exp(s_j)
 * A query that sees no token gets out = 0 and lse = -inf.
 * out: [rows][heads_q][head_dim] of dtype, contiguous, 16-byte aligned; lse:
 * fp32 [rows][heads_q] or NULL.  Rows at or behind cu[batch] keep their
 * contents.  Cache slots that no visible token occupies may hold anything.
 * Scores, softmax sums and outputs accumulate in fp32; codes enter the matrix
 * units exactly, q after an exact shift of its exponent (elements below 2^-17
 * of their row's largest round to 2^-25 of it), probabilities rounded to
 * binary16, each to 2^-12 of itself or 2^-36 of the weight of the largest.
 * max_q, max_len: the largest n_b and lens[b] the caller expects; they choose
 * the kernel and its grid, results are right for any values >= 1.
 * workspace: as sized above, 256-byte aligned, overwritten; NULL when 0.
 * Sums are taken in a fixed order: repeated calls are bit-identical.  Where the
 * splits fall depends on the hints and on all lengths of the batch, so the last
 * bits of a sequence's outputs may change with its company.
 */
slq_status slq_kv_attention(const slq_kv_cache *cache, const slq_kv_seqs *seqs, const void *q,
                            slq_dtype dtype, int64_t rows, int32_t heads_q, int64_t q_row_stride,
                            int64_t q_head_stride, float scale, int32_t window, int64_t max_q,
                            int64_t max_len, void *out, float *lse, void *workspace,
                            slq_stream stream);

/* Workspace bytes slq_sample needs for (rows, vocab); 0 on invalid arguments. */
size_t slq_sample_workspace_bytes(int64_t rows, int64_t vocab);

/*
 * One token per row of logits [rows][vocab] of `dtype` (row stride in
 * elements, aligned to the element), from given uniform numbers u[row] in
 * [0, 1).  NaN logits count as -inf, +inf as the largest finite fp32 value.
 * temperature[row] <= 0 (or NaN): the lowest index of the largest logit,
 * logprob 0.  Otherwise, with w_v = exp((l_v - max l) / temperature) in fp64
 * and tokens ordered by logit descending, equal ones by index, the kept set
 * is the shortest of three prefixes of that order:
 *   the first top_k[row] tokens (<= 0 or >= vocab: all);
 *   the tokens with w_v >= min_p[row] (<= 0 or NaN: all; above 1 counts as 1);
 *   the shortest one holding at least top_p[row] of the mass of the first
 *   top_k tokens (>= 1 or NaN: all; never less than one token).
 * tokens[row] is the first kept index, by index, whose cumulative mass exceeds
 * u[row] * (mass kept); logprobs[row] (or NULL) the log of its share of it.
 * A row whose logits are all -inf gives token -1 and logprob -inf.
 * temperature, top_k, top_p, min_p: [rows] or NULL (1, all, all, all).
 * 1 <= vocab <= 2^24.  workspace: 256-byte aligned, overwritten by the call.
 * Deterministic: repeated calls are bit-identical.
 */
slq_status slq_sample(const void *logits, slq_dtype dtype, int64_t rows, int64_t vocab,
                      int64_t row_stride, const float *u, const float *temperature,
                      const int32_t *top_k, const float *top_p, const float *min_p,
                      int32_t *tokens, float *logprobs, void *workspace, slq_stream stream);

#ifdef __cplusplus
}
#endif
#endif /* SLQ_SERVE_H */
