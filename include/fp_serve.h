/*
 * fp_serve.h -- C ABI of the serving operators next to the prefill path of
 * fp.h (libfp_serve.so, sm_100a): sliding-window attention with sink tokens,
 * a paged key/value cache that can be held in 8 bits, and the attention of new
 * tokens (a prompt's next chunk, or single tokens) over that cache.
 *
 * The conventions are those of fp.h: dense row-major layouts, device memory
 * owned by the caller, no allocation, arguments checked on the host before
 * anything is launched, asynchronous execution on `stream`, problems found on
 * the device recorded in a per-device status word (this library's own, read
 * with fp_serve_last_device_status), no C++ exception across the ABI.  Every
 * call may be captured into a CUDA graph after one eager call of it on the
 * device; a replay reads the current contents of the captured buffers, the
 * lengths and page tables included.  Results do not depend on the timing of
 * the run: there are no floating-point atomics.
 *
 * Visibility.  A query at position i sees the keys j <= i with
 *     window <= 0,  or  i - j < window,  or  j < sinks.
 * Attention is softmax(q.k / sqrt(d)) over the visible keys, in fp32 (bf16
 * inputs: tensor-core products with fp32 accumulation, the softmax weights
 * rounded to bf16 for the product with V, or, for few rows over an 8-bit cache
 * (max_q_len * Hq / Hkv <= 64), weights times the values' scales rounded to fp16 and
 * queries held in fp16 with a power of two for each row; fp32 inputs: fp32
 * throughout, the debug path).  What is not visible has no influence, a NaN or an infinity
 * there included.  A query that sees nothing gets zeros and lse = -inf.  `lse`
 * (or NULL) is the natural-log sum of exponentials of the scaled logits, fp32.
 */
#ifndef FP_SERVE_H_
#define FP_SERVE_H_

#include "fp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A cache element type besides fp_dtype's: 8 bits, 4 of exponent and 3 of
 * mantissa (finite up to 448), with one power-of-two scale per vector. */
enum { FP_E4M3 = 2 };

/*
 * A paged cache.  k and v are [n_pages, Hkv, page_size, d]; a page holds
 * page_size consecutive positions of one sequence.
 *   dtype FP_BF16 or FP_F32: the elements themselves; the exps are NULL.
 *   dtype FP_E4M3: codes, and one byte per vector in k_exps and v_exps
 *     ([n_pages, Hkv, page_size]): the vector's elements are
 *     code * 2^(byte - 127), byte 1 .. 254; byte 255 says that the whole vector
 *     is NaN.  The codes that stand for NaN, 0x7f and 0xff, and a byte of 0 must
 *     not occur in vectors that a token sees or that are read (fp_kv_write makes
 *     none).
 * k, v and the exps must be 16-byte aligned.
 */
typedef struct {
  int n_pages;
  int n_kv_heads; /* Hkv                                     */
  int page_size;  /* 16, 32, 64 or 128                       */
  int head_dim;   /* d: 64 or 128                            */
  int dtype;      /* FP_BF16, FP_F32 or FP_E4M3              */
  void *k;
  void *v;
  uint8_t *k_exps;
  uint8_t *v_exps;
} fp_kv_cache;

/*
 * A batch of sequences and their newest tokens.  Sequence s holds
 * kv_lens[s] tokens, the newest n_s = q_offsets[s + 1] - q_offsets[s] of
 * them included; its new tokens stand at positions kv_lens[s] - n_s ..
 * kv_lens[s] - 1.  Position p is slot p % page_size of page
 * page_table[s, p / page_size].  Entries of the table at or past
 * ceil(kv_lens[s] / page_size) are not read.
 *
 * New tokens are packed: the [H, n_s, d] tensors of the sequences back to
 * back, sequence s starting H * d * q_offsets[s] elements in (the layout of
 * fp_prefill_attn_varlen; with q_offsets NULL, the [Bt, H, N, d] of fp.h with
 * Bt = n_seqs and N = max_q_len).  An lse is packed the same way, [Hq, n_s].
 *
 * The three arrays are in device memory, so a captured call can be replayed
 * with other lengths and pages.  The device checks them: a sequence with
 * q_offsets that decrease or leave 0 .. total_q, with n_s > max_q_len, or with
 * kv_lens[s] < 0 or > max_pages * page_size, is skipped (its rows of the
 * outputs are left as they were); a page outside 0 .. n_pages - 1 is not
 * read or written (its keys are not visible; fp_kv_read gives zeros for it).
 * Either records FP_ERR_DEVICE_CHECK, in fp_paged_attn a page only if some of its
 * keys would be seen: entries of pages that lie behind the window of every new
 * token, and hold no sink, may be anything.  Tokens at negative positions
 * (n_s > kv_lens[s]) are not written by fp_kv_write, see nothing in
 * fp_paged_attn and read as zeros in fp_kv_read.  Rows at or past
 * q_offsets[n_seqs] are left as they were.
 */
typedef struct {
  int n_seqs;
  int max_pages; /* row length of page_table; max_pages * page_size < 2^30 */
  int max_q_len; /* the largest n_s                                        */
  int total_q;   /* rows per head that the packed tensors hold; with
                    q_offsets NULL, n_seqs * max_q_len                     */
  const int32_t *page_table; /* [n_seqs, max_pages] */
  const int32_t *kv_lens;    /* [n_seqs]            */
  const int32_t *q_offsets;  /* [n_seqs + 1] or NULL: every n_s is max_q_len */
} fp_batch;

/*
 * fp_window_attn -- causal attention of whole sequences with a sliding window
 * and sinks: fp_dense_attn's layouts, over the visible keys only.  The shape's
 * block_size is checked and otherwise unused.  bf16: d 64 or 128.  sinks < 0
 * is FP_ERR_PARAM.  No workspace.
 */
fp_status fp_window_attn(const fp_shape *shape, int window, int sinks, const void *q,
                         const void *k, const void *v, void *out, float *lse,
                         fp_stream_t stream);

/*
 * fp_kv_write -- stores the new tokens' k and v (packed, Hkv heads, of type
 * dtype) in their slots of the cache.  An FP_BF16 or FP_F32 cache takes its own
 * type; an FP_E4M3 cache takes either.  Into 8 bits: the exponent is the
 * smallest e >= -126 with max|x| <= 448 * 2^e, the codes are x / 2^e rounded to
 * nearest, ties to even; a vector that holds a NaN or an infinity is held as
 * NaN as a whole.  Slots of no new token keep their contents.  Where two new
 * tokens share a slot (two sequences with the same page), its contents are
 * unspecified.
 */
fp_status fp_kv_write(const fp_kv_cache *cache, const fp_batch *batch, fp_dtype dtype,
                      const void *k, const void *v, fp_stream_t stream);

/*
 * fp_kv_read -- the inverse: the newest n_s tokens of every sequence, packed,
 * of type dtype (the cache's own; FP_BF16 or FP_F32 from FP_E4M3, exact but for
 * bf16 values below 2^-126, and for 2^128, as which values above 248 * 2^120 are
 * held and which reads as an infinity).  With n_s = kv_lens[s]: whole sequences, laid out
 * for the calls of fp.h.
 */
fp_status fp_kv_read(const fp_kv_cache *cache, const fp_batch *batch, fp_dtype dtype, void *k,
                     void *v, fp_stream_t stream);

/*
 * fp_paged_attn -- the new tokens' queries (packed, Hq heads, of type dtype)
 * attend to their sequences in the cache, in which the new tokens' own keys
 * and values have been written.  FP_BF16 queries take FP_BF16 and FP_E4M3
 * caches, FP_F32 queries FP_F32 and FP_E4M3.  out is packed like q.
 * Workspace: fp_paged_attn_workspace bytes (0 for an invalid description, and
 * where none is needed), 256-byte aligned, not shared by calls that may run at
 * the same time; FP_F32 queries need none.  Over an FP_E4M3 cache, chunks
 * (max_q_len * Hq / Hkv > 64) take room there for bf16 copies of
 * min(n_pages, n_seqs * max_pages) pages, of which those that are read are filled
 * in: 4 * Hkv * page_size * d bytes each.  (So over a cache that fills the device,
 * chunks are called with a table of their own sequences only.)
 */
size_t fp_paged_attn_workspace(const fp_kv_cache *cache, const fp_batch *batch, int n_q_heads);
fp_status fp_paged_attn(const fp_kv_cache *cache, const fp_batch *batch, int n_q_heads,
                        fp_dtype dtype, int window, int sinks, const void *q, void *out,
                        float *lse, void *ws, size_t ws_bytes, fp_stream_t stream);

/* fp_last_device_status of this library's kernels. */
fp_status fp_serve_last_device_status(fp_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP_SERVE_H_ */
