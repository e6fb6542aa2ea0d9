/*
 * cf_paged.h -- C ABI of the paged KV cache: the operators that write it and
 * the attention that reads it.
 *
 * Where cf_decode_attn_block keeps one dense cache row of s_max positions per
 * batch row, here keys and values live in pages of `page_size` positions that
 * any sequence may own: position t of sequence b is slot t % page_size of
 * page page_table[b][t / page_size].  Three operators share one handle:
 *
 *   cf_paged_append            rotates new keys (and queries) and writes the
 *                              keys and values to their slots
 *   cf_paged_attention         attention of new tokens over their sequence,
 *                              causal, optionally with a sliding window and
 *                              a few first positions that stay visible
 *   cf_paged_prefix_attention  the same without a window, for a batch whose
 *                              sequences all continue one shared prefix; the
 *                              prefix is read once for the whole batch (fp32:
 *                              once per sequence)
 *
 * A call holds `n_tokens` new tokens of `batch` sequences.  Sequence b has
 * the tokens q_start[b] .. q_start[b+1]-1 (n_b of them, none allowed) and,
 * with them, kv_len[b] positions; its token i sits at position
 *   p = kv_len[b] - n_b + i.
 * q_start == NULL means one token per sequence (n_tokens == batch).  Tokens
 * from q_start[batch] on belong to no sequence and their rows of every
 * output stay as they are.
 *
 * Formulas, per token at position p, head h of KV head g = h / (nq/nkv):
 *   rotation (rotate-half over the first r = rope_dim elements of a head):
 *     a = x_i, b = x_{i+r/2}, angle = P_{axis(i)} * rope_theta^(-2i/r):
 *     x_i <- a cos - b sin,  x_{i+r/2} <- b cos + a sin,    i < r/2
 *   P is p itself, or rope_pos[axis][token] where given
 *   visible(p, j) = 0 <= j <= p  and  (window == 0 or p - j < window or j < n_sinks)
 *   s_j = scale * q_h . k_j,   o_h = sum_j exp(s_j) v_j / sum_j exp(s_j)   over visible j
 *   lse_h = ln sum_j exp(s_j)
 * A row that sees no key (p < 0, also where there is a prefix), or only keys
 * with scores of -infinity, gets o = 0 and lse = -infinity; a score of NaN
 * makes both NaN.  What lies in a slot, be it an infinity or a NaN, reaches
 * the rows that see its position and no other.  An infinity in V gives them an
 * infinity; NaN where one of the other sign is seen too, and where its
 * probability may count as 0 in the product (fp16: below 2^-31 of the row's
 * largest, bf16 2^-115, fp32 2^-126).  Table entries of positions that no row
 * of the sequence sees (past kv_len, behind the window) are not read as pages.
 *
 * Arithmetic: products and sums in fp32 (fp32 storage: plain fp32 FMAs; fp16
 * and bf16: tensor-core products of the stored values).  Probabilities enter
 * the product with V rounded to the storage type (in bf16, with max_q * nq/nkv
 * of 16 at most, as a sum of two such values; in fp16 times 2^15 or, with
 * more, 2^7, which holds them down to 2^-40 or 2^-32); their sum is taken
 * before that rounding.  Outputs are rounded once.  Angles are off by 2^-25 of a turn at
 * most for positions up to 2^28, by 2^-23 for every int32 position (rope_theta
 * of 1 or more).  The same call on the same data gives the same bits.
 *
 * Conventions for every function:
 *   - CF_OK (0) or a negative CF_ERR_* code of cf.h; nothing is printed and no
 *     exception crosses the ABI;
 *   - calls enqueue work on `stream` (a cudaStream_t, NULL = legacy default)
 *     and return; they never allocate, synchronize or copy to the host, so
 *     they can be captured in a CUDA graph;
 *   - the device current at cf_paged_create must be current at every call
 *     (CF_ERR_INVALID_ARG otherwise); the caller owns every tensor;
 *   - not thread-safe per handle.  The attention calls use the handle's
 *     workspace: two of them on one handle must not overlap on the GPU (two
 *     streams, or two graphs replayed at once, need two handles).
 * What the device finds wrong is recorded and read with cf_paged_get_status;
 * the call then still ends, and reads and writes nothing out of bounds:
 *   - a kv_len outside [0, max_pages * page_size] or more tokens in a sequence
 *     than max_q: the sequence's rows get o = 0, lse = -infinity and nothing
 *     is appended for it;
 *   - a needed page number outside [0, num_pages): keys and values of zero
 *     stand for its positions, and nothing is appended to it;
 *   - an appended token with p < 0 is skipped; its q_out row, like that of every
 *     token that is not appended, stays as it was;
 *   - q_start values that decrease or leave [0, n_tokens]: such a sequence
 *     has no tokens, the others have theirs.  Where two sequences then claim a
 *     token, what the call writes is unspecified, though within its outputs.
 */
#ifndef CF_PAGED_H
#define CF_PAGED_H

#include <stdint.h>

#include "cf.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct cf_paged_config {
  int32_t n_q_heads;    /* nq                                                    */
  int32_t n_kv_heads;   /* nkv; nq % nkv == 0                                    */
  int32_t head_dim;     /* d: 64 or 128                                          */
  int32_t page_size;    /* positions per page: a power of two, 1..1024           */
  int32_t num_pages;    /* pages in k_pages and in v_pages                       */
  int32_t max_pages;    /* columns of page_table (pages per sequence, at most)   */
  int32_t max_batch;    /* upper bound on `batch`, 1..65535                      */
  int32_t max_tokens;   /* upper bound on `n_tokens`                             */
  int32_t dtype;        /* cf_dtype of q, k, v, the pages and out                */
  int32_t layout;       /* 0: pages are [page_size, nkv, d]; 1: [nkv, page_size, d] */
  int64_t page_stride;  /* elements from a page to the next: 0 = dense, else at
                           least page_size*nkv*d and a multiple of 16 bytes (a
                           pool that interleaves keys and values has twice it) */
  float rope_theta;     /* base of the rotation                                  */
  int32_t rope_dim;     /* r: elements of a head that are rotated; 0 = head_dim,
                           else a multiple of 16 up to head_dim                  */
  int32_t rope_sections[3]; /* all 0: one axis.  Else the number of the r/2
                           pairs that follow axis 0, 1, 2 (time, height, width);
                           the sum is r/2                                        */
  int32_t rope_interleaved; /* 0: the sections lie one after another.  1: pair i
                           follows axis i % 3 while i / 3 < rope_sections[i % 3],
                           the others axis 0                                     */
  float scale;          /* score scale; 0 = 1/sqrt(head_dim)                     */
} cf_paged_config;

typedef struct cf_paged_handle cf_paged_handle; /* opaque */

/* Validate cfg and allocate the handle's workspace on the current device: an
 * error word and, but for fp32, partial results of split sequences (up to
 * 160,000 * (d + 2) fp32 values, 81 MB for d = 128) and of whole ones beside a
 * prefix (per token of max_tokens up to 2 * nq * (d + 2) fp32 values; calls
 * without a prefix use none of these, but the handle has them all the same).
 * On failure nothing stays allocated and *out is NULL.  Errors: INVALID_ARG
 * (NULL, sizes, strides, sections that do not add up), UNSUPPORTED
 * (head_dim, page_size), CUDA. */
int cf_paged_create(const cf_paged_config* cfg, cf_paged_handle** out);

/* Rotate and append n_tokens new tokens.
 *   q        [n_tokens, nq, d]    rows q_stride elements apart; read
 *   k, v     [n_tokens, nkv, d]   rows kv_stride elements apart; read
 *            (q, k and v may be column ranges of one merged projection)
 *   q_start  [batch+1] int32 or NULL;  kv_len [batch] int32
 *   rope_pos [axes, n_tokens] int32 (axes: 3 with rope_sections, else 1), or
 *            NULL: every axis takes p
 *   page_table [batch, max_pages] int32
 *   k_pages, v_pages              the slots of the new tokens are written; the
 *            pools may alternate by pages, but share none (CF_ERR_ALIAS)
 *   q_out    [n_tokens, nq, d]    rows q_out_stride elements apart; the
 *            rotated queries.  May be q itself (same address and stride; rows
 *            of k and v of that stride may then lie between its own), must
 *            otherwise not overlap an input, nor its rows' gaps (CF_ERR_ALIAS)
 * q and q_out may both be NULL: then only k and v are taken.  Two tokens of
 * one call must not map to the same slot.  Strides are multiples of 16 bytes,
 * pointers to storage 16-byte aligned, int32 arrays 4-byte aligned.
 * n_tokens == 0 or batch == 0 does nothing. */
int cf_paged_append(cf_paged_handle* h, int32_t batch, int32_t n_tokens, const void* q,
                    const void* k, const void* v, int64_t q_stride, int64_t kv_stride,
                    const int32_t* q_start, const int32_t* kv_len, const int32_t* rope_pos,
                    const int32_t* page_table, void* k_pages, void* v_pages, void* q_out,
                    int64_t q_out_stride, void* stream);

/* Attention of n_tokens new tokens, whose keys and values are in the pages.
 *   max_q    upper bound on the tokens of one sequence in this call
 *            (1..n_tokens; ignored, as 1, when q_start is NULL)
 *   q        [n_tokens, nq, d]    rotated queries, rows q_stride elements apart
 *   window   0 = every position up to the token's own, else the number of
 *            last positions that are visible, the token's own among them
 *   n_sinks  first positions that stay visible behind the window (>= 0)
 *   out      [n_tokens, nq, d]    dense; must not overlap an input (CF_ERR_ALIAS)
 *   lse      [n_tokens, nq] fp32, or NULL */
int cf_paged_attention(cf_paged_handle* h, int32_t batch, int32_t n_tokens, int32_t max_q,
                       const void* q, int64_t q_stride, const int32_t* q_start,
                       const int32_t* kv_len, const int32_t* page_table, const void* k_pages,
                       const void* v_pages, int32_t window, int32_t n_sinks, void* out, float* lse,
                       void* stream);

/* Attention of a batch that shares a prefix of prefix_len positions (0 or
 * more; position t is slot t % page_size of page prefix_table[t / page_size]):
 * every token sees the whole prefix and, causally, its own sequence, whose
 * kv_len and page_table do not count the prefix.  Other arguments as above. */
int cf_paged_prefix_attention(cf_paged_handle* h, int32_t batch, int32_t n_tokens, int32_t max_q,
                              const void* q, int64_t q_stride, const int32_t* q_start,
                              const int32_t* kv_len, const int32_t* page_table,
                              const int32_t* prefix_table, int32_t prefix_len,
                              const void* k_pages, const void* v_pages, void* out, float* lse,
                              void* stream);

/* Read and clear the device-side error word (synchronize the stream first):
 * CF_OK, CF_ERR_DEVICE_POS_RANGE (see above), CF_ERR_DEVICE_TIMEOUT or
 * CF_ERR_CUDA. */
int cf_paged_get_status(cf_paged_handle* h);

/* Free the handle and its workspace.  NULL is a no-op. */
void cf_paged_destroy(cf_paged_handle* h);

#ifdef __cplusplus
}
#endif

#endif /* CF_PAGED_H */
