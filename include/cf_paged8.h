/*
 * cf_paged8.h -- C ABI of the paged KV cache held in 8 bits: the operators
 * that write it, the attention that reads it, and one that reads it back.
 *
 * Pages, page tables, tokens, positions, the rotation and what a token sees
 * are those of cf_paged.h.  A slot holds 8-bit codes instead of values, and
 * each (position, KV head) has a scale for its key and one for its value:
 *
 *   k_pages, v_pages  1 byte an element, [num_pages, page_size, nkv, d] or
 *                     [num_pages, nkv, page_size, d] (cf_paged_config.layout)
 *   scales            fp32 [num_pages, nkv, page_size, 2], dense: the key's
 *                     scale, then the value's
 *
 * Half the bytes of a 16-bit cache (d = 128: 264 for 512 bytes per position
 * and KV head), which is what bounds the decode step.
 *
 * Formulas.  A head x (a rotated key, or a value; d elements in fp32) becomes
 *   amax = max |x_i|,  scale = amax / Q,  code_i = round(x_i * (Q / amax))
 *   CF_CODE_INT8: Q = 127, round to nearest even, two's complement
 *   CF_CODE_E4M3: Q = 448, nearest even 8-bit float with 4 exponent bits
 * and stands for code_i * scale.  amax below 2^-100: scale and codes are 0.
 * An infinity or NaN in x: the scale is NaN and the codes are 0, so the whole
 * head counts as NaN.  Attention, with k, v the codes and ks, vs their scales:
 *   s_j = scale * (q . k_j) * ks_j
 *   o   = sum_j exp(s_j) vs_j v_j / sum_j exp(s_j)      over visible j
 *   lse = ln sum_j exp(s_j)
 * A row that sees no key gets o = 0 and lse = -infinity; one that sees a NaN
 * (a scale's or the query's) gets NaN in what it touches: a key's makes o and
 * lse NaN, a value's o alone.  What lies in a slot reaches the rows that see its
 * position and no other.
 *
 * Arithmetic: codes are whole in the products, which run on the tensor cores
 * as fp16 x fp16 with fp32 sums.  The query enters as fp16: bf16 queries are
 * multiplied by a power of two where they need it.  With max_q * nq/nkv of 16 at
 * most that is the same for the rows that share a tile (a sequence's, of one KV
 * head), and an element is off by 2^-39 of the largest of them at most; with more
 * by 2^-25 in a row whose largest lies between 2^-10 and 2^15, else by 2^-39 of
 * that (or by 2^-138).  Scales and softmax statistics are fp32; weights
 * exp(s_j) vs_j enter the second product in fp16, held down to 2^-32 of the row's
 * largest (a scale of 0 counts as 2^-80 there); the sum of exp(s_j) is taken before
 * that rounding and whatever the value scales are.  Outputs are rounded once.  The
 * same call on the same data gives the same bits.
 *
 * Scales are read from 0 to 2^60, value scales from 2^-60 on: a smaller one counts
 * as 0 (what it adds to o is below 2^-70), and a scale above 2^60 or below 0 as
 * NaN.  Appending fp16 stays within that, and so does bf16 between 2^-51 and 2^66;
 * a head of smaller values can be read back (cf_paged8_read) and adds nothing to o.
 * E4m3 codes must not be NaN (0x7f, 0xff; none is appended).
 *
 * Conventions, and what the device records (cf_paged8_get_status), are those
 * of cf_paged.h; scales are 8-byte aligned.
 */
#ifndef CF_PAGED8_H
#define CF_PAGED8_H

#include <stdint.h>

#include "cf_paged.h"

#ifdef __cplusplus
extern "C" {
#endif

enum cf_code { CF_CODE_INT8 = 0, CF_CODE_E4M3 = 1 };

typedef struct cf_paged8_config {
  cf_paged_config cache; /* dtype: of q, k, v and the outputs, CF_F16 or CF_BF16;
                            page_stride: bytes                                   */
  int32_t code;          /* cf_code                                              */
} cf_paged8_config;

typedef struct cf_paged8_handle cf_paged8_handle; /* opaque */

/* Validate cfg and allocate the handle's workspace on the current device: an
 * error word, a word for each sequence and KV head, and partial results of split
 * sequences (with 152 SMs up to (d + 2) * 77,824 fp32 values, 40 MB for d = 128).
 * On failure nothing stays allocated and *out is NULL.  Errors: INVALID_ARG, UNSUPPORTED (head_dim, page_size, fp32),
 * CUDA. */
int cf_paged8_create(const cf_paged8_config* cfg, cf_paged8_handle** out);

/* Rotate, quantise and append n_tokens new tokens: cf_paged_append with codes
 * and scales written in place of the values.  Keys are quantised from the
 * rotated values in fp32. */
int cf_paged8_append(cf_paged8_handle* h, int32_t batch, int32_t n_tokens, const void* q,
                     const void* k, const void* v, int64_t q_stride, int64_t kv_stride,
                     const int32_t* q_start, const int32_t* kv_len, const int32_t* rope_pos,
                     const int32_t* page_table, void* k_pages, void* v_pages, float* scales,
                     void* q_out, int64_t q_out_stride, void* stream);

/* Attention of n_tokens new tokens, whose keys and values are in the pages:
 * single tokens, drafts, or chunks of prompts.  Arguments as in
 * cf_paged_attention. */
int cf_paged8_attention(cf_paged8_handle* h, int32_t batch, int32_t n_tokens, int32_t max_q,
                        const void* q, int64_t q_stride, const int32_t* q_start,
                        const int32_t* kv_len, const int32_t* page_table, const void* k_pages,
                        const void* v_pages, const float* scales, int32_t window, int32_t n_sinks,
                        void* out, float* lse, void* stream);

/* Read positions back into rows of the storage type: code * scale in fp32, then
 * rounded to it.
 *   row_start [batch+1] int32: sequence b has the rows row_start[b] ..
 *             row_start[b+1]-1; rows from row_start[batch] on stay as they are
 *   first     [batch] int32, the position of each sequence's first row, or
 *             NULL: 0
 *   k_out, v_out [n_rows, nkv, d], rows out_stride elements apart (a multiple
 *             of 16 bytes); either may be NULL.  They may be rows of a dense
 *             cache; they must not overlap each other or an input.
 * A position outside [0, max_pages * page_size) is recorded and its row stays
 * as it is; a page outside the pool is recorded and reads as zeros.  n_rows
 * is not bounded by max_tokens, only by 2^30. */
int cf_paged8_read(cf_paged8_handle* h, int32_t batch, int32_t n_rows, const int32_t* row_start,
                   const int32_t* first, const int32_t* page_table, const void* k_pages,
                   const void* v_pages, const float* scales, void* k_out, void* v_out,
                   int64_t out_stride, void* stream);

/* Read and clear the device-side error word, as cf_paged_get_status. */
int cf_paged8_get_status(cf_paged8_handle* h);

/* Free the handle and its workspace.  NULL is a no-op. */
void cf_paged8_destroy(cf_paged8_handle* h);

#ifdef __cplusplus
}
#endif

#endif /* CF_PAGED8_H */
