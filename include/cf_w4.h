/*
 * cf_w4.h -- products of a few rows with a weight matrix held in 4 bits: the
 * projections of a decode step (Q/K/V, output, gate and up, down) at a quarter
 * of their bytes.
 *
 * Formula, per row r of x [rows, K] and column n:
 *   W[k][n] = (code[k][n] - zero[k / group][n]) * scale[k / group][n]
 *   out[r][n] = residual[r][n] + sum_k x[r][k] W[k][n]
 * Codes are whole numbers 0..15.  Without zero points every zero is 8.
 *
 * Arithmetic: x and code - zero enter the tensor cores exactly (fp32 x as a sum
 * of three bf16 values, exact from 2^-110 on), sums are fp32, a group's sum is
 * multiplied by its scale in fp32, and out is rounded once.  (A group's sum of x
 * (code - zero) must itself stay within fp32.)  The same call on the same data
 * gives the same bits.
 *
 * Weights are laid out once, by cf_w4_pack, in the order in which the kernel
 * streams them: for each 128 elements of k and 16 columns one record of 1 KB of
 * codes with their scales and zeros.
 *
 * Conventions: CF_OK or a negative CF_ERR_* code of cf.h, nothing is printed;
 * calls enqueue work on `stream` and return, never allocate or synchronize, and
 * may be captured in a CUDA graph.  The device current at cf_w4_create must be
 * current at every call.  A handle holds its sizes, an error word and no state of a
 * call: one handle serves any number of matrices of its shape, streams and threads.
 */
#ifndef CF_W4_H
#define CF_W4_H

#include <stddef.h>
#include <stdint.h>

#include "cf.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct cf_w4_config {
  int32_t in_features;  /* K: a multiple of group, at most 1 << 20              */
  int32_t out_features; /* N: even, at most 1 << 24                             */
  int32_t group;        /* elements of k that share a scale: 32, 64 or 128      */
  int32_t zeros;        /* 1: weights have zero points                          */
  int32_t max_rows;     /* upper bound on `rows`: 1..64                         */
  int32_t dtype;        /* cf_dtype of x, scales, residual and out              */
} cf_w4_config;

typedef struct cf_w4_handle cf_w4_handle; /* opaque */

/* Validate cfg on the current device.  On failure *out is NULL.  Errors:
 * INVALID_ARG, UNSUPPORTED (group, max_rows), CUDA. */
int cf_w4_create(const cf_w4_config* cfg, cf_w4_handle** out);

/* Bytes of packed weights; 0 for a NULL handle. */
size_t cf_w4_packed_bytes(const cf_w4_handle* h);

/* Lay weights out.
 *   codes   [K, N / 2] bytes, column n in the low (n even) or high half of byte n / 2
 *   scales  [K / group, N]
 *   zeros   [K / group, N] bytes, 0..15 (higher bits are not read); NULL exactly
 *           where the handle has none
 *   packed  cf_w4_packed_bytes, 16-byte aligned; overlaps no input (CF_ERR_ALIAS) */
int cf_w4_pack(cf_w4_handle* h, const uint8_t* codes, const void* scales, const uint8_t* zeros,
               void* packed, void* stream);

/* out = x W (+ residual) for `rows` rows (0 <= rows <= max_rows; 0 does nothing).
 *   x         [rows, K]  rows x_stride elements apart, 16-byte aligned, as the
 *             stride in bytes
 *   residual  [rows, N]  dense, or NULL; may be out itself
 *   out       [rows, N]  dense; must not overlap another input (CF_ERR_ALIAS) */
int cf_w4_matvec(cf_w4_handle* h, int32_t rows, const void* x, int64_t x_stride,
                 const void* packed, const void* residual, void* out, void* stream);

/* Read and clear the device-side error word (synchronize the stream first):
 * CF_OK, CF_ERR_DEVICE_TIMEOUT (a wait that ran out) or CF_ERR_CUDA. */
int cf_w4_get_status(cf_w4_handle* h);

/* NULL is a no-op. */
void cf_w4_destroy(cf_w4_handle* h);

#ifdef __cplusplus
}
#endif

#endif /* CF_W4_H */
