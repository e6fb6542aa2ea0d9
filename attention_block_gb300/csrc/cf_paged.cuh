// cf_paged.cuh -- what the kernels of the paged KV cache share: the call's
// parameters, where a sequence's tokens and visible positions lie, the
// address of a position, and launch entry points (include/cf_paged.h).
#pragma once

#include <stdint.h>

#include "cf.h"
#include "cf_common.cuh"

namespace cf {

constexpr int kMaxPairs = 64;  // rotated pairs of a head (head_dim 128)

// Addressing of the pages, common to every call of a handle.
struct PagedGeom {
  int nq, nkv, G, D;
  int page_shift, page_mask;
  int num_pages, max_pages;
  int64_t page_stride, slot_stride, head_stride;  // elements
};

struct PagedAppendParams {
  PagedGeom g;
  const void *q, *k, *v;
  void *q_out, *k_pages, *v_pages;
  int64_t q_stride, kv_stride, q_out_stride;
  const int *q_start, *kv_len, *rope_pos, *page_table;
  int* errflag;
  int batch, n_tokens, rope_dim, axes;
  uint64_t turn[kMaxPairs];  // theta^(-2i/r) / (2 pi) in 2^-64 of a turn
  uint8_t axis[kMaxPairs];   // which row of rope_pos pair i follows
};

struct PagedAttnParams {
  PagedGeom g;
  const void *q, *k_pages, *v_pages;
  void* out;
  float* lse;
  int64_t q_stride;
  const int *q_start, *kv_len, *page_table, *prefix_table;
  int* errflag;
  int batch, n_tokens, max_q;
  int prefix_len, window, n_sinks;
  float scale_log2;  // score scale * log2(e): softmax in base 2
};

// The tokens of sequence b: first, count and its length; a malformed entry is
// recorded and leaves the sequence without tokens or without keys.
struct PagedSeq {
  int t0, n, len;
};
__device__ __forceinline__ PagedSeq paged_seq(const int* q_start, const int* kv_len, int b,
                                              int n_tokens, int max_q, const PagedGeom& g,
                                              int* errflag) {
  PagedSeq s;
  s.t0 = q_start ? q_start[b] : b;
  const int t1 = q_start ? q_start[b + 1] : b + 1;
  s.len = kv_len[b];
  s.n = t1 - s.t0;
  bool bad = false;
  if (s.t0 < 0 || t1 > n_tokens || t1 < s.t0) {
    s.n = s.t0 = 0;
    bad = true;
  }
  const long long cap = (long long)g.max_pages << g.page_shift;
  if (s.len < 0 || s.len > cap || s.n > max_q) {
    s.len = 0;
    bad = true;
  }
  if (bad) atomicOr(errflag, kDevErrPosRange);
  return s;
}

// Own positions that some row in [p_lo, p_hi] sees: [0, sink) and [lo, hi).
struct PagedRange {
  int sink, lo, hi;
};
__device__ __forceinline__ PagedRange paged_range(int p_lo, int p_hi, int len, int window,
                                                  int n_sinks) {
  PagedRange r;
  r.hi = min(p_hi + 1, len);
  if (r.hi < 0) r.hi = 0;
  r.lo = window > 0 ? max(0, p_lo - window + 1) : 0;
  if (r.lo > r.hi) r.lo = r.hi;
  r.sink = min(n_sinks, r.lo);
  return r;
}

__device__ __forceinline__ bool paged_visible(int p, int j, int window, int n_sinks) {
  return j <= p && (window == 0 || p - j < window || j < n_sinks);
}

// Element offset of position j (KV head 0) through a page table row, or -1 for
// a page number outside the pool (recorded).
__device__ __forceinline__ int64_t paged_offset(const int* table, int j, const PagedGeom& g,
                                                int* errflag) {
  const int page = table[j >> g.page_shift];
  if ((unsigned)page >= (unsigned)g.num_pages) {
    atomicOr(errflag, kDevErrPosRange);
    return -1;
  }
  return (int64_t)page * g.page_stride + (int64_t)(j & g.page_mask) * g.slot_stride;
}

// Host launchers (one translation unit each); false: the launch failed.
bool paged_append_launch(int dtype, const PagedAppendParams& p, int sm_count, cudaStream_t st);
bool paged_attn_simple_launch(int dtype, const PagedAttnParams& p, cudaStream_t st);

}  // namespace cf
