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

// The tiles of TK positions that hold a range: sink tiles from 0, then the
// tiles of [lo, hi); always at least one.
template <int TK>
struct PagedTiles {
  int sink, lo, hi;
  int ns, skip;  // sink tiles, and tiles between them and the window's first
  int tiles;
  __device__ __forceinline__ void set(const PagedRange& r) {
    sink = r.sink;
    lo = r.lo;
    hi = r.hi;
    if (hi <= lo) {  // no key
      sink = ns = skip = 0;
      tiles = 1;
      return;
    }
    const int f = lo / TK, e = (hi + TK - 1) / TK;
    ns = (sink + TK - 1) / TK;
    skip = max(0, f - ns);
    if (skip == 0) ns = 0;
    tiles = e - skip;
  }
  __device__ __forceinline__ int base(int tile) const {
    return (tile < ns ? tile : tile + skip) * TK;
  }
  __device__ __forceinline__ bool sees(int j) const { return (j >= lo && j < hi) || j < sink; }
};

// 16 bytes global -> shared, asynchronously; zeros where there is no source.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// How a kernel's work is cut over its blocks.  The units (key tiles) of all
// items (a sequence or row tile and a KV head) form one line; block c takes
// units [c * upc, (c + 1) * upc).  An item that lies in several blocks leaves
// one partial state (o not normalised, running maximum in base 2, sum) per
// block, in slot 2c where it began in an earlier block and in 2c + 1 where it
// begins in this one.
struct PagedParts {
  float* o;     // [slots][rows][D]
  float2* ml;   // [slots][rows]
  int* tickets; // one per item: partial states written so far (0 between calls)
};

__device__ __forceinline__ void pdl_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void pdl_trigger() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// a / b, in 32 bits where both fit (a 64-bit division is a long chain).
__device__ __forceinline__ long long div_units(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (long long)((uint32_t)a / (uint32_t)b);
  return a / b;
}

// Partial states of one item: the blocks first .. first + n - 1.
struct PagedItemParts {
  long long i0, upc, first;
  int n;
  __device__ __forceinline__ PagedItemParts(long long i0_, long long tiles, long long upc_)
      : i0(i0_), upc(upc_), first(div_units(i0_, upc_)) {
    n = (int)(div_units(i0_ + tiles - 1, upc_) - first) + 1;
  }
  __device__ __forceinline__ long long slot(int k) const {
    const long long c = first + k;
    return 2 * c + (c * upc >= i0 ? 0 : 1);
  }
};

// The shared prefix's partial states, as the kernel that reads the sequences'
// own keys finds them: row R = token * G + (head in the KV head's group) is
// row R % rows of tile R / rows, and item tile * nkv + kv head has `tiles`
// units behind item_cost empty ones.  rows == 0: there is no prefix.
struct PagedPrefixParts {
  const float* o;
  const float2* ml;
  int rows;
  int tiles, item_cost;
  long long upc;
  __device__ __forceinline__ PagedItemParts item(long long index) const {
    return PagedItemParts(index * (tiles + item_cost) + item_cost, tiles, upc);
  }
};

// Softmax state of 4 columns of a row, joined with another one.
struct PagedState4 {
  float m, l;
  float4 o;
  __device__ __forceinline__ void join(float m2, float l2, const float4& o2) {
    const float mn = fmaxf(m, m2);
    if (mn == -INFINITY) return;
    const float a = exp2f(m - mn), b = exp2f(m2 - mn);
    m = mn;
    l = l * a + l2 * b;
    o.x = o.x * a + o2.x * b;
    o.y = o.y * a + o2.y * b;
    o.z = o.z * a + o2.z * b;
    o.w = o.w * a + o2.w * b;
  }
};

// Joins the prefix's states of one row's 4 columns at `col` into s.
template <int D>
__device__ __forceinline__ void paged_join_prefix(PagedState4& s, const PagedPrefixParts& x,
                                                  long long R, int kvh, int nkv, int col) {
  const long long tile = div_units(R, x.rows);
  const int row = (int)(R - tile * x.rows);
  const PagedItemParts parts(x.item(tile * nkv + kvh));
#pragma unroll 4
  for (int k = 0; k < parts.n; ++k) {
    const long long at = parts.slot(k) * x.rows + row;
    const float2 ml = __ldcg(x.ml + at);
    const float4 o = __ldcg(reinterpret_cast<const float4*>(x.o + at * D + col));
    s.join(ml.x, ml.y, o);
  }
}

// Normalises and stores 4 columns of a row, and its lse.
template <typename T, int D>
__device__ __forceinline__ void paged_store4(const PagedState4& s, void* out, float* lse,
                                             long long row, int col) {
  const float inv = s.l == 0.f ? 0.f : 1.f / s.l;
  const float f[4] = {s.o.x * inv, s.o.y * inv, s.o.z * inv, s.o.w * inv};
  store4<T>(static_cast<T*>(out) + row * D + col, f);
  if (lse && col == 0)
    lse[row] = s.m == -INFINITY ? -INFINITY : (s.m + log2f(s.l)) * 0.69314718055994531f;
}

// Host launchers (one translation unit each); false: the launch failed.
struct PagedSplit {  // one kernel's part of a handle's workspace
  float* o = nullptr;
  float2* ml = nullptr;
  int* tickets = nullptr;
  void* meta = nullptr;
  int grid = 0;  // resident blocks the kernel is cut for
};
// Rows (tokens x grouped heads) and resident blocks of the few-row kernel.
constexpr int kFewRows = 16;
int paged_few_grid(int dtype, int head_dim, int sm_count);
// prefix: the call's tokens against the prefix alone, partial states only.
bool paged_few_launch(int dtype, const PagedAttnParams& p, const PagedSplit& ws, bool prefix,
                      const PagedPrefixParts& pre, cudaStream_t st);
// How the few-row kernel cuts the prefix.
PagedPrefixParts paged_few_prefix(const PagedAttnParams& p, const PagedSplit& ws);
bool paged_append_launch(int dtype, const PagedAppendParams& p, int sm_count, cudaStream_t st);
bool paged_attn_simple_launch(int dtype, const PagedAttnParams& p, cudaStream_t st);

// The tensor-core kernel for many rows; the arguments as above.
constexpr int kTcRows = 256;
int paged_tc_grid(int dtype, int head_dim, int sm_count);
size_t paged_tc_meta_bytes(int grid);
bool paged_tc_launch(int dtype, const PagedAttnParams& p, const PagedSplit& ws, bool prefix,
                     const PagedPrefixParts& pre, cudaStream_t st);
PagedPrefixParts paged_tc_prefix(const PagedAttnParams& p, const PagedSplit& ws);

}  // namespace cf
