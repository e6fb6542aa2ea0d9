// cf_paged_host.h -- what the host sides of the paged caches share
// (include/cf_paged.h, include/cf_paged8.h): the checks of a configuration and
// of a call's arguments, and the kernels' parameters made of them.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "cf.h"
#include "cf_paged.cuh"
#include "cf_paged.h"

namespace cf {

// A handle's part that does not depend on what the pages hold.
struct PagedHost {
  cf_paged_config cfg;
  int device = 0, sm_count = 0;
  PagedGeom geom;
  size_t page_es = 0;      // bytes of an element of the pages
  int64_t pool_elems = 0;  // from the first to past the last element of a pool
  uint64_t turn[kMaxPairs];
  uint8_t axis[kMaxPairs];
  float scale_log2 = 0.f;
  size_t pool_bytes() const { return (size_t)pool_elems * page_es; }
  // of the scales of a cache of 8-bit codes
  size_t scale_bytes() const {
    return (size_t)cfg.num_pages * cfg.n_kv_heads * cfg.page_size * sizeof(float2);
  }
};

inline size_t elem_size(int dtype) { return dtype == CF_F32 ? 4 : 2; }

// The largest stride of n rows or pages: what they span, in bytes too, stays
// far below 2^63.
inline int64_t max_stride(int64_t n) {
  return std::min((int64_t)1 << 40, ((int64_t)1 << 56) / n);
}

inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (a == nullptr || b == nullptr || na == 0 || nb == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

inline bool aligned(const void* p, uintptr_t n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

// Which axis pair i follows; false if the sections do not add up.
inline bool assign_axes(const cf_paged_config& c, int pairs, uint8_t* axis) {
  const int* s = c.rope_sections;
  for (int i = 0; i < kMaxPairs; ++i) axis[i] = 0;
  if (s[0] == 0 && s[1] == 0 && s[2] == 0) return true;
  if (s[0] < 0 || s[1] < 0 || s[2] < 0 || (int64_t)s[0] + s[1] + s[2] != pairs) return false;
  int n[3] = {0, 0, 0};
  for (int i = 0; i < pairs; ++i) {
    int a = 0;
    if (c.rope_interleaved)
      a = i / 3 < s[i % 3] ? i % 3 : 0;
    else
      a = i < s[0] ? 0 : (i < s[0] + s[1] ? 1 : 2);
    axis[i] = (uint8_t)a;
    ++n[a];
  }
  return n[0] == s[0] && n[1] == s[1] && n[2] == s[2];
}

// Bytes from the first to past the last element of n rows `stride` apart.
inline size_t rows_bytes(int64_t n, int64_t stride, int64_t row, size_t es) {
  return n > 0 ? (size_t)((n - 1) * stride + row) * es : 0;
}

// Zeros n bytes and waits for that: cudaMemset of device memory may return
// before it is done, and calls on streams that do not wait for the default one
// may follow at once.
inline bool clear(void* p, size_t n) {
  if (cudaMemset(p, 0, n) == cudaSuccess && cudaStreamSynchronize(nullptr) == cudaSuccess)
    return true;
  cudaGetLastError();
  return false;
}

// Whether one of n rows of na bytes from a meets one of n rows of nb bytes from
// b, both `stride` bytes apart.
inline bool rows_meet(const void* a, int64_t na, const void* b, int64_t nb, int64_t n,
                      int64_t stride) {
  const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
  // row i of a and row i + t of b do where -nb < d + t * stride < na: the least
  // t with the left side, in -(n - 1) .. n - 1, decides
  const int64_t x = -nb - d;
  const int64_t floor = x / stride - (x % stride < 0 ? 1 : 0);
  const int64_t t = std::max(floor + 1, 1 - n);
  return t <= n - 1 && d + t * stride < na;
}

// Checks that the handle's calls share; CF_OK or an error.
inline int check_call(const PagedHost& h, int32_t batch, int32_t n_tokens,
                      const int32_t* q_start) {
  const cf_paged_config& c = h.cfg;
  if (batch < 0 || batch > c.max_batch || n_tokens < 0 || n_tokens > c.max_tokens)
    return CF_ERR_INVALID_ARG;
  if (q_start == nullptr && n_tokens != batch) return CF_ERR_INVALID_ARG;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return CF_ERR_CUDA;
  }
  return dev == h.device ? CF_OK : CF_ERR_INVALID_ARG;
}

// Checks c and fills in h for the current device; CF_OK or an error.  page_es:
// bytes of an element of the pages.
inline int paged_host_init(cf_paged_config c, size_t page_es, PagedHost& h) {
  if (c.n_q_heads <= 0 || c.n_kv_heads <= 0 || c.n_q_heads % c.n_kv_heads != 0 ||
      c.head_dim <= 0 || c.page_size <= 0 || c.num_pages <= 0 || c.max_pages <= 0 ||
      c.max_batch <= 0 || c.max_batch > 65535 || c.max_tokens <= 0)
    return CF_ERR_INVALID_ARG;
  if (c.n_q_heads > 65535) return CF_ERR_INVALID_ARG;
  if (c.dtype < CF_F32 || c.dtype > CF_BF16 || c.layout < 0 || c.layout > 1 ||
      c.rope_interleaved < 0 || c.rope_interleaved > 1)
    return CF_ERR_INVALID_ARG;
  if (!(c.rope_theta > 0.f) || !std::isfinite(c.rope_theta) || !(c.scale >= 0.f) ||
      !std::isfinite(c.scale))
    return CF_ERR_INVALID_ARG;
  if (c.head_dim != 64 && c.head_dim != 128) return CF_ERR_UNSUPPORTED;
  if (c.page_size > 1024 || (c.page_size & (c.page_size - 1)) != 0) return CF_ERR_UNSUPPORTED;
  // positions and token rows are 32-bit numbers with room for sums of two
  if ((int64_t)c.max_pages * c.page_size > (1 << 30) || c.max_tokens > (1 << 26) ||
      (int64_t)c.max_tokens * (c.n_q_heads / c.n_kv_heads) > (1 << 30))
    return CF_ERR_INVALID_ARG;
  if (c.rope_dim == 0) c.rope_dim = c.head_dim;
  if (c.rope_dim < 0 || c.rope_dim > c.head_dim || c.rope_dim % 16 != 0) return CF_ERR_INVALID_ARG;
  const int64_t page = (int64_t)c.page_size * c.n_kv_heads * c.head_dim;
  if (c.page_stride == 0) c.page_stride = page;
  if (c.page_stride < page || c.page_stride > max_stride(c.num_pages) ||
      (c.page_stride * (int64_t)page_es) % 16 != 0)
    return CF_ERR_INVALID_ARG;

  h.cfg = c;
  h.page_es = page_es;
  const int pairs = c.rope_dim / 2;
  if (!assign_axes(c, pairs, h.axis)) return CF_ERR_INVALID_ARG;
  for (int i = 0; i < kMaxPairs; ++i) {
    const double two_pi = 6.283185307179586476925286766559;
    const double rate =
        i < pairs ? std::pow((double)c.rope_theta, -2.0 * i / (double)c.rope_dim) / two_pi : 0.0;
    // theta < 1 turns faster than once a position: only the fraction counts
    h.turn[i] = (uint64_t)std::ldexp(rate - std::floor(rate), 64);
  }
  const double scale = c.scale > 0.f ? (double)c.scale : 1.0 / std::sqrt((double)c.head_dim);
  h.scale_log2 = (float)(scale * 1.4426950408889634);
  PagedGeom& g = h.geom;
  g.nq = c.n_q_heads;
  g.nkv = c.n_kv_heads;
  g.G = c.n_q_heads / c.n_kv_heads;
  g.D = c.head_dim;
  g.page_shift = 0;
  while ((1 << g.page_shift) < c.page_size) ++g.page_shift;
  g.page_mask = c.page_size - 1;
  g.num_pages = c.num_pages;
  g.max_pages = c.max_pages;
  g.page_stride = c.page_stride;
  g.slot_stride = c.layout == 0 ? (int64_t)c.n_kv_heads * c.head_dim : c.head_dim;
  g.head_stride = c.layout == 0 ? c.head_dim : (int64_t)c.page_size * c.head_dim;
  h.pool_elems = (int64_t)(c.num_pages - 1) * c.page_stride + page;
  if (cudaGetDevice(&h.device) != cudaSuccess ||
      cudaDeviceGetAttribute(&h.sm_count, cudaDevAttrMultiProcessorCount, h.device) !=
          cudaSuccess) {
    cudaGetLastError();
    return CF_ERR_CUDA;
  }
  return CF_OK;
}

// Checks an attention call's arguments and fills in p; CF_OK or an error.  A
// call that has nothing to do leaves p.n_tokens 0.  scales: NULL but for a
// cache of 8-bit codes, whose caller has checked them.
inline int paged_host_attention(const PagedHost& h, int* errflag, int32_t batch, int32_t n_tokens,
                                int32_t max_q, const void* q, int64_t q_stride,
                                const int32_t* q_start, const int32_t* kv_len,
                                const int32_t* page_table, const int32_t* prefix_table,
                                int32_t prefix_len, const void* k_pages, const void* v_pages,
                                const float* scales, int32_t window, int32_t n_sinks, void* out,
                                float* lse, PagedAttnParams& p) {
  p.n_tokens = 0;
  const int rc = check_call(h, batch, n_tokens, q_start);
  if (rc != CF_OK) return rc;
  const cf_paged_config& c = h.cfg;
  if (window < 0 || n_sinks < 0) return CF_ERR_INVALID_ARG;
  if (prefix_len < 0 || prefix_len > (1 << 30)) return CF_ERR_INVALID_ARG;
  if (batch == 0 || n_tokens == 0) return CF_OK;
  if (q_start == nullptr) max_q = 1;
  if (max_q < 1 || max_q > n_tokens) return CF_ERR_INVALID_ARG;
  const size_t es = elem_size(c.dtype);
  const int64_t qrow = (int64_t)c.n_q_heads * c.head_dim;
  const void* need[] = {q, k_pages, v_pages, out};
  for (const void* p : need)
    if (p == nullptr || !aligned(p, 16)) return CF_ERR_INVALID_ARG;
  const void* ints[] = {kv_len, page_table, prefix_len > 0 ? prefix_table : kv_len};
  for (const void* p : ints)
    if (p == nullptr || !aligned(p, 4)) return CF_ERR_INVALID_ARG;
  if (!aligned(q_start, 4) || !aligned(lse, 4)) return CF_ERR_INVALID_ARG;
  if (q_stride < qrow || q_stride > max_stride(n_tokens) || (q_stride * (int64_t)es) % 16 != 0)
    return CF_ERR_INVALID_ARG;
  const size_t ob = (size_t)n_tokens * qrow * es, lb = (size_t)n_tokens * c.n_q_heads * 4;
  const size_t pool = h.pool_bytes();
  struct {
    const void* p;
    size_t n;
  } in[] = {{q, rows_bytes(n_tokens, q_stride, qrow, es)},
            {k_pages, pool},
            {v_pages, pool},
            {scales, scales ? h.scale_bytes() : 0},
            {q_start, ((size_t)batch + 1) * 4},
            {kv_len, (size_t)batch * 4},
            {page_table, (size_t)batch * c.max_pages * 4},
            {prefix_len > 0 ? prefix_table : nullptr,
             (((size_t)prefix_len + c.page_size - 1) / c.page_size) * 4}};
  for (const auto& x : in)
    if (overlap(out, ob, x.p, x.n) || overlap(lse, lb, x.p, x.n)) return CF_ERR_ALIAS;
  if (overlap(out, ob, lse, lb)) return CF_ERR_ALIAS;

  std::memset(&p, 0, sizeof(p));
  p.g = h.geom;
  p.q = q;
  p.k_pages = k_pages;
  p.v_pages = v_pages;
  p.scales = reinterpret_cast<const float2*>(scales);
  p.out = out;
  p.lse = lse;
  p.q_stride = q_stride;
  p.q_start = q_start;
  p.kv_len = kv_len;
  p.page_table = page_table;
  p.prefix_table = prefix_table;
  p.errflag = errflag;
  p.batch = batch;
  p.n_tokens = n_tokens;
  p.max_q = max_q;
  p.prefix_len = prefix_len;
  p.window = window < (1 << 30) ? window : 0;  // positions stay below 2^30
  p.n_sinks = n_sinks;
  p.scale_log2 = h.scale_log2;
  return CF_OK;
}

// The same of an append's.
inline int paged_host_append(const PagedHost& h, int* errflag, int32_t batch, int32_t n_tokens,
                             const void* q, const void* k, const void* v, int64_t q_stride,
                             int64_t kv_stride, const int32_t* q_start, const int32_t* kv_len,
                             const int32_t* rope_pos, const int32_t* page_table, void* k_pages,
                             void* v_pages, float* scales, void* q_out, int64_t q_out_stride,
                             PagedAppendParams& p) {
  p.n_tokens = 0;
  const int rc = check_call(h, batch, n_tokens, q_start);
  if (rc != CF_OK) return rc;
  const cf_paged_config& c = h.cfg;
  if (batch == 0 || n_tokens == 0) return CF_OK;
  const size_t es = elem_size(c.dtype);
  const int64_t qrow = (int64_t)c.n_q_heads * c.head_dim;
  const int64_t kvrow = (int64_t)c.n_kv_heads * c.head_dim;
  const void* need[] = {k, v, k_pages, v_pages};
  for (const void* p : need)
    if (p == nullptr || !aligned(p, 16)) return CF_ERR_INVALID_ARG;
  if ((q == nullptr) != (q_out == nullptr) || !aligned(q, 16) || !aligned(q_out, 16))
    return CF_ERR_INVALID_ARG;
  if (kv_len == nullptr || page_table == nullptr || !aligned(kv_len, 4) ||
      !aligned(page_table, 4) || !aligned(q_start, 4) || !aligned(rope_pos, 4))
    return CF_ERR_INVALID_ARG;
  auto bad_stride = [&](int64_t s, int64_t row) {
    return s < row || s > max_stride(n_tokens) || (s * (int64_t)es) % 16 != 0;
  };
  if (bad_stride(kv_stride, kvrow)) return CF_ERR_INVALID_ARG;
  if (q != nullptr && (bad_stride(q_stride, qrow) || bad_stride(q_out_stride, qrow)))
    return CF_ERR_INVALID_ARG;
  const bool axes3 = c.rope_sections[0] || c.rope_sections[1] || c.rope_sections[2];
  const size_t pool = h.pool_bytes();
  const size_t ns = scales ? h.scale_bytes() : 0;
  const size_t qo = q ? rows_bytes(n_tokens, q_out_stride, qrow, es) : 0;
  struct {
    const void* p;
    size_t n;
    bool rows;
  } in[] = {{q, q ? rows_bytes(n_tokens, q_stride, qrow, es) : 0, true},
            {k, rows_bytes(n_tokens, kv_stride, kvrow, es), true},
            {v, rows_bytes(n_tokens, kv_stride, kvrow, es), true},
            {q_start, ((size_t)batch + 1) * 4, false},
            {kv_len, (size_t)batch * 4, false},
            {rope_pos, (size_t)n_tokens * (axes3 ? 3 : 1) * 4, false},
            {page_table, (size_t)batch * c.max_pages * 4, false}};
  const bool in_place = q != nullptr && q == q_out && q_stride == q_out_stride;
  // in place the rotated rows may lie between the rows of k and v
  const bool between = in_place && (n_tokens == 1 || q_stride == kv_stride);
  for (const auto& x : in) {
    if (overlap(k_pages, pool, x.p, x.n) || overlap(v_pages, pool, x.p, x.n) ||
        overlap(scales, ns, x.p, x.n))
      return CF_ERR_ALIAS;
    if (in_place && &x == in) continue;  // q itself
    if (between && x.rows ? rows_meet(q, qrow * es, x.p, kvrow * es, n_tokens, q_stride * es)
                          : overlap(q_out, qo, x.p, x.n))
      return CF_ERR_ALIAS;
  }
  if (overlap(q_out, qo, k_pages, pool) || overlap(q_out, qo, v_pages, pool) ||
      overlap(q_out, qo, scales, ns) || overlap(scales, ns, k_pages, pool) ||
      overlap(scales, ns, v_pages, pool))
    return CF_ERR_ALIAS;
  // pools that interleave keys and values overlap as ranges, not as pages
  const int64_t page = (int64_t)c.page_size * kvrow;
  const int64_t pes = (int64_t)h.page_es;
  if (rows_meet(k_pages, page * pes, v_pages, page * pes, c.num_pages, c.page_stride * pes))
    return CF_ERR_ALIAS;

  std::memset(&p, 0, sizeof(p));
  p.g = h.geom;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_out = q_out;
  p.k_pages = k_pages;
  p.v_pages = v_pages;
  p.scales = reinterpret_cast<float2*>(scales);
  p.q_stride = q_stride;
  p.kv_stride = kv_stride;
  p.q_out_stride = q_out_stride;
  p.q_start = q_start;
  p.kv_len = kv_len;
  p.rope_pos = rope_pos;
  p.page_table = page_table;
  p.errflag = errflag;
  p.batch = batch;
  p.n_tokens = n_tokens;
  p.rope_dim = c.rope_dim;
  std::memcpy(p.turn, h.turn, sizeof(p.turn));
  std::memcpy(p.axis, h.axis, sizeof(p.axis));
  return CF_OK;
}

}  // namespace cf
