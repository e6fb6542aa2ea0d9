// cf_paged_api.cu -- host side of include/cf_paged.h: argument checks, the
// handle and its workspace, and which kernel a call launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <new>

#include "cf_paged_host.h"

using namespace cf;

struct cf_paged_handle : PagedHost {
  void* ws = nullptr;
  int* errflag = nullptr;
  PagedSplit few, few_prefix, tc, tc_prefix;
};

namespace {

int attention(cf_paged_handle* h, int32_t batch, int32_t n_tokens, int32_t max_q, const void* q,
              int64_t q_stride, const int32_t* q_start, const int32_t* kv_len,
              const int32_t* page_table, const int32_t* prefix_table, int32_t prefix_len,
              const void* k_pages, const void* v_pages, int32_t window, int32_t n_sinks, void* out,
              float* lse, void* stream) {
  if (h == nullptr) return CF_ERR_INVALID_ARG;
  PagedAttnParams p;
  const int rc = paged_host_attention(*h, h->errflag, batch, n_tokens, max_q, q, q_stride, q_start,
                                      kv_len, page_table, prefix_table, prefix_len, k_pages,
                                      v_pages, nullptr, window, n_sinks, out, lse, p);
  if (rc != CF_OK || p.n_tokens == 0) return rc;
  const cf_paged_config& c = h->cfg;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // fp32 has no tensor-core form.  Up to 16 rows per KV head (tokens of one
  // sequence x grouped heads) share a tile of the few-row kernel; more go to
  // the tensor-core kernel, which takes 76 us for 54 with 4 rows (16 sequences
  // of 4097 positions) and 129 for 100 with 16 (32 of 4004).  For the prefix
  // the rows are the whole call's.
  bool ok;
  if (c.dtype == CF_F32) {
    ok = paged_f32_launch(p, h->few, st);
  } else {
    PagedPrefixParts pre;
    std::memset(&pre, 0, sizeof(pre));
    PagedMode mode = kOwn;
    ok = true;
    if (prefix_len > 0) {
      mode = kOwnAfterPrefix;
      if ((int64_t)n_tokens * p.g.G <= kFewRows) {
        pre = paged_few_prefix(p, h->few_prefix);
        ok = paged_few_launch(c.dtype, p, h->few_prefix, kPrefix, pre, st);
      } else {
        pre = paged_tc_prefix(p, h->tc_prefix);
        ok = paged_tc_launch(c.dtype, p, h->tc_prefix, kPrefix, pre, st);
      }
    }
    if (ok)
      ok = (int64_t)p.max_q * p.g.G <= kFewRows
               ? paged_few_launch(c.dtype, p, h->few, mode, pre, st)
               : paged_tc_launch(c.dtype, p, h->tc, mode, pre, st);
  }
  if (!ok) {
    cudaGetLastError();
    return CF_ERR_CUDA;
  }
  return CF_OK;
}

}  // namespace

extern "C" {

int cf_paged_create(const cf_paged_config* cfg, cf_paged_handle** out) {
  if (out == nullptr) return CF_ERR_INVALID_ARG;
  *out = nullptr;
  if (cfg == nullptr) return CF_ERR_INVALID_ARG;
  cf_paged_handle* h = new (std::nothrow) cf_paged_handle();
  if (h == nullptr) return CF_ERR_CUDA;
  auto fail = [&](int rc) {
    if (h->ws) cudaFree(h->ws);
    delete h;
    return rc;
  };
  const int rc = paged_host_init(*cfg, elem_size(cfg->dtype), *h);
  if (rc != CF_OK) return fail(rc);
  const cf_paged_config& c = h->cfg;
  size_t bytes = 256;
  auto take = [&](size_t n) {
    const size_t at = bytes;
    bytes += (n + 255) & ~(size_t)255;
    return at;
  };
  // The words that start at zero, then the lists, then two sets of states:
  // of the sequences' own keys and of the prefix.  A call uses one attention
  // kernel for each, so the kernels share them.
  h->few.grid = c.dtype == CF_F32 ? paged_f32_grid(c.head_dim, h->sm_count)
                                  : paged_few_grid(c.dtype, c.head_dim, h->sm_count);
  if (h->few.grid == 0) return fail(CF_ERR_CUDA);
  const size_t tickets =
      take(4 * (c.dtype == CF_F32 ? (size_t)h->few.grid + 1 : (size_t)c.max_batch * c.n_kv_heads));
  const size_t redo = take(3 * 4);
  const size_t zero = bytes;
  const int64_t all_rows = (int64_t)c.max_tokens * c.n_q_heads;
  size_t tc_list = 0, at_o[2] = {0, 0}, at_ml[2] = {0, 0};
  const int64_t few_rows = (int64_t)c.max_batch * c.n_kv_heads * kFewRows;
  int64_t slot_rows = 0;
  if (c.dtype != CF_F32) {
    slot_rows = paged_few_part_rows(h->few.grid);
    if ((int64_t)c.max_tokens * h->geom.G > kFewRows) {
      h->tc.grid = paged_tc_grid(c.dtype, c.head_dim, h->sm_count);
      if (h->tc.grid == 0) return fail(CF_ERR_CUDA);
      h->tc.items = ((int64_t)c.max_tokens * h->geom.G / kTcRows + c.max_batch) * c.n_kv_heads;
      tc_list = take(paged_tc_list_bytes(h->tc.grid, h->tc.items));
      slot_rows = std::max<int64_t>(slot_rows, paged_tc_part_rows(h->tc.grid));
    }
    // single rows: the sequences' own before a prefix's are joined, and a prefix's
    const int64_t rows[2] = {slot_rows + (h->tc.grid ? all_rows : std::min(all_rows, few_rows)),
                             slot_rows + all_rows};
    for (int i = 0; i < 2; ++i) {
      at_o[i] = take((size_t)rows[i] * c.head_dim * 4);
      at_ml[i] = take((size_t)rows[i] * 8);
    }
  } else {
    slot_rows = paged_f32_part_rows(h->few.grid);
    at_o[0] = take((size_t)slot_rows * c.head_dim * 4);
    at_ml[0] = take((size_t)slot_rows * 8);
  }
  if (cudaMalloc(&h->ws, bytes) != cudaSuccess) {
    cudaGetLastError();
    h->ws = nullptr;
    return fail(CF_ERR_CUDA);
  }
  if (!clear(h->ws, zero)) return fail(CF_ERR_CUDA);
  uint8_t* ws = static_cast<uint8_t*>(h->ws);
  h->errflag = reinterpret_cast<int*>(ws);
  const PagedParts own = {reinterpret_cast<float*>(ws + at_o[0]),
                          reinterpret_cast<float2*>(ws + at_ml[0]), slot_rows,
                          all_rows <= few_rows};
  const PagedParts prefix = {reinterpret_cast<float*>(ws + at_o[1]),
                             reinterpret_cast<float2*>(ws + at_ml[1]), slot_rows, 1};
  h->few.parts = h->tc.parts = own;
  h->few.tickets = reinterpret_cast<int*>(ws + tickets);
  h->tc.list = ws + tc_list;
  h->tc.tickets = reinterpret_cast<int*>(ws + redo);
  h->few_prefix.parts = h->tc_prefix.parts = prefix;
  h->few_prefix.grid = h->few.grid;
  h->tc_prefix.grid = h->tc.grid;
  *out = h;
  return CF_OK;
}

int cf_paged_append(cf_paged_handle* h, int32_t batch, int32_t n_tokens, const void* q,
                    const void* k, const void* v, int64_t q_stride, int64_t kv_stride,
                    const int32_t* q_start, const int32_t* kv_len, const int32_t* rope_pos,
                    const int32_t* page_table, void* k_pages, void* v_pages, void* q_out,
                    int64_t q_out_stride, void* stream) {
  if (h == nullptr) return CF_ERR_INVALID_ARG;
  PagedAppendParams p;
  const int rc = paged_host_append(*h, h->errflag, batch, n_tokens, q, k, v, q_stride, kv_stride,
                                   q_start, kv_len, rope_pos, page_table, k_pages, v_pages, nullptr,
                                   q_out, q_out_stride, p);
  if (rc != CF_OK || p.n_tokens == 0) return rc;
  if (!paged_append_launch(h->cfg.dtype, p, h->sm_count, static_cast<cudaStream_t>(stream))) {
    cudaGetLastError();
    return CF_ERR_CUDA;
  }
  return CF_OK;
}

int cf_paged_attention(cf_paged_handle* h, int32_t batch, int32_t n_tokens, int32_t max_q,
                       const void* q, int64_t q_stride, const int32_t* q_start,
                       const int32_t* kv_len, const int32_t* page_table, const void* k_pages,
                       const void* v_pages, int32_t window, int32_t n_sinks, void* out, float* lse,
                       void* stream) {
  return attention(h, batch, n_tokens, max_q, q, q_stride, q_start, kv_len, page_table, nullptr, 0,
                   k_pages, v_pages, window, n_sinks, out, lse, stream);
}

int cf_paged_prefix_attention(cf_paged_handle* h, int32_t batch, int32_t n_tokens, int32_t max_q,
                              const void* q, int64_t q_stride, const int32_t* q_start,
                              const int32_t* kv_len, const int32_t* page_table,
                              const int32_t* prefix_table, int32_t prefix_len,
                              const void* k_pages, const void* v_pages, void* out, float* lse,
                              void* stream) {
  return attention(h, batch, n_tokens, max_q, q, q_stride, q_start, kv_len, page_table,
                   prefix_table, prefix_len, k_pages, v_pages, 0, 0, out, lse, stream);
}

int cf_paged_get_status(cf_paged_handle* h) {
  if (h == nullptr) return CF_ERR_INVALID_ARG;
  int flag = 0;
  if (cudaMemcpy(&flag, h->errflag, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess)
    return CF_ERR_CUDA;
  if (flag != 0 && !clear(h->errflag, sizeof(int))) return CF_ERR_CUDA;
  if (flag & kDevErrTimeout) return CF_ERR_DEVICE_TIMEOUT;
  if (flag & kDevErrPosRange) return CF_ERR_DEVICE_POS_RANGE;
  return CF_OK;
}

void cf_paged_destroy(cf_paged_handle* h) {
  if (h == nullptr) return;
  if (h->ws) cudaFree(h->ws);
  delete h;
}

}  // extern "C"
