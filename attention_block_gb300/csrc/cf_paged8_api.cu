// cf_paged8_api.cu -- host side of include/cf_paged8.h: argument checks, the
// handle and its workspace, and which kernel a call launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <new>

#include "cf_paged8.cuh"
#include "cf_paged_host.h"

using namespace cf;

struct cf_paged8_handle : PagedHost {
  int code = 0;
  void* ws = nullptr;
  int* errflag = nullptr;
  PagedSplit few, tc;
};

extern "C" {

int cf_paged8_create(const cf_paged8_config* cfg, cf_paged8_handle** out) {
  if (out == nullptr) return CF_ERR_INVALID_ARG;
  *out = nullptr;
  if (cfg == nullptr || cfg->code < CF_CODE_INT8 || cfg->code > CF_CODE_E4M3)
    return CF_ERR_INVALID_ARG;
  if (cfg->cache.dtype == CF_F32) return CF_ERR_UNSUPPORTED;
  cf_paged8_handle* h = new (std::nothrow) cf_paged8_handle();
  if (h == nullptr) return CF_ERR_CUDA;
  auto fail = [&](int rc) {
    if (h->ws) cudaFree(h->ws);
    delete h;
    return rc;
  };
  const int rc = paged_host_init(cfg->cache, 1, *h);
  if (rc != CF_OK) return fail(rc);
  h->code = cfg->code;
  size_t bytes = 256;
  auto take = [&](size_t n) {
    const size_t at = bytes;
    bytes += (n + 255) & ~(size_t)255;
    return at;
  };
  // The words that start at zero, then the states of split items.
  const cf_paged_config& c = h->cfg;
  h->few.grid = paged8_few_grid(c.dtype, h->code, c.head_dim, h->sm_count);
  if (h->few.grid == 0) return fail(CF_ERR_CUDA);
  const size_t tickets = take(4 * (size_t)c.max_batch * c.n_kv_heads);
  const size_t zero = bytes;
  long long rows = paged_few_part_rows(h->few.grid);
  size_t list = 0;
  if ((int64_t)c.max_tokens * h->geom.G > kFewRows) {
    h->tc.grid = paged8_tc_grid(c.dtype, h->code, c.head_dim, h->sm_count);
    if (h->tc.grid == 0) return fail(CF_ERR_CUDA);
    list = take(paged8_tc_list_bytes(h->tc.grid));
    rows = std::max(rows, paged_tc_part_rows(h->tc.grid));
  }
  const size_t at_o = take((size_t)rows * c.head_dim * 4), at_ml = take((size_t)rows * 8);
  if (cudaMalloc(&h->ws, bytes) != cudaSuccess) {
    cudaGetLastError();
    h->ws = nullptr;
    return fail(CF_ERR_CUDA);
  }
  if (!clear(h->ws, zero)) return fail(CF_ERR_CUDA);
  uint8_t* ws = static_cast<uint8_t*>(h->ws);
  h->errflag = reinterpret_cast<int*>(ws);
  // (a call uses one of the two kernels)
  h->few.parts = h->tc.parts = {reinterpret_cast<float*>(ws + at_o),
                                reinterpret_cast<float2*>(ws + at_ml), rows, 0};
  h->tc.list = ws + list;
  h->few.tickets = reinterpret_cast<int*>(ws + tickets);
  *out = h;
  return CF_OK;
}

int cf_paged8_append(cf_paged8_handle* h, int32_t batch, int32_t n_tokens, const void* q,
                     const void* k, const void* v, int64_t q_stride, int64_t kv_stride,
                     const int32_t* q_start, const int32_t* kv_len, const int32_t* rope_pos,
                     const int32_t* page_table, void* k_pages, void* v_pages, float* scales,
                     void* q_out, int64_t q_out_stride, void* stream) {
  if (h == nullptr) return CF_ERR_INVALID_ARG;
  if (batch > 0 && n_tokens > 0 && (scales == nullptr || !aligned(scales, 8)))
    return CF_ERR_INVALID_ARG;
  PagedAppendParams p;
  const int rc = paged_host_append(*h, h->errflag, batch, n_tokens, q, k, v, q_stride, kv_stride,
                                   q_start, kv_len, rope_pos, page_table, k_pages, v_pages, scales,
                                   q_out, q_out_stride, p);
  if (rc != CF_OK || p.n_tokens == 0) return rc;
  if (!paged8_append_launch(h->cfg.dtype, h->code, p, h->sm_count,
                            static_cast<cudaStream_t>(stream))) {
    cudaGetLastError();
    return CF_ERR_CUDA;
  }
  return CF_OK;
}

int cf_paged8_attention(cf_paged8_handle* h, int32_t batch, int32_t n_tokens, int32_t max_q,
                        const void* q, int64_t q_stride, const int32_t* q_start,
                        const int32_t* kv_len, const int32_t* page_table, const void* k_pages,
                        const void* v_pages, const float* scales, int32_t window, int32_t n_sinks,
                        void* out, float* lse, void* stream) {
  if (h == nullptr) return CF_ERR_INVALID_ARG;
  if (batch > 0 && n_tokens > 0 && (scales == nullptr || !aligned(scales, 8)))
    return CF_ERR_INVALID_ARG;
  PagedAttnParams p;
  const int rc = paged_host_attention(*h, h->errflag, batch, n_tokens, max_q, q, q_stride, q_start,
                                      kv_len, page_table, nullptr, 0, k_pages, v_pages, scales,
                                      window, n_sinks, out, lse, p);
  if (rc != CF_OK || p.n_tokens == 0) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // Up to 16 rows per KV head (tokens of one sequence x grouped heads) go to the
  // few-row kernel; more to the many-row kernel, which takes 99 us for 35 with 4
  // rows (16 sequences of 4097 positions) and 117 for 63 with 16 (32 of 1070-4093).
  if (!((int64_t)p.max_q * p.g.G <= kFewRows
            ? paged8_few_launch(h->cfg.dtype, h->code, p, h->few, st)
            : paged8_tc_launch(h->cfg.dtype, h->code, p, h->tc, st))) {
    cudaGetLastError();
    return CF_ERR_CUDA;
  }
  return CF_OK;
}

int cf_paged8_read(cf_paged8_handle* h, int32_t batch, int32_t n_rows, const int32_t* row_start,
                   const int32_t* first, const int32_t* page_table, const void* k_pages,
                   const void* v_pages, const float* scales, void* k_out, void* v_out,
                   int64_t out_stride, void* stream) {
  if (h == nullptr) return CF_ERR_INVALID_ARG;
  if (n_rows < 0 || n_rows > (1 << 30)) return CF_ERR_INVALID_ARG;
  // (check_call bounds n_tokens by max_tokens; rows have no such bound)
  const int rc = check_call(*h, batch, 0, row_start);
  if (rc != CF_OK) return rc;
  if (batch == 0 || n_rows == 0) return CF_OK;
  const cf_paged_config& c = h->cfg;
  const void* ints[] = {row_start, page_table};
  for (const void* p : ints)
    if (p == nullptr || !aligned(p, 4)) return CF_ERR_INVALID_ARG;
  if (!aligned(first, 4) || scales == nullptr || !aligned(scales, 8)) return CF_ERR_INVALID_ARG;
  const void* pools[] = {k_pages, v_pages};
  for (const void* p : pools)
    if (p == nullptr || !aligned(p, 16)) return CF_ERR_INVALID_ARG;
  if ((k_out == nullptr && v_out == nullptr) || !aligned(k_out, 16) || !aligned(v_out, 16))
    return CF_ERR_INVALID_ARG;
  const int64_t row = (int64_t)c.n_kv_heads * c.head_dim;
  if (out_stride < row || out_stride > max_stride(n_rows) || out_stride % 8 != 0)
    return CF_ERR_INVALID_ARG;
  const size_t ob = rows_bytes(n_rows, out_stride, row, 2), pool = h->pool_bytes();
  struct {
    const void* p;
    size_t n;
  } in[] = {{k_pages, pool},
            {v_pages, pool},
            {scales, h->scale_bytes()},
            {row_start, ((size_t)batch + 1) * 4},
            {first, first ? (size_t)batch * 4 : 0},
            {page_table, (size_t)batch * c.max_pages * 4}};
  for (const auto& x : in)
    if (overlap(k_out, ob, x.p, x.n) || overlap(v_out, ob, x.p, x.n)) return CF_ERR_ALIAS;
  // keys and values may lie side by side in one row
  if (k_out && v_out && rows_meet(k_out, row * 2, v_out, row * 2, n_rows, out_stride * 2))
    return CF_ERR_ALIAS;
  Paged8ReadParams p;
  p.g = h->geom;
  p.k_pages = k_pages;
  p.v_pages = v_pages;
  p.scales = reinterpret_cast<const float2*>(scales);
  p.row_start = row_start;
  p.first = first;
  p.page_table = page_table;
  p.k_out = k_out;
  p.v_out = v_out;
  p.out_stride = out_stride;
  p.errflag = h->errflag;
  p.batch = batch;
  p.n_rows = n_rows;
  if (!paged8_read_launch(c.dtype, h->code, p, static_cast<cudaStream_t>(stream))) {
    cudaGetLastError();
    return CF_ERR_CUDA;
  }
  return CF_OK;
}

int cf_paged8_get_status(cf_paged8_handle* h) {
  if (h == nullptr) return CF_ERR_INVALID_ARG;
  int flag = 0;
  if (cudaMemcpy(&flag, h->errflag, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess)
    return CF_ERR_CUDA;
  if (flag != 0 && !clear(h->errflag, sizeof(int))) return CF_ERR_CUDA;
  if (flag & kDevErrTimeout) return CF_ERR_DEVICE_TIMEOUT;
  if (flag & kDevErrPosRange) return CF_ERR_DEVICE_POS_RANGE;
  return CF_OK;
}

void cf_paged8_destroy(cf_paged8_handle* h) {
  if (h == nullptr) return;
  if (h->ws) cudaFree(h->ws);
  delete h;
}

}  // extern "C"
