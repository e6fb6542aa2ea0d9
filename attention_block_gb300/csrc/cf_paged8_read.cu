// cf_paged8_read.cu -- positions of a cache of 8-bit codes back as rows of
// fp16 or bf16 (cf_paged8_read).
//
// Bound by memory: per head d codes and a scale read, 2 d bytes written.  A
// block takes eight rows: a thread per row looks up where it lies (sequence by
// bisection of the starts, page), then 16 codes at a time are expanded by
// neighbouring threads, four loads ahead.  25,299 positions of 32 heads of 64: 56
// us, 5.6 TB/s (16 rows to a block 59, 32: 68; eight loads ahead 74, two 66).
#include <cuda_runtime.h>

#include <algorithm>

#include "cf_paged8.cuh"

using namespace cf;

namespace {

constexpr int kReadThreads = 256;
constexpr int kReadRows = 8;  // of a block
constexpr int kReadAhead = 4;  // loads of a thread on their way

template <typename T, int D, int CODE>
__global__ void __launch_bounds__(kReadThreads)
    paged8_read_kernel(const __grid_constant__ Paged8ReadParams p) {
  constexpr int C = D / 16;  // 16-byte pieces of a head's codes
  __shared__ int64_t s_code[kReadRows], s_scale[kReadRows];  // -1: zeros, -2: not a row
  __shared__ int s_seq[kReadRows];
  const int tid = threadIdx.x, r0 = blockIdx.x * kReadRows;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0)  // one block reports starts that are out of order
    for (int b = tid; b < p.batch; b += kReadThreads)
      if (!starts_ordered(p.row_start[b], p.row_start[b + 1], p.n_rows))
        atomicOr(p.errflag, kDevErrPosRange);
  // Whether sequence b has the row r.
  auto has = [&](int b, int r) {
    const int t0 = p.row_start[b], t1 = p.row_start[b + 1];
    return starts_ordered(t0, t1, p.n_rows) && t0 <= r && r < t1;
  };
  // Where row r0 + tid of sequence b lies.
  auto look_up = [&](int b) {
    int64_t code = -2, scale = -2;
    const long long j = (long long)(p.first ? p.first[b] : 0) + (r0 + tid - p.row_start[b]);
    if (j < 0 || j >= (long long)p.g.max_pages << p.g.page_shift) {
      atomicOr(p.errflag, kDevErrPosRange);
    } else {
      const int* table = p.page_table + (int64_t)b * p.g.max_pages;
      code = paged_offset(table, (int)j, p.g, p.errflag);
      if (code >= 0) scale = paged8_scale(table, (int)j, p.g);
    }
    s_code[tid] = code;
    s_scale[tid] = scale;
  };
  bool lost = false;  // the bisection finds no sequence for this thread's row
  if (tid < kReadRows) {
    const int r = r0 + tid;
    s_code[tid] = -2;
    s_seq[tid] = -1;
    if (r < p.n_rows) {
      // the last sequence whose start is at or before the row: those behind it
      // begin later
      int lo = 0, hi = p.batch;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (p.row_start[mid] <= r)
          lo = mid + 1;
        else
          hi = mid;
      }
      lost = lo == 0 || !has(lo - 1, r);
      if (!lost) look_up(lo - 1);
    }
  }
  if (__syncthreads_or(lost)) {
    // A row of no sequence or, where starts are out of order, of one that the
    // bisection passed by: all are asked.
    for (int b = tid; b < p.batch; b += kReadThreads) {
      const int t0 = p.row_start[b], t1 = p.row_start[b + 1];
      if (starts_ordered(t0, t1, p.n_rows))
        for (int r = max(t0, r0); r < min(t1, r0 + kReadRows); ++r) atomicMax(&s_seq[r - r0], b);
    }
    __syncthreads();
    if (lost && s_seq[tid] >= 0) look_up(s_seq[tid]);
    __syncthreads();
  }
  // A thread keeps to one piece of a head and walks over the heads of the rows'
  // keys and values, with several loads on their way.
  const int c = tid % C;
  constexpr int step = kReadThreads / C;  // heads of one step of the block
  int side = 0, h = tid / C;              // 2 * row, + 1: its values
  auto fit = [&]() {
    while (h >= p.g.nkv) {
      h -= p.g.nkv;
      ++side;
    }
  };
  fit();
  while (side < 2 * kReadRows) {
    uint4 w[kReadAhead];
    float scale[kReadAhead];
    void* to[kReadAhead];
#pragma unroll
    for (int i = 0; i < kReadAhead; ++i) {
      to[i] = nullptr;
      if (side < 2 * kReadRows) {
        const int row = side >> 1, kv = side & 1;
        void* out = kv ? p.v_out : p.k_out;
        const int64_t code = s_code[row];
        if (out != nullptr && code != -2)
          to[i] = static_cast<T*>(out) + (int64_t)(r0 + row) * p.out_stride + h * D + c * 16;
        w[i] = make_uint4(0, 0, 0, 0);
        scale[i] = 0.f;
        if (to[i] != nullptr && code >= 0) {
          const uint8_t* pool = static_cast<const uint8_t*>(kv ? p.v_pages : p.k_pages);
          w[i] = __ldcs(reinterpret_cast<const uint4*>(pool + code + (int64_t)h * p.g.head_stride +
                                                       c * 16));
          // (coherent, like the codes' load: the append in front may have begun to write them
          // when this launch was here already)
          scale[i] = (&p.scales[s_scale[row] + ((int64_t)h << p.g.page_shift)].x)[kv];
        }
      }
      h += step;
      fit();
    }
#pragma unroll
    for (int i = 0; i < kReadAhead; ++i) {
      if (to[i] == nullptr) continue;
      const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
      uint32_t o[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t first, last;
        code_row4<CODE>(v[e], first, last);
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&first));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&last));
        o[2 * e] = pack2<T>(a.x * scale[i], a.y * scale[i]);
        o[2 * e + 1] = pack2<T>(b.x * scale[i], b.y * scale[i]);
      }
      uint4* dst = static_cast<uint4*>(to[i]);
      dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
      dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

template <typename T, int D>
const void* read_fn(int code) {
  return code == CF_CODE_INT8 ? (const void*)&paged8_read_kernel<T, D, CF_CODE_INT8>
                              : (const void*)&paged8_read_kernel<T, D, CF_CODE_E4M3>;
}

}  // namespace

bool cf::paged8_read_launch(int dtype, int code, const Paged8ReadParams& p, cudaStream_t st) {
  const void* fn = dtype == CF_F16 ? (p.g.D == 64 ? read_fn<__half, 64>(code)
                                                  : read_fn<__half, 128>(code))
                                   : (p.g.D == 64 ? read_fn<__nv_bfloat16, 64>(code)
                                                  : read_fn<__nv_bfloat16, 128>(code));
  Paged8ReadParams pp = p;
  void* args[] = {&pp};
  return launch_pdl(fn, dim3((p.n_rows + kReadRows - 1) / kReadRows), kReadThreads, 0, st, args);
}
