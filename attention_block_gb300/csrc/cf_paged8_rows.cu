// cf_paged8_rows.cu -- attention over a paged cache of 8-bit codes, one warp to
// a row on the CUDA cores (cf_paged8_attention).
//
// A lane forms the whole dot product of one key; then every lane sums its
// columns of 32 weighted values.  Masked positions are never loaded.
#include <cuda_runtime.h>

#include "cf_paged8.cuh"

using namespace cf;

namespace {

constexpr int kRowWarps = 4;

template <typename T, int D, int CODE>
__global__ void __launch_bounds__(kRowWarps * 32)
    paged8_rows_kernel(const __grid_constant__ PagedAttnParams p) {
  constexpr int E = D / 32;  // columns of a lane
  __shared__ float s_q[kRowWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * kRowWarps + warp;
  pdl_wait();
  pdl_trigger();
  if (row >= (long long)p.n_tokens * p.g.nq) return;
  const int t = (int)(row / p.g.nq), h = (int)(row - (long long)t * p.g.nq), kvh = h / p.g.G;
  int b = p.q_start ? -1 : t;
  for (int i = lane; p.q_start && i < p.batch; i += 32)
    if (starts_ordered(p.q_start[i], p.q_start[i + 1], p.n_tokens)) {
      if (p.q_start[i] <= t && t < p.q_start[i + 1]) b = i;
    } else {
      atomicOr(p.errflag, kDevErrPosRange);
    }
  b = __reduce_max_sync(~0u, b);
  if (b < 0) return;
  const PagedSeq s = paged_seq(p.q_start, p.kv_len, b, p.n_tokens, p.max_q, p.g, p.errflag);
  const int pos = s.len - s.n + t - s.t0;
  const PagedRange r = paged_range(pos, pos, s.len, p.window, p.n_sinks);
  const int total = pos < 0 ? 0 : r.sink + r.hi - r.lo;
  const int* table = p.page_table + (int64_t)b * p.g.max_pages;
  float* q = s_q[warp];
  for (int c = lane; c < D; c += 32)
    q[c] = Elem<T>::to_f(static_cast<const T*>(p.q)[(int64_t)t * p.q_stride + (int64_t)h * D + c]);
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int base = 0; base < total; base += 32) {
    const int idx = base + lane;
    int64_t off = -1;  // no page: zeros stand for the key and the value
    float sc = -INFINITY, vs = 0.f;
    if (idx < total) {
      sc = 0.f;
      const int j = idx < r.sink ? idx : r.lo + idx - r.sink;
      off = paged_offset(table, j, p.g, p.errflag);
      if (off >= 0) {
        const float2 ks = p.scales[paged8_scale(table, j, p.g) + ((int64_t)kvh << p.g.page_shift)];
        off += (int64_t)kvh * p.g.head_stride;
        const uint4* k = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.k_pages) + off);
        float acc = 0.f;
        for (int i = 0; i < D / 16; ++i) {
          const uint4 w4 = k[i];
          const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t even, odd;
            code_halves<CODE>(w[e], even, odd);
            const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&even));
            const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&odd));
            const float* qq = q + i * 16 + e * 4;
            acc = fmaf(x.x, qq[0], acc);
            acc = fmaf(y.x, qq[1], acc);
            acc = fmaf(x.y, qq[2], acc);
            acc = fmaf(y.y, qq[3], acc);
          }
        }
        sc = acc * (ks.x * kCodeUnit<CODE> * p.scale_log2);
        vs = ks.y * kCodeUnit<CODE>;
      }
    }
    float mx = sc;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, d));
    const float m_new = fmaxf(m, mx), ref = m_new == -INFINITY ? 0.f : m_new;
    const float pr = exp2f(sc - ref), corr = exp2f(m - ref), w = off >= 0 ? pr * vs : 0.f;
    m = m_new;
    l = l * corr + pr;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= corr;
    const int n = min(32, total - base);
    for (int k = 0; k < n; ++k) {
      const int64_t vo = __shfl_sync(~0u, off, k);
      const float wk = __shfl_sync(~0u, w, k);
      if (vo < 0) continue;
      const uint8_t* v = static_cast<const uint8_t*>(p.v_pages) + vo + lane * E;
      uint32_t x = E == 4 ? *reinterpret_cast<const uint32_t*>(v)
                          : *reinterpret_cast<const uint16_t*>(v);
      uint32_t even, odd;
      code_halves<CODE>(x, even, odd);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&even));
      const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&odd));
      const float vv[4] = {f.x, g.x, f.y, g.y};
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(wk, vv[e], o[e]);
    }
  }
  l = warp_sum(l);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* out = static_cast<T*>(p.out) + row * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = Elem<T>::from_f(o[e] * inv);
  if (p.lse && lane == 0) p.lse[row] = paged_lse(m, l);
}

template <typename T, int D>
const void* rows_fn(int code) {
  return code == CF_CODE_INT8 ? (const void*)&paged8_rows_kernel<T, D, CF_CODE_INT8>
                              : (const void*)&paged8_rows_kernel<T, D, CF_CODE_E4M3>;
}

}  // namespace

bool cf::paged8_rows_launch(int dtype, int code, const PagedAttnParams& p, cudaStream_t st) {
  const void* fn = dtype == CF_F16 ? (p.g.D == 64 ? rows_fn<__half, 64>(code)
                                                  : rows_fn<__half, 128>(code))
                                   : (p.g.D == 64 ? rows_fn<__nv_bfloat16, 64>(code)
                                                  : rows_fn<__nv_bfloat16, 128>(code));
  PagedAttnParams pp = p;
  void* args[] = {&pp};
  const long long rows = (long long)p.n_tokens * p.g.nq;
  return launch_pdl(fn, dim3((unsigned)((rows + kRowWarps - 1) / kRowWarps)), kRowWarps * 32, 0, st,
                    args);
}
