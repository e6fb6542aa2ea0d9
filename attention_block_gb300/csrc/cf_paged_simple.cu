// cf_paged_simple.cu -- attention over the paged cache on the CUDA cores.
//
// One block of four warps per (token, query head).  The keys the row sees
// form one list (prefix, sinks, window); the warps take chunks of 32 of it in
// turn.  A lane forms the whole dot product of one key; then every lane sums
// its columns of the 32 weighted values.  Each warp keeps a running maximum
// and sum (online softmax, base 2) and the four states are joined at the end.
// Masked positions are never loaded.
#include <cuda_runtime.h>

#include <cfloat>

#include "cf_paged.cuh"

using namespace cf;

namespace {

constexpr int kSimpleWarps = 4;

template <typename T, int D>
__global__ void __launch_bounds__(kSimpleWarps * 32)
    paged_attn_simple_kernel(const __grid_constant__ PagedAttnParams p) {
  constexpr int E = D / 32;       // columns of a lane
  constexpr int W = 16 / sizeof(T);
  __shared__ float s_q[D];
  __shared__ float s_o[kSimpleWarps][D];
  __shared__ float s_m[kSimpleWarps], s_l[kSimpleWarps];
  __shared__ int s_seq;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t t = blockIdx.x;
  const int h = blockIdx.y, kvh = h / p.g.G;

  if (tid == 0) s_seq = p.q_start ? -1 : (int)t;
  __syncthreads();
  if (p.q_start) {
    for (int b = tid; b < p.batch; b += kSimpleWarps * 32)
      if (p.q_start[b] <= t && t < p.q_start[b + 1]) s_seq = b;
    __syncthreads();
  }
  const int b = s_seq;
  if (b < 0) return;  // behind the last sequence
  for (int i = tid; i < D; i += kSimpleWarps * 32)
    s_q[i] = Elem<T>::to_f(
        static_cast<const T*>(p.q)[t * p.q_stride + (int64_t)h * D + i]);
  __syncthreads();

  const PagedSeq s =
      paged_seq(p.q_start, p.kv_len, b, p.n_tokens, p.max_q, p.g, p.errflag);
  if (s.n <= 0) return;
  const int pos = s.len - s.n + (int)(t - s.t0);
  const bool bad = s.n > p.max_q || s.len == 0;
  const PagedRange r = paged_range(pos, pos, s.len, p.window, p.n_sinks);
  const int own = pos < 0 || bad ? 0 : r.sink + (r.hi - r.lo);
  const int pre = pos < 0 ? 0 : p.prefix_len;
  const int total = pre + own;
  const int* table = p.page_table + (int64_t)b * p.g.max_pages;

  float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int base = warp * 32; base < total; base += kSimpleWarps * 32) {
    int idx = base + lane;
    int64_t off = -1;  // no page: zeros stand for the key and the value
    float sc = -INFINITY;
    if (idx < total) {
      sc = 0.f;
      if (idx < pre) {
        off = paged_offset(p.prefix_table, idx, p.g, p.errflag);
      } else {
        idx -= pre;
        off = paged_offset(table, idx < r.sink ? idx : r.lo + idx - r.sink, p.g, p.errflag);
      }
    }
    if (off >= 0) {
      off += (int64_t)kvh * p.g.head_stride;
      const T* k = static_cast<const T*>(p.k_pages) + off;
      float acc = 0.f;
#pragma unroll 4
      for (int i = 0; i < D; i += W) {
        float f[W];
        load_cvt<T, W>(k + i, f);
#pragma unroll
        for (int e = 0; e < W; ++e) acc = fmaf(f[e], s_q[i + e], acc);
      }
      sc = acc * p.scale_log2;
    }
    float mx = sc;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, d));
    const float m_new = fmaxf(m, mx);
    const float ref = m_new == -INFINITY ? 0.f : m_new;
    const float pr = exp2f(sc - ref), corr = exp2f(m - ref);
    m = m_new;
    l = l * corr + pr;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= corr;
    const int n = min(32, total - base);
    for (int k = 0; k < n; ++k) {
      const int64_t vo = __shfl_sync(~0u, off, k);
      const float w = __shfl_sync(~0u, pr, k);
      if (vo < 0) continue;
      float f[E];
      const T* v = static_cast<const T*>(p.v_pages) + vo + lane * E;
      if constexpr (E * sizeof(T) >= 4) load_cvt<T, E>(v, f);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(w, f[e], o[e]);
    }
  }
  l = warp_sum(l);
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  __syncthreads();
  float mt = -INFINITY;
#pragma unroll
  for (int w = 0; w < kSimpleWarps; ++w) mt = fmaxf(mt, s_m[w]);
  const float ref = mt == -INFINITY ? 0.f : mt;
  float lt = 0.f;
#pragma unroll
  for (int w = 0; w < kSimpleWarps; ++w) lt += s_l[w] * exp2f(s_m[w] - ref);
  const float inv = lt == 0.f ? 0.f : 1.f / lt;
  T* out = static_cast<T*>(p.out) + (t * p.g.nq + h) * D;
  for (int i = tid; i < D; i += kSimpleWarps * 32) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kSimpleWarps; ++w) v += s_o[w][i] * exp2f(s_m[w] - ref);
    out[i] = Elem<T>::from_f(v * inv);
  }
  if (p.lse && tid == 0)
    p.lse[t * p.g.nq + h] =
        mt == -INFINITY ? -INFINITY : (mt + log2f(lt)) * 0.69314718055994531f;
}

template <typename T>
bool launch(const PagedAttnParams& p, cudaStream_t st) {
  const dim3 grid(p.n_tokens, p.g.nq);
  if (p.g.D == 64)
    paged_attn_simple_kernel<T, 64><<<grid, kSimpleWarps * 32, 0, st>>>(p);
  else
    paged_attn_simple_kernel<T, 128><<<grid, kSimpleWarps * 32, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess;
}

}  // namespace

bool cf::paged_attn_simple_launch(int dtype, const PagedAttnParams& p, cudaStream_t st) {
  switch (dtype) {
    case CF_F32: return launch<float>(p, st);
    case CF_F16: return launch<__half>(p, st);
    default: return launch<__nv_bfloat16>(p, st);
  }
}
