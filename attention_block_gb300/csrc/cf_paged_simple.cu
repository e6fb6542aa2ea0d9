// cf_paged_simple.cu -- attention over the paged cache on the CUDA cores.
//
// One block of four warps per (token, query head); the warps take chunks of 32
// of the keys that the row sees in turn (PagedRow), keep a running maximum and
// sum each (online softmax, base 2), and the four states are joined at the
// end.  fp32 storage has no tensor-core form that keeps its precision; this
// one is for checking models, and bound by the CUDA cores and latency.
#include <cuda_runtime.h>

#include <cfloat>

#include "cf_paged.cuh"

using namespace cf;

namespace {

constexpr int kSimpleWarps = 4;

template <typename T, int D>
__global__ void __launch_bounds__(kSimpleWarps * 32)
    paged_attn_simple_kernel(const __grid_constant__ PagedAttnParams p) {
  constexpr int E = D / 32;  // columns of a lane
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
  // (a sequence with more tokens than the call allows has length 0: pos < 0)
  PagedRow<T, D> x;
  x.run(p, s_q, b, pos, s.len, kvh, warp, kSimpleWarps);
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = x.o[e];
  if (lane == 0) {
    s_m[warp] = x.m;
    s_l[warp] = x.l;
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
