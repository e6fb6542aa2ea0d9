// cf_paged_append.cu -- rotate new keys and queries and write keys and values
// to their pages (cf_paged_append).
//
// The rotation angle is kept as a fraction of a turn in 64-bit fixed point:
// pos * turn_i mod 2^64 is the exact fraction of pos times the host's
// float64 rate, so far positions lose nothing; its top 32 bits go to
// sincospif.  The cosines and sines of a token are formed once per block in
// shared memory and serve all of its heads.
//
// Bound by memory: each element is read once and written once as 16-byte
// vectors.  A unit of work is two vectors: the two halves of W rotated pairs
// (i and i + r/2), or two vectors that are copied.
#include <cuda_runtime.h>

#include "cf_paged.cuh"

using namespace cf;

namespace {

constexpr int kAppendThreads = 128;
constexpr int kMaxTok = 4;  // tokens per block

template <typename T>
__global__ void __launch_bounds__(kAppendThreads)
    paged_append_kernel(const __grid_constant__ PagedAppendParams p, int tok_per_block) {
  constexpr int W = 16 / sizeof(T);
  __shared__ float2 s_cs[kMaxTok][kMaxPairs];
  __shared__ int s_seq[kMaxTok];
  const int tid = threadIdx.x;
  const int t_lo = blockIdx.x * tok_per_block;
  const int nt = min(tok_per_block, p.n_tokens - t_lo);
  const int half = p.rope_dim >> 1;

  if (tid < kMaxTok) s_seq[tid] = p.q_start ? -1 : t_lo + tid;
  __syncthreads();
  if (p.q_start) {
    for (int b = tid; b < p.batch; b += kAppendThreads) {
      const int a = max(p.q_start[b], t_lo), e = min(p.q_start[b + 1], t_lo + nt);
      for (int t = a; t < e; ++t) s_seq[t - t_lo] = b;
    }
    __syncthreads();
  }
  // position, slot and validity of each token (every thread for itself: the
  // loads hit the same addresses)
  int64_t slot[kMaxTok];
  int pos[kMaxTok];
#pragma unroll
  for (int i = 0; i < kMaxTok; ++i) {
    slot[i] = -1;
    pos[i] = 0;
    if (i >= nt || s_seq[i] < 0) continue;
    const int b = s_seq[i];
    const PagedSeq s = paged_seq(p.q_start, p.kv_len, b, p.n_tokens, p.n_tokens, p.g, p.errflag);
    pos[i] = s.len - s.n + (t_lo + i - s.t0);
    if (s.n <= 0 || pos[i] < 0 || pos[i] >= s.len) {
      atomicOr(p.errflag, kDevErrPosRange);
      continue;
    }
    slot[i] = paged_offset(p.page_table + (int64_t)b * p.g.max_pages, pos[i], p.g, p.errflag);
  }
#pragma unroll
  for (int i = 0; i < kMaxTok; ++i) {
    if (i >= nt || slot[i] < 0) continue;
    for (int c = tid; c < half; c += kAppendThreads) {
      const int P = p.rope_pos ? p.rope_pos[(int64_t)p.axis[c] * p.n_tokens + t_lo + i] : pos[i];
      const uint64_t f = (uint64_t)(int64_t)P * p.turn[c];
      const float turns = (float)(int32_t)(uint32_t)(f >> 32) * 0x1p-32f;
      float2 cs;
      sincospif(2.0f * turns, &cs.y, &cs.x);
      s_cs[i][c] = cs;
    }
  }
  __syncthreads();

  const int upd = p.g.D / (2 * W);  // units per head
  const int heads = p.g.nq + 2 * p.g.nkv;
  const int per_tok = heads * upd;
#pragma unroll
  for (int i = 0; i < kMaxTok; ++i) {
    if (i >= nt || slot[i] < 0) continue;
    const int64_t t = t_lo + i;
    for (int u = blockIdx.y * kAppendThreads + tid; u < per_tok; u += gridDim.y * kAppendThreads) {
      const int h = u / upd, c = u - h * upd;
      const T* src;
      T* dst;
      bool rot = c * W < half;
      if (h < p.g.nq) {
        if (p.q == nullptr) continue;
        src = static_cast<const T*>(p.q) + t * p.q_stride + (int64_t)h * p.g.D;
        dst = static_cast<T*>(p.q_out) + t * p.q_out_stride + (int64_t)h * p.g.D;
      } else if (h < p.g.nq + p.g.nkv) {
        const int k = h - p.g.nq;
        src = static_cast<const T*>(p.k) + t * p.kv_stride + (int64_t)k * p.g.D;
        dst = static_cast<T*>(p.k_pages) + slot[i] + k * p.g.head_stride;
      } else {
        const int k = h - p.g.nq - p.g.nkv;
        src = static_cast<const T*>(p.v) + t * p.kv_stride + (int64_t)k * p.g.D;
        dst = static_cast<T*>(p.v_pages) + slot[i] + k * p.g.head_stride;
        rot = false;
      }
      // the unit's two vectors: (c, c + r/2) where rotated; past the rotated
      // part of a q or k head, and for v, two neighbours
      const bool head_rot = h < p.g.nq + p.g.nkv;
      const int e0 = head_rot ? (rot ? c * W : p.rope_dim + 2 * (c * W - half)) : 2 * c * W;
      const int e1 = rot ? e0 + half : e0 + W;
      uint4 a = *reinterpret_cast<const uint4*>(src + e0);
      uint4 b = *reinterpret_cast<const uint4*>(src + e1);
      if (rot) {
        float x[W], y[W];
        Elem<T>::words(reinterpret_cast<const uint32_t*>(&a), 4, x);
        Elem<T>::words(reinterpret_cast<const uint32_t*>(&b), 4, y);
        T o0[W], o1[W];
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const float2 cs = s_cs[i][c * W + e];
          o0[e] = Elem<T>::from_f(x[e] * cs.x - y[e] * cs.y);
          o1[e] = Elem<T>::from_f(y[e] * cs.x + x[e] * cs.y);
        }
        a = *reinterpret_cast<const uint4*>(o0);
        b = *reinterpret_cast<const uint4*>(o1);
      }
      *reinterpret_cast<uint4*>(dst + e0) = a;
      *reinterpret_cast<uint4*>(dst + e1) = b;
    }
  }
}

template <typename T>
bool launch(const PagedAppendParams& p, int sm_count, cudaStream_t st) {
  constexpr int W = 16 / sizeof(T);
  // Few tokens: a token's heads are spread over several blocks, one unit per
  // thread; many: four tokens per block.
  const int units = (p.g.nq + 2 * p.g.nkv) * (p.g.D / (2 * W));
  const int need = (units + kAppendThreads - 1) / kAppendThreads;
  const int tpb = p.n_tokens >= 16 * sm_count ? kMaxTok : 1;
  const int gx = (p.n_tokens + tpb - 1) / tpb;
  const int gy = gx >= 16 * sm_count ? 1 : need;
  paged_append_kernel<T><<<dim3(gx, gy), kAppendThreads, 0, st>>>(p, tpb);
  return cudaGetLastError() == cudaSuccess;
}

}  // namespace

bool cf::paged_append_launch(int dtype, const PagedAppendParams& p, int sm_count,
                             cudaStream_t st) {
  switch (dtype) {
    case CF_F32: return launch<float>(p, sm_count, st);
    case CF_F16: return launch<__half>(p, sm_count, st);
    default: return launch<__nv_bfloat16>(p, sm_count, st);
  }
}
