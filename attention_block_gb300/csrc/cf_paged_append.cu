// cf_paged_append.cu -- rotate new keys and queries and write keys and values
// to their pages (cf_paged_append).
//
// The rotation angle is kept as a fraction of a turn in 64-bit fixed point:
// pos * turn_i mod 2^64 is the exact fraction of pos times the host's
// float64 rate, so far positions lose no more than that rate's rounding (2^-24
// of a turn near 2^31); its top 32 bits go to sincospif as a float (2^-26).
// The cosines and sines of a token are formed once per block in shared memory
// and serve all of its heads.
//
// Bound by memory: each element is read once and written once as 16-byte
// vectors (9600 tokens, 32 + 2 x 8 heads of 128: 36 us, 5.5 TB/s, 0.81 of a
// copy's rate; a single token: 3 us, the launch).  A unit of work is two
// vectors of a head: the halves of W rotated pairs (i and i + r/2), or two
// vectors that are copied.  A thread keeps to one unit of a head and walks over
// the heads of the block's tokens; the first loads are under way before the
// block knows where its tokens go (sequence, length, page: loads that depend on
// one another).
#include <cuda_runtime.h>

#include "cf_paged.cuh"

using namespace cf;

namespace {

constexpr int kAppendThreads = 256;
// Units in flight per thread: few blocks want several, full SMs many warps
// with one each (9600 tokens, 32 + 2 x 8 heads of 128: 42 us with three, 36
// with one and eight blocks per SM; 400 tokens: 4.5 with three, 5.7 with one).
template <int TPB>
constexpr int kBatch = TPB == 1 ? 3 : 1;

template <typename T, int D, int TPB>
__global__ void __launch_bounds__(kAppendThreads, TPB == 1 ? 4 : 8)
    paged_append_kernel(const __grid_constant__ PagedAppendParams p) {
  constexpr int NB = kBatch<TPB>;
  constexpr int W = 16 / sizeof(T), UPH = D / (2 * W);  // units per head
  constexpr int RPI = kAppendThreads / UPH;             // heads per step of the block
  __shared__ float2 s_cs[TPB][kMaxPairs];
  __shared__ int s_seq[TPB], s_pos[TPB];
  __shared__ int64_t s_slot[TPB];
  const int tid = threadIdx.x, c = tid % UPH;
  const int t_lo = blockIdx.x * TPB;
  const int nt = min(TPB, p.n_tokens - t_lo);
  const int half = p.rope_dim >> 1;
  const int heads = p.g.nq + 2 * p.g.nkv;
  const int rows = nt * heads;                 // heads of all the block's tokens
  const int step = gridDim.y * RPI;
  pdl_wait();
  pdl_trigger();

  // this thread's two vectors of a rotated head, and of one that is copied
  const bool rot = c * W < half;
  const int r0 = rot ? c * W : p.rope_dim + 2 * (c * W - half), r1 = rot ? r0 + half : r0 + W;
  int row = blockIdx.y * RPI + tid / UPH;
  int tok = 0, h = row;
  while (h >= heads) {
    h -= heads;
    ++tok;
  }
  uint4 x[NB], y[NB];
  int bt[NB], bh[NB];
  auto load = [&]() {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      bt[i] = row < rows ? tok : -1;
      bh[i] = h;
      if (row < rows) {
        const int64_t t = t_lo + tok;
        const T* src;
        int e0 = r0, e1 = r1;
        if (h < p.g.nq) {
          src = static_cast<const T*>(p.q) + t * p.q_stride + (int64_t)h * D;
          if (p.q == nullptr) bt[i] = -1;
        } else if (h < p.g.nq + p.g.nkv) {
          src = static_cast<const T*>(p.k) + t * p.kv_stride + (int64_t)(h - p.g.nq) * D;
        } else {
          src = static_cast<const T*>(p.v) + t * p.kv_stride + (int64_t)(h - p.g.nq - p.g.nkv) * D;
          e0 = c * W;
          e1 = e0 + D / 2;
        }
        if (bt[i] >= 0) {
          x[i] = *reinterpret_cast<const uint4*>(src + e0);
          y[i] = *reinterpret_cast<const uint4*>(src + e1);
        }
      }
      row += step;
      h += step;
      while (h >= heads) {
        h -= heads;
        ++tok;
      }
    }
  };
  load();

  // ---- where the tokens go, and their angles
  if (tid < TPB) s_seq[tid] = p.q_start ? -1 : t_lo + tid;
  if (p.q_start) {
    __syncthreads();
    for (int b = tid; b < p.batch; b += kAppendThreads) {
      const int t0 = p.q_start[b], t1 = p.q_start[b + 1];
      if (!starts_ordered(t0, t1, p.n_tokens)) {  // claims no token; one block reports it
        if (blockIdx.x + blockIdx.y == 0) atomicOr(p.errflag, kDevErrPosRange);
        continue;
      }
      const int a = max(t0, t_lo), e = min(t1, t_lo + nt);
      for (int t = a; t < e; ++t) atomicMax(&s_seq[t - t_lo], b);
    }
  }
  __syncthreads();
  if (tid < nt) {
    const int b = s_seq[tid];
    int64_t slot = -1;
    int pos = 0;
    if (b >= 0) {
      const PagedSeq s = paged_seq(p.q_start, p.kv_len, b, p.n_tokens, p.n_tokens, p.g, p.errflag);
      pos = s.len - s.n + (t_lo + tid - s.t0);
      if (s.n <= 0 || pos < 0 || pos >= s.len)
        atomicOr(p.errflag, kDevErrPosRange);
      else
        slot = paged_offset(p.page_table + (int64_t)b * p.g.max_pages, pos, p.g, p.errflag);
    }
    s_slot[tid] = slot;
    s_pos[tid] = pos;
  }
  __syncthreads();
  for (int i = tid; i < nt * half; i += kAppendThreads) {
    const int t = i / half, j = i - t * half;
    const int P =
        p.rope_pos ? p.rope_pos[(int64_t)p.axis[j] * p.n_tokens + t_lo + t] : s_pos[t];
    const uint64_t f = (uint64_t)(int64_t)P * p.turn[j];
    const float turns = (float)(int32_t)(uint32_t)(f >> 32) * 0x1p-32f;
    float2 cs;
    sincospif(2.0f * turns, &cs.y, &cs.x);
    s_cs[t][j] = cs;
  }
  __syncthreads();

  while (true) {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      if (bt[i] < 0 || s_slot[bt[i]] < 0) continue;
      const int64_t t = t_lo + bt[i];
      T* dst;
      int e0 = r0, e1 = r1;
      bool turn = rot;
      if (bh[i] < p.g.nq) {
        dst = static_cast<T*>(p.q_out) + t * p.q_out_stride + (int64_t)bh[i] * D;
      } else if (bh[i] < p.g.nq + p.g.nkv) {
        dst = static_cast<T*>(p.k_pages) + s_slot[bt[i]] + (bh[i] - p.g.nq) * p.g.head_stride;
      } else {
        dst = static_cast<T*>(p.v_pages) + s_slot[bt[i]] +
              (bh[i] - p.g.nq - p.g.nkv) * p.g.head_stride;
        e0 = c * W;
        e1 = e0 + D / 2;
        turn = false;
      }
      if (turn) {
        float a[W], b[W];
        Elem<T>::words(reinterpret_cast<const uint32_t*>(&x[i]), 4, a);
        Elem<T>::words(reinterpret_cast<const uint32_t*>(&y[i]), 4, b);
        T o0[W], o1[W];
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const float2 cs = s_cs[bt[i]][c * W + e];
          o0[e] = Elem<T>::from_f(a[e] * cs.x - b[e] * cs.y);
          o1[e] = Elem<T>::from_f(b[e] * cs.x + a[e] * cs.y);
        }
        x[i] = *reinterpret_cast<const uint4*>(o0);
        y[i] = *reinterpret_cast<const uint4*>(o1);
      }
      *reinterpret_cast<uint4*>(dst + e0) = x[i];
      *reinterpret_cast<uint4*>(dst + e1) = y[i];
    }
    if (row >= rows) break;
    load();
  }
}

template <typename T, int D, int TPB>
bool launch_n(const PagedAppendParams& p, int gy, cudaStream_t st) {
  PagedAppendParams pp = p;
  void* args[] = {&pp};
  return launch_pdl((const void*)&paged_append_kernel<T, D, TPB>,
                    dim3((p.n_tokens + TPB - 1) / TPB, gy, 1), kAppendThreads, 0, st, args);
}

template <typename T, int D>
bool launch(const PagedAppendParams& p, int sm_count, cudaStream_t st) {
  // Few tokens: one per block, its heads over several blocks of one step each
  // while the GPU has room.  Many: four per block.
  if (p.n_tokens >= 8 * sm_count) return launch_n<T, D, 4>(p, 1, st);
  constexpr int RPI = kAppendThreads / (D / (2 * (16 / (int)sizeof(T))));
  const int steps = (p.g.nq + 2 * p.g.nkv + RPI - 1) / RPI;
  return launch_n<T, D, 1>(p, p.n_tokens <= sm_count ? steps : (steps + kBatch<1> - 1) / kBatch<1>, st);
}
template <typename T>
bool launch_d(const PagedAppendParams& p, int sm_count, cudaStream_t st) {
  return p.g.D == 64 ? launch<T, 64>(p, sm_count, st) : launch<T, 128>(p, sm_count, st);
}

}  // namespace

bool cf::paged_append_launch(int dtype, const PagedAppendParams& p, int sm_count,
                             cudaStream_t st) {
  switch (dtype) {
    case CF_F32: return launch_d<float>(p, sm_count, st);
    case CF_F16: return launch_d<__half>(p, sm_count, st);
    default: return launch_d<__nv_bfloat16>(p, sm_count, st);
  }
}
