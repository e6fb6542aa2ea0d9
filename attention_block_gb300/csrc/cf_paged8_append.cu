// cf_paged8_append.cu -- rotate new keys and queries, and write the 8-bit codes
// and scales of keys and values to their pages (cf_paged8_append).
//
// Units, angles and lookups are those of cf_paged_append.cu.  The threads of a
// head hold all of it, 16 elements each, find its largest magnitude by shuffles
// and write 8-byte pieces of codes; the first of them writes the scale.
//
// Bound by the reads that are on their way, with issue at half of what it can: 8063
// tokens, 32 + 2 x 8 heads of 128: 41 us, 4.5 TB/s, with five blocks on an SM (48
// registers; half as long again with the eight of cf_paged_append.cu, which spill,
// 43 for 40 with four); a single token: 3 us, the launch.  The source is not shared
// with cf_paged_append.cu: that one took 45 us for 36 when it was.
#include <cuda_runtime.h>

#include "cf_paged.cuh"
#include "cf_paged8.cuh"

using namespace cf;

namespace {

constexpr int kAppendThreads = 256;
// Units in flight per thread (cf_paged_append.cu).
template <int TPB>
constexpr int kBatch = TPB == 1 ? 3 : 1;

// (cos, sin) of f / 2^64 turns, reduced by quarter turns.  What the float that
// sincospif takes rounds off, up to 2^-28 of a turn, is put back by a step of its
// derivative: such errors move more codes over a border than those of the
// rotation's arithmetic do.
__device__ __forceinline__ float2 turn_fine(uint64_t f) {
  const uint32_t hi = (uint32_t)((f + 0x80000000u) >> 32);
  const uint32_t quarter = (hi + 0x20000000u) >> 30;
  const int32_t n = (int32_t)(hi - (quarter << 30));
  const float r = (float)n;
  const float rest = (float)(n - (int32_t)r) * 1.4629180793e-9f;  // 2 pi / 2^32
  float s, c;
  sincospif(r * 0x1p-31f, &s, &c);
  const float s0 = s;
  s = fmaf(rest, c, s);
  c = fmaf(-rest, s0, c);
  const bool swap = quarter & 1u;
  const float x = swap ? s : c, y = swap ? c : s;
  return make_float2(quarter == 1 || quarter == 2 ? -x : x, quarter >= 2 ? -y : y);
}

template <typename T, int D, int TPB, int CODE>
__global__ void __launch_bounds__(kAppendThreads, TPB == 1 ? 3 : 5)
    paged8_append_kernel(const __grid_constant__ PagedAppendParams p) {
  constexpr int NB = kBatch<TPB>;
  constexpr int W = 16 / sizeof(T), UPH = D / (2 * W);  // units per head
  constexpr int RPI = kAppendThreads / UPH;             // heads per step of the block
  __shared__ float2 s_cs[TPB][kMaxPairs];
  __shared__ int s_seq[TPB], s_pos[TPB];
  __shared__ int64_t s_slot[TPB], s_scale[TPB];
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
      if (slot >= 0)
        s_scale[tid] = paged8_scale(p.page_table + (int64_t)b * p.g.max_pages, pos, p.g);
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
    s_cs[t][j] = turn_fine(f);
  }
  __syncthreads();

  while (true) {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      if (bt[i] < 0 || s_slot[bt[i]] < 0) continue;
      const int64_t t = t_lo + bt[i];
      const bool query = bh[i] < p.g.nq, value = bh[i] >= p.g.nq + p.g.nkv;
      const int kvh = bh[i] - p.g.nq - (value ? p.g.nkv : 0);
      const bool turn = rot && !value;
      const int e0 = value ? c * W : r0, e1 = value ? e0 + D / 2 : r1;
      float o[2 * W];  // the two vectors in fp32 (a copy needs none)
      if (turn || !query) {
        Elem<T>::words(reinterpret_cast<const uint32_t*>(&x[i]), 4, o);
        Elem<T>::words(reinterpret_cast<const uint32_t*>(&y[i]), 4, o + W);
      }
      if (turn) {
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const float2 cs = s_cs[bt[i]][c * W + e];
          const float a = o[e], b = o[W + e];
          o[e] = a * cs.x - b * cs.y;
          o[W + e] = b * cs.x + a * cs.y;
        }
      }
      if (!query) {
        float scale;
        uint2 w[2];
        quantise_head<CODE, UPH>(o, scale, w);
        uint8_t* dst = static_cast<uint8_t*>(value ? p.v_pages : p.k_pages) + s_slot[bt[i]] +
                       (int64_t)kvh * p.g.head_stride;
        *reinterpret_cast<uint2*>(dst + e0) = w[0];
        *reinterpret_cast<uint2*>(dst + e1) = w[1];
        if (c == 0) (&p.scales[s_scale[bt[i]] + ((int64_t)kvh << p.g.page_shift)].x)[value] = scale;
        continue;
      }
      T* dst = static_cast<T*>(p.q_out) + t * p.q_out_stride + (int64_t)bh[i] * D;
      if (turn) {
        T v[2 * W];
#pragma unroll
        for (int e = 0; e < 2 * W; ++e) v[e] = Elem<T>::from_f(o[e]);
        x[i] = *reinterpret_cast<const uint4*>(v);
        y[i] = *reinterpret_cast<const uint4*>(v + W);
      }
      *reinterpret_cast<uint4*>(dst + e0) = x[i];
      *reinterpret_cast<uint4*>(dst + e1) = y[i];
    }
    if (row >= rows) break;
    load();
  }
}

template <typename T, int D, int CODE, int TPB>
bool launch_n(const PagedAppendParams& p, int gy, cudaStream_t st) {
  PagedAppendParams pp = p;
  void* args[] = {&pp};
  return launch_pdl((const void*)&paged8_append_kernel<T, D, TPB, CODE>,
                    dim3((p.n_tokens + TPB - 1) / TPB, gy, 1), kAppendThreads, 0, st, args);
}

template <typename T, int D, int CODE>
bool launch(const PagedAppendParams& p, int sm_count, cudaStream_t st) {
  // Few tokens: one per block, its heads over several blocks of one step each
  // while the GPU has room.  Many: four per block (one and four per block, us: 300
  // tokens 4.7 and 6.6, 800 8.1 and 8.3, 1300 11.4 and 9.9, 2400 20.6 and 14.3).
  if (p.n_tokens >= 8 * sm_count) return launch_n<T, D, CODE, 4>(p, 1, st);
  constexpr int RPI = kAppendThreads / (D / (2 * (16 / (int)sizeof(T))));
  const int steps = (p.g.nq + 2 * p.g.nkv + RPI - 1) / RPI;
  return launch_n<T, D, CODE, 1>(
      p, p.n_tokens <= sm_count ? steps : (steps + kBatch<1> - 1) / kBatch<1>, st);
}
template <typename T, int CODE>
bool launch_d(const PagedAppendParams& p, int sm_count, cudaStream_t st) {
  return p.g.D == 64 ? launch<T, 64, CODE>(p, sm_count, st) : launch<T, 128, CODE>(p, sm_count, st);
}
template <typename T>
bool launch_code(int code, const PagedAppendParams& p, int sm_count, cudaStream_t st) {
  return code == CF_CODE_INT8 ? launch_d<T, CF_CODE_INT8>(p, sm_count, st)
                              : launch_d<T, CF_CODE_E4M3>(p, sm_count, st);
}

}  // namespace

bool cf::paged8_append_launch(int dtype, int code, const PagedAppendParams& p, int sm_count,
                              cudaStream_t st) {
  return dtype == CF_F16 ? launch_code<__half>(code, p, sm_count, st)
                         : launch_code<__nv_bfloat16>(code, p, sm_count, st);
}
