// cf_paged_f32.cu -- attention over the paged cache for fp32 storage, on the
// CUDA cores: no tensor-core form keeps its precision.
//
// Bound by the cache's bytes for few rows, by the fp32 units (and the shared
// memory that feeds them) for many.  A block has R packed (token, grouped
// head) rows of one KV head, 4 or 16, and its warps take tiles of 32 positions
// in turn: each has a K and a V buffer of its own that cp.async refills as
// soon as it is read, so one is on its way while the other is worked on.  For
// the scores a lane has 4 rows and R / 4 positions: a vector from shared memory
// fills 4 cycles of its port even where lanes share it, so each has to serve
// several products (16 rows to a lane's one position: 331 us for 2 prompts of
// 512, 32 / 8 heads of 128; 4 x 4: 260 us).  For the sum a lane has D / 32
// columns and all R rows.  The warps' states are joined in a fixed order.
// A block finds its row tile by the tile's number, from the starts where those
// are in order.  Where they are not the row tiles are counted up over the batch.
// Where the row tiles do not fill the GPU, several blocks share each one's
// positions, and the last of them to finish joins their states in order.
// 16 sequences of 4097 positions: 99 us, 5.4 TB/s; one of 32769: 52 us.
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "cf_paged.cuh"

using namespace cf;

namespace {

constexpr int kF32Warps = 6;
constexpr int kF32Threads = kF32Warps * 32;
constexpr int kTK = 32;  // positions of a tile: a lane each

template <int D, int R>
struct F32Shape {
  static constexpr int TILE = kTK * D * 4;
  static constexpr int WARP = 2 * TILE + kTK * R * 4;  // K, V, P
  static constexpr int SMEM = kF32Warps * WARP + R * D * 4;
  static_assert(SMEM <= 224 * 1024 && R * D * 4 <= TILE, "shared memory");
};

struct F32Args {
  PagedAttnParams p;
  PagedParts ws;  // R rows per (row tile, KV head, split)
  int* tickets;   // one per (row tile, KV head); zero between calls
  const int* disorder;  // batches of more than kF32Threads: whether starts are out of order
};

__device__ __forceinline__ float4 lds4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

template <int D, int R>
__global__ void __launch_bounds__(kF32Threads, D == 64 ? 2 : 1)
    paged_f32_kernel(const __grid_constant__ F32Args a) {
  using S = F32Shape<D, R>;
  constexpr int E = D / 32, C = D / 4;  // columns of a lane, 16-byte chunks of a row
  constexpr int RPI = 32 / C;           // rows of one copy instruction
  constexpr int RG = R / 4, KG = 32 / RG;  // the lanes' grid over rows and positions
  const PagedAttnParams& p = a.p;
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ float2 s_ml[kF32Warps][R];
  __shared__ long long s_sum[kF32Warps];
  __shared__ int s_seq, s_no, s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int kvh = blockIdx.y, G = p.g.G;
  const int rg = lane / KG, kg = lane % KG;  // rows 4 rg .. + 3, positions kg + n KG
  float* sq = reinterpret_cast<float*>(sm + kF32Warps * S::WARP);

  auto start = [&](int b) { return p.q_start ? p.q_start[b] : b; };
  auto first_no = [&](int b, int t0) { return (int)((long long)t0 * G / R) + b; };
  // Row tiles of sequence b.
  auto row_tiles = [&](int b) {
    const int t0 = start(b), t1 = p.q_start ? p.q_start[b + 1] : b + 1;
    return starts_ordered(t0, t1, p.n_tokens) ? ((t1 - t0) * G + R - 1) / R : 0;
  };
  bool disorder = false;
  if (p.q_start)
    disorder = p.batch > kF32Threads
                   ? *a.disorder != 0
                   : __syncthreads_or(tid < p.batch && !starts_ordered(start(tid), start(tid + 1),
                                                                       p.n_tokens)) != 0;
  if (tid == 0) s_seq = -1;
  __syncthreads();
  if (!disorder) {
    // Row tile j of sequence b has the number t0 * G / R + b + j: unique, below
    // T * G / R + batch, and the first ones increase.  So this block's sequence
    // is the last whose first number is not above its own; a round of the search
    // leaves a 192nd of the batch.
    int lo = 0, hi = p.batch;
    while (hi - lo > kF32Threads) {
      const int w = (hi - lo + kF32Threads - 1) / kF32Threads, b = lo + tid * w;
      if (tid == 0) s_seq = lo;
      __syncthreads();
      if (b < hi && first_no(b, start(b)) <= (int)blockIdx.x) atomicMax(&s_seq, b);
      __syncthreads();
      lo = s_seq;
      hi = min(hi, lo + w);
      __syncthreads();
      if (tid == 0) s_seq = -1;
      __syncthreads();
    }
    if (lo + tid < hi) {
      const int b = lo + tid, no = first_no(b, start(b)), j = (int)blockIdx.x - no;
      if (j >= 0 && j < row_tiles(b)) {
        s_seq = b;
        s_no = no;
      }
    }
  } else {
    // The tile with this number when all are counted up.  They are as few as
    // above unless sequences claim a token twice.
    long long no = 0;
    for (int b0 = 0; b0 < p.batch; b0 += kF32Threads) {
      const int n = b0 + tid < p.batch ? row_tiles(b0 + tid) : 0;
      long long incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(~0u, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) s_sum[warp] = incl;
      __syncthreads();
      long long before = no + incl - n;
#pragma unroll
      for (int w = 0; w < kF32Warps; ++w) {
        if (w < warp) before += s_sum[w];
        no += s_sum[w];
      }
      if (before <= blockIdx.x && blockIdx.x < before + n) {
        s_seq = b0 + tid;
        s_no = (int)before;
      }
      __syncthreads();
    }
    if (blockIdx.x + blockIdx.y + blockIdx.z == 0 && tid == 0)
      atomicOr(p.errflag, kDevErrPosRange);
  }
  __syncthreads();
  const int b = s_seq;
  if (b < 0) return;  // no row tile has this number
  const PagedSeq s = paged_seq(p.q_start, p.kv_len, b, p.n_tokens, p.max_q, p.g, p.errflag);
  const int r0 = ((int)blockIdx.x - s_no) * R;
  const int nr = min(R, s.n * G - r0);
  const int p0 = s.len - s.n;
  const int plo = p0 + r0 / G, phi = p0 + (r0 + nr - 1) / G;

  for (int i = tid; i < R * C; i += kF32Threads) {
    const int r = i / C, c = i - r * C;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < nr) {
      const int tok = (r0 + r) / G, h = kvh * G + (r0 + r) - tok * G;
      v = *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) +
                                           (int64_t)(s.t0 + tok) * p.q_stride + (int64_t)h * D +
                                           4 * c);
    }
    reinterpret_cast<float4*>(sq)[r * C + (c ^ (r >> 2))] = v;  // no bank conflicts over rg
  }
  __syncthreads();

  // ---- the tiles: the prefix's, then the sequence's own
  PagedTiles<kTK> own;
  own.set(paged_range(max(plo, 0), phi, phi + 1, p.window, p.n_sinks));
  const int n_pre = phi >= 0 ? (p.prefix_len + kTK - 1) / kTK : 0;
  const int n_all = n_pre + (own.hi > own.lo ? own.tiles : 0);
  const int step = gridDim.z * kF32Warps;
  const int* table = p.page_table + (int64_t)b * p.g.max_pages;
  uint8_t* mine = sm + warp * S::WARP;
  const uint32_t sk = smem_u32(mine), sv = sk + S::TILE, sp = sv + S::TILE, sqa = smem_u32(sq);
  // Where this lane's position of a tile lies, -1: zeros stand for it.
  auto locate = [&](int t) -> int64_t {
    if (t >= n_all) return -1;
    int64_t off = -1;
    if (t < n_pre) {
      const int j = t * kTK + lane;
      if (j < p.prefix_len) off = paged_offset(p.prefix_table, j, p.g, p.errflag);
    } else {
      const int j = own.base(t - n_pre) + lane;
      if (own.sees(j)) off = paged_offset(table, j, p.g, p.errflag);
    }
    return off < 0 ? -1 : off + (int64_t)kvh * p.g.head_stride;
  };
  const int cr = lane / C, cc = lane % C;
  auto copy = [&](const void* pages, uint32_t dst, int64_t off, bool swizzle) {
#pragma unroll 8
    for (int y = 0; y < kTK; y += RPI) {
      const int row = y + cr;
      const int64_t o = __shfl_sync(~0u, off, row);
      cp16(dst + row * (D * 4) + ((swizzle ? cc ^ (row & 7) : cc) << 4),
           static_cast<const float*>(pages) + (o < 0 ? 0 : o + 4 * cc), o >= 0);
    }
    cp_commit();
  };

  float m[4], l[4], o[R][E];  // of the lane's rows for scores, of all rows
  int pos[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    m[x] = -INFINITY;
    l[x] = 0.f;
    pos[x] = p0 + (r0 + 4 * rg + x) / G;
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int e = 0; e < E; ++e) o[r][e] = 0.f;
  int t = blockIdx.z * kF32Warps + warp;
  int64_t off = locate(t);
  if (t < n_all) {
    copy(p.k_pages, sk, off, true);
    copy(p.v_pages, sv, off, false);
  }
  for (; t < n_all; t += step) {
    const int next = t + step;
    off = locate(next);
    cp_wait<1>();  // K is there
    __syncwarp();
    float sc[4][RG];
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int n = 0; n < RG; ++n) sc[x][n] = 0.f;
#pragma unroll 2
    for (int i = 0; i < C; ++i) {
      float4 k[RG];
#pragma unroll
      for (int n = 0; n < RG; ++n) {
        const int row = kg + n * KG;
        k[n] = lds4(sk + row * (D * 4) + ((i ^ (row & 7)) << 4));
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float4 q = lds4(sqa + ((4 * rg + x) * C + (i ^ rg)) * 16);
#pragma unroll
        for (int n = 0; n < RG; ++n)
          sc[x][n] = fmaf(k[n].x, q.x,
                          fmaf(k[n].y, q.y, fmaf(k[n].z, q.z, fmaf(k[n].w, q.w, sc[x][n]))));
      }
    }
    __syncwarp();
    if (next < n_all)
      copy(p.k_pages, sk, off, true);
    else
      cp_commit();

    // ---- softmax; what a row does not see gets -1 for its probability
    const bool pre = t < n_pre;
    const int base = pre ? t * kTK : own.base(t - n_pre);
    const bool full = pre ? base + kTK <= p.prefix_len && plo >= 0
                          : base + kTK - 1 <= plo && (p.window == 0 || phi - base < p.window ||
                                                      base + kTK <= p.n_sinks);
    float corr[4];
    bool grown = false;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      bool vis[RG];
      float mx = -INFINITY;
#pragma unroll
      for (int n = 0; n < RG; ++n) {
        const int j = base + kg + n * KG;
        vis[n] = full || (pre ? j < p.prefix_len && pos[x] >= 0
                              : paged_visible(pos[x], j, p.window, p.n_sinks));
        sc[x][n] = vis[n] ? sc[x][n] * p.scale_log2 : -INFINITY;
        mx = fmaxf(mx, sc[x][n]);
      }
#pragma unroll
      for (int d = KG / 2; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, d));
      const float m_new = fmaxf(m[x], mx), ref = m_new == -INFINITY ? 0.f : m_new;
      grown |= m_new != m[x];
      corr[x] = m_new != m[x] ? exp2f(m[x] - ref) : 1.f;
      l[x] *= corr[x];
      m[x] = m_new;
#pragma unroll
      for (int n = 0; n < RG; ++n) {
        sc[x][n] = vis[n] ? exp2f(sc[x][n] - ref) : -1.f;
        if (vis[n]) l[x] += sc[x][n];
      }
    }
    if (__any_sync(~0u, grown)) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float f = __shfl_sync(~0u, corr[r & 3], (r >> 2) * KG);
#pragma unroll
        for (int e = 0; e < E; ++e) o[r][e] *= f;
      }
    }
#pragma unroll
    for (int n = 0; n < RG; ++n)
      *reinterpret_cast<float4*>(mine + 2 * S::TILE + ((kg + n * KG) * R + 4 * rg) * 4) =
          make_float4(sc[0][n], sc[1][n], sc[2][n], sc[3][n]);
    cp_wait<1>();  // V is there
    __syncwarp();
    auto weigh = [&](auto guard) {
#pragma unroll 4
      for (int k = 0; k < kTK; ++k) {
        float v[E];
        if constexpr (E == 4) {
          const float4 x = lds4(sv + k * (D * 4) + lane * 16);
          v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(mine + S::TILE + k * (D * 4) + lane * 8);
          v[0] = x.x, v[1] = x.y;
        }
#pragma unroll
        for (int r = 0; r < R; r += 4) {
          const float4 w = lds4(sp + (k * R + r) * 4);
          const float ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            if (decltype(guard)::value && ww[x] < 0.f) continue;
#pragma unroll
            for (int e = 0; e < E; ++e) o[r + x][e] = fmaf(ww[x], v[e], o[r + x][e]);
          }
        }
      }
    };
    if (full)
      weigh(std::false_type{});
    else
      weigh(std::true_type{});
    __syncwarp();
    if (next < n_all)
      copy(p.v_pages, sv, off, false);
    else
      cp_commit();
  }
  cp_wait<0>();
  __syncwarp();

  // ---- the warps' states, over their K buffers
#pragma unroll
  for (int x = 0; x < 4; ++x) {
#pragma unroll
    for (int d = KG / 2; d >= 1; d >>= 1) l[x] += __shfl_xor_sync(~0u, l[x], d);
    if (kg == 0) s_ml[warp][4 * rg + x] = make_float2(m[x], l[x]);
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int e = 0; e < E; ++e)
      reinterpret_cast<float*>(mine)[r * D + lane * E + e] = o[r][e];
  __syncthreads();
  const int splits = gridDim.z;
  const long long item = (long long)blockIdx.x * p.g.nkv + kvh;
  auto out_row = [&](int r) {
    const int tok = (r0 + r) / G;
    return (long long)(s.t0 + tok) * p.g.nq + kvh * G + (r0 + r) - tok * G;
  };
  for (int i = tid; i < nr * C; i += kF32Threads) {
    const int r = i / C, col = (i - r * C) * 4;
    PagedState4 x{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll
    for (int w = 0; w < kF32Warps; ++w)
      x.join(s_ml[w][r].x, s_ml[w][r].y,
             *reinterpret_cast<const float4*>(sm + w * S::WARP + (r * D + col) * 4));
    if (splits == 1) {
      paged_store4<float, D>(x, p.out, p.lse, out_row(r), col);
    } else {
      const long long at = (item * splits + blockIdx.z) * R + r;
      __stcg(reinterpret_cast<float4*>(a.ws.o + at * D + col), x.o);
      if (col == 0) __stcg(a.ws.ml + at, make_float2(x.m, x.l));
    }
  }
  if (splits == 1) return;
  __threadfence();
  __syncthreads();
  if (tid == 0) s_last = atomicAdd(a.tickets + item, 1) == splits - 1;
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  if (tid == 0) a.tickets[item] = 0;
  for (int i = tid; i < nr * C; i += kF32Threads) {
    const int r = i / C, col = (i - r * C) * 4;
    PagedState4 x{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll 4
    for (int z = 0; z < splits; ++z) {
      const long long at = (item * splits + z) * R + r;
      const float2 ml = __ldcg(a.ws.ml + at);
      x.join(ml.x, ml.y, __ldcg(reinterpret_cast<const float4*>(a.ws.o + at * D + col)));
    }
    paged_store4<float, D>(x, p.out, p.lse, out_row(r), col);
  }
}

// Whether starts are out of order, for the blocks of a large batch: 3 to 8 us of
// 33 for 700 single tokens, of 208 for 300 x 4, of 409 for 700 x 2.
__global__ void __launch_bounds__(1024)
    paged_f32_order_kernel(const int* q_start, int batch, int n_tokens, int* disorder) {
  bool bad = false;
  for (int b = threadIdx.x; b < batch; b += 1024)
    bad |= !starts_ordered(q_start[b], q_start[b + 1], n_tokens);
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) *disorder = any;
}

struct F32Fn {
  void (*fn)(F32Args);
  int smem;
};
F32Fn f32_fn(int d, int rows) {
  if (d == 64)
    return rows == 4 ? F32Fn{paged_f32_kernel<64, 4>, F32Shape<64, 4>::SMEM}
                     : F32Fn{paged_f32_kernel<64, 16>, F32Shape<64, 16>::SMEM};
  return rows == 4 ? F32Fn{paged_f32_kernel<128, 4>, F32Shape<128, 4>::SMEM}
                   : F32Fn{paged_f32_kernel<128, 16>, F32Shape<128, 16>::SMEM};
}

}  // namespace

int cf::paged_f32_grid(int head_dim, int sm_count) {
  int per_sm = 0;
  for (int rows : {4, 16}) {
    const F32Fn f = f32_fn(head_dim, rows);
    if (cudaFuncSetAttribute(f.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, f.smem) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, f.fn, kF32Threads, f.smem) !=
            cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
  }
  return per_sm * sm_count;
}

// a launch that splits has at most 2 * grid blocks
long long cf::paged_f32_part_rows(int grid) { return 2LL * grid * 16; }

bool cf::paged_f32_launch(const PagedAttnParams& p, const PagedSplit& ws, cudaStream_t st) {
  // 4 rows where a call's sequences have no more: 99 us for 16 sequences of
  // 4097 positions, 32 / 8 heads of 128; with 16 rows, all in use, 198.
  const int rows = (long long)p.max_q * p.g.G <= 4 ? 4 : 16;
  const F32Fn f = f32_fn(p.g.D, rows);
  const long long tiles = (long long)p.n_tokens * p.g.G / rows + p.batch;
  // Twice the resident blocks, since the row tiles are an upper bound: one
  // sequence of 32769 positions 52 us, with once 89; 1025 positions 11.6, 10.1.
  const long long splits =
      std::max<long long>(1, std::min<long long>(64, 2LL * ws.grid / (tiles * p.g.nkv)));
  F32Args a;
  a.p = p;
  a.ws = ws.parts;
  a.tickets = ws.tickets;
  a.disorder = ws.tickets + ws.grid;
  if (p.q_start && p.batch > kF32Threads) {
    int* disorder = ws.tickets + ws.grid;
    void* order[] = {&a.p.q_start, &a.p.batch, &a.p.n_tokens, &disorder};
    if (cudaLaunchKernel((const void*)&paged_f32_order_kernel, dim3(1), dim3(1024), order, 0, st) !=
        cudaSuccess)
      return false;
  }
  void* args[] = {&a};
  return cudaLaunchKernel((const void*)f.fn, dim3((unsigned)tiles, p.g.nkv, (unsigned)splits),
                          dim3(kF32Threads), args, f.smem, st) == cudaSuccess;
}
