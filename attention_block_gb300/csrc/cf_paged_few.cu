// cf_paged_few.cu -- attention over the paged cache for few rows per KV head:
// single tokens and short drafts (tokens x grouped heads <= 16), fp16 / bf16.
//
// Bound by the cache's bytes: every visible key and value is read once, all
// rows of a KV head share it, and the tensor cores (mma.sync m16n8k16; a
// 16-row tile leaves tcgen05's 128 rows empty) have far more than the 16
// flops a byte needs.
//
// The key tiles of all (sequence, KV head) items are one line of units that
// the blocks share evenly (PagedParts), so ragged lengths and small batches
// fill the GPU; the last block to finish a split item joins its parts in a
// fixed order.  A block has four warps; each takes a quarter of a tile's
// positions through a cp.async ring of its own and keeps its own softmax
// state, so nothing but an item's end synchronises them, and the ring runs
// ahead across items.  A position that no row sees is not read: its slot is
// filled with zeros by the copy (source size 0), so what lies there cannot
// reach a product.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "cf_mma.cuh"
#include "cf_paged.cuh"

using namespace cf;

namespace {

constexpr int kFewWarps = 4;
constexpr int kFewThreads = kFewWarps * 32;
constexpr int kFewStages = 3;
constexpr int kBlocksPerSm = 2;
constexpr int kMaxParts = 64;  // per item: the last block joins them alone

template <int D>
struct Shape {
  static constexpr int KS = 2048 / D;             // positions of a warp's stage: 8 KB of K and V
  static constexpr int TK = KS * kFewWarps;          // positions of a unit
  static constexpr int STAGE = 2 * KS * D * 2;    // bytes
  static constexpr int RING = kFewWarps * kFewStages * STAGE;
  static constexpr int BUF = kFewWarps * 8 * D * 4;  // eight rows of each warp's o
  static constexpr int SMEM = RING + BUF;
  static_assert(kBlocksPerSm * (SMEM + 2048) <= 228 * 1024, "two blocks on an SM");
};

// A sequence's tokens and its key tiles; at least one tile where there are
// tokens: rows that see nothing are written too.
template <int TK>
struct Work : PagedTiles<TK> {
  int t0, n, p0;  // tokens, position of the first
};

template <int TK, bool PRE>
__device__ __forceinline__ Work<TK> work_of(const PagedAttnParams& p, int b) {
  Work<TK> w;
  if constexpr (PRE) {
    w.t0 = 0;
    w.n = p.n_tokens;
    w.p0 = p.prefix_len;
    w.set(PagedRange{0, 0, p.prefix_len});
  } else {
    const PagedSeq s = paged_seq(p.q_start, p.kv_len, b, p.n_tokens, p.max_q, p.g, p.errflag);
    w.t0 = s.t0;
    w.n = s.n;
    w.p0 = s.len - s.n;
    if (s.n <= 0) {
      w.n = w.tiles = 0;
      return w;
    }
    w.set(paged_range(max(w.p0, 0), s.len - 1, s.len, p.window, p.n_sinks));
  }
  return w;
}

// A walk over a block's units: sequence b, KV head h, tile, and the item's
// first unit i0.
template <int TK, bool PRE>
struct Cursor {
  Work<TK> w;
  int b, h, tile;
  long long u, i0;
  __device__ __forceinline__ void next(const PagedAttnParams& p, long long end) {
    ++u;
    if (++tile < w.tiles) return;
    tile = 0;
    i0 = u;
    if (++h < p.g.nkv) return;
    h = 0;
    if (u >= end) return;
    do {
      ++b;
      w = work_of<TK, PRE>(p, b);
    } while (w.tiles == 0);
  }
};

template <typename T, int D, bool PRE>
__global__ void __launch_bounds__(kFewThreads, kBlocksPerSm)
    paged_few_kernel(const __grid_constant__ PagedAttnParams p, const PagedParts ws,
                     const PagedPrefixParts pre, int max_blocks) {
  using S = Shape<D>;
  constexpr int KS = S::KS, TK = S::TK;
  constexpr int C = D / 8;         // 16-byte chunks of a row
  constexpr int NT = KS / 8;       // key octets of a stage
  constexpr int NO = D / 8;        // column octets of o
  using M = MmaKind<T>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_scan[kFewWarps];
  __shared__ int s_max[kFewWarps];
  __shared__ uint32_t s_valid[kFewWarps][kFewStages];
  __shared__ float2 s_ml[kFewWarps][kFewRows];
  __shared__ long long s_start_i0;
  __shared__ int s_start_b, s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gq = lane >> 2, tq = lane & 3;
  float* buf = reinterpret_cast<float*>(smem + S::RING);

  pdl_wait();
  pdl_trigger();

  // Units of every sequence, summed up over the batch: each thread has a run
  // of sequences.
  const int nseq = PRE ? 1 : p.batch;
  const int per = (nseq + kFewThreads - 1) / kFewThreads;
  const int b_lo = min(nseq, tid * per), b_hi = min(nseq, b_lo + per);
  long long mine = 0;
  int top = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const int t = work_of<TK, PRE>(p, b).tiles;
    mine += (long long)t * p.g.nkv;
    top = max(top, t);
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(~0u, incl, o);
    if (lane >= o) incl += v;
    top = max(top, __shfl_xor_sync(~0u, top, o));
  }
  if (lane == 31) s_scan[warp] = incl;
  if (lane == 0) s_max[warp] = top;
  __syncthreads();
  long long before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kFewWarps; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
    top = max(top, s_max[w]);
  }
  const long long upc = max(div_units(total + max_blocks - 1, max_blocks),
                            (long long)((top + kMaxParts - 1) / kMaxParts));
  const long long u0 = blockIdx.x * upc, u1 = min(total, u0 + upc);
  if (u0 >= u1) return;
  if (before <= u0 && u0 < before + mine) {
    long long at = before;
    for (int b = b_lo; b < b_hi; ++b) {
      const long long n = (long long)work_of<TK, PRE>(p, b).tiles * p.g.nkv;
      if (u0 < at + n) {
        s_start_b = b;
        s_start_i0 = at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();

  Cursor<TK, PRE> cur;
  cur.b = s_start_b;
  cur.w = work_of<TK, PRE>(p, cur.b);
  cur.u = u0;
  {
    const long long off = u0 - s_start_i0;
    cur.h = (int)div_units(off, cur.w.tiles);
    cur.tile = (int)(off - (long long)cur.h * cur.w.tiles);
    cur.i0 = u0 - cur.tile;
  }
  Cursor<TK, PRE> ld = cur;  // runs ahead of cur

  const char* kbase = static_cast<const char*>(p.k_pages);
  const char* vbase = static_cast<const char*>(p.v_pages);
  uint8_t* ring = smem + warp * kFewStages * S::STAGE;
  const uint32_t ring_s = smem_u32(ring);

  // The page of this lane's position in the tile that ld stands on, fetched
  // one tile before its copies are issued.
  int ld_pos = -1, ld_page = -1;
  auto fetch_page = [&]() {
    ld_pos = -1;
    if (ld.u >= u1 || lane >= KS) return;
    const int j = ld.w.base(ld.tile) + warp * KS + lane;
    if (!ld.w.sees(j)) return;
    ld_pos = j;
    const int* table = PRE ? p.prefix_table : p.page_table + (int64_t)ld.b * p.g.max_pages;
    ld_page = __ldg(table + (j >> p.g.page_shift));
  };
  auto issue = [&](int stage) {
    if (ld.u < u1) {
      int64_t off = -1;  // no copy: zeros
      if (ld_pos >= 0) {
        if ((unsigned)ld_page >= (unsigned)p.g.num_pages)
          atomicOr(p.errflag, kDevErrPosRange);
        else
          off = ((int64_t)ld_page * p.g.page_stride +
                 (int64_t)(ld_pos & p.g.page_mask) * p.g.slot_stride +
                 (int64_t)ld.h * p.g.head_stride) * 2;
      }
      const uint32_t valid = __ballot_sync(~0u, ld_pos >= 0);
      if (lane == 0) s_valid[warp][stage] = valid;
      const uint32_t dst = ring_s + stage * S::STAGE;
      if (valid) {
#pragma unroll
        for (int i = 0; i < KS * C / 32; ++i) {
          const int row = i * (32 / C) + lane / C, c = lane % C;
          const int64_t o = __shfl_sync(~0u, off, row);
          const bool there = o >= 0;
          const int64_t at = there ? o + c * 16 : 0;
          const uint32_t d = dst + row * (D * 2) + ((c ^ (row & 7)) << 4);
          cp16(d, kbase + at, there);
          cp16(d + KS * D * 2, vbase + at, there);
        }
      }
      ld.next(p, u1);
      fetch_page();
    }
    cp_commit();
  };

  fetch_page();
#pragma unroll
  for (int s = 0; s < kFewStages - 1; ++s) issue(s);

  int stage = 0;
  uint32_t qf[D / 16][4];
  float o[NO][4], m[2], l[2];
  int pos[2];  // positions of this thread's two rows
  bool fresh = true;
  int first_tile = cur.tile;

  while (cur.u < u1) {
    const int nrows = cur.w.n * p.g.G;
    if (fresh) {
      fresh = false;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = gq + 8 * r;
        const int i = row / p.g.G;
        pos[r] = cur.w.p0 + i;
        const T* src = static_cast<const T*>(p.q) + (int64_t)(cur.w.t0 + i) * p.q_stride +
                       (int64_t)(cur.h * p.g.G + row - i * p.g.G) * D + 2 * tq;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          qf[k][r] = row < nrows ? *reinterpret_cast<const uint32_t*>(src + k * 16) : 0u;
          qf[k][r + 2] = row < nrows ? *reinterpret_cast<const uint32_t*>(src + k * 16 + 8) : 0u;
        }
        m[r] = -INFINITY;
        l[r] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < NO; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[k][e] = 0.f;
    }
    issue(stage == 0 ? kFewStages - 1 : stage - 1);
    cp_wait<kFewStages - 1>();
    __syncwarp();
    const uint32_t valid = s_valid[warp][stage];
    if (valid) {
      const uint32_t ks = ring_s + stage * S::STAGE, vs = ks + KS * D * 2;
      float c[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) c[nt][e] = 0.f;
#pragma unroll
        for (int k2 = 0; k2 < D / 32; ++k2) {
          const int row = nt * 8 + (lane & 7), ch = k2 * 4 + (lane >> 3);
          uint32_t r0, r1, r2, r3;
          ldsm_x4(r0, r1, r2, r3, ks + row * (D * 2) + ((ch ^ (row & 7)) << 4));
          M::mma(c[nt], qf[2 * k2], r0, r1);
          M::mma(c[nt], qf[2 * k2 + 1], r2, r3);
        }
      }
      // mask, running maximum
      const int j0 = cur.w.base(cur.tile) + warp * KS;
      float mx[2] = {m[0], m[1]};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int jj = nt * 8 + 2 * tq + (e & 1);
          bool see = (valid >> jj) & 1;
          if (!PRE && cur.w.n > 1)
            see = see && paged_visible(pos[e >> 1], j0 + jj, p.window, p.n_sinks);
          c[nt][e] = see ? c[nt][e] * p.scale_log2 : -INFINITY;
          mx[e >> 1] = fmaxf(mx[e >> 1], c[nt][e]);
        }
      float corr[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(~0u, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(~0u, mx[r], 2));
        const float ref = mx[r] == -INFINITY ? 0.f : mx[r];
        corr[r] = exp2f(m[r] - ref);
        m[r] = mx[r];
        mx[r] = ref;
        l[r] *= corr[r];
      }
      if (__any_sync(~0u, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
        for (int k = 0; k < NO; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[k][e] *= corr[e >> 1];
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          c[nt][e] = exp2f(c[nt][e] - mx[e >> 1]);
          l[e >> 1] += c[nt][e];
        }
      // o += P V; bf16 probabilities enter as hi + lo pairs (the tensor cores
      // have the time), fp16 ones with their 11 bits
#pragma unroll
      for (int kk = 0; kk < KS / 16; ++kk) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
          M::split2(c[2 * kk + (x >> 1)][2 * (x & 1)], c[2 * kk + (x >> 1)][2 * (x & 1) + 1],
                    hi[x], lo[x]);
#pragma unroll
        for (int n2 = 0; n2 < NO / 2; ++n2) {
          const int row = kk * 16 + (lane & 15), ch = n2 * 2 + (lane >> 4);
          uint32_t r0, r1, r2, r3;
          ldsm_x4_trans(r0, r1, r2, r3, vs + row * (D * 2) + ((ch ^ (row & 7)) << 4));
          M::mma(o[2 * n2], hi, r0, r1);
          M::mma(o[2 * n2 + 1], hi, r2, r3);
          if constexpr (M::kAttnHiLo) {
            M::mma(o[2 * n2], lo, r0, r1);
            M::mma(o[2 * n2 + 1], lo, r2, r3);
          }
        }
      }
    }
    __syncwarp();  // the stage is read before its next copies are issued
    stage = stage + 1 == kFewStages ? 0 : stage + 1;

    const bool item_done = cur.tile + 1 == cur.w.tiles;
    if (!item_done && cur.u + 1 < u1) {
      cur.next(p, u1);
      continue;
    }

    // ---- the block's part of the item is complete: join the warps
    const bool whole = item_done && first_tile == 0;
    const PagedItemParts parts(cur.i0, cur.w.tiles, upc);
    const long long slot = parts.slot((int)(blockIdx.x - parts.first));
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(~0u, l[r], 1);
      l[r] += __shfl_xor_sync(~0u, l[r], 2);
      if (tq == 0) s_ml[warp][gq + 8 * r] = make_float2(m[r], l[r]);
    }
    const long long ticket = ((long long)cur.b * p.g.nkv + cur.h);
    constexpr int C4 = D / 4;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (8 * r >= nrows) break;
      float* dst = buf + (warp * 8 + gq) * D + 2 * tq;
#pragma unroll
      for (int k = 0; k < NO; ++k)
        *reinterpret_cast<float2*>(dst + k * 8) = make_float2(o[k][2 * r], o[k][2 * r + 1]);
      __syncthreads();
      const int rows = min(8, nrows - 8 * r);
      for (int x = tid; x < rows * C4; x += kFewThreads) {
        const int rr = x / C4, col = (x - rr * C4) * 4, row = 8 * r + rr;
        PagedState4 s{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) {
          const float2 ml = s_ml[w][row];
          s.join(ml.x, ml.y, *reinterpret_cast<const float4*>(buf + (w * 8 + rr) * D + col));
        }
        if (PRE || !whole) {
          const long long at = slot * kFewRows + row;
          __stcg(reinterpret_cast<float4*>(ws.o + at * D + col), s.o);
          if (col == 0) __stcg(ws.ml + at, make_float2(s.m, s.l));
        } else {
          const int i = row / p.g.G, g = row - i * p.g.G;
          const long long t = cur.w.t0 + i;
          if (pre.rows && cur.w.p0 + i >= 0)
            paged_join_prefix<D>(s, pre, t * p.g.G + g, cur.h, p.g.nkv, col);
          paged_store4<T, D>(s, p.out, p.lse, t * p.g.nq + cur.h * p.g.G + g, col);
        }
      }
      __syncthreads();
    }
    if (!PRE && !whole) {
      // the last block to write its part of the item joins all of them
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const int before_me = atomicAdd(ws.tickets + ticket, 1);
        s_last = before_me == parts.n - 1;
        if (s_last) ws.tickets[ticket] = 0;
      }
      __syncthreads();
      if (s_last) {
        __threadfence();
        for (int x = tid; x < min(nrows, kFewRows) * C4; x += kFewThreads) {
          const int row = x / C4, col = (x - row * C4) * 4;
          PagedState4 s{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll 4
          for (int k = 0; k < parts.n; ++k) {
            const long long at = parts.slot(k) * kFewRows + row;
            const float2 ml = __ldcg(ws.ml + at);
            s.join(ml.x, ml.y, __ldcg(reinterpret_cast<const float4*>(ws.o + at * D + col)));
          }
          const int i = row / p.g.G, g = row - i * p.g.G;
          const long long t = cur.w.t0 + i;
          if (pre.rows && cur.w.p0 + i >= 0)
            paged_join_prefix<D>(s, pre, t * p.g.G + g, cur.h, p.g.nkv, col);
          paged_store4<T, D>(s, p.out, p.lse, t * p.g.nq + cur.h * p.g.G + g, col);
        }
      }
    }
    // a sequence with more tokens than the call allows: recorded, all rows zero
    for (int x = kFewRows * C4 + tid; !PRE && x < nrows * C4; x += kFewThreads) {
      const int row = x / C4, col = (x - row * C4) * 4, i = row / p.g.G, g = row - i * p.g.G;
      const PagedState4 none{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
      paged_store4<T, D>(none, p.out, p.lse, (long long)(cur.w.t0 + i) * p.g.nq + cur.h * p.g.G + g,
                         col);
    }
    cur.next(p, u1);
    fresh = true;
    first_tile = cur.tile;
  }
  cp_wait<0>();
}

using Fn = void (*)(PagedAttnParams, PagedParts, PagedPrefixParts, int);

template <typename T, bool PRE>
const void* fn_d(int d) {
  return d == 64 ? (const void*)&paged_few_kernel<T, 64, PRE>
                 : (const void*)&paged_few_kernel<T, 128, PRE>;
}
const void* fn_of(int dtype, int d, bool prefix) {
  if (dtype == CF_F16) return prefix ? fn_d<__half, true>(d) : fn_d<__half, false>(d);
  return prefix ? fn_d<__nv_bfloat16, true>(d) : fn_d<__nv_bfloat16, false>(d);
}
int smem_of(int d) { return d == 64 ? Shape<64>::SMEM : Shape<128>::SMEM; }

}  // namespace

int cf::paged_few_grid(int dtype, int head_dim, int sm_count) {
  const int smem = smem_of(head_dim);
  for (int prefix = 0; prefix < 2; ++prefix)
    if (cudaFuncSetAttribute(fn_of(dtype, head_dim, prefix != 0),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
  return kBlocksPerSm * sm_count;  // __launch_bounds__ and Shape see to it that they fit
}

PagedPrefixParts cf::paged_few_prefix(const PagedAttnParams& p, const PagedSplit& ws) {
  const int TK = p.g.D == 64 ? Shape<64>::TK : Shape<128>::TK;
  PagedPrefixParts x;
  x.o = ws.o;
  x.ml = ws.ml;
  x.rows = kFewRows;
  x.tiles = (p.prefix_len + TK - 1) / TK;
  x.item_cost = 0;
  const long long total = (long long)x.tiles * p.g.nkv;
  x.upc = std::max((total + ws.grid - 1) / ws.grid,
                   (long long)((x.tiles + kMaxParts - 1) / kMaxParts));
  return x;
}

bool cf::paged_few_launch(int dtype, const PagedAttnParams& p, const PagedSplit& ws, bool prefix,
                          const PagedPrefixParts& pre, cudaStream_t st) {
  PagedAttnParams pp = p;
  PagedParts parts{ws.o, ws.ml, ws.tickets};
  PagedPrefixParts pr = pre;
  int grid = ws.grid;
  void* args[] = {&pp, &parts, &pr, &grid};
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.gridDim = dim3(grid, 1, 1);
  lc.blockDim = dim3(kFewThreads, 1, 1);
  lc.dynamicSmemBytes = smem_of(p.g.D);
  lc.stream = st;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelExC(&lc, fn_of(dtype, p.g.D, prefix), args) == cudaSuccess;
}
