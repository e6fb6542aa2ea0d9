// cf_paged_few.cu -- attention over the paged cache for few rows per KV head:
// single tokens and short drafts (tokens x grouped heads <= 16), fp16 / bf16.
//
// Bound by the cache's bytes: every visible key and value is read once, all
// rows of a KV head share it, and the tensor cores (mma.sync m16n8k16; a
// 16-row tile leaves tcgen05's 128 rows empty) have far more than the 16
// flops a byte needs.
//
// The key tiles of all (sequence, KV head) items are one line of units, cut
// into pieces (PagedParts).  A worker is one warp: it takes whole tiles
// through a cp.async ring of its own, which runs ahead across items and
// pieces, keeps its own softmax state and never waits for another warp.
// Ragged lengths and small batches thereby fill the GPU.  A second kernel
// joins the parts of split items, in a fixed order: which warp computed a
// part does not matter.  A position that no row sees is not read: its slot
// is filled with zeros by the copy (source size 0), so what lies there cannot
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
constexpr int kPieces = 3;      // pieces per warp where there is work for them ...
constexpr int kFineUnits = 12;  // ... which is from this many units per warp on
constexpr int kJoinThreads = 256;

template <int D>
struct Shape {
  static constexpr int KS = 2048 / D;           // positions of a unit: 8 KB of K and V
  static constexpr int STAGE = 2 * KS * D * 2;  // bytes
  static constexpr int SMEM = kFewWarps * kFewStages * STAGE;
  // 1 KB of static shared memory and 1 KB that the system takes for a block
  static_assert(kBlocksPerSm * (SMEM + 2048) <= 228 * 1024, "two blocks on an SM");
};

// Units of a piece.  Memory serves some SMs faster than others: with one piece
// per warp the fast ones idle at the end, so a long line is cut finer and the
// later pieces go to whoever is free.
__host__ __device__ inline long long few_upc(long long total, int warps) {
  const long long n = total >= (long long)kFineUnits * warps ? (long long)kPieces * warps : warps;
#ifdef __CUDA_ARCH__
  return div_units(total + n - 1, n);
#else
  return (total + n - 1) / n;
#endif
}

// An item for the joining kernel.
struct alignas(16) FewItem {
  long long i0;
  int tiles, t0, p0, n, b, h;
};
// Head of the list of such items.
struct alignas(16) FewList {
  long long upc;
  int pad[2];
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

// A walk over units: sequence b, KV head h, tile, the item's first unit i0,
// and the end of the piece.
template <int TK, bool PRE>
struct Cursor {
  Work<TK> w;
  int b, h, tile;
  long long u, i0, end;
  __device__ __forceinline__ void next(const PagedAttnParams& p) {
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

struct FewArgs {
  PagedAttnParams p;
  PagedPrefixParts pre;
  PagedParts ws;
  FewList* head;
  FewItem* list;
  int* counter;  // pieces handed out, warps done, items listed, joining blocks done
  int row_limit;  // rows per item, at most
  int split;      // the joining kernel's lane groups per row
};

template <typename T, int D, int MODE>
__global__ void __launch_bounds__(kFewThreads, kBlocksPerSm)
    paged_few_kernel(const __grid_constant__ FewArgs a) {
  using S = Shape<D>;
  constexpr bool PRE = MODE == kPrefix;
  constexpr int KS = S::KS;
  constexpr int C = D / 8;   // 16-byte chunks of a row
  constexpr int NT = KS / 8;  // key octets of a stage
  constexpr int NO = D / 8;   // column octets of o
  using M = MmaKind<T>;
  const PagedAttnParams& p = a.p;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_first[32];  // first unit of every fourth thread's sequences
  __shared__ long long s_scan[kFewWarps];
  __shared__ uint32_t s_valid[kFewWarps][kFewStages];
  __shared__ int s_piece[kFewWarps][4];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gq = lane >> 2, tq = lane & 3;

  pdl_wait();
  pdl_trigger();

  // Units of every sequence, summed up over the batch: each thread has a run
  // of sequences.
  const int nseq = PRE ? 1 : p.batch;
  const int per = (nseq + kFewThreads - 1) / kFewThreads;
  long long mine = 0;
  for (int b = tid * per; b < min(nseq, (tid + 1) * per); ++b)
    mine += (long long)work_of<KS, PRE>(p, b).tiles * p.g.nkv;
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(~0u, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  long long before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kFewWarps; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  if (tid % kFewWarps == 0) s_first[tid / kFewWarps] = before;
  const int workers = gridDim.x * kFewWarps, me = blockIdx.x * kFewWarps + warp;
  const long long upc = PRE ? a.pre.upc : few_upc(total, workers);
  // pieces 0 .. workers - 1 are dealt out, the others fetched from a counter
  const bool fine = upc > 0 && total > upc * workers;
  if (!PRE && blockIdx.x == 0 && tid == 0) a.head->upc = upc;
  __syncthreads();

  // The walk's start in a piece; past the last one it has no units.
  auto locate = [&](Cursor<KS, PRE>& c, int piece) {
    c.u = (long long)piece * upc;
    c.end = min(total, c.u + upc);
    if (c.u >= total) {
      c.end = c.u = total;
      return;
    }
    // the last run of sequences that begins at or before unit u
    const int n = __popc(__ballot_sync(~0u, s_first[lane] <= c.u));
    long long at = s_first[n - 1];
    int b = (n - 1) * kFewWarps * per;
    while (true) {
      c.w = work_of<KS, PRE>(p, b);
      const long long len = (long long)c.w.tiles * p.g.nkv;
      if (c.u < at + len) break;
      at += len;
      ++b;
    }
    c.b = b;
    const long long off = c.u - at;
    c.h = (int)div_units(off, c.w.tiles);
    c.tile = (int)(off - (long long)c.h * c.w.tiles);
    c.i0 = c.u - c.tile;
  };

  const char* kbase = static_cast<const char*>(p.k_pages);
  const char* vbase = static_cast<const char*>(p.v_pages);
  const uint32_t ring_s = smem_u32(smem + warp * kFewStages * S::STAGE);

  int seq = 0, ld_seq = 0;  // pieces begun so far, less one; the copies run ahead
  int upcoming = 0;         // lane 0: the piece after the one the copies are in
  auto fetch_piece = [&]() {
    if (lane == 0) upcoming = fine ? workers + atomicAdd(a.counter, 1) : 1 << 30;
  };
  Cursor<KS, PRE> cur;
  locate(cur, me);
  if (lane == 0) s_piece[warp][0] = me;
  if (cur.u < cur.end) fetch_piece();
  Cursor<KS, PRE> ld = cur;  // runs ahead of cur

  // The page of this lane's position in the tile that ld stands on, fetched
  // one tile before its copies are issued.
  int ld_pos = -1, ld_page = -1;
  auto fetch_page = [&]() {
    ld_pos = -1;
    if (ld.u >= ld.end || lane >= KS) return;
    const int j = ld.w.base(ld.tile) + lane;
    if (!ld.w.sees(j)) return;
    ld_pos = j;
    const int* table = PRE ? p.prefix_table : p.page_table + (int64_t)ld.b * p.g.max_pages;
    ld_page = __ldg(table + (j >> p.g.page_shift));
  };
  auto issue = [&](int stage) {
    if (ld.u < ld.end) {
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
      const int ob = ld.b, oh = ld.h;
      ld.next(p);
      if (ld.u >= ld.end && ld.end < total) {  // later pieces lie further on
        ++ld_seq;
        const int piece = __shfl_sync(~0u, upcoming, 0);
        if (lane == 0) s_piece[warp][ld_seq & 3] = piece;
        locate(ld, piece);
        if (ld.u < ld.end) fetch_piece();
      }
      fetch_page();
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
      if (ld.u < ld.end && (ld.b != ob || ld.h != oh)) {  // the next item's queries
        const int row = lane * 64 / D, i = row / p.g.G;
        if (row < ld.w.n * p.g.G)
          prefetch_line(static_cast<const T*>(p.q) + (int64_t)(ld.w.t0 + i) * p.q_stride +
                        (int64_t)(ld.h * p.g.G + row - i * p.g.G) * D + lane * 64 % D);
      }
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

  while (cur.u < cur.end) {
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
      const int j0 = cur.w.base(cur.tile);
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
    if (!item_done && cur.u + 1 < cur.end) {
      cur.next(p);
      continue;
    }

    // ---- the warp's part of the item is complete
    const bool whole = item_done && first_tile == 0;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(~0u, l[r], 1);
      l[r] += __shfl_xor_sync(~0u, l[r], 2);
    }
    // (a sequence with more tokens than the call allows has no keys: all rows zero)
    if ((MODE != kOwn || !whole) && (PRE || cur.w.n <= p.max_q)) {
      const long long piece = s_piece[warp][seq & 3];
      const long long slot = 2 * piece + (piece * upc >= cur.i0 ? 0 : 1);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = gq + 8 * r, i = row / p.g.G;
        if (row >= nrows) continue;
        long long at = slot * kFewRows + row;
        if (whole)
          at = a.ws.state_base +
               (a.ws.by_token
                    ? (long long)(cur.w.t0 + i) * p.g.nq + cur.h * p.g.G + row - i * p.g.G
                    : ((long long)cur.b * p.g.nkv + cur.h) * kFewRows + row);
        if (tq == 0) __stcg(a.ws.ml + at, make_float2(m[r], l[r]));
        float* dst = a.ws.o + at * D + 2 * tq;
#pragma unroll
        for (int k = 0; k < NO; ++k)
          __stcg(reinterpret_cast<float2*>(dst + 8 * k), make_float2(o[k][2 * r], o[k][2 * r + 1]));
      }
      if (!PRE && first_tile == 0 && lane == 0) {
        FewItem x;
        x.i0 = cur.i0;
        x.tiles = cur.w.tiles;
        x.t0 = cur.w.t0;
        x.p0 = cur.w.p0;
        x.n = cur.w.n;
        x.b = cur.b;
        x.h = cur.h;
        a.list[atomicAdd(a.counter + 2, 1)] = x;
      }
    } else {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = gq + 8 * r, i = row / p.g.G;
        const long long at = (long long)(cur.w.t0 + i) * p.g.nq + cur.h * p.g.G + row - i * p.g.G;
        const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
        T* dst = static_cast<T*>(p.out) + at * D + 8 * tq;
#pragma unroll
        for (int k = 0; k < NO; k += 4) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = pack2<T>(o[k + e][2 * r] * inv, o[k + e][2 * r + 1] * inv);
          quad_transpose(w, tq);  // lane q: the 8 columns of octet k + q
          if (row < nrows)
            *reinterpret_cast<uint4*>(dst + 8 * k) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (p.lse && row < nrows && tq == 0)
          p.lse[at] = m[r] == -INFINITY ? -INFINITY : (m[r] + log2f(l[r])) * 0.69314718055994531f;
      }
    }
    for (int x = kFewRows * (D / 4) + lane; !PRE && x < nrows * (D / 4); x += 32) {
      const int row = x / (D / 4), col = (x - row * (D / 4)) * 4, i = row / p.g.G;
      const PagedState4 none{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
      paged_store4<T, D>(none, p.out, p.lse,
                         (long long)(cur.w.t0 + i) * p.g.nq + cur.h * p.g.G + row - i * p.g.G, col);
    }
    const bool piece_done = cur.u + 1 == cur.end;
    cur.next(p);
    if (piece_done && cur.end < total) {
      ++seq;
      locate(cur, s_piece[warp][seq & 3]);
    }
    fresh = true;
    first_tile = cur.tile;
  }
  cp_wait<0>();
  // the last warp out leaves the counters at zero for the next call
  if (fine && lane == 0 && atomicAdd(a.counter + 1, 1) == workers - 1) {
    a.counter[0] = 0;
    a.counter[1] = 0;
  }
}

// Joins the states of the listed items, and the prefix's: one row per group of
// D / 4 lanes, or per block, whose groups then share the row's parts.
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) paged_few_join_kernel(const __grid_constant__ FewArgs a) {
  constexpr int W = D / 4, NG = kJoinThreads / W;
  __shared__ float4 s_o[NG][W];
  __shared__ float2 s_ml[NG];
  const PagedAttnParams& p = a.p;
  const int tid = threadIdx.x, grp = tid / W, col = (tid % W) * 4;
  pdl_wait();
  pdl_trigger();
  const long long rows = (long long)a.counter[2] * a.row_limit;
  const long long upc = a.head->upc;
  const int split = a.split;  // groups per row: 1 or NG
  const long long step = (long long)gridDim.x * NG / split;
  for (long long x0 = (long long)blockIdx.x * NG / split; x0 < rows; x0 += step) {
    const long long x = split == 1 ? x0 + grp : x0;
    PagedState4 s{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    long long at = -1;
    if (x < rows) {
      const long long item = div_units(x, a.row_limit);
      const int row = (int)(x - item * a.row_limit);
      const FewItem it = a.list[item];
      const int i = row / p.g.G, gi = row - i * p.g.G;
      if (i < it.n) {
        const long long t = it.t0 + i;
        at = t * p.g.nq + it.h * p.g.G + gi;
        const PagedRowParts own(PagedItemParts(it.i0, it.tiles, upc), kFewRows, row,
                                a.ws.state_base +
                                    (a.ws.by_token
                                         ? at
                                         : ((long long)it.b * p.g.nkv + it.h) * kFewRows + row));
        const bool with_pre = a.pre.rows && it.p0 + i >= 0;
        if (split == 1) {
          paged_join_row<D>(s, a.ws.o, a.ws.ml, own, col);
          if (with_pre)
            paged_join_row<D>(s, a.pre.o, a.pre.ml, paged_prefix_row(a.pre, p.g, t, it.h, gi), col);
        } else {
#pragma unroll 4
          for (int k = grp; k < own.n; k += NG) {
            const long long r = own.row(k);
            const float2 ml = __ldcg(a.ws.ml + r);
            s.join(ml.x, ml.y, __ldcg(reinterpret_cast<const float4*>(a.ws.o + r * D + col)));
          }
          if (with_pre) {
            const PagedRowParts pr = paged_prefix_row(a.pre, p.g, t, it.h, gi);
#pragma unroll 4
            for (int k = grp; k < pr.n; k += NG) {
              const long long r = pr.row(k);
              const float2 ml = __ldcg(a.pre.ml + r);
              s.join(ml.x, ml.y, __ldcg(reinterpret_cast<const float4*>(a.pre.o + r * D + col)));
            }
          }
        }
      }
    }
    if (split != 1) {
      s_o[grp][tid % W] = s.o;
      if (col == 0) s_ml[grp] = make_float2(s.m, s.l);
      __syncthreads();
      if (grp == 0) {
#pragma unroll
        for (int g = 1; g < NG; ++g) s.join(s_ml[g].x, s_ml[g].y, s_o[g][tid % W]);
      }
      __syncthreads();
    }
    if (at >= 0 && (split == 1 || grp == 0)) paged_store4<T, D>(s, p.out, p.lse, at, col);
  }
  // the last block out empties the list for the next call
  __syncthreads();
  if (tid == 0 && atomicAdd(a.counter + 3, 1) == (int)gridDim.x - 1) {
    a.counter[2] = 0;
    a.counter[3] = 0;
  }
}

struct FewFns {
  const void *main, *join;
  int smem;
};
template <typename T, int D>
FewFns few_fns_td(int mode) {
  const void* main = mode == kPrefix ? (const void*)&paged_few_kernel<T, D, kPrefix>
                     : mode == kOwn  ? (const void*)&paged_few_kernel<T, D, kOwn>
                                     : (const void*)&paged_few_kernel<T, D, kOwnAfterPrefix>;
  return FewFns{main, (const void*)&paged_few_join_kernel<T, D>, Shape<D>::SMEM};
}
FewFns few_fns(int dtype, int d, int mode) {
  if (dtype == CF_F16) return d == 64 ? few_fns_td<__half, 64>(mode) : few_fns_td<__half, 128>(mode);
  return d == 64 ? few_fns_td<__nv_bfloat16, 64>(mode) : few_fns_td<__nv_bfloat16, 128>(mode);
}

bool launch_pdl(const void* fn, int grid, int threads, int smem, cudaStream_t st, void** args) {
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.gridDim = dim3(grid, 1, 1);
  lc.blockDim = dim3(threads, 1, 1);
  lc.dynamicSmemBytes = smem;
  lc.stream = st;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelExC(&lc, fn, args) == cudaSuccess;
}

}  // namespace

int cf::paged_few_grid(int dtype, int head_dim, int sm_count) {
  for (int mode = kOwn; mode <= kOwnAfterPrefix; ++mode) {
    const FewFns f = few_fns(dtype, head_dim, mode);
    if (cudaFuncSetAttribute(f.main, cudaFuncAttributeMaxDynamicSharedMemorySize, f.smem) !=
        cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
  }
  return kBlocksPerSm * sm_count;  // __launch_bounds__ and Shape see to it that they fit
}

long long cf::paged_few_part_rows(int grid) {
  return 2LL * kPieces * grid * kFewWarps * kFewRows;
}

size_t cf::paged_few_list_bytes(long long items) {
  return sizeof(FewList) + (size_t)items * sizeof(FewItem);
}

PagedPrefixParts cf::paged_few_prefix(const PagedAttnParams& p, const PagedSplit& ws) {
  const int KS = p.g.D == 64 ? Shape<64>::KS : Shape<128>::KS;
  PagedPrefixParts x;
  x.o = ws.parts.o;
  x.ml = ws.parts.ml;
  x.state_base = ws.parts.state_base;
  x.rows = kFewRows;
  x.tiles = (p.prefix_len + KS - 1) / KS;
  x.item_cost = 0;
  x.upc = few_upc((long long)x.tiles * p.g.nkv, ws.grid * kFewWarps);
  return x;
}

bool cf::paged_few_launch(int dtype, const PagedAttnParams& p, const PagedSplit& ws, PagedMode mode,
                          const PagedPrefixParts& pre, cudaStream_t st) {
  const FewFns f = few_fns(dtype, p.g.D, mode);
  FewArgs a;
  a.p = p;
  a.pre = pre;
  a.ws = ws.parts;
  a.head = static_cast<FewList*>(ws.list);
  a.list = reinterpret_cast<FewItem*>(a.head + 1);
  a.counter = ws.counter;
  a.row_limit = std::min(kFewRows, p.max_q * p.g.G);
  // a block per row while the rows may not fill the GPU's lane groups anyway
  const int ng = kJoinThreads / (p.g.D / 4), blocks = ws.grid * 4;
  const long long rows = (long long)p.batch * p.g.nkv * a.row_limit;
  a.split = rows <= 2LL * blocks ? ng : 1;
  void* args[] = {&a};
  if (!launch_pdl(f.main, ws.grid, kFewThreads, f.smem, st, args)) return false;
  if (mode == kPrefix) return true;
  const long long want = a.split == 1 ? (rows + ng - 1) / ng : rows;
  return launch_pdl(f.join, (int)std::min<long long>(blocks, want), kJoinThreads, 0, st, args);
}
