// cf_paged_few.cu -- attention over the paged cache for few rows per KV head:
// single tokens and short drafts (tokens x grouped heads <= 16), fp16 / bf16.
//
// Bound by the cache's bytes: every visible key and value is read once, all
// rows of a KV head share it, and the tensor cores (mma.sync m16n8k16; a
// 16-row tile leaves tcgen05's 128 rows empty) have far more than the 16
// flops a byte needs.  16 sequences of 4097 positions, 32 / 8 heads of 128: 54
// us, 5.0 TB/s; one sequence of 131072 positions: 93 us, 5.7 TB/s; what is left
// to the copy rate is a fixed 9-14 us of schedule, first loads and joins.
//
// The key tiles of all (sequence, KV head) items are one line of units that
// the warps share evenly (PagedParts), so ragged lengths and small batches
// fill the GPU.  A warp takes its whole run of tiles through a cp.async ring
// of its own that runs ahead across items, keeps its own softmax state, and
// waits for nobody until its run is done.  Then the block joins the parts of
// items that several of its warps share, and the last block to finish a part
// of an item that lies in several blocks joins those, in a fixed order.
// A position that no row sees is not read: its slot is filled with zeros by
// the copy (source size 0), so what lies there cannot reach a product.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "cf_mma.cuh"
#include "cf_paged_few.cuh"

using namespace cf;

namespace {

constexpr int kFewWarps = 8;  // one block per SM
constexpr int kFewThreads = kFewWarps * 32;
constexpr int kJoinThreads = 256;

template <int D>
struct Shape {
  static constexpr int KS = 2048 / D;   // positions of a unit
  static constexpr int SLOT = KS * D * 2;  // bytes of its K or V: 4 KB
  // K and V of two units: a slot is refilled as soon as it is read, so three
  // are on their way while one is worked on
  static constexpr int RING = 4 * SLOT;
  static constexpr int ROWS = kFewRows * D * 4;  // o of a part
  static constexpr int WARP = RING + ROWS;
  static constexpr int SMEM = kFewWarps * WARP;
  static_assert(ROWS <= RING && SMEM <= 224 * 1024, "shared memory");
};

struct FewArgs {
  PagedAttnParams p;
  PagedPrefixParts pre;
  PagedParts ws;
  int* tickets;   // per item: parts written so far
  int row_limit;  // rows per item, at most
};

// Row of an item's own state.
__device__ __forceinline__ long long state_row(const FewArgs& a, const FewItem& it, int row) {
  return a.ws.state_base + (a.ws.by_token ? out_row(a.p, it, row)
                                          : ((long long)it.b * a.p.g.nkv + it.h) * kFewRows + row);
}

// Two probabilities in 16 bits: fp16 rounds them.  bf16 takes hi + lo, hi cut off
// and lo the rest, at least 2^-18 of the whole: both are positive where the
// probability is (from 2^-115 on), so an infinity in V keeps its sign in both
// products, where a lo of 0 or below would make it NaN.  The sum is off by 2^-16.
template <typename T>
__device__ __forceinline__ void split_weights(float a, float b, uint32_t& hi, uint32_t& lo) {
  if constexpr (MmaKind<T>::kAttnHiLo) {
    const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
    hi = __byte_perm(x, y, 0x7632);
    lo = pack2<T>(fmaxf(a - __uint_as_float(x & 0xffff0000u), a * 0x1p-18f),
                  fmaxf(b - __uint_as_float(y & 0xffff0000u), b * 0x1p-18f));
  } else {
    hi = pack2<T>(a, b);
  }
}

template <typename T, int D, int MODE>
__global__ void __launch_bounds__(kFewThreads, 1)
    paged_few_kernel(const __grid_constant__ FewArgs a) {
  using S = Shape<D>;
  constexpr bool PRE = MODE == kPrefix;
  constexpr int KS = S::KS;
  constexpr int C = D / 8;   // 16-byte chunks of a row
  constexpr int NT = KS / 8;  // key octets of a stage
  constexpr int NO = D / 8;   // column octets of o
  using M = MmaKind<T>;
  constexpr int LIFT = weight_lift<T>(0);
  const PagedAttnParams& p = a.p;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_first[kFewThreads];  // first unit of each thread's sequences
  __shared__ long long s_scan[kFewWarps];
  __shared__ int s_top[kFewWarps];
  __shared__ uint32_t s_valid[kFewWarps][2];
  // per warp: the part of an item that began before its run (F), and of one
  // that goes on behind it (L; if it also began before, there is no F)
  __shared__ FewItem s_item[2][kFewWarps];
  __shared__ float2 s_ml[2][kFewWarps][kFewRows];
  __shared__ int s_has[2][kFewWarps];
  __shared__ int s_last[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gq = lane >> 2, tq = lane & 3;

  // After a prefix launch this one reads only what that launch has waited for
  // already (pdl_wait), so it starts beside its last blocks and waits for it at
  // the end.
  if constexpr (MODE != kOwnAfterPrefix) pdl_wait();
  pdl_trigger();

  // Units of every sequence, summed up over the batch: each thread has a run
  // of sequences.
  const int nseq = PRE ? 1 : p.batch;
  const int per = (nseq + kFewThreads - 1) / kFewThreads;
  long long mine = 0;
  int top = 0;  // units of the longest item
  for (int b = tid * per; b < min(nseq, (tid + 1) * per); ++b) {
    const int t = work_of<KS, PRE>(p, b).tiles;
    mine += (long long)t * p.g.nkv;
    top = max(top, t);
  }
  top = __reduce_max_sync(~0u, top);
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(~0u, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) {
    s_scan[warp] = incl;
    s_top[warp] = top;
  }
  __syncthreads();
  long long before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kFewWarps; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
    top = max(top, s_top[w]);
  }
  s_first[tid] = before;
  const long long block_upc =
      PRE ? a.pre.upc : div_units(total + gridDim.x * kFewWarps - 1, gridDim.x * kFewWarps) * kFewWarps;
  if (lane == 0) s_has[0][warp] = s_has[1][warp] = 0;
  __syncthreads();

  // A cursor at unit u of the line.
  auto locate = [&](Cursor<KS, PRE>& c, long long u) {
    // the last run of sequences that begins at or before unit u
    int n = 0;
#pragma unroll
    for (int i = 0; i < kFewThreads / 32; ++i)
      n += __popc(__ballot_sync(~0u, s_first[i * 32 + lane] <= u));
    long long at = s_first[n - 1];
    int b = (n - 1) * per;
    while (true) {
      c.w = work_of<KS, PRE>(p, b);
      const long long len = (long long)c.w.tiles * p.g.nkv;
      if (u < at + len || b + 1 >= nseq) break;
      at += len;
      ++b;
    }
    c.b = b;
    const long long off = u - at;
    c.h = (int)div_units(off, max(c.w.tiles, 1));
    c.tile = (int)(off - (long long)c.h * c.w.tiles);
    c.i0 = u - c.tile;
    c.u = u;
  };
  // This block's units.  Where items are short, by themselves or beside a
  // block's share, a block takes the items that begin in its share, whole:
  // one item more at most, and nothing to join across blocks.  That takes about
  // 4 us for 4 rows and 10 us for 16, the time of 24 and 60 units.
  Cursor<KS, PRE> cur;
  long long lo = min(total, blockIdx.x * block_upc), hi = min(total, lo + block_upc);
  const bool snap = !PRE && block_upc >= 3LL * top && (top <= 16 + 2 * a.row_limit || block_upc >= 8LL * top);
  if (snap) {
    if (lo < total) {
      locate(cur, lo);
      if (cur.tile) lo = cur.i0 + cur.w.tiles;
    }
    if (hi < total) {
      locate(cur, hi);
      if (cur.tile) hi = cur.i0 + cur.w.tiles;
    }
  }
  if (lo >= hi) {
    if constexpr (MODE == kOwnAfterPrefix) pdl_wait();
    return;
  }
  // and this warp's run of them
  const int run = (int)((hi - lo + kFewWarps - 1) / kFewWarps);
  cur.u = lo + (long long)warp * run;
  cur.end = min(hi, cur.u + run);
  if (cur.u < cur.end) locate(cur, cur.u);

  const char* kbase = static_cast<const char*>(p.k_pages);
  const char* vbase = static_cast<const char*>(p.v_pages);
  uint8_t* mem = smem + warp * S::WARP;
  const uint32_t ring_s = smem_u32(mem);

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
  // Copies a unit's K or V into a slot; lane i holds position i's byte offset,
  // or -1 (zeros).
  constexpr int RP = 32 / C;  // rows of one copy instruction
  const int r0 = lane / C, c0 = lane % C;
  const uint32_t d0 = ring_s + r0 * (D * 2) + ((c0 ^ r0) << 4);
  const int64_t ss = p.g.slot_stride * 2;
  const bool octets = p.g.page_shift >= 3;
  auto copy = [&](int slot, const char* src, int64_t off) {
    const uint32_t d = d0 + slot * S::SLOT;
    if (octets && __all_sync(~0u, off >= 0 || lane >= KS)) {
      // eight consecutive positions lie in one page: one lookup serves them
#pragma unroll
      for (int y = 0; y < KS / 8; ++y) {
        const char* at = src + __shfl_sync(~0u, off, 8 * y) + r0 * ss + c0 * 16;
#pragma unroll
        for (int z = 0; z < 8 / RP; ++z) {
          cp16((d + (8 * y + z * RP) * (D * 2)) ^ ((z * RP) << 4), at);
          at += RP * ss;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < KS / RP; ++i) {
        const int64_t o = __shfl_sync(~0u, off, i * RP + r0);
        cp16((d + i * RP * (D * 2)) ^ (((i * RP) & 7) << 4), src + (o >= 0 ? o + c0 * 16 : 0),
             o >= 0);
      }
    }
  };
  int64_t v_off = -1;  // of the unit whose V is still to be copied
  bool v_some = false;
  auto issue_k = [&](int pair) {
    v_some = false;
    if (ld.u < ld.end) {
      v_off = -1;  // no copy: zeros
      if (ld_pos >= 0) {
        if ((unsigned)ld_page >= (unsigned)p.g.num_pages)
          atomicOr(p.errflag, kDevErrPosRange);
        else
          v_off = ((int64_t)ld_page * p.g.page_stride +
                   (int64_t)(ld_pos & p.g.page_mask) * p.g.slot_stride +
                   (int64_t)ld.h * p.g.head_stride) * 2;
      }
      const uint32_t valid = __ballot_sync(~0u, ld_pos >= 0);
      if (lane == 0) s_valid[warp][pair] = valid;
      v_some = valid != 0;
      const int ob = ld.b, oh = ld.h;
      ld.next(p);
      fetch_page();
      if (v_some) copy(2 * pair, kbase, v_off);
      if (ld.u < ld.end && (ld.b != ob || ld.h != oh)) {  // the next item's queries
        const int row = lane * 64 / D, i = row / p.g.G;
        if (row < ld.w.n * p.g.G)
          prefetch_line(static_cast<const T*>(p.q) + (int64_t)(ld.w.t0 + i) * p.q_stride +
                        (int64_t)(ld.h * p.g.G + row - i * p.g.G) * D + lane * 64 % D);
      }
    }
    cp_commit();
  };
  auto issue_v = [&](int pair) {
    if (v_some) copy(2 * pair + 1, vbase, v_off);
    cp_commit();
  };

  fetch_page();
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    issue_k(s);
    issue_v(s);
  }

  int pair = 0;
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
    cp_wait<3>();  // K has landed
    __syncwarp();
    const uint32_t valid = s_valid[warp][pair];
    const uint32_t ks = ring_s + 2 * pair * S::SLOT, vs = ks + S::SLOT;
    float c[NT][4];
    bool edge = false;  // do the rows see different parts of this tile?
    if (valid) {
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
    }
    __syncwarp();  // K is read before its next copies are issued
    issue_k(pair);
    if (valid) {
      // mask, running maximum
      const int j0 = cur.w.base(cur.tile);
      edge = !PRE && cur.w.n > 1 &&
                        (j0 + KS - 1 > cur.w.p0 ||
                         (p.window != 0 && cur.w.p0 + cur.w.n - 1 - j0 >= p.window));
      float mx[2] = {m[0], m[1]};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int jj = nt * 8 + 2 * tq + (e & 1);
          bool see = (valid >> jj) & 1;
          if (edge) see = see && paged_visible(pos[e >> 1], j0 + jj, p.window, p.n_sinks);
          c[nt][e] = see ? c[nt][e] * p.scale_log2 : -INFINITY;
          mx[e >> 1] = fmaxf(mx[e >> 1], c[nt][e]);
        }
      float corr[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(~0u, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(~0u, mx[r], 2));
        const float ref = mx[r] == -INFINITY ? 0.f : mx[r];
        corr[r] = ex2(m[r] - ref);
        m[r] = mx[r];
        mx[r] = ref - LIFT;
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
          c[nt][e] = ex2(c[nt][e] - mx[e >> 1]);
          l[e >> 1] += c[nt][e];
        }
    }
    cp_wait<3>();  // V has landed
    __syncwarp();
    if (valid) {
      // Where rows see different parts of a tile, an infinity or NaN in V that
      // one row sees would reach the others as 0 * inf: such a tile is summed
      // without the tensor cores, by the rows that see it.
      bool apart = false;
      if (edge) {
        bool bad = false;
#pragma unroll
        for (int i = 0; i < S::SLOT / 512; ++i) {
          uint32_t w[4];
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                       : "r"(vs + (i * 32 + lane) * 16));
#pragma unroll
          for (int e = 0; e < 4; ++e) bad |= nonfinite2<T>(w[e]);
        }
        apart = __any_sync(~0u, bad);
      }
      if (apart) {
        const int j0 = cur.w.base(cur.tile);
#pragma unroll
        for (int x = 0; x < NT * 2; ++x) {
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            const int jj = (x >> 1) * 8 + 2 * q + (x & 1);
            const float w0 = __shfl_sync(~0u, c[x >> 1][x & 1], gq * 4 + q);
            const float w1 = __shfl_sync(~0u, c[x >> 1][2 + (x & 1)], gq * 4 + q);
            const bool there = (valid >> jj) & 1;
            const bool s0 = there && paged_visible(pos[0], j0 + jj, p.window, p.n_sinks);
            const bool s1 = there && paged_visible(pos[1], j0 + jj, p.window, p.n_sinks);
#pragma unroll
            for (int k = 0; k < NO; ++k) {
              uint32_t v;
              asm volatile("ld.shared.u32 %0, [%1];"
                           : "=r"(v)
                           : "r"(vs + jj * (D * 2) + ((k ^ (jj & 7)) << 4) + tq * 4));
              float f[2];
              Elem<T>::words(&v, 1, f);
              if (s0) {
                o[k][0] = fmaf(w0, f[0], o[k][0]);
                o[k][1] = fmaf(w0, f[1], o[k][1]);
              }
              if (s1) {
                o[k][2] = fmaf(w1, f[0], o[k][2]);
                o[k][3] = fmaf(w1, f[1], o[k][3]);
              }
            }
          }
        }
      } else {
      // o += P V; bf16 probabilities enter as hi + lo pairs (the tensor cores
      // have the time), fp16 ones with their 11 bits, times 2^LIFT
#pragma unroll
      for (int kk = 0; kk < KS / 16; ++kk) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
          split_weights<T>(c[2 * kk + (x >> 1)][2 * (x & 1)],
                           c[2 * kk + (x >> 1)][2 * (x & 1) + 1], hi[x], lo[x]);
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
    }
    __syncwarp();
    issue_v(pair);
    pair ^= 1;

    const bool item_done = cur.tile + 1 == cur.w.tiles;
    if (!item_done && cur.u + 1 < cur.end) {
      cur.next(p);
      continue;
    }

    // ---- the warp's part of the item is complete
    const bool begins = first_tile == 0;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(~0u, l[r], 1);
      l[r] += __shfl_xor_sync(~0u, l[r], 2);
    }
    if constexpr (LIFT != 0) {
      constexpr float back = 1.f / (1 << LIFT);
      l[0] *= back;
      l[1] *= back;
#pragma unroll
      for (int k = 0; k < NO; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[k][e] *= back;
    }
    FewItem it;
    it.i0 = cur.i0;
    it.tiles = cur.w.tiles;
    it.t0 = cur.w.t0;
    it.p0 = cur.w.p0;
    it.n = cur.w.n;
    it.b = cur.b;
    it.h = cur.h;
    if (!begins || !item_done) {
      // kept in shared memory until the block's warps are done; the ring is
      // free at the run's end, where an L is left
      const int kind = item_done ? 0 : 1;
      if (kind) {
        cp_wait<0>();
        __syncwarp();
      }
      float* dst = reinterpret_cast<float*>(kind ? mem : mem + S::RING);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (gq + 8 * r >= nrows) continue;
        if (tq == 0) s_ml[kind][warp][gq + 8 * r] = make_float2(m[r], l[r]);
#pragma unroll
        for (int k = 0; k < NO; ++k)
          *reinterpret_cast<float2*>(dst + (gq + 8 * r) * D + 8 * k + 2 * tq) =
              make_float2(o[k][2 * r], o[k][2 * r + 1]);
      }
      if (lane == 0) {
        s_item[kind][warp] = it;
        s_has[kind][warp] = 1;
      }
    } else if (MODE != kOwn && (PRE || it.n <= p.max_q)) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = gq + 8 * r;
        if (row >= nrows) continue;
        const long long at = state_row(a, it, row);
        if (tq == 0) __stcg(a.ws.ml + at, make_float2(m[r], l[r]));
#pragma unroll
        for (int k = 0; k < NO; ++k)
          __stcg(reinterpret_cast<float2*>(a.ws.o + at * D + 8 * k + 2 * tq),
                 make_float2(o[k][2 * r], o[k][2 * r + 1]));
      }
    } else {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = gq + 8 * r;
        const long long at = out_row(p, it, row);
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
        if (p.lse && row < nrows && tq == 0) p.lse[at] = paged_lse(m[r], l[r]);
      }
      // a sequence with more tokens than the call allows has no keys: its
      // other rows are zero too
      for (int x = kFewRows * (D / 4) + lane; !PRE && x < nrows * (D / 4); x += 32) {
        const PagedState4 none{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
        paged_store4<T, D>(none, p.out, p.lse, out_row(p, it, x / (D / 4)), x % (D / 4) * 4);
      }
    }
    cur.next(p);
    fresh = true;
    first_tile = cur.tile;
  }
  cp_wait<0>();
  __syncthreads();

  // ---- items that several warps share.  The parts of one lie side by side:
  // L of the warp that begins it, L of those it runs through, F of the last.
  constexpr int C4 = D / 4;
  auto finish = [&](PagedState4& s, const FewItem& it, int row, int col) {
    if (MODE == kOwn) {
      paged_store4<T, D>(s, p.out, p.lse, out_row(p, it, row), col);
    } else {
      const long long at = state_row(a, it, row);
      __stcg(reinterpret_cast<float4*>(a.ws.o + at * D + col), s.o);
      if (col == 0) __stcg(a.ws.ml + at, make_float2(s.m, s.l));
    }
  };
  if (tid < 2) s_last[tid] = 0;
  FewItem cut[2];                 // items that go on in other blocks: the first's, the last's
  bool has_cut[2] = {false, false};
  int task = 0;
  for (int w0 = 0, k0 = 0; w0 < kFewWarps;) {
    if (!s_has[k0][w0]) {
      w0 += k0;
      k0 ^= 1;
      continue;
    }
    const FewItem it = s_item[k0][w0];
    int last = w0, kind = k0;  // of the item's last part in this block
    while (kind == 1 && last + 1 < kFewWarps) {
      ++last;
      kind = s_has[0][last] ? 0 : 1;
    }
    const bool here = it.i0 >= lo;  // begins in this block
    const long long slot = 2 * (long long)blockIdx.x + (lo >= it.i0 ? 0 : 1);
    // rows are dealt out to the warps across items
    const int nrows = it.n * p.g.G, col = (lane % C4) * 4;
    for (int row0 = 0; row0 < nrows; row0 += 32 / C4, ++task) {
      const int row = row0 + lane / C4;
      if (task % kFewWarps != warp || row >= nrows) continue;
      PagedState4 s{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
      for (int w = w0; w <= last; ++w) {
        const int k = w == last ? kind : 1;
        const float* src =
            reinterpret_cast<const float*>(smem + w * S::WARP + (k ? 0 : S::RING)) + row * D + col;
        s.join(s_ml[k][w][row].x, s_ml[k][w][row].y, *reinterpret_cast<const float4*>(src));
      }
      if (here && kind == 0) {
        finish(s, it, row, col);
      } else {
        const long long at = slot * kFewRows + row;
        __stcg(reinterpret_cast<float4*>(a.ws.o + at * D + col), s.o);
        if (col == 0) __stcg(a.ws.ml + at, make_float2(s.m, s.l));
      }
    }
    if (!here || kind != 0) {
      cut[here ? 1 : 0] = it;
      has_cut[here ? 1 : 0] = true;
    }
    // on to what follows that part: after an F its warp's L, if any
    w0 = kind == 0 ? last : kFewWarps;
    k0 = 1;
  }
  if constexpr (MODE == kOwnAfterPrefix) pdl_wait();
  if (PRE || !(has_cut[0] || has_cut[1])) return;
  __syncthreads();
  if (tid < 2 && has_cut[tid]) {
    __threadfence();
    const FewItem it = cut[tid];
    const PagedItemParts parts(it.i0, it.tiles, block_upc);
    int* ticket = a.tickets + (long long)it.b * p.g.nkv + it.h;
    if (atomicAdd(ticket, 1) == parts.n - 1) {
      *ticket = 0;
      s_last[tid] = 1;
      __threadfence();
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (!s_last[i]) continue;
    const PagedItemParts parts(cut[i].i0, cut[i].tiles, block_upc);
    for (int x = tid; x < cut[i].n * p.g.G * C4; x += kFewThreads) {
      const int row = x / C4, col = (x - row * C4) * 4;
      PagedState4 s{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
      paged_join_row<D>(s, a.ws.o, a.ws.ml, PagedRowParts(parts, kFewRows, row, -1), col);
      finish(s, cut[i], row, col);
    }
  }
}

// Joins the own states of every row and the prefix's: a row per D / 4 lanes.
// Eight parts in flight per lane at two blocks on an SM: 51 us for 64 sequences
// behind 8192 shared positions (32 / 8 heads of 128), 197 for 128 of 4 tokens
// behind 16385; four at more blocks: 53 and 190.
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads, 2)
    paged_few_join_kernel(const __grid_constant__ FewArgs a) {
  constexpr int W = D / 4, NG = kJoinThreads / W;
  const PagedAttnParams& p = a.p;
  const int tid = threadIdx.x, col = (tid % W) * 4;
  pdl_wait();
  pdl_trigger();
  const long long rows = (long long)p.batch * p.g.nkv * a.row_limit;
  for (long long x = (long long)blockIdx.x * NG + tid / W; x < rows; x += (long long)gridDim.x * NG) {
    const long long pair = div_units(x, a.row_limit);
    const int row = (int)(x - pair * a.row_limit);
    FewItem it;
    it.b = (int)div_units(pair, p.g.nkv);
    it.h = (int)(pair - (long long)it.b * p.g.nkv);
    const PagedSeq q = paged_seq(p.q_start, p.kv_len, it.b, p.n_tokens, p.max_q, p.g, p.errflag);
    // (a sequence with more tokens than the call allows is written already)
    if (row >= q.n * p.g.G || q.n > p.max_q) continue;
    it.t0 = q.t0;
    const long long at = state_row(a, it, row);
    const float2 ml = __ldcg(a.ws.ml + at);
    PagedState4 s{ml.x, ml.y, __ldcg(reinterpret_cast<const float4*>(a.ws.o + at * D + col))};
    const int i = row / p.g.G;
    if (q.len - q.n + i >= 0)
      paged_join_row<D>(s, a.pre.o, a.pre.ml,
                        paged_prefix_row(a.pre, p.g, it.t0 + i, it.h, row - i * p.g.G), col);
    paged_store4<T, D>(s, p.out, p.lse, out_row(p, it, row), col);
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
  return sm_count;
}

long long cf::paged_few_part_rows(int grid) { return 2LL * grid * kFewRows; }

PagedPrefixParts cf::paged_few_prefix(const PagedAttnParams& p, const PagedSplit& ws) {
  const int KS = p.g.D == 64 ? Shape<64>::KS : Shape<128>::KS;
  const long long warps = (long long)ws.grid * kFewWarps;
  PagedPrefixParts x;
  x.o = ws.parts.o;
  x.ml = ws.parts.ml;
  x.state_base = ws.parts.state_base;
  x.rows = kFewRows;
  x.tiles = (p.prefix_len + KS - 1) / KS;
  x.item_cost = 0;
  x.upc = ((long long)x.tiles * p.g.nkv + warps - 1) / warps * kFewWarps;  // a block's
  return x;
}

bool cf::paged_few_launch(int dtype, const PagedAttnParams& p, const PagedSplit& ws, PagedMode mode,
                          const PagedPrefixParts& pre, cudaStream_t st) {
  const FewFns f = few_fns(dtype, p.g.D, mode);
  FewArgs a;
  a.p = p;
  a.pre = pre;
  a.ws = ws.parts;
  a.tickets = ws.tickets;
  a.row_limit = std::min(kFewRows, p.max_q * p.g.G);
  void* args[] = {&a};
  if (!launch_pdl(f.main, dim3(ws.grid), kFewThreads, f.smem, st, args)) return false;
  if (mode != kOwnAfterPrefix) return true;
  const int ng = kJoinThreads / (p.g.D / 4);
  const long long rows = (long long)p.batch * p.g.nkv * a.row_limit;
  return launch_pdl(f.join, dim3((unsigned)std::min<long long>(8LL * ws.grid, (rows + ng - 1) / ng)),
                    kJoinThreads, 0, st, args);
}
