// cf_paged8_few.cu -- attention over the paged cache of 8-bit codes for few
// rows per KV head: single tokens and short drafts (tokens x grouped heads <=
// 16).
//
// 16 sequences of 4097 positions, 32 / 8 heads of 128: 35 us, 4.0 TB/s (the 16-bit
// cache: 54); 32 of 2383-32504: 186-200, 5.8-6.2 TB/s; one of 1025, 32 heads: 12; 4
// draft tokens of 32 sequences of 1070-4093 (16 rows): 63.  Half the bytes to the
// arithmetic of the 16-bit cache: the work per byte decides the form.  Keys and values are
// the A operand of mma.sync m16n8k16 and the rows its B operand, in octets:
// S^T = K Q^T (16 keys x 8 rows) and O^T = V^T P^T (16 columns x 8 rows), so
// up to 8 rows cost half the products, exponentials and registers of a 16-row
// tile.  Codes become fp16 in registers, four at a time; the order of a head's
// elements in the products is free, so a lane's keys are 16-byte reads without
// a transposition, and the pairs of columns that a transposing load gives for
// V are two rows of O^T.
//
// Scales: with a_j = scale ks_j log2(e) and b_j = log2 vs_j, the weight of
// value j is exp(s_j) vs_j = 2^(a_j q.k_j + b_j), so one fused product, one
// maximum and one exponential serve the weights, whatever the scales are; the
// sum of exp(s_j) takes the weight times 1 / vs_j, or where scales lie far apart an
// exponential of its own (ValueScale).  Weights enter the second product as one
// fp16 value: a relative 2^-12 each, by which results in fp16 are off 2.2e-4 of their
// norm for the 2.1e-4 of their own rounding; a second value for the rest would double
// that product.
//
// A unit of 32 positions takes a warp 820 instructions (e4m3, 8 rows), 55 % of the
// SM's issue slots at the copy rate, but 5500 cycles: with three warps to a
// scheduler the chains are not hidden.  16 warps of 128 registers spill (40 us for
// 36), 10 with two units on their way have fewer to switch between (41).  A fixed
// 10-12 us are the schedule, the first loads and the joins.
//
// The cut of the work, rings and joins are those of cf_paged_few.cu: the key
// tiles of all (sequence, KV head) items are one line that the warps share
// evenly; a warp runs through its tiles with a cp.async ring of its own; the
// block joins what its warps share, the last block of a split item the rest.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "cf_mma.cuh"
#include "cf_paged8.cuh"
#include "cf_paged_few.cuh"

using namespace cf;

namespace {

constexpr int KS = 32;  // positions of a unit

// One block per SM.
// NT octets of rows: with one the kernel takes 36 us for 4 rows (16 sequences of
// 4097 positions), with two 44.
template <int D, int NT>
struct Shape8 {
  static constexpr int WARPS = NT == 1 ? 12 : 8, THREADS = 32 * WARPS;
  static constexpr int SLOT = KS * D;              // bytes of a unit's K or V
  static constexpr int PAIRS = D == 128 ? NT : 2;   // units whose K and V are on their way
  static constexpr int SCALES = KS * 8;
  static constexpr int PREP = KS * 16;             // what the weights take of a unit's scales
  static constexpr int RING = PAIRS * (2 * SLOT + SCALES) + PREP;
  static constexpr int ROWS = 8 * NT * D * 4;      // o of a part
  static constexpr int WARP = RING + ROWS;
  static constexpr int SMEM = WARPS * WARP;
  static_assert(ROWS <= PAIRS * 2 * SLOT && SMEM <= 220 * 1024, "shared memory");
};

struct Few8Args {
  PagedAttnParams p;
  PagedParts ws;
  int* tickets;   // per item: parts written so far
  int row_limit;  // rows per item, at most
};

__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 w;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
               : "r"(at));
  return w;
}
template <typename T, int D, int CODE, int NT>
__global__ void __launch_bounds__(Shape8<D, NT>::THREADS, 1)
    paged8_few_kernel(const __grid_constant__ Few8Args a) {
  using S = Shape8<D, NT>;
  using M = MmaKind<__half>;
  constexpr int MT = KS / 16;     // key tiles of a unit
  constexpr int NH = D / 64;      // 64-element pieces of a head
  constexpr int NJ = D / 16;      // 16-column tiles of o
  constexpr int PAIRS = S::PAIRS, WARPS = S::WARPS, THREADS = S::THREADS;
  constexpr int LIFT = weight_lift<__half>(0);
  const PagedAttnParams& p = a.p;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_first[THREADS];  // first unit of each thread's sequences
  __shared__ long long s_scan[WARPS];
  __shared__ int s_top[WARPS];
  // per warp: the part of an item that began before its run (F), and of one
  // that goes on behind it (L; if it also began before, there is no F)
  __shared__ FewItem s_item[2][WARPS];
  __shared__ float2 s_ml[2][WARPS][kFewRows];
  __shared__ int s_has[2][WARPS];
  __shared__ int s_last[2];
  // each warp's place, and that of its copies, ahead of it: too much for
  // registers.  One lane moves them on.
  __shared__ Cursor<KS, false> s_cur[WARPS], s_ld[WARPS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gq = lane >> 2, tq = lane & 3;

  pdl_wait();
  pdl_trigger();

  // Units of every sequence, summed up over the batch: each lane of every warp
  // has one or, with more than 32, each thread a run of them.
  const bool small = p.batch <= 32;
  const int per = small ? 1 : (p.batch + THREADS - 1) / THREADS;
  const int mine0 = small ? lane : tid * per;
  long long mine = 0;
  int top = 0;  // units of the longest item
  for (int b = mine0; b < min(p.batch, mine0 + per); ++b) {
    const int t = work_of<KS, false>(p, b).tiles;
    mine += (long long)t * p.g.nkv;
    top = max(top, t);
  }
  const int own_tiles = top;  // (of the lane's one sequence)
  top = __reduce_max_sync(~0u, top);
  auto scan = [&](long long x) {  // sums up to each lane's
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(~0u, x, o);
      if (lane >= o) x += v;
    }
    return x;
  };
  long long incl = scan(mine);
  long long before = incl - mine, total = __shfl_sync(~0u, incl, 31);
  if (!small) {
    if (lane == 31) {
      s_scan[warp] = incl;
      s_top[warp] = top;
    }
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) before += s_scan[w];
      total += s_scan[w];
      top = max(top, s_top[w]);
    }
    s_first[tid] = before;
  }
  const long long block_upc = div_units(total + gridDim.x * WARPS - 1, gridDim.x * WARPS) * WARPS;
  if (lane == 0) s_has[0][warp] = s_has[1][warp] = 0;
  if (!small) __syncthreads();
  // Where there is little work and the blocks are enough for it, an item takes whole
  // ones: it is cut into fewer parts, and no block has parts of two.  Without and
  // with, us: one sequence of 4097 positions, 32 / 8 heads of 128, 14.1 and 12.8, of
  // 101 10.1 and 8.4; 24 of 301, 16 / 4 heads, 13.0 and 9.3; 2 of 8001, 32 heads, 34.3
  // and 34.3.  Where they are not enough, the question costs 0.1 (32 heads, 8 of
  // 301-901, 19.7 and 19.8; 4 of 501-2001, 21.4 and 21.6).
  int pad = 0;
  if (small && total > 0 && block_upc <= 4 * WARPS) {
    const int n = (int)block_upc, blocks = (own_tiles + n - 1) / n * p.g.nkv;
    const uint32_t all = __reduce_add_sync(~0u, (uint32_t)blocks);
    if (all <= gridDim.x) {
      pad = n;
      mine = (long long)blocks * n;
      before = scan(mine) - mine;
      total = (long long)all * n;
    }
  }
  auto units = [&](int tiles) { return pad ? (tiles + pad - 1) / pad * pad : tiles; };

  // A cursor at unit u of the line.
  auto locate = [&](Cursor<KS, false>& c, long long u) {
    // the last run of sequences that begins at or before unit u
    int n = 0;
    long long at;
    if (small) {
      n = __popc(__ballot_sync(~0u, lane < p.batch && before <= u));
      at = __shfl_sync(~0u, before, n - 1);
    } else {
#pragma unroll
      for (int i = 0; i < THREADS / 32; ++i)
        n += __popc(__ballot_sync(~0u, s_first[i * 32 + lane] <= u));
      at = s_first[n - 1];
    }
    int b = (n - 1) * per;
    while (true) {
      c.w = work_of<KS, false>(p, b);
      const long long len = (long long)units(c.w.tiles) * p.g.nkv;
      if (u < at + len || b + 1 >= p.batch) break;
      at += len;
      ++b;
    }
    c.b = b;
    const long long off = u - at;
    const int wide = units(c.w.tiles);
    c.h = (int)div_units(off, max(wide, 1));
    c.tile = (int)(off - (long long)c.h * wide);
    c.i0 = u - c.tile;
    c.u = u;
  };
  // This block's units.  Where items are short, by themselves or beside a
  // block's share, a block takes the items that begin in its share, whole:
  // one item more at most, and nothing to join across blocks.
  Cursor<KS, false> at;
  long long lo = min(total, blockIdx.x * block_upc), hi = min(total, lo + block_upc);
  const bool snap =
      !pad && block_upc >= 3LL * top && (top <= 16 + 2 * a.row_limit || block_upc >= 8LL * top);
  if (snap) {
    if (lo < total) {
      locate(at, lo);
      if (at.tile) lo = at.i0 + at.w.tiles;
    }
    if (hi < total) {
      locate(at, hi);
      if (at.tile) hi = at.i0 + at.w.tiles;
    }
  }
  if (lo >= hi) return;
  if (pad) {  // without what only fills the last block
    locate(at, lo);
    hi = min(hi, at.i0 + at.w.tiles);
  }
  // and this warp's run of them
  const int run = (int)((hi - lo + WARPS - 1) / WARPS);
  at.u = lo + (long long)warp * run;
  at.end = min(hi, at.u + run);
  if (at.u < at.end) locate(at, at.u);
  Cursor<KS, false>&cur = s_cur[warp], &ld = s_ld[warp];
  if (lane == 0) cur = ld = at;
  __syncwarp();

  uint8_t* mem = smem + warp * S::WARP;
  const uint32_t ring_s = smem_u32(mem);
  const uint32_t scale_s = ring_s + PAIRS * 2 * S::SLOT, prep_s = scale_s + PAIRS * S::SCALES;

  // The unit whose copies are next: ld stands on its item's first one in this
  // run or on the one itself, ld_tile and ld_left say which, and how many units
  // of the item are left to this run.
  int ld_tile = ld.tile, ld_left = 0;
  if (ld.u < ld.end) ld_left = (int)min((long long)(ld.w.tiles - ld.tile), ld.end - ld.u);
  // The page of this lane's position in it, fetched one unit before its copies
  // are issued (a coherent load: the launch in front may have written the table).
  int ld_pos = -1, ld_page = -1;
  auto fetch_page = [&]() {
    ld_pos = -1;
    if (ld_left == 0) return;
    const int j = ld.w.base(ld_tile) + lane;
    if (!ld.w.sees(j)) return;
    ld_pos = j;
    ld_page = p.page_table[(int64_t)ld.b * p.g.max_pages + (j >> p.g.page_shift)];
  };
  // Copies a unit's K or V into a slot; lane i holds position i's byte offset,
  // or -1 (zeros).  Chunks of 16 bytes are swizzled so that the reads below
  // are free of bank conflicts: keys by two rows, values by eight.
  constexpr int C = D / 16;   // chunks of a row
  constexpr int RP = 32 / C;  // rows of one copy instruction
  const int r0 = lane / C, c0 = lane % C;
  const uint32_t k0 = ring_s + r0 * D + ((D == 128 ? c0 ^ ((r0 & 1) << 2) : c0) << 4);
  const uint32_t v0 =
      ring_s + S::SLOT + r0 * D + ((D == 128 ? c0 ^ r0 : c0 ^ ((r0 >> 1) & 3)) << 4);
  const char* kbase = static_cast<const char*>(p.k_pages) + c0 * 16;
  const char* vbase = static_cast<const char*>(p.v_pages) + c0 * 16;
  const int64_t step = RP * p.g.slot_stride, own = r0 * p.g.slot_stride;
  const bool octets = p.g.page_shift >= 3;
  auto copy = [&](uint32_t d, bool values, const char* src, int64_t off) {
    // the swizzle of a later row of the same lane (D = 128: rows 4 apart)
    const uint32_t d4 = values && D == 128 ? d ^ 64u : d;
    if (octets && __all_sync(~0u, off >= 0)) {
      // eight consecutive positions lie in one page: one lookup serves them
#pragma unroll
      for (int y = 0; y < KS / 8; ++y) {
        const char* at = src + own + __shfl_sync(~0u, off, 8 * y);
        cp16(d + 8 * y * D, at);
        if constexpr (RP == 4) cp16(d4 + (8 * y + 4) * D, at + step);
      }
    } else {
#pragma unroll
      for (int i = 0; i < KS / RP; ++i) {
        const int64_t o = __shfl_sync(~0u, off, i * RP + r0);
        cp16((i * RP & 4 ? d4 : d) + i * RP * D, src + (o >= 0 ? o : 0), o >= 0);
      }
    }
  };
  int64_t v_off = -1;  // of the unit whose V is still to be copied
  bool v_some = false;
  auto issue_k = [&](int pair) {
    v_some = false;
    if (ld_left) {
      v_off = -1;  // no copy: zeros
      int64_t sc = 0;
      if (ld_pos >= 0) {
        if ((unsigned)ld_page >= (unsigned)p.g.num_pages) {
          atomicOr(p.errflag, kDevErrPosRange);
        } else {
          const int slot = ld_pos & p.g.page_mask;
          v_off = (int64_t)ld_page * p.g.page_stride + (int64_t)slot * p.g.slot_stride +
                  (int64_t)ld.h * p.g.head_stride;
          sc = (((int64_t)ld_page * p.g.nkv + ld.h) << p.g.page_shift) + slot;
        }
      }
      v_some = ld.w.hi > ld.w.lo;  // (a sequence without keys has one tile)
      bool other = false;
      if (--ld_left) {
        ++ld_tile;
      } else {
        __syncwarp();
        if (lane == 0) {
          const int passed = ld_tile - ld.tile;
          ld.u += passed;
          ld.tile = ld_tile;
          ld.next(p);
        }
        __syncwarp();
        if (ld.u < ld.end) {
          ld_tile = ld.tile;
          ld_left = (int)min((long long)(ld.w.tiles - ld.tile), ld.end - ld.u);
          other = true;
        }
      }
      fetch_page();
      if (v_some) {
        cp8(scale_s + pair * S::SCALES + lane * 8, p.scales + sc, v_off >= 0);
        copy(k0 + 2 * pair * S::SLOT, false, kbase, v_off);
      }
      if (other) {  // the next item's queries
        const int row = lane * 64 / D, i = row / p.g.G;
        if (row < ld.w.n * p.g.G)
          prefetch_line(static_cast<const T*>(p.q) + (int64_t)(ld.w.t0 + i) * p.q_stride +
                        (int64_t)(ld.h * p.g.G + row - i * p.g.G) * D + lane * 64 % D);
      }
    }
    cp_commit();
  };
  auto issue_v = [&](int pair) {
    if (v_some) copy(v0 + 2 * pair * S::SLOT, true, vbase, v_off);
    cp_commit();
  };

  fetch_page();
#pragma unroll
  for (int s = 0; s < PAIRS; ++s) {
    issue_k(s);
    issue_v(s);
  }

  // where this lane's pieces of K (of key gq) and V (of position lane % 16) lie;
  // their swizzles are whole in the bits that a piece's number is put to by ^
  const uint32_t k_lane = ring_s + gq * D + ((D == 128 ? tq ^ ((gq & 1) << 2) : tq) << 4);
  const uint32_t v_lane =
      ring_s + S::SLOT + (lane & 15) * D +
      (((lane >> 4) ^ (D == 128 ? lane & 7 : (lane >> 1) & 3)) << 4);
  int pair = 0;
  uint32_t qf[NT][D / 16][2];
  float o[NT][NJ][4], m[NT][2], l[NT][2];
  int pos[NT][2];  // positions of rows 8 nt + 2 tq and + 1: this thread's
  float qk = 0.f;  // what q.k is multiplied by beside the key's scale
  int tile = 0, left = 0;  // of the item: the unit in work, units left to this run
  bool high = false;       // has it shown a high value scale (ValueScale)?

  while (cur.u < cur.end) {
    const int nrows = cur.w.n * p.g.G;
    if (left == 0) {
      tile = cur.tile;
      left = (int)min((long long)(cur.w.tiles - tile), cur.end - cur.u);
      high = false;
      uint32_t top2 = 0;  // bf16: largest finite magnitude of the rows, as bits
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int row = gq + 8 * nt, i = row / p.g.G;
        const T* src = static_cast<const T*>(p.q) + (int64_t)(cur.w.t0 + i) * p.q_stride +
                       (int64_t)(cur.h * p.g.G + row - i * p.g.G) * D + 16 * tq;
#pragma unroll
        for (int k = 0; k < NH * 2; ++k) {  // 8 elements: two steps
          const uint4 w = row < nrows
                              ? *reinterpret_cast<const uint4*>(src + (k >> 1) * 64 + (k & 1) * 8)
                              : make_uint4(0, 0, 0, 0);
          qf[nt][2 * k][0] = w.x;
          qf[nt][2 * k][1] = w.y;
          qf[nt][2 * k + 1][0] = w.z;
          qf[nt][2 * k + 1][1] = w.w;
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          pos[nt][r] = cur.w.p0 + (8 * nt + 2 * tq + r) / p.g.G;
          m[nt][r] = -INFINITY;
          l[nt][r] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < NJ; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][k][e] = 0.f;
      }
      float back = 1.f;
      if constexpr (sizeof(T) == 2 && MmaKind<T>::kBf16) {
        // to fp16: times the power of two that takes the largest to 2^14..2^15
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t x = qf[nt][k][e] & 0x7fff7fffu;
              const uint32_t y = x & 0xffffu, z = x >> 16;
              if (y < 0x7f80u) top2 = max(top2, y);
              if (z < 0x7f80u) top2 = max(top2, z);
            }
        top2 = __reduce_max_sync(~0u, top2);
        // exponent of the largest, kept where 2^(14 - e) and its inverse are normal
        const int e = min(max((int)(top2 >> 7) - 127, -100), 127);
        const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
        back = __uint_as_float((uint32_t)(127 - 14 + e) << 23);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float f[2];
              Elem<T>::words(&qf[nt][k][x], 1, f);
              qf[nt][k][x] = pack2<__half>(f[0] * up, f[1] * up);
            }
      }
      qk = back * p.scale_log2;
    }
    cp_wait<2 * PAIRS - 1>();  // K and the scales have landed
    __syncwarp();
    const bool some = cur.w.hi > cur.w.lo;
    const uint32_t k_at = k_lane + 2 * pair * S::SLOT, v_at = v_lane + 2 * pair * S::SLOT;
    const int j0 = cur.w.base(tile);
    float c[MT][NT][4];
    uint32_t apart = 0;  // positions that the sum takes apart (ValueScale)
    if (some) {
      {  // each lane's position: a, b, 1 / vs
        const bool there = cur.w.sees(j0 + lane);
        float k, v;
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                     : "=f"(k), "=f"(v)
                     : "r"(scale_s + pair * S::SCALES + lane * 8));
        const ValueScale vs(v);
        bool alone = false;
        if (__any_sync(~0u, there && !vs.plain)) {
          high |= __any_sync(~0u, there && ValueScale::high(v));
          alone = there && ((ValueScale::low(v) && high) || !scale_is_read(v));
          apart = __ballot_sync(~0u, alone);
        }
        const float ak = there ? key_scale(k) * qk : 0.f, bk = there ? vs.log2 : -INFINITY;
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(prep_s + lane * 16), "f"(ak),
                     "f"(bk), "f"(alone ? 0.f : vs.inv), "f"(there ? v : 0.f)
                     : "memory");
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) c[mt][nt][e] = 0.f;
#pragma unroll
        for (int hf = 0; hf < NH; ++hf) {
          const uint32_t at = (k_at ^ (hf << 6)) + mt * 16 * D;
          const uint4 x = lds16(at), y = lds16(at + 8 * D);
          const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t f[4];
            code_row4<CODE>(xw[w], f[0], f[2]);
            code_row4<CODE>(yw[w], f[1], f[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              M::mma(c[mt][nt], f, qf[nt][hf * 4 + w][0], qf[nt][hf * 4 + w][1]);
          }
        }
      }
    }
    __syncwarp();  // K and the scales are read before their next copies are issued
    issue_k(pair);
    uint32_t pf[MT][NT][2];
    if (some) {
      // mask, running maximum
      const bool edge =  // do the rows see different parts of this tile?
          cur.w.n > 1 && (j0 + KS - 1 > cur.w.p0 ||
                          (p.window != 0 && cur.w.p0 + cur.w.n - 1 - j0 >= p.window));
      float inv[MT][2];  // 1 / vs
      float mx[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mx[nt][0] = m[nt][0];
        mx[nt][1] = m[nt][1];
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int jj = mt * 16 + 8 * r + gq;
          const uint4 w = lds16(prep_s + jj * 16);
          const float ak = __uint_as_float(w.x), bk = __uint_as_float(w.y);
          inv[mt][r] = __uint_as_float(w.z);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float& x = c[mt][nt][2 * r + e];
              x = fmaf(x, ak, bk);
              if (edge && !paged_visible(pos[nt][e], j0 + jj, p.window, p.n_sinks)) x = -INFINITY;
              mx[nt][e] = fmaxf(mx[nt][e], x);
            }
        }
      float corr[NT][2];  // at first the square roots
      bool moved = apart != 0;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int d = 4; d <= 16; d <<= 1)
            mx[nt][e] = fmaxf(mx[nt][e], __shfl_xor_sync(~0u, mx[nt][e], d));
          const float ref = mx[nt][e] == -INFINITY ? 0.f : mx[nt][e];
          // (by halves: with value scales far apart, what the sum is multiplied by can be
          // below 2^-126 and the sum still count)
          corr[nt][e] = ex2(0.5f * (m[nt][e] - ref));
          moved |= corr[nt][e] != 1.f;
          m[nt][e] = mx[nt][e];
          mx[nt][e] = ref - LIFT;
        }
      if (__any_sync(~0u, moved)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            l[nt][e] = l[nt][e] * corr[nt][e] * corr[nt][e];
            corr[nt][e] *= corr[nt][e];
          }
#pragma unroll
          for (int k = 0; k < NJ; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][k][e] *= corr[nt][e & 1];
        }
        if (apart) {  // 2^(s - reference) of those positions
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const int jj = mt * 16 + 8 * r + gq;
              if (!((apart >> jj) & 1)) continue;
              const float b = __uint_as_float(lds16(prep_s + jj * 16).y);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) l[nt][e] += ex2(c[mt][nt][2 * r + e] - b - mx[nt][e]);
            }
          // a value of NaN: o of the rows that see it
          const float v = __uint_as_float(lds16(prep_s + lane * 16).w);
          const uint32_t odd = __ballot_sync(~0u, !scale_is_read(v));
          if (odd) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                bool hit = !edge;
                for (uint32_t w = odd; w; w &= w - 1)
                  hit |= paged_visible(pos[nt][e], j0 + __ffs(w) - 1, p.window, p.n_sinks);
                if (!hit) continue;
#pragma unroll
                for (int k = 0; k < NJ; ++k)
                  o[nt][k][e] = o[nt][k][e + 2] = __uint_as_float(0x7fc00000u);
              }
          }
        }
      }
      // weights, and their sums without the value scales
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float& x = c[mt][nt][e];
            x = ex2(x - mx[nt][e & 1]);
            l[nt][e & 1] = fmaf(x, inv[mt][e >> 1], l[nt][e & 1]);
          }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            pf[mt][nt][r] =
                movmatrix_trans(pack2<__half>(c[mt][nt][2 * r], c[mt][nt][2 * r + 1]));
    }
    cp_wait<2 * PAIRS - 1>();  // V has landed
    __syncwarp();
    if (some) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < NJ; j += 2) {
          uint32_t w[4];
          ldsm_x4_trans(w[0], w[1], w[2], w[3], (v_at ^ (j << 4)) + mt * 16 * D);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t f[4];
            code_halves<CODE>(w[2 * x], f[0], f[1]);
            code_halves<CODE>(w[2 * x + 1], f[2], f[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              M::mma(o[nt][j + x], f, pf[mt][nt][0], pf[mt][nt][1]);
          }
        }
    }
    __syncwarp();
    issue_v(pair);
    if (++pair == PAIRS) pair = 0;

    if (--left) {
      ++tile;
      continue;
    }

    // ---- the warp's part of the item is complete
    const bool begins = cur.tile == 0, item_done = tile + 1 == cur.w.tiles;
    constexpr float back = 1.f / (1 << LIFT);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) l[nt][e] += __shfl_xor_sync(~0u, l[nt][e], d);
        l[nt][e] *= back;
      }
#pragma unroll
      for (int k = 0; k < NJ; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][k][e] *= back;
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
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = 8 * nt + 2 * tq + e;
          if (row >= nrows) continue;
          if (gq == 0) s_ml[kind][warp][row] = make_float2(m[nt][e], l[nt][e]);
#pragma unroll
          for (int k = 0; k < NJ; ++k)
            *reinterpret_cast<float2*>(dst + row * D + 16 * k + 2 * gq) =
                make_float2(o[nt][k][e], o[nt][k][e + 2]);
        }
      if (lane == 0) {
        s_item[kind][warp] = it;
        s_has[kind][warp] = 1;
      }
    } else {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = 8 * nt + 2 * tq + e;
          if (row >= nrows) continue;
          const long long at = out_row(p, it, row);
          const float n = l[nt][e] == 0.f ? 0.f : 1.f / l[nt][e];
#pragma unroll
          for (int k = 0; k < NJ; ++k)
            *reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + at * D + 16 * k + 2 * gq) =
                pack2<T>(o[nt][k][e] * n, o[nt][k][e + 2] * n);
          if (p.lse && gq == 0) p.lse[at] = paged_lse(m[nt][e], l[nt][e]);
        }
      // a sequence with more tokens than the call allows has no keys: its
      // other rows are zero too
      for (int x = 8 * NT * (D / 4) + lane; x < nrows * (D / 4); x += 32) {
        const PagedState4 none{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
        paged_store4<T, D>(none, p.out, p.lse, out_row(p, it, x / (D / 4)), x % (D / 4) * 4);
      }
    }
    __syncwarp();
    if (lane == 0) {
      cur.u += tile - cur.tile;
      cur.tile = tile;
      cur.next(p);
    }
    __syncwarp();
  }
  cp_wait<0>();
  __syncthreads();

  // ---- items that several warps share.  The parts of one lie side by side:
  // L of the warp that begins it, L of those it runs through, F of the last.
  constexpr int C4 = D / 4;
  if (tid < 2) s_last[tid] = 0;
  FewItem cut[2];                 // items that go on in other blocks: the first's, the last's
  bool has_cut[2] = {false, false};
  int task = 0;
  for (int w0 = 0, k0 = 0; w0 < WARPS;) {
    if (!s_has[k0][w0]) {
      w0 += k0;
      k0 ^= 1;
      continue;
    }
    const FewItem it = s_item[k0][w0];
    int last = w0, kind = k0;  // of the item's last part in this block
    while (kind == 1 && last + 1 < WARPS) {
      ++last;
      kind = s_has[0][last] ? 0 : 1;
    }
    const bool here = it.i0 >= lo;  // begins in this block
    const long long slot = 2 * (long long)blockIdx.x + (lo >= it.i0 ? 0 : 1);
    // rows are dealt out to the warps across items
    const int nrows = it.n * p.g.G, col = (lane % C4) * 4;
    for (int row0 = 0; row0 < nrows; row0 += 32 / C4, ++task) {
      const int row = row0 + lane / C4;
      if (task % WARPS != warp || row >= nrows) continue;
      PagedState4 s{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
      for (int w = w0; w <= last; ++w) s.m = fmaxf(s.m, s_ml[w == last ? kind : 1][w][row].x);
      const float ref = s.m == -INFINITY ? 0.f : s.m;
#pragma unroll 4
      for (int w = w0; w <= last; ++w) {
        const int k = w == last ? kind : 1;
        const float2 ml = s_ml[k][w][row];
        const float4 o4 = *reinterpret_cast<const float4*>(
            reinterpret_cast<const float*>(smem + w * S::WARP + (k ? 0 : S::RING)) + row * D + col);
        const float half = ex2(0.5f * (ml.x - ref)), x = half * half;
        s.l = fmaf(ml.y * half, half, s.l);
        s.o.x = fmaf(o4.x, x, s.o.x);
        s.o.y = fmaf(o4.y, x, s.o.y);
        s.o.z = fmaf(o4.z, x, s.o.z);
        s.o.w = fmaf(o4.w, x, s.o.w);
      }
      if (here && kind == 0) {
        paged_store4<T, D>(s, p.out, p.lse, out_row(p, it, row), col);
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
    w0 = kind == 0 ? last : WARPS;
    k0 = 1;
  }
  if (!(has_cut[0] || has_cut[1])) return;
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
    for (int x = tid; x < cut[i].n * p.g.G * C4; x += THREADS) {
      const int row = x / C4, col = (x - row * C4) * 4;
      PagedState4 s{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
      paged_join_row<D, 8, true>(s, a.ws.o, a.ws.ml, PagedRowParts(parts, kFewRows, row, -1), col);
      paged_store4<T, D>(s, p.out, p.lse, out_row(p, cut[i], row), col);
    }
  }
}

struct Few8Fn {
  const void* main;
  int threads, smem;
};
template <typename T, int D, int NT>
Few8Fn few8_code(int code) {
  return Few8Fn{code == CF_CODE_INT8
                    ? (const void*)&paged8_few_kernel<T, D, CF_CODE_INT8, NT>
                    : (const void*)&paged8_few_kernel<T, D, CF_CODE_E4M3, NT>,
                Shape8<D, NT>::THREADS, Shape8<D, NT>::SMEM};
}
template <typename T>
Few8Fn few8_d(int code, int d, int rows) {
  if (d == 64) return rows <= 8 ? few8_code<T, 64, 1>(code) : few8_code<T, 64, 2>(code);
  return rows <= 8 ? few8_code<T, 128, 1>(code) : few8_code<T, 128, 2>(code);
}
// rows: of an item, at most.
Few8Fn few8_fn(int dtype, int code, int d, int rows) {
  return dtype == CF_F16 ? few8_d<__half>(code, d, rows) : few8_d<__nv_bfloat16>(code, d, rows);
}

}  // namespace

int cf::paged8_few_grid(int dtype, int code, int head_dim, int sm_count) {
  for (int rows = 8; rows <= kFewRows; rows += 8) {
    const Few8Fn f = few8_fn(dtype, code, head_dim, rows);
    if (cudaFuncSetAttribute(f.main, cudaFuncAttributeMaxDynamicSharedMemorySize, f.smem) !=
        cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
  }
  return sm_count;
}

bool cf::paged8_few_launch(int dtype, int code, const PagedAttnParams& p, const PagedSplit& ws,
                           cudaStream_t st) {
  Few8Args a;
  a.p = p;
  a.ws = ws.parts;
  a.tickets = ws.tickets;
  a.row_limit = std::min(kFewRows, p.max_q * p.g.G);
  const Few8Fn f = few8_fn(dtype, code, p.g.D, a.row_limit);
  void* args[] = {&a};
  return launch_pdl(f.main, dim3(ws.grid), f.threads, f.smem, st, args);
}
