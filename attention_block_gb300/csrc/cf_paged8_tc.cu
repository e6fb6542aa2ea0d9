// cf_paged8_tc.cu -- attention over the paged cache of 8-bit codes for many
// rows per KV head: chunks of prompts and long drafts, on the fifth-generation
// tensor cores.
//
// Items, units, the line of units and the alternation of the two halves are
// those of cf_paged_tc.cu: 256 packed (token, grouped head) rows of a KV head
// against tiles of 128 positions, P written back to TMEM over S.  What differs
// is that codes become fp16 on their way into shared memory.  Both products
// are fp16 x fp16; a code is exact in fp16, and scales do not touch the
// operands: with a_j = scale ks_j log2(e) and b_j = log2 vs_j the weight of
// value j is 2^(a_j q.k_j + b_j), and the sum of exp(s_j) takes that weight
// times c_j = 1 / vs_j, or where scales lie far apart an exponential of its own
// (ValueScale).
//
// Roles of a block's 16 warps:
//   0-3, 4-7  softmax of half 0 / 1, a thread per row
//   8-11      codes of K and V: copied into shared memory ahead (cp.async, each
//             thread what it will read itself), then as fp16 into the swizzled
//             tiles; a, b, c of a tile's positions
//   12        one thread issues S = Q K^T and O += P V
//   13-15     queries: copied, and where they are bf16 turned into fp16 in
//             place, a row that would leave fp16's range times a power of two
//             (of the first item together with the softmax warps)
// What a row does not see gets a weight of exactly 0, and codes are finite, so
// nothing that lies in a slot reaches a row that does not see it; a NaN among
// a tile's value scales is set in the scores of the rows that see it.  Weights
// enter the second product as one fp16 value (cf_paged8_few.cu); over short contexts
// results in fp16 are off 2.8e-4 of their norm, 2.1e-4 of it their own rounding.
//
// 512 tokens behind 15872 (32 / 8 heads of 128): 160 us, 845 TFLOP/s; 4 chunks of
// 820-1024 tokens behind 195-1752, 32 heads: 186; one prompt of 8192 638.  The 16-bit
// cache takes 113, 154 and 402 for the same: its kernel loads tiles as they are, this
// one expands each again for every 256 rows, through three slots for five (what each
// of these costs is not measured).
//
// A half's tiles are a chain: when they took 171 and 207 us, 3450 cycles softmax and
// 1950 until the next scores were there (products of both halves 2050).  A branch for
// NaN behind each 32 columns was 11-20 us of that: what is rare stands in the block
// that the maximum's growth enters (in blocks of its own 172-190 and 214-233).
// Measured before that was found: reading the positions' a, b, c takes up to a sixth
// of the softmax (without them 150 and 205 of 171 and 207).  Accumulator fragments,
// with which a thread needs a quarter of them, take 186 and 316 (205 and 272 in two
// passes of 32 columns each): their chains are longer.  code x scale rounded to fp16
// as operand, with powers of two alone in the softmax, takes 163 and 215, but puts
// 2.7 times the error of an fp16 result on it.  An item's result takes 5500-7500
// cycles, its queries 8000 (bf16: 18000), some behind the last tiles.  Queries by
// halves, and half 1's last product behind the next item's first scores, let the
// halves fall out of step: 4 chunks of bf16, GQA, 199 us for 190.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "cf_paged8.cuh"
#include "cf_paged_tc.cuh"

using namespace cf;

namespace {

// Scales of what no row of an item sees: masked, and nothing for the sum to take
// apart.  (A page outside the pool reads as zeros.)
__device__ const float2 kUnseen = {0.f, 1.f};

template <int D>
struct Tc8Shape {
  static constexpr int TILE = kBN * D * 2;         // bytes of a K, V or Q tile
  static constexpr int SLOTS = D == 128 ? 3 : 7;  // K and V tiles
  static constexpr int RAW = D == 128 ? 3 : 6;    // tiles of codes on their way
  static constexpr int SMEM = (2 + SLOTS) * TILE + RAW * kBN * D;  // 1024-aligned
  // The scales of tile j are written when its K has a slot.  With an odd number
  // of slots that was V's of tile j - (SLOTS + 1) / 2: the products with it are
  // complete, and so is that tile's softmax.
  static constexpr int BUFS = (SLOTS + 1) / 2;
  static_assert(SLOTS % 2 == 1, "K takes V's slot");
  static constexpr int AHEAD = RAW / 2 + 2;  // units whose scales are on their way
  static constexpr uint32_t S_COL = 0, O_COL = 2 * kBN;  // TMEM columns
};

// Of a tile's positions: a, b, c; whether 32 of them have low (1), high (2) or odd
// (4) value scales (ValueScale), and which are odd.
struct Tc8Scales {
  float a[kBN], b[kBN], c[kBN];
  uint32_t kinds[kBN / 32], odd[kBN / 32];
};

// What an item costs apart from its tiles, in tiles: its queries, its result, the
// halves out of step.  4 chunks of 820-1024 tokens, 32 heads: 186.3 us with 3, 186.2
// with 4, 189.1 with 5; one chunk of 512 behind 15872: 161.2, 159.3, 161.3; one prompt
// of 8192: 724, 639, 635.
constexpr int kItemCost8 = 4;
using Cursor = TcCursor<false, kItemCost8>;

struct Tc8Args {
  PagedAttnParams p;
  PagedParts ws;
  TcMeta* meta;
  int slots;  // upper bound on the row tiles' numbers
  int grid;   // blocks of the main kernel
};

__device__ __forceinline__ float4 lds4(const float* at) {
  return *reinterpret_cast<const float4*>(at);
}
__device__ __forceinline__ void sts16(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

// Maxima of the 16-bit halves.
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  asm("max.u16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
  return a;
}

template <typename T, int D, int CODE>
__global__ void __launch_bounds__(kTcThreads, 1)
    paged8_tc_kernel(const __grid_constant__ Tc8Args a) {
  using S = Tc8Shape<D>;
  constexpr int LIFT = weight_lift<__half>(kGrow);
  constexpr float BACK = 1.f / (1 << LIFT);
  // Warps that bring the first item's queries: turning them takes longer than the
  // softmax warps' help costs (bf16, 512 behind 15872 159.3 us, with 3 161.5; fp16, 4
  // chunks 189.1, with 3 186.2).
  constexpr int FIRST = kIsBf16<T> ? 11 : 3;
  const PagedAttnParams& p = a.p;
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ long long s_scan[kTcThreads / 32];
  __shared__ Cursor s_cur;
  __shared__ Cursor s_wcur[16];  // each warp's place: too much for registers
  __shared__ __align__(8) uint64_t s_full[S::SLOTS], s_empty[S::SLOTS];
  __shared__ __align__(8) uint64_t s_qfirst, s_qfull, s_qempty, s_done;
  __shared__ __align__(8) uint64_t s_sfull[2], s_pfull[2], s_ofull[2];
  __shared__ uint32_t s_tmem;
  __shared__ __align__(16) Tc8Scales s_scale[S::BUFS];
  __shared__ __align__(8) float2 s_raw[S::AHEAD][kBN];  // scales on their way
  __shared__ float s_qf[2][2 * kHalf];  // what a row's queries were divided by; items take turns
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sq = smem_u32(sm);                   // Q, two tiles
  const uint32_t skv = sq + 2 * S::TILE;              // K and V slots
  int* err = p.errflag;

  if (sq & 1023u) {  // the swizzle goes by the address
    if (tid == 0) atomicOr(err, kDevErrTimeout);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < S::SLOTS; ++i) {
      mbar_init(&s_full[i], 4);
      mbar_init(&s_empty[i], 1);
    }
    mbar_init(&s_qfirst, FIRST);  // of the first item
    mbar_init(&s_qfull, 3);
    mbar_init(&s_qempty, 1);
    mbar_init(&s_done, 1);
    for (int h = 0; h < 2; ++h) {
      mbar_init(&s_sfull[h], 1);
      mbar_init(&s_pfull[h], 4);
      mbar_init(&s_ofull[h], 1);
    }
    fence_mbar_init_cluster();
  }
  pdl_wait();
  pdl_trigger();

  // ---- this block's units
  // the lookups below depend on one another: have their lines on the way
  for (int b = tid; b < p.batch; b += kTcThreads) {
    if (p.q_start) prefetch_line(p.q_start + b + 1);
    prefetch_line(p.kv_len + b);
  }
  TcShare<false> share(p, a.slots, true, tid);
  long long mine, incl;
  RowTile mine_t;  // the last of this thread's row tiles: with one each, the one
#pragma unroll 1
  while (true) {
    mine = 0;
    share.walk(p, [&](const RowTile& t) {
      mine += (long long)(t.tiles + kItemCost8) * p.g.nkv;
      mine_t = t;
      return false;
    });
    incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(~0u, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s_scan[warp] = incl;
    bool done = true;
    if (p.q_start && share.ordered)
      for (int b = tid; b < p.batch; b += kTcThreads)
        done &= starts_ordered(p.q_start[b], p.q_start[b + 1], p.n_tokens);
    if (__syncthreads_and(done)) break;
    share = TcShare<false>(p, a.slots, false, tid);  // the sum was over numbers that mean nothing
  }
  long long before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kTcThreads / 32; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  const long long upc = div_units(total + gridDim.x - 1, gridDim.x);
  const long long u0 = blockIdx.x * upc, u1 = min(total, u0 + upc);
  if (tid == 0) a.meta[blockIdx.x].tiles = 0;
  if (u0 >= u1) return;
  if (before <= u0 && u0 < before + mine) {
    long long at = before;
    if (share.ordered && share.per == 1)
      start_in(p, mine_t, u0, at, s_cur);
    else
      share.walk(p, [&](const RowTile& t) { return start_in(p, t, u0, at, s_cur); });
  }
  if (warp == 12) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }
  tc05_fence_before();
  __syncthreads();
  tc05_fence_after();
  const uint32_t tmem = s_tmem;

  // The queries of cur's item: this warp's part of them, every `warps`th group of
  // rows from `first` on.
  constexpr int C = D / 8;    // 16-byte chunks of a row
  constexpr int RP = 32 / C;  // rows of one copy
  constexpr int NG = 2 * kHalf / RP;
  const int r0 = lane / C, c0 = lane % C;
  auto chunk = [&](int row) {
    return sq + (row >= kHalf ? S::TILE : 0) +
           (uint32_t)((c0 >> 3) * (kBN * 128) + (row & (kHalf - 1)) * 128 +
                      (((c0 & 7) ^ (row & 7)) << 4));
  };
  // x / G for a row's place behind the first token of its tile
  const uint32_t over = 0xffffffffu / (uint32_t)p.g.G + 1u;
  constexpr int U = 4;  // copies, and rows' chunks in work, at a time
  auto queries = [&](const Cursor& cur, uint32_t turn, int first, int warps) {
    const RowTile& t = cur.t;
    // in registers: the first products wait for the queries
    const int gr0 = t.j * 2 * kHalf, i0 = gr0 / p.g.G, rem = gr0 - i0 * p.g.G;
    const int left = t.rows - gr0;
    const T* q = static_cast<const T*>(p.q) + (int64_t)(t.t0 + i0) * p.q_stride +
                 (int64_t)cur.h * p.g.G * D + c0 * 8;
#pragma unroll 1
    for (int g0 = first; g0 < NG; g0 += warps * U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int g = g0 + warps * u, row = g * RP + r0;
        if (g >= NG) break;
        const int x = rem + row, i = p.g.G == 1 ? x : (int)__umulhi(x, over);
        const T* src = q + i * p.q_stride + (x - i * p.g.G) * D;
        cp16(chunk(row), row < left ? src : static_cast<const T*>(p.q), row < left);
      }
    }
    cp_commit();
    cp_wait<0>();
    if constexpr (kIsBf16<T>) {
      // a thread's own chunks, in place
#pragma unroll 1
      for (int g0 = first; g0 < NG; g0 += warps * U) {
        uint32_t x[U][4], top[U];  // largest finite magnitudes of the rows, as bits
#pragma unroll
        for (int u = 0; u < U; ++u)  // (behind the last chunk: the first again)
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(x[u][0]), "=r"(x[u][1]), "=r"(x[u][2]), "=r"(x[u][3])
                       : "r"(chunk((g0 + warps * u < NG ? g0 + warps * u : g0) * RP + r0)));
#pragma unroll
        for (int u = 0; u < U; ++u) {
          uint32_t y = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) y = max2(y, x[u][e] & 0x7fff7fffu);
          top[u] = max(y & 0xffffu, y >> 16);
          if (top[u] >= 0x7f80u) {  // infinities and NaN do not count
            top[u] = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t lo = x[u][e] & 0x7fffu, hi = (x[u][e] >> 16) & 0x7fffu;
              if (lo < 0x7f80u) top[u] = max(top[u], lo);
              if (hi < 0x7f80u) top[u] = max(top[u], hi);
            }
          }
        }
#pragma unroll
        for (int d = C / 2; d >= 1; d >>= 1)
#pragma unroll
          for (int u = 0; u < U; ++u) top[u] = max(top[u], __shfl_xor_sync(~0u, top[u], d));
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int g = g0 + warps * u, row = g * RP + r0;
          if (g >= NG) break;
          // exponents -10 .. 14 of the largest stay: what is lost then is below 2^-25
          const int e = (int)(top[u] >> 7) - 127;
          float up = 1.f, down = 1.f;
          if (top[u] != 0 && (e > 14 || e < -10)) {
            const int s = min(max(14 - e, -113), 113);
            up = __uint_as_float((uint32_t)(127 + s) << 23);
            down = __uint_as_float((uint32_t)(127 - s) << 23);
          }
#pragma unroll
          for (int e2 = 0; e2 < 4; ++e2) {
            float f[2];
            Elem<T>::words(&x[u][e2], 1, f);
            x[u][e2] = pack2<__half>(f[0] * up, f[1] * up);
          }
          sts16(chunk(row), x[u][0], x[u][1], x[u][2], x[u][3]);
          if (c0 == 0) s_qf[turn][row] = down;
        }
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
  };

  if (warp < 8) {
    // ------------------------------------------------------------ softmax --
    // 72 for the others (512 behind 15872 159.3 us, 4 chunks, 32 heads, 186.2, 32 of 8
    // tokens 109.9; with 88 for the codes and 56 for the rest 157.8, 185.6 and 111.9; with
    // 176 here and 80 there 164.8, 181.9 and 106.6).
    set_regs_up<184>();
    const int hf = warp >> 2;                   // half
    const int r = (warp & 3) * 32 + lane;       // row of the half = TMEM lane
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + S::S_COL + hf * kBN;
    const uint32_t to = tmem + lanes + S::O_COL + hf * D;
    Cursor& cur = s_wcur[warp];
    if (lane == 0) cur = s_cur;
    __syncwarp();
    if constexpr (kIsBf16<T>) {  // nothing else to do before the first scores
      if (cur.u < u1) {
        queries(cur, 0, 3 + warp, FIRST);
        if (lane == 0) mbar_arrive(&s_qfirst);
      }
    }
    uint32_t n_tiles = 0;  // active tiles so far: parity of the barriers
    uint32_t items = 0;
    int buf = S::BUFS - 1;  // of the tile's scales
    while (cur.u < u1) {
      const RowTile& t = cur.t;
      const int gr = t.j * 2 * kHalf + hf * kHalf + r;  // row of the sequence
      const int pos = t.p0 + gr / p.g.G;
      const PagedRange rng = t.half[hf];
      const int plo = t.plo[hf], phi = t.phi[hf];
      const int first = cur.tile, count = (int)min((long long)(t.tiles - first), u1 - cur.u);
      const int ns = t.ns, skip = t.skip;
      float m = -INFINITY, l = 0.f;
      bool some = false;  // O holds something
      uint32_t ask = 4;   // kinds of value scales for which the sum is taken apart
#pragma unroll 1
      for (int tile = first; tile < first + count; ++tile) {
        const int base = (tile < ns ? tile : tile + skip) * kBN;
        if (++buf == S::BUFS) buf = 0;
        if (tile_active(rng, base)) {
          const Tc8Scales& sc = s_scale[buf];
          wait_bar(&s_sfull[hf], n_tiles & 1, err);
          tc05_fence_after();
          float s[kBN];
#pragma unroll
          for (int k = 0; k < kBN / 32; ++k) tmem_ld32(ts + 32 * k, s + 32 * k);
          tmem_wait_ld();
          float qf = 1.f;
          if constexpr (kIsBf16<T>) {  // rows whose queries were brought into fp16's range
            qf = s_qf[items & 1][hf * kHalf + r];
            if (__any_sync(~0u, qf != 1.f)) {
#pragma unroll
              for (int k = 0; k < kBN; ++k) s[k] *= qf;
            }
          }
#pragma unroll
          for (int k = 0; k < kBN; k += 4) {
            const float4 av = lds4(sc.a + k), bv = lds4(sc.b + k);
            const float2 x = fma2(make_float2(s[k], s[k + 1]), make_float2(av.x, av.y),
                                  make_float2(bv.x, bv.y));
            const float2 y = fma2(make_float2(s[k + 2], s[k + 3]), make_float2(av.z, av.w),
                                  make_float2(bv.z, bv.w));
            s[k] = x.x;
            s[k + 1] = x.y;
            s[k + 2] = y.x;
            s[k + 3] = y.y;
          }
          const bool full = half_full<false>(p, plo, phi, base);
          // bit k: this row sees position j0 + k
          auto sees = [&](int j0) {
            uint32_t see = low_bits(pos + 1 - j0);
            if (p.window != 0)
              see &= ~low_bits(pos - p.window + 1 - j0) | low_bits(p.n_sinks - j0);
            return see;
          };
          if (!full) {
#pragma unroll
            for (int c = 0; c < kBN / 32; ++c) {
              const uint32_t see = sees(base + 32 * c);
              if (__all_sync(~0u, see == ~0u)) continue;
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!((see >> k) & 1u)) s[32 * c + k] = -INFINITY;
            }
          }
          float mx4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int k = 4; k < kBN - 4; k += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e) mx4[e] = max3(mx4[e], s[k + e], s[k + 4 + e]);
#pragma unroll
          for (int e = 0; e < 4; ++e) mx4[e] = fmaxf(mx4[e], s[kBN - 4 + e]);
          const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
          const float m_new = fmaxf(m, mx);
          // (one question for both: another branch on every tile's way costs 2-11 %)
          const uint4 kd = *reinterpret_cast<const uint4*>(sc.kinds);
          const uint32_t kinds = kd.x | kd.y | kd.z | kd.w;
          ask |= (kinds >> 1) & 1u;  // low ones count from the first high one on
          const bool apart = (kinds & ask) != 0;
          const bool grow = m_new - m > (float)kGrow || apart;  // also from -inf
          float l_apart = 0.f;
          if (__any_sync(~0u, grow)) {
            // (by halves: with value scales far apart, what the sum is multiplied by can be
            // below 2^-126 and the sum still count)
            const float half = m_new == -INFINITY ? 1.f : ex2(0.5f * (m - m_new));
            const float corr = half * half;
            if (some) {
              wait_bar(&s_ofull[hf], (n_tiles - 1) & 1, err);
              tc05_fence_after();
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                uint32_t o[16];
                tmem_ld_32x32b_x16_nowait(to + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
                tmem_st16(to + c, o);
              }
            }
            l = l * half * half;
            m = m_new;
            if (apart) {  // the sum over this tile as 2^(s - reference)
              const float at = (m == -INFINITY ? 0.f : m) - LIFT;
              l_apart = l;
#pragma unroll 1
              for (int c = 0; c < kBN; c += 16) {
                const uint32_t see = sees(base + c);
                uint32_t x[16];
                tmem_ld_32x32b_x16_nowait(ts + c, x);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                  const float4 av = lds4(sc.a + c + e);
                  const float y[4] = {av.x, av.y, av.z, av.w};
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const float s2 = fmaf(__uint_as_float(x[e + i]) * qf, y[i], -at);
                    l_apart += ex2((see >> (e + i)) & 1u ? s2 : -INFINITY);
                  }
                }
              }
              // values of NaN: for the rows that see them
              if ((sc.odd[0] | sc.odd[1] | sc.odd[2] | sc.odd[3]) != 0) {
#pragma unroll
                for (int k = 0; k < kBN / 32; ++k) {
                  const uint32_t hit = sc.odd[k] & sees(base + 32 * k);
#pragma unroll
                  for (int e = 0; e < 32; ++e)
                    if ((hit >> e) & 1u) s[32 * k + e] = __uint_as_float(0x7fc00000u);
                }
              }
            }
          }
          const float ref = (m == -INFINITY ? 0.f : m) - LIFT;
          const float2 ref2 = make_float2(-ref, -ref);
          float2 sum[2] = {make_float2(l, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int k = 0; k < kBN / 32; ++k) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const float4 cv = lds4(sc.c + 32 * k + 2 * e);
#pragma unroll
              for (int x2 = 0; x2 < 2; ++x2) {
                float2 x = add2(make_float2(s[32 * k + 2 * (e + x2)], s[32 * k + 2 * (e + x2) + 1]),
                                ref2);
                x.x = ex2(x.x);
                x.y = ex2(x.y);
                sum[x2] = fma2(x, x2 ? make_float2(cv.z, cv.w) : make_float2(cv.x, cv.y), sum[x2]);
                w[e + x2] = pack2<__half>(x.x, x.y);
              }
            }
            tmem_st16(ts + 16 * k, w);
          }
          tmem_wait_st();
          tc05_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_pfull[hf]);
          l = apart ? l_apart : (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          some = true;
          ++n_tiles;
        }
      }
      // ---- the block's part of the item
      const bool whole = first == 0 && count == t.tiles;
      if (some) {
        wait_bar(&s_ofull[hf], (n_tiles - 1) & 1, err);
        tc05_fence_after();
      }
      l *= BACK;
      const bool part = !whole;  // leaves a state, not a result
      // this block's slot for the item (PagedParts)
      const long long prow0 =
          (2 * (long long)blockIdx.x + (u0 >= cur.i0 ? 0 : 1)) * (2 * kHalf) + hf * kHalf;
      const int q4 = lane & 3;
      // this lane's own row: where it goes, and what its values are scaled by
      long long my_row = -1;
      float my_inv = 1.f;
      if (gr < t.rows) {
        const int i = gr / p.g.G;
        my_row = ((long long)t.t0 + i) * p.g.nq + cur.h * p.g.G + gr - i * p.g.G;
        if (part) {
          my_row = prow0 + r;
          __stcg(a.ws.ml + my_row, make_float2(m, l));
        } else {
          my_inv = l == 0.f ? 0.f : BACK / l;
          if (p.lse) p.lse[my_row] = paged_lse(m, l);
        }
      }
#pragma unroll 1
      for (int hh = 0; hh < 2; ++hh) {  // 16 rows of the warp at a time
        float inv[2];
        long long orow[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int src = hh * 16 + e * 8 + (lane >> 2);  // lane that has this row
          orow[e] = __shfl_sync(~0u, my_row, src);
          inv[e] = __shfl_sync(~0u, my_inv, src);
        }
#pragma unroll 1
        for (int c64 = 0; c64 < D; c64 += 64) {
          float o2[2][16];
          if (some) {
            tmem_ld_frag(to + ((uint32_t)(16 * hh) << 16) + c64, o2[0]);
            tmem_ld_frag(to + ((uint32_t)(16 * hh) << 16) + c64 + 32, o2[1]);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int x = 0; x < 32; ++x) o2[x >> 4][x & 15] = 0.f;
          }
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int c = c64 + 32 * y;
            const float(&o)[16] = o2[y];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (part) {
                // of two octets A, B the even lanes of a quad store A's words,
                // the odd ones B's, 16 bytes each
#pragma unroll
                for (int b2 = 0; b2 < 2; ++b2) {
                  const float A0 = o[8 * b2 + 2 * e] * BACK, A1 = o[8 * b2 + 2 * e + 1] * BACK;
                  const float B0 = o[8 * b2 + 4 + 2 * e] * BACK, B1 = o[8 * b2 + 5 + 2 * e] * BACK;
                  const bool odd = q4 & 1;
                  const float g0 = __shfl_xor_sync(~0u, odd ? A0 : B0, 1);
                  const float g1 = __shfl_xor_sync(~0u, odd ? A1 : B1, 1);
                  if (orow[e] >= 0)
                    __stcg(reinterpret_cast<float4*>(a.ws.o + orow[e] * D + c + 16 * b2 +
                                                     8 * (q4 & 1) + 4 * (q4 >> 1)),
                           odd ? make_float4(g0, g1, B0, B1) : make_float4(A0, A1, g0, g1));
                }
              } else {
                uint32_t w[4];
#pragma unroll
                for (int b = 0; b < 4; ++b)
                  w[b] = pack2<T>(o[4 * b + 2 * e] * inv[e], o[4 * b + 2 * e + 1] * inv[e]);
                quad_transpose(w, q4);  // lane q: the 8 columns of octet q
                if (orow[e] >= 0)
                  *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + orow[e] * D + c + 8 * q4) =
                      make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          }
        }
      }
      if (part && first == 0 && tid == 0) {
        TcMeta x;
        x.i0 = cur.i0;
        x.upc = upc;
        x.tiles = t.tiles;
        x.t0 = t.t0;
        x.p0 = t.p0;
        x.rows = t.rows;
        x.j = t.j;
        x.h = cur.h;
        a.meta[blockIdx.x] = x;
      }
      tc05_fence_before();  // O is read before the next item's first product
      __syncwarp();
      if (lane == 0) {
        cur.u += count - 1;
        cur.tile += count - 1;
        cur.next(p, u1);
      }
      __syncwarp();
      ++items;
    }
  } else if (warp < 12) {
    // -------------------------------------------------------------- codes --
    set_regs_down<72>();
    const int lw = warp - 8;  // rows 32 lw .. 32 lw + 31 of every tile
    Cursor& cur = s_wcur[warp];
    if (lane == 0) cur = s_cur;
    __syncwarp();
    constexpr int C = D / 16;    // 16-byte pieces of a row's codes
    constexpr int RP = 32 / C;   // rows of one load
    constexpr int NP = 32 / RP;  // loads of a tile
    // A piece becomes the 16-byte chunks 2 c0 and 2 c0 + 1 of its row.  Eight
    // neighbouring lanes have four pieces of one slab from an even and an odd
    // row: their stores meet in no bank.
    const int r0 = (lane >> 2) & (RP - 1), c0 = (lane & 3) | (D == 128 ? (lane >> 4) << 2 : 0);
    const uint32_t d0 = skv + (uint32_t)((c0 >> 2) * (kBN * 128) + (lw * 32 + r0) * 128);
    const uint32_t x0 = (uint32_t)((2 * c0) & 7);
    const char* kbase = static_cast<const char*>(p.k_pages) + c0 * 16;
    const char* vbase = static_cast<const char*>(p.v_pages) + c0 * 16;
    // A ring of tiles of codes.  A thread reads what it copied itself: its own
    // groups of copies are all that it waits for.
    const uint32_t raw = skv + S::SLOTS * S::TILE + (tid - 256) * 16;
    // Copies the pieces of the rows that lie at the lanes' offsets; -1: zeros.
    auto load = [&](int r, const char* src, int64_t off) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int64_t o = __shfl_sync(~0u, off, i * RP + r0);
        cp16(raw + (r * NP + i) * (kCopyThreads * 16), src + (o >= 0 ? o : 0), o >= 0);
      }
    };
    auto convert = [&](int r, uint32_t slot) {
      uint32_t c[NP][4];  // all of them first: a store might be to what a load behind it reads
#pragma unroll
      for (int i = 0; i < NP; ++i)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(c[i][0]), "=r"(c[i][1]), "=r"(c[i][2]), "=r"(c[i][3])
                     : "r"(raw + (r * NP + i) * (kCopyThreads * 16)));
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) code_row4<CODE>(c[i][e], h[2 * e], h[2 * e + 1]);
        const uint32_t row = d0 + slot * S::TILE + i * RP * 128;
        const uint32_t sw = (uint32_t)((i * RP + r0) & 7);
        sts16(row + ((x0 ^ sw) << 4), h[0], h[1], h[2], h[3]);
        sts16(row + (((x0 + 1) ^ sw) << 4), h[4], h[5], h[6], h[7]);
      }
    };
    // The page of this lane's position, looked up one tile ahead of its loads (a coherent
    // load: the launch in front may have written the table).
    int f_pos = -1, f_page = 0;
    auto look_up = [&]() {
      f_pos = -1;
      if (cur.u >= u1) return;
      const int j = cur.t.base(cur.tile) + lw * 32 + lane;
      if (!cur.t.sees(j)) return;
      f_pos = j;
      f_page = p.page_table[(int64_t)cur.t.b * p.g.max_pages + (j >> p.g.page_shift)];
    };
    // K and V of the units in turn, RAW tiles ahead of their conversion; cur runs
    // with the copies.
    int64_t off = -1;     // of this lane's position in the unit whose copies are next
    bool value = false;   // its V is next
    int in = 0, in_unit = 0, left = 0;  // ring places; tiles to be converted
    const int row = lw * 32 + lane;
    auto issue = [&]() {
      if (value) {
        load(in, vbase, off);
        value = false;
        ++left;
        if (++in == S::RAW) in = 0;
      } else if (cur.u < u1) {
        off = -1;
        const float2* scale = &kUnseen;
        const bool seen = f_pos >= 0;
        if (seen) {
          if ((unsigned)f_page >= (unsigned)p.g.num_pages) {
            atomicOr(err, kDevErrPosRange);
          } else {
            const int slot = f_pos & p.g.page_mask;
            off = (int64_t)f_page * p.g.page_stride + (int64_t)slot * p.g.slot_stride +
                  (int64_t)cur.h * p.g.head_stride;
            scale = p.scales + (((int64_t)f_page * p.g.nkv + cur.h) << p.g.page_shift) + slot;
          }
        }
        __syncwarp();
        if (lane == 0) cur.next(p, u1);
        __syncwarp();
        look_up();
        cp8(smem_u32(&s_raw[in_unit][row]), scale, off >= 0 || !seen);
        if (++in_unit == S::AHEAD) in_unit = 0;
        load(in, kbase, off);
        value = true;
        ++left;
        if (++in == S::RAW) in = 0;
      }
      cp_commit();
    };
    RingPos ring(0, S::SLOTS);
    uint32_t use = 0;  // slots taken so far
    int buf = 0, out = 0, out_unit = 0;
    look_up();
#pragma unroll 1
    for (int i = 0; i < S::RAW; ++i) issue();
#pragma unroll 1
    for (bool key = true; left > 0; key = !key) {
      cp_wait<S::RAW - 1>();
      if (use >= S::SLOTS) wait_bar(&s_empty[ring.slot], ring.phase ^ 1u, err);
      ++use;
      if (key) {
        const float2 scale = s_raw[out_unit][row];
        if (++out_unit == S::AHEAD) out_unit = 0;
        const ValueScale vs(scale.y);
        Tc8Scales& sc = s_scale[buf];
        sc.a[row] = key_scale(scale.x) * p.scale_log2;
        sc.b[row] = vs.log2;
        sc.c[row] = vs.inv;
        uint32_t kinds = 0, odd = 0;
        if (__any_sync(~0u, !vs.plain)) {
          odd = __ballot_sync(~0u, !scale_is_read(scale.y));
          kinds = (__any_sync(~0u, ValueScale::low(scale.y)) ? 1u : 0u) |
                  (__any_sync(~0u, ValueScale::high(scale.y)) ? 2u : 0u) | (odd ? 4u : 0u);
        }
        if (lane == 0) {
          sc.kinds[lw] = kinds;
          sc.odd[lw] = odd;
        }
        if (++buf == S::BUFS) buf = 0;
      }
      convert(out, ring.slot);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_full[ring.slot]);
      ring.next(S::SLOTS);
      if (++out == S::RAW) out = 0;
      --left;
      issue();
    }
    cp_wait<0>();
  } else if (warp > 12) {
    // ------------------------------------------------------------ queries --
    set_regs_down<72>();
    const int qw = warp - 13;
    Cursor& cur = s_wcur[warp];
    if (lane == 0) cur = s_cur;
    __syncwarp();
    uint32_t items = 0;
    while (cur.u < u1) {
      const int count = (int)min((long long)(cur.t.tiles - cur.tile), u1 - cur.u);
      if (items) wait_bar(&s_qempty, (items - 1) & 1, err);
      queries(cur, items & 1, qw, items ? 3 : FIRST);
      if (lane == 0) {
        mbar_arrive(items ? &s_qfull : &s_qfirst);
        cur.u += count - 1;
        cur.tile += count - 1;
        cur.next(p, u1);
      }
      __syncwarp();
      ++items;
    }
  } else {
    // ---------------------------------------------------------------- mma --
    set_regs_down<72>();
    // The whole warp walks (its operands then lie in uniform registers); one
    // elected thread issues.
    {
      constexpr uint32_t id_s = idesc_kind_f16(false, kHalf, kBN);
      constexpr uint32_t id_o = idesc_kind_f16(false, kHalf, D) | (1u << 16);  // B is N-major
      Cursor& cur = s_wcur[12];
      if (lane == 0) cur = s_cur;
      __syncwarp();
      const bool leader = elect_one();
      // descriptors of slot 0 and of Q; addresses count in 16 bytes
      const uint64_t dk0 = smem_desc_k_sw128(skv, 1024), dq0 = smem_desc_k_sw128(sq, 1024);
      const uint64_t dv0 = smem_desc_mn_sw128(skv, kBN * 128, 1024);
      RingPos ring(0, S::SLOTS);
      uint32_t items = 0, n_tiles[2] = {0, 0};
      auto scores = [&](int h, int slot) {
        if (leader) {
          const uint64_t dk = dk0 + slot * (S::TILE / 16), dq = dq0 + h * (S::TILE / 16);
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            const uint32_t off = ((x >> 2) * (kBN * 128) + (x & 3) * 32) / 16;
            tc05_mma_f16(tmem + S::S_COL + h * kBN, dq + off, dk + off, id_s, x > 0);
          }
          tc05_commit(&s_sfull[h]);
        }
        __syncwarp();
      };
      // O of half h (+)= P V; frees the slot where it is V's last reader
      auto values = [&](int h, int slot, bool acc, bool free_slot) {
        wait_bar(&s_pfull[h], n_tiles[h] & 1, err);
        tc05_fence_after();
        if (leader) {
          const uint64_t dv = dv0 + slot * (S::TILE / 16);
#pragma unroll
          for (int x = 0; x < kBN / 16; ++x)
            tc05_mma_f16_ts(tmem + S::O_COL + h * D, tmem + S::S_COL + h * kBN + x * 8,
                            dv + x * (16 * 128 / 16), id_o, acc || x > 0);
          tc05_commit(&s_ofull[h]);
          if (free_slot) tc05_commit(&s_empty[slot]);
        }
        __syncwarp();
        ++n_tiles[h];
      };
      while (cur.u < u1) {
        const TileCheck<false> tc(cur.t);
        const int ns = cur.t.ns, skip = cur.t.skip, first = cur.tile;
        const int count = (int)min((long long)(cur.t.tiles - first), u1 - cur.u);
        // the tiles that both halves see whole, but for the run's last
        int mid_lo, mid_hi;
        tc.middle(p, first, first + count - 1, ns, skip, mid_lo, mid_hi);
        wait_bar(items ? &s_qfull : &s_qfirst, items ? (items - 1) & 1 : 0, err);
        ++items;
        tc05_fence_after();
        bool acc0 = false, acc1 = false;
        bool pend = false;  // half 1's O += P V of the last tile is still to come
        int pend_slot = 0;
        // One tile: the scores of half 0, O of half 1 for the tile before, the
        // scores of half 1, O of half 0.  This warp's own instructions are on
        // the critical path, so the usual tile has its own copy of the code,
        // without any question.
        auto step = [&](bool act0, bool act1, bool last) {
          const int kslot = ring.slot;
          wait_bar(&s_full[kslot], ring.phase, err);
          ring.next(S::SLOTS);
          tc05_fence_after();
          if (act0) scores(0, kslot);
          if (pend) {
            values(1, pend_slot, acc1, true);
            acc1 = true;
            pend = false;
          }
          if (act1) scores(1, kslot);
          if (leader) {
            tc05_commit(&s_empty[kslot]);
            if (last) tc05_commit(&s_qempty);
          }
          __syncwarp();
          const int vslot = ring.slot;
          wait_bar(&s_full[vslot], ring.phase, err);
          ring.next(S::SLOTS);
          tc05_fence_after();
          if (act0) {
            values(0, vslot, acc0, !act1);
            acc0 = true;
          }
          if (act1 && !last) {
            pend = true;
            pend_slot = vslot;
          } else if (act1) {
            values(1, vslot, acc1, true);
          } else if (!act0) {
            if (leader) tc05_commit(&s_empty[vslot]);
            __syncwarp();
          }
        };
#pragma unroll 1
        for (int tile = first; tile < first + count; ++tile) {
          if (tile == mid_lo && mid_lo < mid_hi) {
#pragma unroll 1
            for (; tile < mid_hi; ++tile) step(true, true, false);
          }
          const int base = (tile < ns ? tile : tile + skip) * kBN;
          step(tc.active(0, base), tc.active(1, base), tile + 1 == first + count);
        }
        if (lane == 0) {
          cur.u += count - 1;
          cur.tile += count - 1;
          cur.next(p, u1);
        }
        __syncwarp();
      }
      if (leader) tc05_commit(&s_done);
      __syncwarp();
      wait_bar(&s_done, 0, err);
    }
  }
  __syncthreads();
  if (warp == 12) tmem_dealloc(tmem, 512);
}

// Joins the states of split items, one to a block of the main kernel at most: a row
// per D / 4 lanes, gridDim.y blocks to an item.
constexpr int kTc8JoinY = 16;
template <typename T, int D>
__global__ void __launch_bounds__(256, 4) paged8_tc_join_kernel(const __grid_constant__ Tc8Args a) {
  const PagedAttnParams& p = a.p;
  constexpr int C4 = D / 4;
  pdl_wait();
  pdl_trigger();
  const TcMeta x = a.meta[blockIdx.x];
  // (an item that ends behind the line: lengths changed under the call)
  if (x.tiles == 0 || x.i0 + x.tiles > x.upc * a.grid) return;
  const int rows = min(2 * kHalf, x.rows - x.j * 2 * kHalf);
  const PagedItemParts parts(x.i0, x.tiles, x.upc);
  for (int e = blockIdx.y * 256 + threadIdx.x; e < rows * C4; e += gridDim.y * 256) {
    const int r = e / C4, col = (e - r * C4) * 4;
    PagedState4 s{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    const int gr = x.j * 2 * kHalf + r, i = gr / p.g.G, g = gr - i * p.g.G;
    const long long row = ((long long)x.t0 + i) * p.g.nq + x.h * p.g.G + g;
    paged_join_row<D, 4, true>(s, a.ws.o, a.ws.ml, PagedRowParts(parts, 2 * kHalf, r, -1), col);
    paged_store4<T, D>(s, p.out, p.lse, row, col);
  }
}

struct Tc8Fns {
  const void *main, *join;
  int smem;
};
template <typename T, int D>
Tc8Fns tc8_code(int code) {
  return Tc8Fns{code == CF_CODE_INT8 ? (const void*)&paged8_tc_kernel<T, D, CF_CODE_INT8>
                                     : (const void*)&paged8_tc_kernel<T, D, CF_CODE_E4M3>,
                (const void*)&paged8_tc_join_kernel<T, D>, Tc8Shape<D>::SMEM};
}
Tc8Fns tc8_fns(int dtype, int code, int d) {
  if (dtype == CF_F16) return d == 64 ? tc8_code<__half, 64>(code) : tc8_code<__half, 128>(code);
  return d == 64 ? tc8_code<__nv_bfloat16, 64>(code) : tc8_code<__nv_bfloat16, 128>(code);
}

}  // namespace

int cf::paged8_tc_grid(int dtype, int code, int head_dim, int sm_count) {
  const Tc8Fns f = tc8_fns(dtype, code, head_dim);
  if (cudaFuncSetAttribute(f.main, cudaFuncAttributeMaxDynamicSharedMemorySize, f.smem) !=
      cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return sm_count;
}

size_t cf::paged8_tc_list_bytes(int grid) { return (size_t)grid * sizeof(TcMeta); }

bool cf::paged8_tc_launch(int dtype, int code, const PagedAttnParams& p, const PagedSplit& ws,
                          cudaStream_t st) {
  const Tc8Fns f = tc8_fns(dtype, code, p.g.D);
  Tc8Args a;
  a.p = p;
  a.ws = ws.parts;
  a.meta = static_cast<TcMeta*>(ws.list);
  a.slots = (int)((long long)p.n_tokens * p.g.G / kTcRows) + p.batch;
  a.grid = ws.grid;
  void* args[] = {&a};
  if (!launch_pdl(f.main, dim3(ws.grid), kTcThreads, f.smem, st, args)) return false;
  // fewer blocks to an item where its rows are fewer
  const long long rows = std::min<long long>(kTcRows, (long long)p.max_q * p.g.G);
  const int y = (int)std::min<long long>(kTc8JoinY, (rows * (p.g.D / 4) + 255) / 256);
  return launch_pdl(f.join, dim3(ws.grid, y), 256, 0, st, args);
}
