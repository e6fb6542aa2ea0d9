// cf_paged_tc.cu -- attention over the paged cache for many rows per KV head:
// prompts, long drafts, and a whole batch against its shared prefix, fp16 or
// bf16, on the fifth-generation tensor cores.
//
// A KV head's rows are the packed (token, grouped head) pairs, so grouped
// heads share every key tile.  An item is 256 rows (two halves of 128, the
// tensor core's M) of one KV head; its units are tiles of 128 positions.  All
// items' units form one line that the blocks, one per SM, share evenly
// (PagedParts): causal triangles, windows, ragged batches and few long items
// all fill the GPU.  An item that lies in several blocks leaves partial
// states, joined by a second small kernel.
//
// Roles of a block's 16 warps:
//   0-3, 4-7  softmax of half 0 / 1, a thread per row: S from TMEM, mask,
//             running maximum, exp2, P (16 bits) back into TMEM over S, sum
//             of P before its rounding; the final o
//   8-11      copy Q, K and V through the page table into shared memory
//             (cp.async; positions that no row sees become zeros, so what
//             lies there reaches no product): tiles of 64-column slabs, rows
//             of 128 bytes, the 16-byte chunks of a row swizzled
//   12        one thread issues S = Q K^T (operands in shared memory) and
//             O += P V (P from TMEM, V as an N-major operand).  Where the rows
//             of a tile see different parts of it, the warp looks for
//             infinities and NaN in its V, which would reach the rows that do
//             not see them as 0 * inf: such an item is listed and computed
//             again, row by row, by the joining kernel
// The halves alternate: while one is in its softmax the tensor core works on
// the other.  TMEM: S (or P) and O of both halves, 512 columns.
//
// O is rescaled only where a row's maximum grew by more than 2^8 since its
// last rescale: P then stays below 2^8 (fp16 holds it times 2^7) and keeps its
// relative precision in 16-bit floating point, and most tiles pass without
// touching O.
//
// Bound by the tensor core where items are long (one prompt of 8192 tokens, 32
// / 8 heads of 128: 399 us, 1380 TFLOP/s, 0.72 of a library product's rate),
// by the softmax's chain otherwise: 1.65 us a unit, 1.07 of them products, and
// an item's masked tiles, wait for O and result, which weigh about 5 units
// (kItemCost).  With 64 columns exp2 and masks take longer than the products
// (8191 tokens, window 1024, 32 heads: 189 us).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "cf_paged.cuh"
#include "cf_tc05.cuh"
#include "cf_test.h"

using namespace cf;

namespace {

constexpr int kTcThreads = 512;
constexpr int kCopyThreads = 128;
constexpr int kHalf = 128;     // rows of a half
constexpr int kBN = 128;       // positions of a tile
// What an item costs beside its tiles, in tiles.  4 prompts of 517-2048 tokens
// (32 / 8 heads of 128): 241 us with 0, 155 with 2, 145 with 5, 150 with 8.
constexpr int kItemCost = 5;
constexpr int kPagedRunInts = 9;  // of a run that cf_test_paged_line reports
constexpr int kGrow = 8;       // log2 of the growth that forces a rescale

template <int D>
struct TcShape {
  static constexpr int TILE = kBN * D * 2;                   // bytes of a K, V or Q tile
  static constexpr int SLOTS = D == 128 ? 5 : 10;            // K and V tiles in flight
  static constexpr int SMEM = (2 + SLOTS) * TILE;  // 1024-aligned; 3 KB are left for the rest
  static constexpr uint32_t S_COL = 0, O_COL = 2 * kBN;      // TMEM columns
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
// The lowest n bits, n any number.
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u);
}
// Arrives on bar when this thread's copies so far have landed (the barrier's
// count includes the arrival).
__device__ __forceinline__ void cp_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, "
      "%10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
// 32 columns of 16 TMEM lanes as mma accumulator fragments: of column octet b,
// r[4b], r[4b+1] are row lane / 4, columns 2 (lane % 4) and + 1, and r[4b+2],
// r[4b+3] the same of row lane / 4 + 8.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, float (&v)[16]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// D[tmem] (+)= A[tmem] . B[bdesc] for one K step of 16.
__device__ __forceinline__ void tc05_mma_f16_ts(uint32_t dtmem, uint32_t atmem, uint64_t bdesc,
                                                uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(dtmem),
      "r"(atmem), "l"(bdesc), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}

// mbar_wait without a call: a called function would need registers that
// setmaxnreg moves.  Bounded like it, and as quick to give up once any wait
// has recorded a timeout.
__device__ __forceinline__ void wait_bar(uint64_t* bar, uint32_t parity, int* err) {
  const uint32_t a = smem_u32(bar);
  if (mbar_try_wait_cta(a, parity)) return;
  const long long t0 = clock64();
  for (uint32_t spins = 1; !mbar_try_wait_cta(a, parity); ++spins) {
    if ((spins & 1023u) != 0) continue;
    if (*reinterpret_cast<volatile int*>(err) & kDevErrTimeout) return;
    if (clock64() - t0 > kWaitLimitCycles) {
      atomicOr(err, kDevErrTimeout);
      return;
    }
  }
}

template <typename T>
constexpr bool kIsBf16 = false;
template <>
constexpr bool kIsBf16<__nv_bfloat16> = true;

template <int N>
__device__ __forceinline__ void set_regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A row tile (256 rows of a sequence, or of the whole call for the prefix)
// and its key tiles.  Where the starts are in order, row tile j of sequence b
// has the number t0 * G / 256 + b + j: unique, increasing, below
// T * G / 256 + batch.
struct RowTile : PagedTiles<kBN> {
  int b, j, jn;        // sequence, row tile, row tiles of the sequence
  int t0, p0, rows;    // first token, its position, rows of the sequence
  PagedRange half[2];  // what each half's rows see together
  int plo[2], phi[2];  // positions of a half's first and last row
};

template <bool PRE>
CF_HOST_DEVICE void seq_of(const PagedAttnParams& p, int b, RowTile& t) {
  t.b = b;
  if constexpr (PRE) {
    t.t0 = t.p0 = 0;
    t.rows = p.n_tokens * p.g.G;
  } else {
    const PagedSeq s = paged_seq(p.q_start, p.kv_len, b, p.n_tokens, p.max_q, p.g, p.errflag);
    t.t0 = s.t0;
    t.p0 = s.len - s.n;
    t.rows = s.n * p.g.G;
  }
  t.jn = (t.rows + 2 * kHalf - 1) / (2 * kHalf);
}

// Fills in row tile j of the sequence that seq_of() set.
template <bool PRE>
CF_HOST_DEVICE void tile_of(const PagedAttnParams& p, int j, RowTile& t) {
  t.j = j;
  PagedRange u{0, 0, 0};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r0 = j * 2 * kHalf + h * kHalf, r1 = min(r0 + kHalf, t.rows) - 1;
    t.half[h] = PagedRange{0, 0, 0};
    t.plo[h] = t.phi[h] = 0;
    if (r0 > r1) continue;
    if constexpr (PRE) {
      t.half[h].hi = p.prefix_len;
    } else {
      t.plo[h] = t.p0 + r0 / p.g.G;
      t.phi[h] = t.p0 + r1 / p.g.G;
      // p0 + tokens is the sequence's length: no row sees past it
      t.half[h] = paged_range(max(t.plo[h], 0), t.phi[h], t.phi[h] + 1, p.window, p.n_sinks);
    }
    if (h == 0) {
      u = t.half[0];
    } else {
      // half 1 has the later rows: it sees as far or farther, and its window
      // starts as late or later
      const PagedRange a = t.half[0], c = t.half[1];
      u = a.hi <= a.lo ? c : PagedRange{max(a.sink, min(c.sink, a.lo)), a.lo, c.hi};
    }
  }
  t.set(u);
}

// Whether a half has rows that see part of the tile at `base`.
__device__ __forceinline__ bool tile_active(const PagedRange& r, int base) {
  return r.hi > r.lo && ((base < r.hi && base + kBN > r.lo) || base < r.sink);
}

// Whether all rows of half h see the whole tile at `base`.
template <bool PRE>
__device__ __forceinline__ bool half_full(const PagedAttnParams& p, int plo, int phi, int base) {
  if constexpr (PRE) return base + kBN <= p.prefix_len;
  return base + kBN - 1 <= plo &&
         (p.window == 0 || phi - base < p.window || base + kBN <= p.n_sinks);
}
// What a launch asks about a row tile's key tiles, one by one.  V is looked
// through where an active half does not see the tile whole.  (All rows see the
// prefix alike.)
template <bool PRE>
struct TileCheck {
  PagedRange h[2];
  int plo[2], phi[2];
  __device__ __forceinline__ explicit TileCheck(const RowTile& t)
      : h{t.half[0], t.half[1]}, plo{t.plo[0], t.plo[1]}, phi{t.phi[0], t.phi[1]} {}
  __device__ __forceinline__ bool active(int i, int base) const { return tile_active(h[i], base); }
  // Of the tiles [lo, hi): the longest run behind the sink tiles that both
  // halves see whole.
  __device__ __forceinline__ void middle(const PagedAttnParams& p, int lo, int hi, int ns, int skip,
                                         int& mid_lo, int& mid_hi) const {
    mid_lo = max(lo, ns);
    mid_hi = mid_lo;
    if (h[0].hi <= h[0].lo || h[1].hi <= h[1].lo) return;
    if constexpr (PRE) {
      mid_hi = max(mid_lo, min(hi, p.prefix_len / kBN));
    } else {
      // half_full: base + kBN - 1 <= plo, and behind the window's start
      mid_hi = (min(plo[0], plo[1]) + 1) / kBN - skip;
      if (p.window != 0)
        mid_lo = max(mid_lo, (max(0, max(phi[0], phi[1]) - p.window + 1) + kBN - 1) / kBN - skip);
      mid_hi = max(mid_lo, min(hi, mid_hi));
    }
  }
  // Rows [lo, hi) of the tile's V to look through, none if lo >= hi: of the
  // positions that some row sees and some does not, behind the first row's
  // position or where the windows start.
  __device__ __forceinline__ void look(const PagedAttnParams& p, int base, int& lo, int& hi) const {
    lo = kBN;
    hi = 0;
    if constexpr (PRE) return;
    const bool a0 = active(0, base), a1 = active(1, base);
    if (!a0 && !a1) return;
    const int first = a0 ? plo[0] : plo[1], last = a1 ? phi[1] : phi[0];
    if (last > first && last >= base && first + 1 < base + kBN) {
      lo = max(0, first + 1 - base);
      hi = min(kBN, last + 1 - base);
    }
    const int w0 = max(first - p.window + 1, p.n_sinks), w1 = last - p.window + 1;
    if (p.window != 0 && w0 < w1 && w1 > base && w0 < base + kBN) {
      lo = min(lo, max(0, w0 - base));
      hi = max(hi, min(kBN, w1 - base));
    }
  }
};

// A walk over a block's units: row tiles, KV heads, key tiles.  On the line of
// units an item has kItemCost empty ones before its tiles, so that blocks with
// many small items get fewer of them.
template <bool PRE>
struct TcCursor {
  RowTile t;
  int h, tile;
  long long u, i0;  // this unit, the item's first
  // true when the unit left was the last of its item in this walk
  CF_HOST_DEVICE bool next(const PagedAttnParams& p, long long end) {
    ++u;
    if (++tile < t.tiles) return u >= end;
    tile = 0;
    u += kItemCost;
    i0 = u;
    if (++h < p.g.nkv) return true;
    h = 0;
    if (u >= end) return true;
    int j = t.j + 1;
    while (j >= t.jn) {
      if (PRE || t.b + 1 >= p.batch) {  // only where starts or lengths change under the call: stop
        u = end;
        return true;
      }
      seq_of<PRE>(p, t.b + 1, t);
      j = 0;
    }
    tile_of<PRE>(p, j, t);
    return true;
  }
};

// A thread's share of the row tiles while the block finds its units: those of
// some numbers or, where starts are out of order (numbers then mean nothing),
// of some sequences.  All threads' shares, one after another, are all row tiles
// in the order of TcCursor, whatever the starts are.
template <bool PRE>
struct TcShare {
  bool ordered;
  int lo, hi, per;  // numbers, or sequences, lo .. hi - 1
  CF_HOST_DEVICE TcShare(const PagedAttnParams& p, int slots, bool ordered_, int thread)
      : ordered(ordered_) {
    const int n = ordered ? slots : p.batch;
    per = (n + kTcThreads - 1) / kTcThreads;
    lo = min(n, thread * per);
    hi = min(n, lo + per);
  }
  static CF_HOST_DEVICE int first_no(const PagedAttnParams& p, int b) {
    const int t0 = p.q_start ? min(max(p.q_start[b], 0), p.n_tokens) : b;
    return (int)((long long)t0 * p.g.G / (2 * kHalf)) + b;
  }
  // Calls f(tile) for the share's row tiles, in order, until it says stop.
#pragma nv_exec_check_disable  // f runs where walk does
  template <typename F>
  CF_HOST_DEVICE void walk(const PagedAttnParams& p, F&& f) const {
    if (lo >= hi) return;
    RowTile t;
    if constexpr (PRE) {
      seq_of<PRE>(p, 0, t);
      for (int j = lo; j < hi; ++j) {
        tile_of<PRE>(p, j, t);
        if (f(t)) return;
      }
    } else {
      int b = lo, end = hi;
      if (ordered) {  // the last sequence whose first number is <= lo
        int e = p.batch - 1;
        b = 0;
        end = p.batch;
        while (b < e) {
          const int mid = (b + e + 1) >> 1;
          if (first_no(p, mid) <= lo)
            b = mid;
          else
            e = mid - 1;
        }
      }
      for (; b < end; ++b) {
        const int no = ordered ? first_no(p, b) : 0;
        if (ordered && no >= hi) return;
        seq_of<PRE>(p, b, t);
        const int j1 = ordered ? min(t.jn, hi - no) : t.jn;
        for (int j = ordered ? max(0, lo - no) : 0; j < j1; ++j) {
          tile_of<PRE>(p, j, t);
          if (f(t)) return;
        }
      }
    }
  }
};

// Sets c to unit u of the line if that lies in the row tile t, whose units
// begin at `at`; else at moves on behind the row tile.
template <bool PRE>
CF_HOST_DEVICE bool start_in(const PagedAttnParams& p, const RowTile& t, long long u, long long& at,
                             TcCursor<PRE>& c) {
  const int len = t.tiles + kItemCost;
  const long long n = (long long)len * p.g.nkv;
  if (u >= at + n) {
    at += n;
    return false;
  }
  c.t = t;
  c.h = (int)div_units(u - at, len);
  c.i0 = at + (long long)c.h * len + kItemCost;
  c.tile = u > c.i0 ? (int)(u - c.i0) : 0;
  c.u = c.i0 + c.tile;
  return true;
}

// An item whose states the joining kernel takes up, written by the block that
// begins it: a split one (one per block at most, at the block's place), and
// after a prefix every one (in a list, in no order).
struct alignas(16) TcMeta {
  long long i0, upc;
  int tiles;  // 0: this block begins no split item
  int t0, p0, rows, j, h;
};

// Items to be computed again.
struct TcRedo {
  int b, t0, p0, rows, j, h;
};

struct TcArgs {
  PagedAttnParams p;
  PagedPrefixParts pre;
  PagedParts ws;
  TcMeta* meta;
  int n_meta, max_redo;  // places of the lists: short only where starts contradict themselves
  TcRedo* redo;
  // Items to be computed again, blocks that are done with them, items listed
  // in meta; all 0 between calls.
  int* n_redo;
  int slots;  // upper bound on the row tiles' numbers
  int grid;   // blocks of the main kernel
};

template <typename T, int D, int MODE>
__global__ void __launch_bounds__(kTcThreads, 1) paged_tc_kernel(const __grid_constant__ TcArgs a) {
  constexpr bool PRE = MODE == kPrefix, JOIN = MODE == kOwnAfterPrefix;
  using S = TcShape<D>;
  constexpr int C = D / 8;  // 16-byte chunks of a row
  constexpr int LIFT = weight_lift<T>(kGrow);
  constexpr float BACK = 1.f / (1 << LIFT);
  const PagedAttnParams& p = a.p;
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ long long s_scan[kTcThreads / 32];
  __shared__ TcCursor<PRE> s_cur;
  __shared__ TcCursor<PRE> s_wcur[13];  // each working warp's place: too much for registers
  __shared__ __align__(8) uint64_t s_full[S::SLOTS], s_empty[S::SLOTS];
  __shared__ __align__(8) uint64_t s_qfull, s_qempty, s_done;
  __shared__ __align__(8) uint64_t s_sfull[2], s_pfull[2], s_ofull[2];
  __shared__ uint32_t s_tmem;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sq = smem_u32(sm);                   // Q, two tiles
  const uint32_t skv = sq + 2 * S::TILE;              // K and V slots
  int* err = p.errflag;

  if (sq & 1023u) {  // the swizzle goes by the address
    if (tid == 0) atomicOr(err, kDevErrTimeout);
    if constexpr (JOIN) pdl_wait();
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < S::SLOTS; ++i) {
      mbar_init(&s_full[i], kCopyThreads);
      mbar_init(&s_empty[i], 1);
    }
    mbar_init(&s_qfull, kCopyThreads);
    mbar_init(&s_qempty, 1);
    mbar_init(&s_done, 1);
    for (int h = 0; h < 2; ++h) {
      mbar_init(&s_sfull[h], 1);
      mbar_init(&s_pfull[h], 4);
      mbar_init(&s_ofull[h], 1);
    }
    fence_mbar_init_cluster();
  }
  // After a prefix launch this one reads only what that launch has waited for
  // already (pdl_wait), so it starts on the SMs that it leaves and waits for it
  // at the end.
  if constexpr (!JOIN) pdl_wait();
  pdl_trigger();

  // ---- this block's units
  if constexpr (!PRE)  // the lookups below depend on one another: have their lines on the way
    for (int b = tid; b < p.batch; b += kTcThreads) {
      if (p.q_start) prefetch_line(p.q_start + b + 1);
      prefetch_line(p.kv_len + b);
    }
  const int nslots = PRE ? (p.n_tokens * p.g.G + 255) / 256 : a.slots;
  TcShare<PRE> share(p, nslots, true, tid);
  long long mine, incl;
  RowTile mine_t;  // the last of this thread's row tiles: with one each, the one
#pragma unroll 1
  while (true) {
    mine = 0;
    share.walk(p, [&](const RowTile& t) {
      mine += (long long)(t.tiles + kItemCost) * p.g.nkv;
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
    if (!PRE && p.q_start && share.ordered)
      for (int b = tid; b < p.batch; b += kTcThreads)
        done &= starts_ordered(p.q_start[b], p.q_start[b + 1], p.n_tokens);
    if (__syncthreads_and(done)) break;
    share = TcShare<PRE>(p, nslots, false, tid);  // the sum was over numbers that mean nothing
  }
  long long before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kTcThreads / 32; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  const long long upc = PRE ? a.pre.upc : div_units(total + gridDim.x - 1, gridDim.x);
  const long long u0 = blockIdx.x * upc, u1 = min(total, u0 + upc);
  if (MODE == kOwn && tid == 0) a.meta[blockIdx.x].tiles = 0;
  if (u0 >= u1) {
    if constexpr (JOIN) pdl_wait();
    return;
  }
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

  if (warp < 8) {
    // ------------------------------------------------------------ softmax --
    set_regs_up<184>();
    const int hf = warp >> 2;                   // half
    const int r = (warp & 3) * 32 + lane;       // row of the half = TMEM lane
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + S::S_COL + hf * kBN;
    const uint32_t to = tmem + lanes + S::O_COL + hf * D;
    const float sc = p.scale_log2;
    TcCursor<PRE>& cur = s_wcur[warp];
    if (lane == 0) cur = s_cur;
    __syncwarp();
    uint32_t n_tiles = 0;  // active tiles so far: parity of the barriers
    while (cur.u < u1) {
      const RowTile& t = cur.t;
      const int gr = t.j * 2 * kHalf + hf * kHalf + r;  // row of the sequence
      const int pos = PRE ? 0 : t.p0 + gr / p.g.G;
      const PagedRange rng = t.half[hf];
      const int plo = t.plo[hf], phi = t.phi[hf];
      const int first = cur.tile, count = (int)min((long long)(t.tiles - first), u1 - cur.u);
      const int ns = t.ns, skip = t.skip;
      float m = -INFINITY, l = 0.f;
      bool some = false;  // O holds something
#pragma unroll 1
      for (int tile = first; tile < first + count; ++tile) {
        const int base = (tile < ns ? tile : tile + skip) * kBN;
        if (tile_active(rng, base)) {
          wait_bar(&s_sfull[hf], n_tiles & 1, err);
          tc05_fence_after();
          float s[kBN];
#pragma unroll
          for (int k = 0; k < kBN / 32; ++k) tmem_ld32(ts + 32 * k, s + 32 * k);
          tmem_wait_ld();
          const bool full = half_full<PRE>(p, plo, phi, base);
          if (!full) {
#pragma unroll
            for (int c = 0; c < kBN / 32; ++c) {
              // bit k: this row sees position base + 32 c + k
              const int j0 = base + 32 * c;
              uint32_t see = low_bits((PRE ? p.prefix_len : pos + 1) - j0);
              if (!PRE && p.window != 0)
                see &= ~low_bits(pos - p.window + 1 - j0) | low_bits(p.n_sinks - j0);
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
          const bool grow = (m_new - m) * sc > (float)kGrow;  // also from -inf
          if (__any_sync(~0u, grow)) {
            const float corr = m_new == -INFINITY ? 1.f : ex2((m - m_new) * sc);
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
            l *= corr;
            m = m_new;
          }
          const float ref = (m == -INFINITY ? 0.f : m * sc) - LIFT;
          const float2 sc2 = make_float2(sc, sc), ref2 = make_float2(-ref, -ref);
          float2 sum[2] = {make_float2(l, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int k = 0; k < kBN / 32; ++k) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float2 x = fma2(make_float2(s[32 * k + 2 * e], s[32 * k + 2 * e + 1]), sc2, ref2);
              x.x = ex2(x.x);
              x.y = ex2(x.y);
              sum[e & 1] = add2(sum[e & 1], x);
              w[e] = pack2<T>(x.x, x.y);
            }
            tmem_st16(ts + 16 * k, w);
          }
          tmem_wait_st();
          tc05_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_pfull[hf]);
          l = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
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
      const float m2 = m * sc;  // base 2
      l *= BACK;
      const bool part = MODE != kOwn || !whole;  // leaves a state, not a result
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
          my_row = whole ? a.ws.state_base + my_row : prow0 + r;
          __stcg(a.ws.ml + my_row, make_float2(m2, l));
        } else {
          my_inv = l == 0.f ? 0.f : BACK / l;
          if (p.lse) p.lse[my_row] = paged_lse(m2, l);
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
      if (!PRE && part && first == 0 && tid == 0) {
        TcMeta x;
        x.i0 = cur.i0;
        x.upc = upc;
        x.tiles = t.tiles;
        x.t0 = t.t0;
        x.p0 = t.p0;
        x.rows = t.rows;
        x.j = t.j;
        x.h = cur.h;
        const int at = JOIN ? atomicAdd(a.n_redo + 2, 1) : blockIdx.x;
        if (at < a.n_meta) a.meta[at] = x;
      }
      tc05_fence_before();  // O is read before the next item's first product
      __syncwarp();
      if (lane == 0) {
        cur.u += count - 1;
        cur.tile += count - 1;
        cur.next(p, u1);
      }
      __syncwarp();
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------- copies --
    set_regs_down<80>();
    const int lw = warp - 8;  // rows 32 lw .. 32 lw + 31 of every tile
    TcCursor<PRE>& cur = s_wcur[warp];
    if (lane == 0) cur = s_cur;
    __syncwarp();
    constexpr int RP = 32 / C;                      // rows of one copy instruction
    const int r0 = lane / C, c0 = lane % C;
    const uint32_t d0 = (uint32_t)((c0 >> 3) * (kBN * 128) + (lw * 32 + r0) * 128);
    const uint32_t x0 = (uint32_t)(((c0 & 7) ^ r0) << 4);
    const int64_t ss = p.g.slot_stride * 2;
    // Copies 32 rows; lane i holds row i's byte offset in src, or -1 (zeros).
    auto copy = [&](uint32_t dst, const char* src, int64_t off, bool octets) {
      if (octets && __all_sync(~0u, off >= 0)) {
        // eight consecutive positions lie in one page: one lookup serves them
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const char* at = src + __shfl_sync(~0u, off, 8 * y) + r0 * ss + c0 * 16;
#pragma unroll
          for (int z = 0; z < 8 / RP; ++z) {
            cp16(dst + d0 + (8 * y + z * RP) * 128 + (x0 ^ ((z * RP) << 4)), at);
            at += RP * ss;
          }
        }
      } else {
#pragma unroll 8
        for (int x = 0; x < C; ++x) {
          const int64_t o = __shfl_sync(~0u, off, x * RP + r0);
          cp16(dst + d0 + x * RP * 128 + (x0 ^ (((x * RP) & 7) << 4)),
               src + (o >= 0 ? o + c0 * 16 : 0), o >= 0);
        }
      }
    };
    const char* kbase = static_cast<const char*>(p.k_pages);
    const char* vbase = static_cast<const char*>(p.v_pages);
    const char* qbase = static_cast<const char*>(p.q);
    const bool octets = p.g.page_shift >= 3;
    // The page of this lane's position, looked up one tile ahead of its copies.
    int f_pos = -1, f_page = 0;
    auto look_up = [&]() {
      const int j = cur.t.base(cur.tile) + lw * 32 + lane;
      f_pos = -1;
      if (cur.u >= u1 || !cur.t.sees(j)) return;
      f_pos = j;
      f_page = __ldg((PRE ? p.prefix_table : p.page_table + (int64_t)cur.t.b * p.g.max_pages) +
                     (j >> p.g.page_shift));
    };
    RingPos ring(0, S::SLOTS);
    uint32_t use = 0;  // slots taken so far
    uint32_t items = 0;
    bool fresh = true;
    look_up();
    while (cur.u < u1) {
      // a new item's Q: this lane's rows
      int64_t qoff[2] = {-1, -1};
      const bool new_q = fresh;
      if (new_q) {
        const RowTile& t = cur.t;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int gr = t.j * 2 * kHalf + h * kHalf + lw * 32 + lane;
          const int i = gr / p.g.G;
          if (gr < t.rows)
            qoff[h] =
                ((int64_t)(t.t0 + i) * p.q_stride + (int64_t)(cur.h * p.g.G + gr - i * p.g.G) * D) * 2;
        }
      }
      int64_t off = -1;
      if (f_pos >= 0) {
        if ((unsigned)f_page >= (unsigned)p.g.num_pages)
          atomicOr(err, kDevErrPosRange);
        else
          off = ((int64_t)f_page * p.g.page_stride +
                 (int64_t)(f_pos & p.g.page_mask) * p.g.slot_stride +
                 (int64_t)cur.h * p.g.head_stride) * 2;
      }
      __syncwarp();
      if (lane == 0) fresh = cur.next(p, u1);
      fresh = __shfl_sync(~0u, fresh, 0);
      __syncwarp();  // the cursor lies in shared memory; a shuffle orders nothing there
      look_up();
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        if (use >= S::SLOTS) wait_bar(&s_empty[ring.slot], ring.phase ^ 1u, err);
        copy(skv + ring.slot * S::TILE, kv ? vbase : kbase, off, octets);
        cp_arrive(&s_full[ring.slot]);
        ring.next(S::SLOTS);
        ++use;
      }
      // Q last: its buffer is free only when the previous item's scores are done
      if (new_q) {
        if (items) wait_bar(&s_qempty, (items - 1) & 1, err);
        copy(sq, qbase, qoff[0], false);
        copy(sq + S::TILE, qbase, qoff[1], false);
        cp_arrive(&s_qfull);
        ++items;
      }
    }
  } else {
    // ---------------------------------------------------------------- mma --
    set_regs_down<64>();
    // The whole warp walks (its operands then lie in uniform registers); one
    // elected thread issues.
    if (__shfl_sync(~0u, warp, 0) == 12) {
      constexpr uint32_t id_s = idesc_kind_f16(kIsBf16<T>, kHalf, kBN);
      constexpr uint32_t id_o = idesc_kind_f16(kIsBf16<T>, kHalf, D) | (1u << 16);  // B is N-major
      TcCursor<PRE>& cur = s_wcur[12];
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
        const TileCheck<PRE> tc(cur.t);
        const int ns = cur.t.ns, skip = cur.t.skip, first = cur.tile;
        const int count = (int)min((long long)(cur.t.tiles - first), u1 - cur.u);
        wait_bar(&s_qfull, items & 1, err);
        ++items;
        fence_proxy_async_smem();  // the copies wrote as ordinary stores
        bool bad = false;  // an infinity or NaN in a tile that was looked through
        bool acc0 = false, acc1 = false;
        bool pend = false;  // half 1's O += P V of the last tile is still to come
        int pend_slot = 0;
        // One tile: the scores of half 0, O of half 1 for the tile before, the
        // scores of half 1, O of half 0.  This warp's own instructions are on
        // the critical path, so the usual tile has its own copy of the code,
        // without any question.
        auto step = [&](bool act0, bool act1, int look_lo, int look_hi, bool last) {
          const int kslot = ring.slot;
          wait_bar(&s_full[kslot], ring.phase, err);
          ring.next(S::SLOTS);
          fence_proxy_async_smem();
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
          if (look_lo < look_hi) {  // the softmax of these scores is under way
            const uint32_t v0 = skv + vslot * S::TILE + lane * 16;
            uint32_t top[4] = {0u, 0u, 0u, 0u};  // largest magnitudes, 16 bits each
#pragma unroll
            for (int slab = 0; slab < D / 64; ++slab) {
#pragma unroll 4
              for (int i = (look_lo & ~3) * 128; i < look_hi * 128; i += 512) {  // four rows
                uint32_t w[4];
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                             : "r"(v0 + slab * (kBN * 128) + i));
#pragma unroll
                for (int e = 0; e < 4; ++e) top[e] = __vmaxu2(top[e], w[e] & 0x7fff7fffu);
              }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) bad |= nonfinite2<T>(top[e]);
          }
          fence_proxy_async_smem();
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
        // the tiles that both halves see whole, but for the run's last
        int mid_lo, mid_hi;
        tc.middle(p, first, first + count - 1, ns, skip, mid_lo, mid_hi);
#pragma unroll 1
        for (int tile = first; tile < first + count; ++tile) {
          if (tile == mid_lo && mid_lo < mid_hi) {
#pragma unroll 1
            for (; tile < mid_hi; ++tile) step(true, true, kBN, 0, false);
          }
          const int base = (tile < ns ? tile : tile + skip) * kBN;
          int look_lo, look_hi;
          tc.look(p, base, look_lo, look_hi);
          step(tc.active(0, base), tc.active(1, base), look_lo, look_hi, tile + 1 == first + count);
        }
        if (!PRE && __any_sync(~0u, bad) && lane == 0) {
          TcRedo x;
          x.b = cur.t.b;
          x.t0 = cur.t.t0;
          x.p0 = cur.t.p0;
          x.rows = cur.t.rows;
          x.j = cur.t.j;
          x.h = cur.h;
          const int at = atomicAdd(a.n_redo, 1);
          if (at < a.max_redo) a.redo[at] = x;
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
  if constexpr (JOIN) pdl_wait();
}

// Joins the states of the listed items, and the prefix's to them: a row per
// D / 4 lanes, gridDim.y blocks to an item.  Then computes again the items
// where that was asked for.  Bound by the launch and by reads of the states
// that are in L2; four blocks on an SM with four parts in flight per lane and
// up to 16 blocks to an item take 2-15 us less than eight in flight at two or
// three blocks with 32 to an item (with the main kernel, 8191 tokens, window
// 1024: 202 -> 185 us; 4 prompts of 517-2048 behind 0-2049: 150 -> 143).  That
// all items after a prefix are joined here, and none by the main kernel with a
// thread to a row, is 312 -> 167 us for 128 sequences of 8 tokens behind 8192
// shared positions (32 / 8 heads of 128).
constexpr int kTcJoinY = 16;
template <typename T, int D>
__global__ void __launch_bounds__(256, 4) paged_tc_join_kernel(const __grid_constant__ TcArgs a) {
  __shared__ float s_q[8][D];
  const PagedAttnParams& p = a.p;
  const int tid = threadIdx.x, lane = tid & 31;
  pdl_wait();
  pdl_trigger();
  const bool prefix = a.pre.rows != 0;
  const int n_redo = min(a.n_redo[0], a.max_redo);
  const int n_items = prefix ? min(a.n_redo[2], a.n_meta) : a.n_meta;
  constexpr int C4 = D / 4;
  for (int item = blockIdx.x; item < n_items; item += gridDim.x) {
    const TcMeta x = a.meta[item];
    // (an item that ends behind the line: lengths changed under the call)
    bool join = x.tiles != 0 && x.i0 + x.tiles <= x.upc * a.grid;
    for (int i = 0; i < n_redo && join; ++i)
      join = a.redo[i].t0 != x.t0 || a.redo[i].j != x.j || a.redo[i].h != x.h;
    if (!join) continue;
    const int rows = min(2 * kHalf, x.rows - x.j * 2 * kHalf);
    const PagedItemParts parts(x.i0, x.tiles, x.upc);
    for (int e = blockIdx.y * 256 + tid; e < rows * C4; e += gridDim.y * 256) {
      const int r = e / C4, col = (e - r * C4) * 4;
      PagedState4 s{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
      const int gr = x.j * 2 * kHalf + r, i = gr / p.g.G, g = gr - i * p.g.G;
      const long long t = x.t0 + i;
      const long long row = t * p.g.nq + x.h * p.g.G + g;
      paged_join_row<D, 4>(s, a.ws.o, a.ws.ml,
                           PagedRowParts(parts, 2 * kHalf, r, a.ws.state_base + row), col);
      if (prefix && x.p0 + i >= 0)
        paged_join_row<D, 4>(s, a.pre.o, a.pre.ml, paged_prefix_row(a.pre, p.g, t, x.h, g), col);
      paged_store4<T, D>(s, p.out, p.lse, row, col);
    }
  }
  if (n_redo == 0 && !prefix) return;
  const int warps = gridDim.x * gridDim.y * 8;
  float* q = s_q[tid >> 5];
  for (int e = (blockIdx.y * gridDim.x + blockIdx.x) * 8 + (tid >> 5); e < n_redo * 2 * kHalf;
       e += warps) {
    const TcRedo it = a.redo[e / (2 * kHalf)];
    const int gr = it.j * 2 * kHalf + e % (2 * kHalf);
    if (gr >= it.rows) continue;
    const int i = gr / p.g.G;
    const long long t = it.t0 + i, h = it.h * p.g.G + gr - i * p.g.G;
    __syncwarp();
    for (int c = lane; c < D; c += 32)
      q[c] = Elem<T>::to_f(static_cast<const T*>(p.q)[t * p.q_stride + h * D + c]);
    __syncwarp();
    PagedRow<T, D> r;
    r.run(p, q, it.b, it.p0 + i, it.p0 + it.rows / p.g.G, it.h, 0, 1);
    const float inv = r.l == 0.f ? 0.f : 1.f / r.l;
    T* out = static_cast<T*>(p.out) + (t * p.g.nq + h) * D + lane * (D / 32);
#pragma unroll
    for (int c = 0; c < D / 32; ++c) out[c] = Elem<T>::from_f(r.o[c] * inv);
    if (p.lse && lane == 0) p.lse[t * p.g.nq + h] = paged_lse(r.m, r.l);
  }
  // the last block out empties the lists
  __syncthreads();
  if (tid == 0 && atomicAdd(a.n_redo + 1, 1) == (int)(gridDim.x * gridDim.y) - 1) {
    a.n_redo[0] = 0;
    a.n_redo[1] = 0;
    a.n_redo[2] = 0;
  }
}

struct TcFns {
  const void *main, *join;
  int smem;
};
template <typename T, int D>
TcFns fns_td(int mode) {
  const void* main = mode == kPrefix ? (const void*)&paged_tc_kernel<T, D, kPrefix>
                     : mode == kOwn  ? (const void*)&paged_tc_kernel<T, D, kOwn>
                                     : (const void*)&paged_tc_kernel<T, D, kOwnAfterPrefix>;
  return TcFns{main, (const void*)&paged_tc_join_kernel<T, D>, TcShape<D>::SMEM};
}
TcFns tc_fns(int dtype, int d, int mode) {
  if (dtype == CF_F16) return d == 64 ? fns_td<__half, 64>(mode) : fns_td<__half, 128>(mode);
  return d == 64 ? fns_td<__nv_bfloat16, 64>(mode) : fns_td<__nv_bfloat16, 128>(mode);
}

}  // namespace

int cf::paged_tc_grid(int dtype, int head_dim, int sm_count) {
  for (int mode = kOwn; mode <= kOwnAfterPrefix; ++mode) {
    const TcFns f = tc_fns(dtype, head_dim, mode);
    if (cudaFuncSetAttribute(f.main, cudaFuncAttributeMaxDynamicSharedMemorySize, f.smem) !=
        cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
  }
  return sm_count;
}

long long cf::paged_tc_part_rows(int grid) { return 2LL * grid * kTcRows; }

size_t cf::paged_tc_list_bytes(int grid, long long items) {
  // every part of an item can be listed for another pass
  return (size_t)std::max<long long>(grid, items) * sizeof(TcMeta) +
         (size_t)(items + grid) * sizeof(TcRedo);
}

PagedPrefixParts cf::paged_tc_prefix(const PagedAttnParams& p, const PagedSplit& ws) {
  PagedPrefixParts x;
  x.o = ws.parts.o;
  x.ml = ws.parts.ml;
  x.state_base = ws.parts.state_base;
  x.rows = kTcRows;
  x.tiles = (p.prefix_len + kBN - 1) / kBN;
  x.item_cost = kItemCost;
  const long long row_tiles = ((long long)p.n_tokens * p.g.G + kTcRows - 1) / kTcRows;
  x.upc = std::max<long long>(
      1, (row_tiles * p.g.nkv * (x.tiles + kItemCost) + ws.grid - 1) / ws.grid);
  return x;
}

bool cf::paged_tc_launch(int dtype, const PagedAttnParams& p, const PagedSplit& ws, PagedMode mode,
                         const PagedPrefixParts& pre, cudaStream_t st) {
  const TcFns f = tc_fns(dtype, p.g.D, mode);
  TcArgs a;
  a.p = p;
  a.pre = pre;
  a.ws = ws.parts;
  a.meta = static_cast<TcMeta*>(ws.list);
  const long long n_list = std::max<long long>(ws.grid, ws.items);
  a.n_meta = (int)(mode == kOwn ? ws.grid : n_list);
  a.max_redo = (int)(ws.items + ws.grid);
  a.redo = reinterpret_cast<TcRedo*>(a.meta + n_list);
  a.n_redo = ws.tickets;
  a.slots = (int)((long long)p.n_tokens * p.g.G / kTcRows) + p.batch;
  a.grid = ws.grid;
  void* args[] = {&a};
  if (!launch_pdl(f.main, dim3(ws.grid), kTcThreads, f.smem, st, args)) return false;
  if (mode == kPrefix) return true;
  // fewer blocks to an item where its rows are fewer
  const long long rows = std::min<long long>(kTcRows, (long long)p.max_q * p.g.G);
  const int y = (int)std::min<long long>(kTcJoinY, (rows * (p.g.D / 4) + 255) / 256);
  return launch_pdl(f.join, dim3(ws.grid * (kTcJoinY / y), y), 256, 0, st, args);
}

extern "C" int cf_test_paged_line(int32_t batch, int32_t n_tokens, int32_t max_q, int32_t group,
                                  int32_t n_kv_heads, int32_t window, int32_t n_sinks, int32_t grid,
                                  const int32_t* q_start, const int32_t* kv_len, int32_t max_runs,
                                  int32_t* runs, int64_t* line) {
  if (batch < 1 || n_tokens < 1 || max_q < 1 || group < 1 || n_kv_heads < 1 || grid < 1 ||
      window < 0 || n_sinks < 0 || kv_len == nullptr || runs == nullptr || line == nullptr)
    return CF_ERR_INVALID_ARG;
  int err = 0;
  PagedAttnParams p;
  std::memset(&p, 0, sizeof(p));
  p.g.nkv = n_kv_heads;
  p.g.G = group;
  p.g.max_pages = 1 << 20;
  p.g.page_shift = 10;
  p.q_start = q_start;
  p.kv_len = kv_len;
  p.errflag = &err;
  p.batch = batch;
  p.n_tokens = n_tokens;
  p.max_q = max_q;
  p.window = window;
  p.n_sinks = n_sinks;
  bool ordered = true;
  for (int b = 0; q_start && b < batch; ++b)
    ordered &= starts_ordered(q_start[b], q_start[b + 1], n_tokens);
  const int slots = (int)((long long)n_tokens * group / kTcRows) + batch;
  long long first[kTcThreads + 1] = {0};
  for (int t = 0; t < kTcThreads; ++t) {
    long long mine = 0;
    TcShare<false>(p, slots, ordered, t).walk(p, [&](const RowTile& r) {
      mine += (long long)(r.tiles + kItemCost) * n_kv_heads;
      return false;
    });
    first[t + 1] = first[t] + mine;
  }
  const long long total = first[kTcThreads], upc = div_units(total + grid - 1, grid);
  line[0] = total;
  line[1] = upc;
  int n = 0;
  for (int block = 0; block < grid; ++block) {
    const long long u0 = block * upc, u1 = min(total, u0 + upc);
    if (u0 >= u1) break;
    TcCursor<false> c;
    bool found = false;
    for (int t = 0; t < kTcThreads && !found; ++t)
      if (first[t] <= u0 && u0 < first[t + 1]) {
        long long at = first[t];
        TcShare<false>(p, slots, ordered, t).walk(p, [&](const RowTile& r) {
          return found = start_in(p, r, u0, at, c);
        });
      }
    if (!found) return CF_ERR_DEVICE_POS_RANGE;
    while (c.u < u1) {
      const int count = (int)min((long long)(c.t.tiles - c.tile), u1 - c.u);
      const PagedItemParts parts(c.i0, c.t.tiles, upc);
      if (n < max_runs) {
        const int32_t run[kPagedRunInts] = {block, c.t.b, c.t.j, c.h, c.t.tiles, c.tile, count,
                                            parts.slot(0), parts.slot(parts.n - 1)};
        std::memcpy(runs + (size_t)n * kPagedRunInts, run, sizeof(run));
      }
      ++n;
      c.u += count - 1;
      c.tile += count - 1;
      c.next(p, u1);
    }
  }
  return n;
}
