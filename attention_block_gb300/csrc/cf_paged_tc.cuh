// cf_paged_tc.cuh -- what the many-row attention kernels of the paged caches
// share (16-bit values and 8-bit codes): small PTX wrappers, row tiles and their
// key tiles, and the walk over the line of units.
#pragma once

#include "cf_paged.cuh"
#include "cf_tc05.cuh"

namespace cf {

constexpr int kTcThreads = 512;
constexpr int kCopyThreads = 128;
constexpr int kHalf = 128;     // rows of a half
constexpr int kBN = 128;       // positions of a tile
// What an item costs beside its tiles, in tiles.  4 prompts of 517-2048 tokens
// (32 / 8 heads of 128): 241 us with 0, 155 with 2, 145 with 5, 150 with 8.
constexpr int kItemCost = 5;
constexpr int kGrow = 8;       // log2 of the growth that forces a rescale

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
// units an item has COST empty ones before its tiles, so that blocks with
// many small items get fewer of them.
template <bool PRE, int COST = kItemCost>
struct TcCursor {
  RowTile t;
  int h, tile;
  long long u, i0;  // this unit, the item's first
  // true when the unit left was the last of its item in this walk
  CF_HOST_DEVICE bool next(const PagedAttnParams& p, long long end) {
    ++u;
    if (++tile < t.tiles) return u >= end;
    tile = 0;
    u += COST;
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
template <bool PRE, int COST>
CF_HOST_DEVICE bool start_in(const PagedAttnParams& p, const RowTile& t, long long u, long long& at,
                             TcCursor<PRE, COST>& c) {
  const int len = t.tiles + COST;
  const long long n = (long long)len * p.g.nkv;
  if (u >= at + n) {
    at += n;
    return false;
  }
  c.t = t;
  c.h = (int)div_units(u - at, len);
  c.i0 = at + (long long)c.h * len + COST;
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

}  // namespace cf
