// cf_paged_few.cuh -- items and their key tiles, as the few-row attention
// kernels of the paged caches walk over them (16-bit values and 8-bit codes).
#pragma once

#include "cf_paged.cuh"

namespace cf {

// An item, as far as those need it that join its parts.
struct alignas(16) FewItem {
  long long i0;
  int tiles, t0, p0, n, b, h;
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
      if (PRE || b + 1 >= p.batch) {  // only where lengths change under the call: stop
        u = end;
        return;
      }
      w = work_of<TK, PRE>(p, ++b);
    } while (w.tiles == 0);
  }
};

// Row of out (and of the prefix's states) of an item's row.
__device__ __forceinline__ long long out_row(const PagedAttnParams& p, const FewItem& it, int row) {
  const int i = row / p.g.G;
  return (long long)(it.t0 + i) * p.g.nq + it.h * p.g.G + row - i * p.g.G;
}

}  // namespace cf
