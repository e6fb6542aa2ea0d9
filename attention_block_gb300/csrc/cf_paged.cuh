// cf_paged.cuh -- what the kernels of the paged KV cache share: the call's
// parameters, where a sequence's tokens and visible positions lie, the
// address of a position, and launch entry points (include/cf_paged.h).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "cf.h"
#include "cf_common.cuh"

namespace cf {

constexpr int kMaxPairs = 64;  // rotated pairs of a head (head_dim 128)

// How a call's work is cut is computed by functions that also run on the host,
// where a test walks them over any starts and lengths.
#define CF_HOST_DEVICE __host__ __device__ __forceinline__
CF_HOST_DEVICE void record_error(int* errflag, int bits) {
#ifdef __CUDA_ARCH__
  atomicOr(errflag, bits);
#else
  *errflag |= bits;
#endif
}

// Addressing of the pages, common to every call of a handle.
struct PagedGeom {
  int nq, nkv, G, D;
  int page_shift, page_mask;
  int num_pages, max_pages;
  int64_t page_stride, slot_stride, head_stride;  // elements
};

struct PagedAppendParams {
  PagedGeom g;
  const void *q, *k, *v;
  void *q_out, *k_pages, *v_pages;
  float2* scales;  // of a cache of 8-bit codes
  int64_t q_stride, kv_stride, q_out_stride;
  const int *q_start, *kv_len, *rope_pos, *page_table;
  int* errflag;
  int batch, n_tokens, rope_dim;
  uint64_t turn[kMaxPairs];  // theta^(-2i/r) / (2 pi) in 2^-64 of a turn
  uint8_t axis[kMaxPairs];   // which row of rope_pos pair i follows
};

struct PagedAttnParams {
  PagedGeom g;
  const void *q, *k_pages, *v_pages;
  const float2* scales;  // of a cache of 8-bit codes
  void* out;
  float* lse;
  int64_t q_stride;
  const int *q_start, *kv_len, *page_table, *prefix_table;
  int* errflag;
  int batch, n_tokens, max_q;
  int prefix_len, window, n_sinks;
  float scale_log2;  // score scale * log2(e): softmax in base 2
};

// Whether a sequence's starts are in order and within the call's tokens.
CF_HOST_DEVICE bool starts_ordered(int t0, int t1, int n_tokens) {
  return t0 >= 0 && t1 >= t0 && t1 <= n_tokens;
}

// The tokens of sequence b: first, count and its length; a malformed entry is
// recorded and leaves the sequence without tokens or without keys.
struct PagedSeq {
  int t0, n, len;
};
CF_HOST_DEVICE PagedSeq paged_seq(const int* q_start, const int* kv_len, int b, int n_tokens,
                                  int max_q, const PagedGeom& g, int* errflag) {
  PagedSeq s;
  s.t0 = q_start ? q_start[b] : b;
  const int t1 = q_start ? q_start[b + 1] : b + 1;
  s.len = kv_len[b];
  bool bad = !starts_ordered(s.t0, t1, n_tokens);
  s.n = bad ? 0 : t1 - s.t0;
  if (bad) s.t0 = 0;
  const long long cap = (long long)g.max_pages << g.page_shift;
  if (s.len < 0 || s.len > cap || s.n > max_q) {
    s.len = 0;
    bad = true;
  }
  if (bad) record_error(errflag, kDevErrPosRange);
  return s;
}

// Own positions that some row in [p_lo, p_hi] sees: [0, sink) and [lo, hi).
struct PagedRange {
  int sink, lo, hi;
};
CF_HOST_DEVICE PagedRange paged_range(int p_lo, int p_hi, int len, int window, int n_sinks) {
  PagedRange r;
  r.hi = min(p_hi + 1, len);
  if (r.hi < 0) r.hi = 0;
  r.lo = window > 0 ? max(0, p_lo - window + 1) : 0;
  if (r.lo > r.hi) r.lo = r.hi;
  r.sink = min(n_sinks, r.lo);
  return r;
}

__device__ __forceinline__ bool paged_visible(int p, int j, int window, int n_sinks) {
  return j <= p && (window == 0 || p - j < window || j < n_sinks);
}

// Element offset of position j (KV head 0) through a page table row, or -1 for
// a page number outside the pool (recorded).
__device__ __forceinline__ int64_t paged_offset(const int* table, int j, const PagedGeom& g,
                                                int* errflag) {
  const int page = table[j >> g.page_shift];
  if ((unsigned)page >= (unsigned)g.num_pages) {
    atomicOr(errflag, kDevErrPosRange);
    return -1;
  }
  return (int64_t)page * g.page_stride + (int64_t)(j & g.page_mask) * g.slot_stride;
}

// The tiles of TK positions that hold a range: sink tiles from 0, then the
// tiles of [lo, hi); always at least one.
template <int TK>
struct PagedTiles {
  int sink, lo, hi;
  int ns, skip;  // sink tiles, and tiles between them and the window's first
  int tiles;
  CF_HOST_DEVICE void set(const PagedRange& r) {
    sink = r.sink;
    lo = r.lo;
    hi = r.hi;
    if (hi <= lo) {  // no key
      sink = ns = skip = 0;
      tiles = 1;
      return;
    }
    const int f = lo / TK, e = (hi + TK - 1) / TK;
    ns = (sink + TK - 1) / TK;
    skip = max(0, f - ns);
    if (skip == 0) ns = 0;
    tiles = e - skip;
  }
  __device__ __forceinline__ int base(int tile) const {
    return (tile < ns ? tile : tile + skip) * TK;
  }
  __device__ __forceinline__ bool sees(int j) const { return (j >= lo && j < hi) || j < sink; }
};

// 16 bytes global -> shared, asynchronously; zeros where there is no source.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// How a kernel's work is cut.  The units (key tiles) of all items (a sequence
// or row tile and a KV head) form one line, cut into pieces: piece c takes
// units [c * upc, (c + 1) * upc).  An item that lies in several pieces leaves
// one partial state (o not normalised, running maximum in base 2, sum) per
// piece, in slot 2c where it began in an earlier piece and in 2c + 1 where it
// begins in this one.  Where states are wanted of every item (a prefix's, and
// own keys' before the prefix is joined), one that lies within a piece has
// rows of its own from state_base on: the prefix's at token * nq + head; own
// ones too, or at 16 rows per (sequence, KV head) where those are fewer.
struct PagedParts {
  float* o;              // [rows][D]: slots of a fixed number of rows, then single rows
  float2* ml;            // [rows]
  long long state_base;
  int by_token;
};

// Starts a load into L1 without waiting for it.
__device__ __forceinline__ void prefetch_line(const void* at) {
  asm volatile("{\n\t.reg .u32 v;\n\tld.global.ca.u32 v, [%0];\n\t}" ::"l"(at));
}
// Waits until the launch in front has ended and what it wrote can be seen.
// Every kernel here calls it before it triggers the next (pdl_trigger), so one
// that has begun knows that everything before the launch in front has ended
// too.  The one exception is the launch behind a prefix's (kOwnAfterPrefix): it
// triggers first and waits at its end, and until then reads nothing that the
// prefix's launch writes, and writes nothing that it uses.  That needs the
// prefix's launch to wait before it triggers.
__device__ __forceinline__ void pdl_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void pdl_trigger() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// a / b, in 32 bits where both fit (a 64-bit division is a long chain).
CF_HOST_DEVICE long long div_units(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (long long)((uint32_t)a / (uint32_t)b);
  return a / b;
}

// Slots of one item's partial states, in the order of its n pieces.
struct PagedItemParts {
  int first, odd, n;
  CF_HOST_DEVICE PagedItemParts(long long i0, long long tiles, long long upc) {
    const long long c = div_units(i0, upc);
    first = (int)(2 * c);
    odd = c * upc >= i0 ? 0 : 1;  // later pieces all begin behind i0
    n = (int)(div_units(i0 + tiles - 1, upc) - c) + 1;
  }
  CF_HOST_DEVICE int slot(int k) const { return first + 2 * k + (k == 0 ? odd : 0); }
};

// The shared prefix's states, as the kernels that join them to the sequences'
// own find them: row R = token * G + (head in the KV head's group) is row
// R % rows of tile R / rows, and item tile * nkv + kv head has `tiles` units
// behind item_cost empty ones.  rows == 0: there is no prefix.
struct PagedPrefixParts {
  const float* o;
  const float2* ml;
  long long state_base;
  int rows;
  int tiles, item_cost;
  long long upc;
};

// Where one row's states of an item lie: row() of the arrays for part k < n.
struct PagedRowParts {
  PagedItemParts parts;
  int rows, r, n;
  long long state;
  __device__ __forceinline__ PagedRowParts(const PagedItemParts& p, int rows_, int r_,
                                           long long state_)
      : parts(p), rows(rows_), r(r_), n(p.n), state(state_) {}
  __device__ __forceinline__ long long row(int k) const {
    return n == 1 ? state : (long long)parts.slot(k) * rows + r;
  }
};
__device__ __forceinline__ PagedRowParts paged_prefix_row(const PagedPrefixParts& x,
                                                          const PagedGeom& g, long long token,
                                                          int kvh, int gi) {
  const long long R = token * g.G + gi, tile = div_units(R, x.rows);
  const long long index = tile * g.nkv + kvh;
  return PagedRowParts(
      PagedItemParts(index * (x.tiles + x.item_cost) + x.item_cost, x.tiles, x.upc), x.rows,
      (int)(R - tile * x.rows), x.state_base + token * g.nq + kvh * g.G + gi);
}

// Softmax state of 4 columns of a row, joined with another one.
struct PagedState4 {
  float m, l;
  float4 o;
  __device__ __forceinline__ void join(float m2, float l2, const float4& o2) {
    const float mn = fmaxf(m, m2), ref = mn == -INFINITY ? 0.f : mn;
    const float a = exp2f(m - ref), b = exp2f(m2 - ref);
    m = mn;
    l = l * a + l2 * b;
    o.x = o.x * a + o2.x * b;
    o.y = o.y * a + o2.y * b;
    o.z = o.z * a + o2.z * b;
    o.w = o.w * a + o2.w * b;
  }
};

// Joins a row's states into s: the D / 4 lanes that share the row call it
// together, each for its 4 columns at `col`.  Each lane fetches one part's
// maximum and sum, and the parts' values come B at a time, the first ones
// together with the maxima.  HALVES: what a sum is multiplied by can be below 2^-126
// and the sum still count, as the maxima hold value scales that lie far apart.
template <int D, int B = 8, bool HALVES = false>
__device__ __forceinline__ void paged_join_row(PagedState4& s, const float* o, const float2* ml,
                                               const PagedRowParts& x, int col) {
  constexpr int W = D / 4;
  const int lane = threadIdx.x & 31, gl = lane % W;
  const uint32_t mask = W == 32 ? ~0u : 0xffffu << (lane & 16);
  for (int k0 = 0; k0 < x.n; k0 += W) {
    const int n = min(W, x.n - k0);
    float2 v = make_float2(-INFINITY, 0.f);
    if (gl < n) v = __ldcg(ml + x.row(k0 + gl));
    float4 y[B];
    auto fetch = [&](int k) {
#pragma unroll
      for (int i = 0; i < B; ++i)
        y[i] = k + i < n ? __ldcg(reinterpret_cast<const float4*>(o + x.row(k0 + k + i) * D + col))
                         : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    fetch(0);
    float mx = v.x;
#pragma unroll
    for (int d = W / 2; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(mask, mx, d));
    const float mn = fmaxf(s.m, mx), ref = mn == -INFINITY ? 0.f : mn;
    float a, w, l, ha = 1.f;
    if constexpr (HALVES) {
      const float hw = exp2f(0.5f * (v.x - ref));
      ha = exp2f(0.5f * (s.m - ref));
      a = ha * ha;
      w = hw * hw;
      l = v.y * hw * hw;
    } else {
      a = exp2f(s.m - ref), w = exp2f(v.x - ref);
      l = v.y * w;
    }
#pragma unroll
    for (int d = W / 2; d >= 1; d >>= 1) l += __shfl_xor_sync(mask, l, d);
    s.m = mn;
    if constexpr (HALVES)
      s.l = s.l * ha * ha + l;
    else
      s.l = s.l * a + l;
    s.o = make_float4(s.o.x * a, s.o.y * a, s.o.z * a, s.o.w * a);
    for (int k = 0; k < n; k += B) {
      if (k) fetch(k);
#pragma unroll
      for (int i = 0; i < B; ++i) {
        const float wk = __shfl_sync(mask, w, (k + i) % W, W);
        s.o.x = fmaf(y[i].x, wk, s.o.x);
        s.o.y = fmaf(y[i].y, wk, s.o.y);
        s.o.z = fmaf(y[i].z, wk, s.o.z);
        s.o.w = fmaf(y[i].w, wk, s.o.w);
      }
    }
  }
}

// A row's lse from its maximum in base 2 and its sum.  The sum decides: where
// every score is NaN the maximum is still -infinity.
__device__ __forceinline__ float paged_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

// Normalises and stores 4 columns of a row, and its lse.
template <typename T, int D>
__device__ __forceinline__ void paged_store4(const PagedState4& s, void* out, float* lse,
                                             long long row, int col) {
  const float inv = s.l == 0.f ? 0.f : 1.f / s.l;
  const float f[4] = {s.o.x * inv, s.o.y * inv, s.o.z * inv, s.o.w * inv};
  store4<T>(static_cast<T*>(out) + row * D + col, f);
  if (lse && col == 0) lse[row] = paged_lse(s.m, s.l);
}

// Transposes w over a quad of lanes: lane q ends with word q of lanes 0..3.
__device__ __forceinline__ void quad_transpose(uint32_t (&w)[4], int q) {
  const bool a = q & 1, b = q & 2;
#pragma unroll
  for (int i = 0; i < 4; i += 2) {  // pairs (0, 1) and (2, 3)
    const uint32_t x = __shfl_xor_sync(~0u, a ? w[i] : w[i + 1], 1);
    if (a)
      w[i] = x;
    else
      w[i + 1] = x;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {  // pairs (0, 2) and (1, 3)
    const uint32_t x = __shfl_xor_sync(~0u, b ? w[i] : w[i + 2], 2);
    if (b)
      w[i] = x;
    else
      w[i + 2] = x;
  }
}

template <typename T>
struct MmaExp;  // exponent bits of a 16-bit type
template <>
struct MmaExp<__half> {
  static constexpr uint32_t mask = 0x7c00u;
};
template <>
struct MmaExp<__nv_bfloat16> {
  static constexpr uint32_t mask = 0x7f80u;
};

// Whether one of the two 16-bit values in w is an infinity or NaN.
template <typename T>
__device__ __forceinline__ bool nonfinite2(uint32_t w) {
  const uint32_t e = MmaExp<T>::mask;
  return (w & e) == e || ((w >> 16) & e) == e;
}

// 2^x, off by 2 ulp; results below 2^-126 are 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// One row of attention by one warp on the CUDA cores: the row at position pos
// of sequence b sees, in one list, the prefix, its sinks and its window.  A
// lane forms the whole dot product of one key; then every lane sums its
// columns of 32 weighted values.  Masked positions are never loaded.  The
// warp takes the chunks of 32 keys w, w + step, ..; q: the row's query in
// fp32, shared memory.
template <typename T, int D>
struct PagedRow {
  static constexpr int E = D / 32;  // columns of a lane
  float m, l, o[E];                 // running maximum (base 2), the lane's share of the sum, o
  __device__ __forceinline__ void run(const PagedAttnParams& p, const float* q, int b, int pos,
                                      int len, int kvh, int w, int step) {
    constexpr int W = 16 / sizeof(T);
    const int lane = threadIdx.x & 31;
    const PagedRange r = paged_range(pos, pos, len, p.window, p.n_sinks);
    const int pre = pos < 0 ? 0 : p.prefix_len;
    const int total = pos < 0 ? 0 : pre + r.sink + (r.hi - r.lo);
    const int* table = p.page_table + (int64_t)b * p.g.max_pages;
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int base = w * 32; base < total; base += step * 32) {
      int idx = base + lane;
      int64_t off = -1;  // no page: zeros stand for the key and the value
      float sc = -INFINITY;
      if (idx < total) {
        sc = 0.f;
        if (idx < pre) {
          off = paged_offset(p.prefix_table, idx, p.g, p.errflag);
        } else {
          idx -= pre;
          off = paged_offset(table, idx < r.sink ? idx : r.lo + idx - r.sink, p.g, p.errflag);
        }
      }
      if (off >= 0) {
        off += (int64_t)kvh * p.g.head_stride;
        const T* k = static_cast<const T*>(p.k_pages) + off;
        float acc = 0.f;
#pragma unroll 4
        for (int i = 0; i < D; i += W) {
          float f[W];
          load_cvt<T, W>(k + i, f);
#pragma unroll
          for (int e = 0; e < W; ++e) acc = fmaf(f[e], q[i + e], acc);
        }
        sc = acc * p.scale_log2;
      }
      float mx = sc;
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, d));
      const float m_new = fmaxf(m, mx);
      const float ref = m_new == -INFINITY ? 0.f : m_new;
      const float pr = exp2f(sc - ref), corr = exp2f(m - ref);
      m = m_new;
      l = l * corr + pr;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= corr;
      const int n = min(32, total - base);
      for (int k = 0; k < n; ++k) {
        const int64_t vo = __shfl_sync(~0u, off, k);
        const float wk = __shfl_sync(~0u, pr, k);
        if (vo < 0) continue;
        float f[E];
        load_cvt<T, E>(static_cast<const T*>(p.v_pages) + vo + lane * E, f);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(wk, f[e], o[e]);
      }
    }
    l = warp_sum(l);
  }
};

// log2 of what weights are multiplied by before they become 16-bit operands,
// where none is above 2^largest: fp16 has few exponents, and weights below
// 2^-25 would count in their sum and not in the product.  Times 2^(15 - largest)
// it holds them down to 2^(largest - 40).  A part's states are scaled back.
template <typename T>
CF_HOST_DEVICE constexpr int weight_lift(int largest) {
  return MmaExp<T>::mask == 0x7c00u ? 15 - largest : 0;
}

// What a launch attends to: the sequences' own keys; the shared prefix (it
// leaves states only); own keys, joined with the prefix's states.
enum PagedMode { kOwn = 0, kPrefix = 1, kOwnAfterPrefix = 2 };

// An attention kernel's part of a handle's workspace.
struct PagedSplit {
  PagedParts parts;
  void* list = nullptr;    // items for a joining kernel
  int* tickets = nullptr;  // words that are zero between calls: few rows, one per (sequence,
                           // KV head); many, three
  int grid = 0;            // resident blocks
  long long items = 0;     // that the lists have room for
};

// Launches a kernel that may begin before the one in front of it in the stream
// has ended (and waits for that one itself, pdl_wait); false: it failed.
inline bool launch_pdl(const void* fn, dim3 grid, int threads, int smem, cudaStream_t st,
                       void** args) {
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.gridDim = grid;
  lc.blockDim = dim3(threads, 1, 1);
  lc.dynamicSmemBytes = smem;
  lc.stream = st;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelExC(&lc, fn, args) == cudaSuccess;
}

// Host launchers (one translation unit each); false: the launch failed.
bool paged_append_launch(int dtype, const PagedAppendParams& p, int sm_count, cudaStream_t st);

// The fp32 kernel.  grid: resident blocks, 0 on failure; part_rows: workspace;
// a ticket per resident block and a word more.
int paged_f32_grid(int head_dim, int sm_count);
long long paged_f32_part_rows(int grid);
bool paged_f32_launch(const PagedAttnParams& p, const PagedSplit& ws, cudaStream_t st);

// The kernel for few rows (tokens x grouped heads), and the one on the fifth
// generation's tensor cores for many.  grid: resident blocks, 0 on failure;
// part_rows and list_bytes: workspace; launch with kPrefix: the call's tokens
// against the prefix alone; prefix: how such a launch cuts it.
constexpr int kFewRows = 16;
int paged_few_grid(int dtype, int head_dim, int sm_count);
long long paged_few_part_rows(int grid);
PagedPrefixParts paged_few_prefix(const PagedAttnParams& p, const PagedSplit& ws);
bool paged_few_launch(int dtype, const PagedAttnParams& p, const PagedSplit& ws, PagedMode mode,
                      const PagedPrefixParts& pre, cudaStream_t st);

constexpr int kTcRows = 256;
int paged_tc_grid(int dtype, int head_dim, int sm_count);
long long paged_tc_part_rows(int grid);
size_t paged_tc_list_bytes(int grid, long long items);
PagedPrefixParts paged_tc_prefix(const PagedAttnParams& p, const PagedSplit& ws);
bool paged_tc_launch(int dtype, const PagedAttnParams& p, const PagedSplit& ws, PagedMode mode,
                     const PagedPrefixParts& pre, cudaStream_t st);

}  // namespace cf
