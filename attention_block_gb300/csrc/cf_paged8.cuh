// cf_paged8.cuh -- what the kernels of the paged cache of 8-bit codes share:
// where scales lie, codes from values and back, and launch entry points
// (include/cf_paged8.h).
#pragma once

#include "cf_paged.cuh"
#include "cf_paged8.h"

namespace cf {

// Index of the scales of position j, KV head 0: a KV head's are page_size
// apart.  The page must lie in the pool (paged_offset).
__device__ __forceinline__ int64_t paged8_scale(const int* table, int j, const PagedGeom& g) {
  return (((int64_t)table[j >> g.page_shift] * g.nkv) << g.page_shift) + (j & g.page_mask);
}

// Largest magnitude of a code.
template <int CODE>
constexpr float kCodeTop = CODE == CF_CODE_INT8 ? 127.f : 448.f;

// Four codes of values that are within the codes' range.
template <int CODE>
__device__ __forceinline__ uint32_t code4(const float* f) {
  if constexpr (CODE == CF_CODE_INT8) {
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) w |= (uint32_t)(__float2int_rn(f[e]) & 0xff) << (8 * e);
    return w;
  } else {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(f[1]), "f"(f[0]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(f[3]), "f"(f[2]));
    return (uint32_t)lo | (uint32_t)hi << 16;
  }
}

// Codes and scale of a head that LANES neighbouring lanes hold, 16 values each:
// w[0] the codes of the first eight, w[1] of the others.
template <int CODE, int LANES>
__device__ __forceinline__ void quantise_head(const float (&f)[16], float& scale, uint2 (&w)[2]) {
  const uint32_t group = (uint32_t)((1ull << LANES) - 1) << (threadIdx.x & 31 & ~(LANES - 1));
  uint32_t top = 0;  // as whole numbers magnitudes are in order, NaN last
#pragma unroll
  for (int e = 0; e < 16; ++e) top = max(top, __float_as_uint(f[e]) & 0x7fffffffu);
#pragma unroll
  for (int d = LANES / 2; d >= 1; d >>= 1) top = max(top, __shfl_xor_sync(group, top, d));
  const float amax = __uint_as_float(top);
  const bool finite = top < 0x7f800000u, zero = amax < 0x1p-100f;
  scale = finite ? (zero ? 0.f : amax / kCodeTop<CODE>) : __uint_as_float(0x7fc00000u);
  const float inv = finite && !zero ? kCodeTop<CODE> / amax : 0.f;
  float y[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) y[e] = finite ? f[e] * inv : 0.f;
  w[0] = make_uint2(code4<CODE>(y), code4<CODE>(y + 4));
  w[1] = make_uint2(code4<CODE>(y + 8), code4<CODE>(y + 12));
}

// Four codes as two words of fp16 values: of codes 0 and 2, and of 1 and 3.
// Both are exact; an e4m3 NaN becomes a NaN.  (Whole numbers set into the mantissa of
// a power of two, which is then subtracted: a published way with weights of 8 and 4
// bits, Kim et al., 2022; the constants follow from the format.)
template <int CODE>
__device__ __forceinline__ void code_halves(uint32_t w, uint32_t& even, uint32_t& odd) {
  if constexpr (CODE == CF_CODE_INT8) {
    // 1024 + (code + 128) is the fp16 with those low bits
    const uint32_t u = w ^ 0x80808080u;
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    const uint32_t e = __byte_perm(u, 0x64646464u, 0x4240), o = __byte_perm(u, 0x64646464u, 0x4341);
    const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&e), bias);
    const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&o), bias);
    even = *reinterpret_cast<const uint32_t*>(&a);
    odd = *reinterpret_cast<const uint32_t*>(&b);
  } else {
    const uint32_t t = __byte_perm(w, 0u, 0x3120);
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(even), "=r"(odd)
        : "r"(t));
  }
}

// The same of codes 0 and 1, and of 2 and 3.
template <int CODE>
__device__ __forceinline__ void code_row4(uint32_t w, uint32_t& first, uint32_t& last) {
  if constexpr (CODE == CF_CODE_INT8) {
    const uint32_t u = w ^ 0x80808080u;
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    const uint32_t e = __byte_perm(u, 0x64646464u, 0x4140), o = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&e), bias);
    const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&o), bias);
    first = *reinterpret_cast<const uint32_t*>(&a);
    last = *reinterpret_cast<const uint32_t*>(&b);
  } else {
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(first), "=r"(last)
        : "r"(w));
  }
}

// log2 x and 1 / x, off by a few ulp (log2 by 2^-22 near 1).
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Value scales in the weights.  A position's weight takes log2 vs into its
// exponent; the sum of exp(s) takes the weight times 1 / vs.  That is whole while the
// scales of a row lie within 2^79 of one another: what is flushed then has an exp(s)
// below 2^-54 of the largest, and 2^30 of them are 2^-24 of the sum.  So it is from
// 2^-80 to 2^-1 (values of 63 with int8, 224 with e4m3), and from 2^-19 to the largest
// scale, 2^60.  Where an item has shown a scale above 2^-1 (high), the positions with
// one below 2^-19 (low) are added to the sum apart, as 2^(s - reference).
//
// A scale of zero enters the exponent as 2^-80: the codes are zero, so it only has to
// be too small to raise the maximum (20 octaves below the least scale), and leaves
// 2^(s - reference) room for a sum of 2^30 (2^(80 + 15 + 30) at most).
//
// What lies outside the scales that are read: below 2^-60 a value scale counts as 0
// (its codes may be other than zero: what 2^-80 of them adds is below 2^-70); above
// 2^60 or below 0 a scale counts as NaN (odd).
struct ValueScale {
  float log2;      // of what stands for the scale in the exponent
  float inv;       // 1 / that: what the sum multiplies a weight by
  bool plain;      // neither low nor high nor odd
  __device__ __forceinline__ explicit ValueScale(float v) {
    const float vv = v >= 0x1p-60f ? fminf(v, 0x1p60f) : 0x1p-80f;
    log2 = lg2(vv);
    inv = rcp(vv);
    plain = v >= 0x1p-19f && v <= 0.5f;
  }
  static __device__ __forceinline__ bool low(float v) { return v < 0x1p-19f; }
  static __device__ __forceinline__ bool high(float v) { return v > 0.5f; }
};
__device__ __forceinline__ bool scale_is_read(float v) { return v >= 0.f && v <= 0x1p60f; }
__device__ __forceinline__ float key_scale(float k) {
  return scale_is_read(k) ? k : __uint_as_float(0x7fc00000u);
}

// 8 bytes global -> shared, asynchronously; zeros where there is no source.
__device__ __forceinline__ void cp8(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src),
               "r"(there ? 8 : 0)
               : "memory");
}

// Host launchers; false: the launch failed.
bool paged8_append_launch(int dtype, int code, const PagedAppendParams& p, int sm_count,
                          cudaStream_t st);
struct Paged8ReadParams {
  PagedGeom g;
  const void *k_pages, *v_pages;
  const float2* scales;
  const int *row_start, *first, *page_table;
  void *k_out, *v_out;
  int64_t out_stride;
  int* errflag;
  int batch, n_rows;
};
bool paged8_read_launch(int dtype, int code, const Paged8ReadParams& p, cudaStream_t st);

// The kernel for few rows (tokens x grouped heads, at most kFewRows).  grid:
// resident blocks, 0 on failure; its parts take as many rows as
// paged_few_part_rows says.
int paged8_few_grid(int dtype, int code, int head_dim, int sm_count);
bool paged8_few_launch(int dtype, int code, const PagedAttnParams& p, const PagedSplit& ws,
                       cudaStream_t st);

// The kernel for many rows; its parts take as many rows as paged_tc_part_rows
// says, and its list of items paged8_tc_list_bytes.
int paged8_tc_grid(int dtype, int code, int head_dim, int sm_count);
size_t paged8_tc_list_bytes(int grid);
bool paged8_tc_launch(int dtype, int code, const PagedAttnParams& p, const PagedSplit& ws,
                      cudaStream_t st);

}  // namespace cf
