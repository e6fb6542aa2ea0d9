// cf_w4.cu -- products of a few rows with weights of 4 bits (include/cf_w4.h):
// the layout of the weights, the product, and the host side.
//
// The weights are the tensor core's A operand (16 columns of W by 16 elements
// of k), the rows of x its B operand (8 rows), so one row costs as many
// instructions as eight.  A code c becomes the 16-bit float 1024 + c (fp16) or
// 128 + c (bf16) by setting bits, and c - zero by one exact subtraction; a
// group's sum is scaled in fp32.
//
// A record holds 64 columns x 128 elements of k.  Its codes: for each block of
// 16 columns and each 64 of k, a 16-byte vector per lane, word s the A fragment
// of step s.  Lane (g, t) of step s stands for columns g and g + 8 and for
// k = 32 (s / 2) + 8 t + 4 (s % 2) + 0..3: any order of k will do as long as x
// follows it, and in this one a lane's x are 16-byte vectors and no step mixes
// two groups.  Of a word, nibble i and nibble i + 4 are the two halves of the
// fragment's register i.  Behind the codes the groups' scales, then their
// zeros, columns g and g + 8 of a block side by side.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <new>

#include "cf_common.cuh"
#include "cf_mma.cuh"
#include "cf_paged.cuh"
#include "cf_w4.h"

using namespace cf;

namespace {

constexpr int kUnitK = 128;   // elements of k of a record
constexpr int kTileN = 64;    // columns of a record
constexpr int kCodeBytes = kUnitK * kTileN / 2;
constexpr int kW4Threads = 256;

struct W4Shape {
  int K, N, group, zeros, es;
  int units, tiles;       // records along k and along n
  int record;             // bytes
  __host__ __device__ int groups() const { return kUnitK / group; }  // of a record
};

// ------------------------------------------------------------------- layout --
__global__ void __launch_bounds__(kW4Threads)
    w4_pack_kernel(W4Shape s, const uint8_t* codes, const uint8_t* scales, const uint8_t* zeros,
                   uint8_t* packed) {
  const int unit = blockIdx.x % s.units, tile = blockIdx.x / s.units;
  uint8_t* out = packed + (int64_t)blockIdx.x * s.record;
  pdl_wait();
  for (int w = threadIdx.x; w < kCodeBytes / 4; w += kW4Threads) {
    const int step = w & 3, lane = (w >> 2) & 31, half = (w >> 7) & 1, block = w >> 8;
    const int g = lane >> 2, t = lane & 3;
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // register i & 3, its low (i < 4) or high half
      const int n = tile * kTileN + block * 16 + g + 8 * (i & 1);
      const int k = unit * kUnitK + half * 64 + 32 * (step >> 1) + 8 * t + 4 * (step & 1) +
                    2 * ((i >> 1) & 1) + (i >> 2);
      uint32_t c = 0;
      if (n < s.N && k < s.K) c = (codes[(int64_t)k * (s.N / 2) + n / 2] >> (4 * (n & 1))) & 15u;
      word |= c << (4 * i);
    }
    reinterpret_cast<uint32_t*>(out)[w] = word;
  }
  // scales and zeros: place x of a group is column (x / 16) * 16 + (x % 16) / 2 + 8 (x % 2)
  const int places = s.groups() * kTileN;
  for (int e = threadIdx.x; e < places; e += kW4Threads) {
    const int x = e % kTileN;
    const int n = tile * kTileN + (x & ~15) + ((x & 15) >> 1) + 8 * (x & 1);
    const int k = unit * kUnitK + (e / kTileN) * s.group;
    const bool there = n < s.N && k < s.K;
    const int64_t at = (int64_t)(k / s.group) * s.N + n;
    if (s.es == 2)
      reinterpret_cast<uint16_t*>(out + kCodeBytes)[e] =
          there ? reinterpret_cast<const uint16_t*>(scales)[at] : 0;
    else
      reinterpret_cast<uint32_t*>(out + kCodeBytes)[e] =
          there ? reinterpret_cast<const uint32_t*>(scales)[at] : 0u;
    if (s.zeros) out[kCodeBytes + places * s.es + e] = there ? zeros[at] & 15u : 0;
  }
}

// ------------------------------------------------------------------ product --
// How codes and x enter the tensor core.
template <typename T>
struct W4Type;
template <>
struct W4Type<__half> {
  using M = MmaKind<__half>;
  static constexpr uint32_t kBias = 0x64006400u;  // 1024, ulp 1
  static constexpr int PARTS = 1;
  static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
    const __half2 r = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};
template <>
struct W4Type<__nv_bfloat16> {
  using M = MmaKind<__nv_bfloat16>;
  static constexpr uint32_t kBias = 0x43004300u;  // 128, ulp 1
  static constexpr int PARTS = 1;
  static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r =
        __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};
template <>
struct W4Type<float> : W4Type<__nv_bfloat16> {
  static constexpr int PARTS = 3;  // x = the sum of three bf16 values
};

struct W4Args {
  W4Shape s;
  const void *x, *residual;
  const uint8_t* packed;
  void* out;
  int64_t x_stride;
  int rows;
};

// x of one lane for the two steps of 32 elements of k: words [step][half]
// (PARTS of them).
template <typename T>
struct XFrag {
  uint32_t w[W4Type<T>::PARTS][4];
  __device__ __forceinline__ void load(const T* at, bool there) {
    if constexpr (sizeof(T) == 2) {
      const uint4 v = there ? *reinterpret_cast<const uint4*>(at) : make_uint4(0, 0, 0, 0);
      w[0][0] = v.x;
      w[0][1] = v.y;
      w[0][2] = v.z;
      w[0][3] = v.w;
    } else {
      float f[8];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 v = there ? reinterpret_cast<const float4*>(at)[i] : make_float4(0, 0, 0, 0);
        f[4 * i] = v.x;
        f[4 * i + 1] = v.y;
        f[4 * i + 2] = v.z;
        f[4 * i + 3] = v.w;
      }
#pragma unroll
      for (int part = 0; part < 3; ++part)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // cut off, not rounded: what is left is exact, and an infinity leaves nothing
          const uint32_t a = __float_as_uint(f[2 * i]), b = __float_as_uint(f[2 * i + 1]);
          w[part][i] = __byte_perm(a, b, 0x7632);
          f[2 * i] = rest(f[2 * i]);
          f[2 * i + 1] = rest(f[2 * i + 1]);
        }
    }
  }
  static __device__ __forceinline__ float rest(float f) {
    const float hi = __uint_as_float(__float_as_uint(f) & 0xffff0000u);
    return fabsf(f) < INFINITY ? f - hi : 0.f;
  }
};

// A block takes 64 columns: warp w the 16 columns w % 4, and every other record
// along k from w / 4 on.
template <typename T, int NT>
__global__ void __launch_bounds__(kW4Threads) w4_kernel(const __grid_constant__ W4Args a) {
  using W = W4Type<T>;
  __shared__ float s_part[4][16][8 * NT];
  const W4Shape& s = a.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int block = warp & 3, tile = blockIdx.x;
  const uint8_t* stream = a.packed + (int64_t)tile * s.units * s.record;
  const int places = s.groups() * kTileN;
  pdl_wait();
  pdl_trigger();
  float y[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) y[i][e] = 0.f;
  for (int u = warp >> 2; u < s.units; u += 2) {
    const uint8_t* rec = stream + (int64_t)u * s.record;
    float acc[NT][4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {  // 32 elements of k
      if ((q * 32) % s.group == 0) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
      }
      const int gr = q * 32 / s.group, place = gr * kTileN + block * 16 + 2 * g;
      const uint2 c = *reinterpret_cast<const uint2*>(
          rec + ((block * 2 + (q >> 1)) * 32 + lane) * 16 + (q & 1) * 8);
      uint32_t z0 = W::kBias + 0x00080008u, z1 = z0;
      if (s.zeros) {
        const uint8_t* z = rec + kCodeBytes + places * s.es + place;
        z0 = W::kBias + z[0] * 0x00010001u;
        z1 = W::kBias + z[1] * 0x00010001u;
      }
      uint32_t A[2][4];
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          A[st][i] = W::sub((((st ? c.y : c.x) >> (4 * i)) & 0x000f000fu) | W::kBias, i & 1 ? z1 : z0);
      const int k = u * kUnitK + q * 32;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int row = i * 8 + g;
        XFrag<T> x;
        x.load(static_cast<const T*>(a.x) + row * a.x_stride + k + t * 8, row < a.rows && k < s.K);
#pragma unroll
        for (int part = 0; part < W::PARTS; ++part)
#pragma unroll
          for (int st = 0; st < 2; ++st)
            W::M::mma(acc[i], A[st], x.w[part][2 * st], x.w[part][2 * st + 1]);
      }
      if ((q * 32 + 32) % s.group == 0) {
        const T* sc = reinterpret_cast<const T*>(rec + kCodeBytes) + place;
        const float s0 = Elem<T>::to_f(sc[0]), s1 = Elem<T>::to_f(sc[1]);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          y[i][0] = fmaf(acc[i][0], s0, y[i][0]);
          y[i][1] = fmaf(acc[i][1], s0, y[i][1]);
          y[i][2] = fmaf(acc[i][2], s1, y[i][2]);
          y[i][3] = fmaf(acc[i][3], s1, y[i][3]);
        }
      }
    }
  }
  if (warp >= 4) {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        s_part[block][g + 8 * (e >> 1)][i * 8 + 2 * t + (e & 1)] = y[i][e];
  }
  __syncthreads();
  if (warp >= 4) return;
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int n = tile * kTileN + block * 16 + g + 8 * (e >> 1), row = i * 8 + 2 * t + (e & 1);
      if (n >= s.N || row >= a.rows) continue;
      float v = y[i][e] + s_part[block][g + 8 * (e >> 1)][row];
      const int64_t at = (int64_t)row * s.N + n;
      if (a.residual) v += Elem<T>::to_f(static_cast<const T*>(a.residual)[at]);
      static_cast<T*>(a.out)[at] = Elem<T>::from_f(v);
    }
}

template <typename T>
const void* w4_fn(int rows) {
  return rows <= 8    ? (const void*)&w4_kernel<T, 1>
         : rows <= 16 ? (const void*)&w4_kernel<T, 2>
         : rows <= 32 ? (const void*)&w4_kernel<T, 4>
                      : (const void*)&w4_kernel<T, 8>;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (a == nullptr || b == nullptr || na == 0 || nb == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

struct cf_w4_handle {
  cf_w4_config cfg;
  W4Shape s;
  int device = 0, sm_count = 0;
};

namespace {

// CF_OK where the handle's device is the current one.
int on_device(const cf_w4_handle* h) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return CF_ERR_CUDA;
  }
  return dev == h->device ? CF_OK : CF_ERR_INVALID_ARG;
}

}  // namespace

extern "C" {

int cf_w4_create(const cf_w4_config* cfg, cf_w4_handle** out) {
  if (out == nullptr) return CF_ERR_INVALID_ARG;
  *out = nullptr;
  if (cfg == nullptr) return CF_ERR_INVALID_ARG;
  const cf_w4_config& c = *cfg;
  if (c.in_features <= 0 || c.in_features > (1 << 20) || c.out_features <= 0 ||
      c.out_features > (1 << 24) || c.out_features % 2 != 0 || c.group <= 0 || c.zeros < 0 ||
      c.zeros > 1 || c.max_rows <= 0 || c.dtype < CF_F32 || c.dtype > CF_BF16)
    return CF_ERR_INVALID_ARG;
  if ((c.group != 32 && c.group != 64 && c.group != 128) || c.max_rows > 64)
    return CF_ERR_UNSUPPORTED;
  if (c.in_features % c.group != 0) return CF_ERR_INVALID_ARG;
  cf_w4_handle* h = new (std::nothrow) cf_w4_handle();
  if (h == nullptr) return CF_ERR_CUDA;
  h->cfg = c;
  W4Shape& s = h->s;
  s.K = c.in_features;
  s.N = c.out_features;
  s.group = c.group;
  s.zeros = c.zeros;
  s.es = c.dtype == CF_F32 ? 4 : 2;
  s.units = (s.K + kUnitK - 1) / kUnitK;
  s.tiles = (s.N + kTileN - 1) / kTileN;
  s.record = kCodeBytes + s.groups() * kTileN * (s.es + s.zeros);
  if ((int64_t)s.units * s.tiles > INT32_MAX) {  // the grid of the layout's kernel
    delete h;
    return CF_ERR_INVALID_ARG;
  }
  if (cudaGetDevice(&h->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&h->sm_count, cudaDevAttrMultiProcessorCount, h->device) !=
          cudaSuccess) {
    cudaGetLastError();
    delete h;
    return CF_ERR_CUDA;
  }
  *out = h;
  return CF_OK;
}

size_t cf_w4_packed_bytes(const cf_w4_handle* h) {
  return h == nullptr ? 0 : (size_t)h->s.units * h->s.tiles * h->s.record;
}

int cf_w4_pack(cf_w4_handle* h, const uint8_t* codes, const void* scales, const uint8_t* zeros,
               void* packed, void* stream) {
  if (h == nullptr) return CF_ERR_INVALID_ARG;
  const int rc = on_device(h);
  if (rc != CF_OK) return rc;
  const W4Shape& s = h->s;
  if (codes == nullptr || scales == nullptr || (zeros != nullptr) != (s.zeros != 0) ||
      packed == nullptr || !aligned(packed, 16) || !aligned(scales, s.es))
    return CF_ERR_INVALID_ARG;
  const size_t n = cf_w4_packed_bytes(h), groups = (size_t)(s.K / s.group) * s.N;
  if (overlap(packed, n, codes, (size_t)s.K * (s.N / 2)) ||
      overlap(packed, n, scales, groups * s.es) || overlap(packed, n, zeros, zeros ? groups : 0))
    return CF_ERR_ALIAS;
  W4Shape sh = s;
  const uint8_t* sc = static_cast<const uint8_t*>(scales);
  uint8_t* pk = static_cast<uint8_t*>(packed);
  void* args[] = {&sh, &codes, &sc, &zeros, &pk};
  if (!launch_pdl((const void*)&w4_pack_kernel, dim3((unsigned)(s.units * s.tiles)), kW4Threads, 0,
                  static_cast<cudaStream_t>(stream), args)) {
    cudaGetLastError();
    return CF_ERR_CUDA;
  }
  return CF_OK;
}

int cf_w4_matvec(cf_w4_handle* h, int32_t rows, const void* x, int64_t x_stride,
                 const void* packed, const void* residual, void* out, void* stream) {
  if (h == nullptr || rows < 0 || rows > h->cfg.max_rows) return CF_ERR_INVALID_ARG;
  const int rc = on_device(h);
  if (rc != CF_OK || rows == 0) return rc;
  const W4Shape& s = h->s;
  if (x == nullptr || packed == nullptr || out == nullptr || !aligned(x, 16) ||
      !aligned(packed, 16) || !aligned(out, s.es) || !aligned(residual, s.es))
    return CF_ERR_INVALID_ARG;
  if (x_stride < s.K || x_stride > (1LL << 40) || (x_stride * s.es) % 16 != 0)
    return CF_ERR_INVALID_ARG;
  const size_t ob = (size_t)rows * s.N * s.es;
  if (overlap(out, ob, x, ((size_t)(rows - 1) * x_stride + s.K) * s.es) ||
      overlap(out, ob, packed, cf_w4_packed_bytes(h)) ||
      (residual != out && overlap(out, ob, residual, ob)))
    return CF_ERR_ALIAS;
  W4Args a;
  a.s = s;
  a.x = x;
  a.residual = residual;
  a.packed = static_cast<const uint8_t*>(packed);
  a.out = out;
  a.x_stride = x_stride;
  a.rows = rows;
  void* args[] = {&a};
  const void* fn = h->cfg.dtype == CF_F32   ? w4_fn<float>(rows)
                   : h->cfg.dtype == CF_F16 ? w4_fn<__half>(rows)
                                            : w4_fn<__nv_bfloat16>(rows);
  if (!launch_pdl(fn, dim3(s.tiles), kW4Threads, 0, static_cast<cudaStream_t>(stream), args)) {
    cudaGetLastError();
    return CF_ERR_CUDA;
  }
  return CF_OK;
}

void cf_w4_destroy(cf_w4_handle* h) { delete h; }

}  // extern "C"
