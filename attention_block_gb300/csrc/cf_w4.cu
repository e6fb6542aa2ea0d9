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
//
// Bound by the weights' bytes for few rows.  A block takes a tile of 64 columns,
// or a part of its k; its eight warps take the records in turn, each through a
// ring of its own that bulk copies fill (records lie one after another), so no
// warp waits for another before the sums are joined.  Within a record a warp has
// four independent chains of products, and its x serve four blocks of columns.
// Where tiles are few, k is split over the blocks of a cluster, which exchange
// their sums through distributed shared memory; all sums are joined in a fixed
// order.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <new>

#include "cf_cluster.cuh"
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
  int* errflag;
  int rows, split;
};

// Two neighbouring elements in fp32.
__device__ __forceinline__ void load_cvt2(const float* p, float (&f)[2]) {
  const float2 v = *reinterpret_cast<const float2*>(p);
  f[0] = v.x;
  f[1] = v.y;
}
template <typename T>
__device__ __forceinline__ void load_cvt2(const T* p, float (&f)[2]) {
  load_cvt<T, 2>(p, f);
}

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

constexpr int kWarps = kW4Threads / 32;
constexpr int kStages = 2;     // records of a warp's ring
constexpr int kMaxSplit = 8;
constexpr int kPitch = kTileN + 4;  // of a row of sums

// Asks for n bytes (a multiple of 16) to be brought to L2.
__device__ __forceinline__ void prefetch_l2(const void* at, uint32_t n) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at), "r"(n) : "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

// Block `blockIdx.x % split` of its cluster takes its share of the records of
// tile blockIdx.x / split.  With 64 rows the sums of a tile are too many for a
// warp: two warps share a record, each with two blocks of columns.
template <typename T, int NT>
__global__ void __launch_bounds__(kW4Threads, NT * W4Type<T>::PARTS <= 2 ? 2 : 1)
    w4_kernel(const __grid_constant__ W4Args a) {
  using W = W4Type<T>;
  constexpr int BL = NT <= 4 ? 4 : 2;          // blocks of columns of a warp
  constexpr int STREAMS = kWarps * BL / 4;     // records that are in work
  constexpr bool AHEAD = NT * W::PARTS <= 2;   // there are registers for x ahead
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(8) uint64_t s_full[kWarps][kStages];
  const W4Shape& s = a.s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int tile = blockIdx.x / a.split, part = blockIdx.x - tile * a.split;
  const int u0 = (int)((long long)s.units * part / a.split);
  const int u1 = (int)((long long)s.units * (part + 1) / a.split);
  const int first = u0 + warp % STREAMS;                    // this warp's records
  const int n = first < u1 ? (u1 - first + STREAMS - 1) / STREAMS : 0;
  const int b0 = BL == 4 ? 0 : warp / STREAMS * BL;         // and blocks
  constexpr int kPart = BL * 1024;                          // bytes of their codes
  const int extra = s.record - kCodeBytes;                  // of scales and zeros
  const int slot_bytes = kPart + extra;
  const uint8_t* stream = a.packed + ((int64_t)tile * s.units + first) * s.record;
  uint8_t* mem = ring + warp * kStages * slot_bytes;
  const int64_t stride = (int64_t)STREAMS * s.record;
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&s_full[warp][i], 1);
    fence_mbar_init_cluster();
    // what lies in L2 is what memory holds: this may run ahead of the launch in front
    if (b0 == 0)
      for (int i = 0; i < min(n, 2 * kStages); ++i) prefetch_l2(stream + i * stride, s.record);
  }
  __syncwarp();
  pdl_wait();
  pdl_trigger();
  const uint64_t policy = policy_evict_first();
  auto copy = [&](int i) {  // by one lane
    const int slot = i % kStages;
    const uint8_t* rec = stream + i * stride;
    mbar_arrive_expect_tx(&s_full[warp][slot], slot_bytes);
    if (BL == 4) {
      bulk_load_1d(mem + slot * slot_bytes, rec, slot_bytes, &s_full[warp][slot], policy);
    } else {
      bulk_load_1d(mem + slot * slot_bytes, rec + b0 * 1024, kPart, &s_full[warp][slot], policy);
      bulk_load_1d(mem + slot * slot_bytes + kPart, rec + kCodeBytes, extra, &s_full[warp][slot],
                   policy);
    }
  };
  if (lane == 0)
    for (int i = 0; i < min(n, kStages); ++i) copy(i);

  // x of this lane for half a record: rows g + 8 j, k = 32 q + 8 t
  struct Half {
    XFrag<T> f[NT][2];
  };
  auto load_x = [&](Half& x, int i, int half) {
    const int k = (first + i * STREAMS) * kUnitK + half * 64 + t * 8;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int q = 0; q < 2; ++q)
        x.f[j][q].load(static_cast<const T*>(a.x) + (int64_t)(j * 8 + g) * a.x_stride + k + q * 32,
                       j * 8 + g < a.rows && k + q * 32 < s.K);
  };
  float y[BL][NT][4];
#pragma unroll
  for (int b = 0; b < BL; ++b)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) y[b][j][e] = 0.f;
  const bool fine = s.group == 32;
  const int shift = s.group == 128 ? 1 : 0;  // groups of a record's half: 1 / 2, 1, 2
  const int places = s.groups() * kTileN;
  Half x[AHEAD ? 2 : 1];
  if (AHEAD && n > 0) load_x(x[0], 0, 0);
  for (int i = 0; i < n; ++i) {
    const int slot = i % kStages;
    if (!AHEAD) load_x(x[0], i, 0);
    mbar_wait(&s_full[warp][slot], (i / kStages) & 1, a.errflag);
    const uint8_t* rec = mem + slot * slot_bytes;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if constexpr (AHEAD) {
        if (half == 0)
          load_x(x[1], i, 1);
        else if (i + 1 < n)
          load_x(x[0], i + 1, 0);
      } else if (half == 1) {
        load_x(x[0], i, 1);
      }
      const Half& h = x[AHEAD ? half : 0];
      const int gr = fine ? 2 * half : half >> shift;
#pragma unroll
      for (int b = 0; b < BL; ++b) {
        const uint4 c = *reinterpret_cast<const uint4*>(rec + ((b * 2 + half) * 32 + lane) * 16);
        const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
        float sc[2];
        uint32_t z[2] = {W::kBias + 0x00080008u, W::kBias + 0x00080008u};
        auto scales = [&](int gr) {
          const int place = gr * kTileN + (b0 + b) * 16 + 2 * g;
          load_cvt2(reinterpret_cast<const T*>(rec + kPart) + place, sc);
          if (s.zeros) {
            const uint32_t zz =
                *reinterpret_cast<const uint16_t*>(rec + kPart + places * s.es + place);
            z[0] = W::kBias + (zz & 0xffu) * 0x00010001u;
            z[1] = W::kBias + (zz >> 8) * 0x00010001u;
          }
        };
        scales(gr);
        float acc[NT][4];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (q == 1 && fine) scales(gr + 1);
          if (q == 0 || fine) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
          }
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            uint32_t A[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              A[e] = W::sub(((cw[2 * q + st] >> (4 * e)) & 0x000f000fu) | W::kBias, z[e & 1]);
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int w = 0; w < W::PARTS; ++w)
                W::M::mma(acc[j], A, h.f[j][q].w[w][2 * st], h.f[j][q].w[w][2 * st + 1]);
          }
          if (q == 1 || fine) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) y[b][j][e] = fmaf(acc[j][e], sc[e >> 1], y[b][j][e]);
          }
        }
      }
    }
    __syncwarp();  // the slot is read
    if (lane == 0 && i + kStages < n) copy(i + kStages);
  }
  __syncthreads();  // every record is read: the rings take the sums

  // [stream][row][column of the tile]
  float* sums = reinterpret_cast<float*>(ring);
  constexpr int kRows = 8 * NT;
#pragma unroll
  for (int b = 0; b < BL; ++b)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        sums[(warp % STREAMS * kRows + j * 8 + 2 * t + (e & 1)) * kPitch + (b0 + b) * 16 + g +
             8 * (e >> 1)] = y[b][j][e];
  __syncthreads();
  auto finish = [&](int row, int col, float v) {
    const int n0 = tile * kTileN + col;
    if (n0 >= s.N) return;
    const int64_t o = (int64_t)row * s.N + n0;
    if (a.residual) v += Elem<T>::to_f(static_cast<const T*>(a.residual)[o]);
    static_cast<T*>(a.out)[o] = Elem<T>::from_f(v);
  };
  for (int e = tid; e < a.rows * kTileN; e += kW4Threads) {
    const int row = e / kTileN, col = e - row * kTileN, at = row * kPitch + col;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < STREAMS; ++w) v += sums[w * kRows * kPitch + at];
    if (a.split == 1)
      finish(row, col, v);
    else
      sums[at] = v;
  }
  if (a.split == 1) return;
  cluster_sync_all();
  const uint32_t base = smem_u32(sums);
  for (int e = part * kW4Threads + tid; e < a.rows * kTileN; e += a.split * kW4Threads) {
    const int row = e / kTileN, col = e - row * kTileN;
    float v = 0.f;
    for (int r = 0; r < a.split; ++r) v += ld_cluster(mapa(base, r) + (row * kPitch + col) * 4);
    finish(row, col, v);
  }
  cluster_sync_all();  // no block leaves while its sums are read
}

// Rows of a launch, at most: fp32 x as three values of 64 rows leave no registers.
int launch_rows(int dtype) { return dtype == CF_F32 ? 32 : 64; }

template <typename T>
const void* w4_fn(int rows) {
  if (rows <= 8) return (const void*)&w4_kernel<T, 1>;
  if (rows <= 16) return (const void*)&w4_kernel<T, 2>;
  if constexpr (W4Type<T>::PARTS == 1)
    if (rows > 32) return (const void*)&w4_kernel<T, 8>;
  return (const void*)&w4_kernel<T, 4>;
}
const void* w4_fn_of(int dtype, int rows) {
  return dtype == CF_F32   ? w4_fn<float>(rows)
         : dtype == CF_F16 ? w4_fn<__half>(rows)
                           : w4_fn<__nv_bfloat16>(rows);
}
// Shared memory of a launch: the rings, then the sums.
int w4_smem(const W4Shape& s, int rows) {
  const int nt = rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 32 ? 4 : 8, bl = nt <= 4 ? 4 : 2;
  const int ring = kWarps * kStages * (bl * 1024 + s.record - kCodeBytes);
  return std::max(ring, kWarps * bl / 4 * 8 * nt * kPitch * 4);
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
  int device = 0;
  int split = 1;  // blocks of a cluster
  int* errflag = nullptr;
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
  int sms = 0;
  auto fail = [&]() {
    cudaGetLastError();
    if (h->errflag) cudaFree(h->errflag);
    delete h;
    return CF_ERR_CUDA;
  };
  if (cudaGetDevice(&h->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess)
    return fail();
  // Few tiles leave SMs without one: k is split until there are three blocks to
  // two SMs (two fit on each), or a block has four records left.
  while (h->split < kMaxSplit && s.tiles * h->split * 2 < 3 * sms && s.units >= 8 * h->split)
    h->split *= 2;
  for (int rows = 8; rows <= launch_rows(c.dtype); rows *= 2)
    if (cudaFuncSetAttribute(w4_fn_of(c.dtype, rows), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             100 * 1024) != cudaSuccess)
      return fail();
  if (cudaMalloc(&h->errflag, sizeof(int)) != cudaSuccess ||
      cudaMemset(h->errflag, 0, sizeof(int)) != cudaSuccess ||
      cudaStreamSynchronize(nullptr) != cudaSuccess)
    return fail();
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
  a.packed = static_cast<const uint8_t*>(packed);
  a.x_stride = x_stride;
  a.errflag = h->errflag;
  a.split = h->split;
  void* args[] = {&a};
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)h->split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  lc.gridDim = dim3((unsigned)(s.tiles * h->split));
  lc.blockDim = dim3(kW4Threads);
  lc.stream = static_cast<cudaStream_t>(stream);
  lc.attrs = attr;
  lc.numAttrs = h->split > 1 ? 2 : 1;
  const int step = launch_rows(h->cfg.dtype);
  for (int r0 = 0; r0 < rows; r0 += step) {
    a.rows = std::min(step, rows - r0);
    a.x = static_cast<const uint8_t*>(x) + r0 * x_stride * s.es;
    a.out = static_cast<uint8_t*>(out) + (int64_t)r0 * s.N * s.es;
    a.residual = residual ? static_cast<const uint8_t*>(residual) + (int64_t)r0 * s.N * s.es
                          : nullptr;
    lc.dynamicSmemBytes = w4_smem(s, a.rows);
    if (cudaLaunchKernelExC(&lc, w4_fn_of(h->cfg.dtype, a.rows), args) != cudaSuccess) {
      cudaGetLastError();
      return CF_ERR_CUDA;
    }
  }
  return CF_OK;
}

int cf_w4_get_status(cf_w4_handle* h) {
  if (h == nullptr) return CF_ERR_INVALID_ARG;
  int flag = 0;
  if (cudaMemcpy(&flag, h->errflag, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess)
    return CF_ERR_CUDA;
  if (flag != 0 && cudaMemset(h->errflag, 0, sizeof(int)) != cudaSuccess) return CF_ERR_CUDA;
  return flag != 0 ? CF_ERR_DEVICE_TIMEOUT : CF_OK;
}

void cf_w4_destroy(cf_w4_handle* h) {
  if (h == nullptr) return;
  if (h->errflag) cudaFree(h->errflag);
  delete h;
}

}  // extern "C"
