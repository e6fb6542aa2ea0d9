// cf_w4.cu -- products of a few rows with weights of 4 bits (include/cf_w4.h):
// the layout of the weights, the product, and the host side.
//
// The weights are the tensor core's A operand (16 columns of W by 16 elements
// of k), the rows of x its B operand (8 rows), so one row costs as many
// instructions as eight.  A code c becomes the 16-bit float 1024 + c (fp16) or
// 128 + c (bf16) by setting bits, and c - zero by one exact subtraction (a published
// way with weights of few bits, Kim et al., 2022); a group's sum is scaled in fp32.
//
// A record holds 16 columns x 128 elements of k.  Its codes: for each 64 of k a
// 16-byte vector per lane, word s the A fragment of step s.  Lane (g, t) of step
// s stands for columns g and g + 8 and for k = 32 (s / 2) + 8 t + 4 (s % 2) + 0..3:
// any order of k will do as long as x follows it, and in this one a lane's x are
// 16-byte vectors and no step mixes two groups.  Of a word, nibble i and nibble
// i + 4 are the two halves of the fragment's register i.  Behind the codes the
// groups' scales, then what is subtracted for their zeros, as 16-bit floats,
// columns g and g + 8 side by side.  Records of
// neighbouring columns lie one after another, then the next 128 of k.
//
// Bound by the weights' bytes for few rows.  The columns, in blocks of 16, are
// shared evenly over as many thread blocks as the SMs hold, so all of them end at
// about one time; one takes its columns four blocks at a time.  Its eight warps
// take k in turn, each through a ring of its own that bulk copies fill ahead, over
// the next columns too, so no warp waits for another before the sums are joined.
// Within a step a warp has up to four independent chains of products, and its x
// serve them all.  Where columns are few, k is split over the blocks of a
// cluster, which exchange their sums through distributed shared memory; all sums
// are joined in a fixed order.
//
// One row, 4096 x 12288 in fp16: 8.1-8.5 us with the weights in DRAM, 3.1 TB/s; 4096 x
// 22016 in bf16: 14.3, 3.3 TB/s; 16 rows, 11008 x 4096: 12.4.  2-3 us of it are the
// launch, the first records and the sums.  Of the rest no pipe is full (one row and 16
// rows: integer 38 and 27 %, issue 48 and 35, DRAM 26 and 17, tensor cores 18): a
// warp's steps are chains from copy over unpacking (a word of eight codes takes 4
// masks and 3 shifts in bf16, 4 and 1 in fp16) to product and scale, and 16 warps on
// an SM do not hide them.  With more rows x and the products (mma.sync) grow, the
// weights' share falls: 4096 x 12288, 32 rows 23, 64 rows 41.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <new>
#include <type_traits>

#include "cf_cluster.cuh"
#include "cf_common.cuh"
#include "cf_mma.cuh"
#include "cf_paged.cuh"
#include "cf_paged_host.h"
#include "cf_w4.h"

using namespace cf;

namespace {

constexpr int kUnitK = 128;   // elements of k of a record
constexpr int kBlockN = 16;   // columns of a record
constexpr int kCodeBytes = kUnitK * kBlockN / 2;
constexpr int kW4Threads = 256;

struct W4Shape {
  int K, N, group, zeros, es;
  int half;               // fp16 operands, else bf16
  int units, blocks;      // records along k and along n
  int record;             // bytes
  __host__ __device__ int groups() const { return kUnitK / group; }  // of a record
};

// ------------------------------------------------------------------- layout --
// The 16-bit float that is subtracted from a code of a column with this zero:
// fp16, columns g (0) and g + 8 (1) of a block, or bf16.
__host__ __device__ constexpr uint32_t zero_half(bool half, uint32_t zero, int column) {
  return !half ? 0x4300u + zero : column == 0 ? 0x6400u + zero : 0x5400u + (zero << 4);
}

constexpr int kPackThreads = 128;
__global__ void __launch_bounds__(kPackThreads)
    w4_pack_kernel(W4Shape s, const uint8_t* codes, const uint8_t* scales, const uint8_t* zeros,
                   uint8_t* packed) {
  const int unit = blockIdx.x / s.blocks, block = blockIdx.x - unit * s.blocks;
  uint8_t* out = packed + (int64_t)blockIdx.x * s.record;
  pdl_wait();
  for (int w = threadIdx.x; w < kCodeBytes / 4; w += kPackThreads) {
    const int step = w & 3, lane = (w >> 2) & 31, half = w >> 7;
    const int g = lane >> 2, t = lane & 3;
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // register i & 3, its low (i < 4) or high half
      const int n = block * kBlockN + g + 8 * (i & 1);
      const int k = unit * kUnitK + half * 64 + 32 * (step >> 1) + 8 * t + 4 * (step & 1) +
                    2 * ((i >> 1) & 1) + (i >> 2);
      uint32_t c = 0;
      if (n < s.N && k < s.K) c = (codes[(int64_t)k * (s.N / 2) + n / 2] >> (4 * (n & 1))) & 15u;
      word |= c << (4 * i);
    }
    reinterpret_cast<uint32_t*>(out)[w] = word;
  }
  // scales and zeros: place x of a group is column x / 2 + 8 (x % 2)
  const int places = s.groups() * kBlockN;
  for (int e = threadIdx.x; e < places; e += kPackThreads) {
    const int x = e % kBlockN;
    const int n = block * kBlockN + (x >> 1) + 8 * (x & 1);
    const int k = unit * kUnitK + (e / kBlockN) * s.group;
    const bool there = n < s.N && k < s.K;
    const int64_t at = (int64_t)(k / s.group) * s.N + n;
    if (s.es == 2)
      reinterpret_cast<uint16_t*>(out + kCodeBytes)[e] =
          there ? reinterpret_cast<const uint16_t*>(scales)[at] : 0;
    else
      reinterpret_cast<uint32_t*>(out + kCodeBytes)[e] =
          there ? reinterpret_cast<const uint32_t*>(scales)[at] : 0u;
    if (s.zeros)
      reinterpret_cast<uint16_t*>(out + kCodeBytes + places * s.es)[e] =
          (uint16_t)zero_half(s.half, there ? zeros[at] & 15u : 0u, x & 1);
  }
}

// ------------------------------------------------------------------ product --
// How codes and x enter the tensor core.
template <typename T>
struct W4Type;

// (w & mask) | bias in one instruction: both from registers, as the compiler
// takes two with constants.
struct W4Mask {
  uint32_t low, high, bias;
  __device__ __forceinline__ explicit W4Mask(uint32_t b) {
    asm("mov.b32 %0, 0x000f000f;" : "=r"(low));
    asm("mov.b32 %0, 0x00f000f0;" : "=r"(high));
    asm("mov.b32 %0, %1;" : "=r"(bias) : "r"(b));
  }
  static __device__ __forceinline__ uint32_t take(uint32_t w, uint32_t mask, uint32_t bias) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(w), "r"(mask), "r"(bias));
    return d;
  }
};

template <>
struct W4Type<__half> {
  using M = MmaKind<__half>;
  // M::mma onto zero
  static __device__ __forceinline__ void first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  }
  static constexpr uint32_t kBias = 0x64006400u;  // 1024, ulp 1
  static constexpr int PARTS = 1;
  // The fragment of a word; z: bias + zero of columns g and g + 8.  Nibbles 1
  // and 3 stay four bits up, as 1024 + 16 c, and one fused operation takes the
  // sixteenth and subtracts.
  static __device__ __forceinline__ void fragment(uint32_t w, const W4Mask& m,
                                                  const uint32_t (&z)[2], uint32_t (&A)[4]) {
    const uint32_t v = w >> 8;
    A[0] = sub(W4Mask::take(w, m.low, m.bias), z[0]);
    A[1] = sub16(W4Mask::take(w, m.high, m.bias), z[1]);
    A[2] = sub(W4Mask::take(v, m.low, m.bias), z[0]);
    A[3] = sub16(W4Mask::take(v, m.high, m.bias), z[1]);
  }
  static constexpr bool kHalf = true;
  static __device__ __forceinline__ uint32_t sub16(uint32_t a, uint32_t b) {
    const uint32_t sixteenth = 0x2c002c00u;
    const __half2 r = __hfma2(*reinterpret_cast<__half2*>(&a),
                              *reinterpret_cast<const __half2*>(&sixteenth),
                              __hneg2(*reinterpret_cast<__half2*>(&b)));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
    const __half2 r = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};
template <>
struct W4Type<__nv_bfloat16> {
  using M = MmaKind<__nv_bfloat16>;
  static __device__ __forceinline__ void first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  }
  static constexpr uint32_t kBias = 0x43004300u;  // 128, ulp 1
  static constexpr int PARTS = 1;
  static __device__ __forceinline__ void fragment(uint32_t w, const W4Mask& m,
                                                  const uint32_t (&z)[2], uint32_t (&A)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      A[e] = sub(W4Mask::take(w >> (4 * e), m.low, m.bias), z[e & 1]);
  }
  static constexpr bool kHalf = false;
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
  int shares;  // column shares: blocks of the grid without the split
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
// (PARTS of them).  Coherent loads: the launch in front, which may still have been
// writing x when this one began, has to be seen.
template <typename T>
struct XFrag {
  uint32_t w[W4Type<T>::PARTS][4];
  __device__ __forceinline__ void load(const T* at, bool there = true) {
    if constexpr (sizeof(T) == 2) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (there) v = *reinterpret_cast<const uint4*>(at);
      w[0][0] = v.x;
      w[0][1] = v.y;
      w[0][2] = v.z;
      w[0][3] = v.w;
    } else {
      float f[8];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (there) v = reinterpret_cast<const float4*>(at)[i];
        f[4 * i] = v.x;
        f[4 * i + 1] = v.y;
        f[4 * i + 2] = v.z;
        f[4 * i + 3] = v.w;
      }
#pragma unroll
      for (int part = 0; part < 3; ++part)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // cut off, not rounded: what is left is exact; an infinity leaves nothing, and
          // a NaN, whose upper half may be an infinity's, a NaN
          const uint32_t a = __float_as_uint(f[2 * i]), b = __float_as_uint(f[2 * i + 1]);
          w[part][i] = __byte_perm(a, b, 0x7632);
          f[2 * i] = rest(f[2 * i]);
          f[2 * i + 1] = rest(f[2 * i + 1]);
        }
    }
  }
  static __device__ __forceinline__ float rest(float f) {
    const float hi = __uint_as_float(__float_as_uint(f) & 0xffff0000u);
    return fabsf(f) == INFINITY ? 0.f : f - hi;
  }
};

constexpr int kWarps = kW4Threads / 32;
constexpr int kStages = 2;     // records of a warp's ring
constexpr int kMaxSplit = 8;

// Asks for n bytes (a multiple of 16) to be brought to L2.
__device__ __forceinline__ void prefetch_l2(const void* at, uint32_t n) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at), "r"(n) : "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

// How many thread blocks of w4_kernel<T, NT> an SM holds, and how many blocks of
// columns a warp has sums of at a time.
template <typename T, int NT>
constexpr int kPerSm = NT * W4Type<T>::PARTS <= 2 ? 2 : 1;
template <int NT>
constexpr int kWide = NT == 1 || NT == 4 ? 4 : 2;

// Block `blockIdx.x % split` of its cluster takes its share of k for column
// share blockIdx.x / split.
template <typename T, int NT>
__global__ void __launch_bounds__(kW4Threads, kPerSm<T, NT>)
    w4_kernel(const __grid_constant__ W4Args a) {
  using W = W4Type<T>;
  constexpr int BL = kWide<NT>;
  constexpr bool AHEAD = NT * W::PARTS <= 2;  // there are registers for x ahead
  constexpr int kPitch = BL * kBlockN + 4;    // of a row of sums
  constexpr int kRows = 8 * NT;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(8) uint64_t s_full[kWarps][kStages];
  const W4Shape& s = a.s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int share = blockIdx.x / a.split, part = blockIdx.x - share * a.split;
  const int u0 = (int)((long long)s.units * part / a.split) + warp;
  const int u1 = (int)((long long)s.units * (part + 1) / a.split);
  const int n = u0 < u1 ? (u1 - u0 + kWarps - 1) / kWarps : 0;  // this warp's steps along k
  const int c0 = (int)((long long)s.blocks * share / a.shares);
  const int c1 = (int)((long long)s.blocks * (share + 1) / a.shares);
  // the columns in passes of nearly equal width
  const int passes = (c1 - c0 + BL - 1) / BL;
  auto pass_at = [&](int i) { return c0 + (int)((long long)(c1 - c0) * i / passes); };
  const int slot_bytes = BL * s.record;
  uint8_t* mem = ring + warp * kStages * slot_bytes;
  float* sums = reinterpret_cast<float*>(ring + kWarps * kStages * slot_bytes);
  const int64_t stride = (int64_t)s.blocks * s.record;  // from a unit to the next
  const uint64_t policy = policy_evict_first();

  // Copies run ahead of the products: the next one's pass and step, its records,
  // and which of the ring's slots it takes.
  int in_pass = 0, in_step = 0, in = 0, in_bytes;
  const uint8_t* in_at;
  auto in_begin = [&]() {
    const int b = pass_at(in_pass);
    in_bytes = (pass_at(in_pass + 1) - b) * s.record;
    in_at = a.packed + u0 * stride + (int64_t)b * s.record;
  };
  auto copy = [&](bool hint) {  // by one lane
    if (hint) {
      prefetch_l2(in_at, in_bytes);
    } else {
      mbar_arrive_expect_tx(&s_full[warp][in], in_bytes);
      bulk_load_1d(mem + in * slot_bytes, in_at, in_bytes, &s_full[warp][in], policy);
      if (++in == kStages) in = 0;
    }
    in_at += kWarps * stride;
    if (++in_step == n) {
      in_step = 0;
      if (++in_pass < passes) in_begin();
    }
  };
  const int total = n * passes;
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&s_full[warp][i], 1);
    fence_mbar_init_cluster();
    // what lies in L2 is what memory holds: this may run ahead of the launch in front
    in_begin();
    for (int i = 0; i < min(total, 2 * kStages); ++i) copy(true);
    in_pass = in_step = 0;
    in_begin();
  }
  __syncwarp();
  pdl_wait();
  pdl_trigger();
  if (lane == 0)
    for (int i = 0; i < min(total, kStages); ++i) copy(false);

  // x of this lane for half a record: rows g + 8 j, k = 32 q + 8 t
  struct Half {
    XFrag<T> f[NT][2];
  };
  // (a row behind the last gives columns that nobody reads: any row will do)
  const T* row[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
    row[j] = static_cast<const T*>(a.x) + (int64_t)min(j * 8 + g, a.rows - 1) * a.x_stride + t * 8;
  auto load_x = [&](Half& x, int step, int half) {
    const int k = (u0 + step * kWarps) * kUnitK + half * 64;
    if (k + 64 <= s.K) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int q = 0; q < 2; ++q) x.f[j][q].load(row[j] + k + q * 32);
    } else {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int q = 0; q < 2; ++q) x.f[j][q].load(row[j] + k + q * 32, k + q * 32 < s.K);
    }
  };
  // A record's half has two groups (fine), one, or half of one.  Where its
  // scales and zeros begin for this lane, and how far the second half's are.
  const bool fine = s.group == 32, zeros = s.zeros != 0;
  const int places = s.groups() * kBlockN;
  const int half_at = fine ? 2 * kBlockN : s.group == 64 ? kBlockN : 0;
  const uint8_t* scale0 = mem + kCodeBytes + 2 * g * (int)sizeof(T);
  const uint8_t* zero0 = mem + kCodeBytes + places * (int)sizeof(T) + 4 * g;
  const W4Mask mask(W::kBias);
  Half x[AHEAD ? 2 : 1];
  if (AHEAD && n > 0) load_x(x[0], 0, 0);
  int slot = 0, phase = 0;
  for (int pass = 0; pass < passes; ++pass) {
    const int first = pass_at(pass), wide = pass_at(pass + 1) - first;
    float y[BL][NT][4];
#pragma unroll
    for (int b = 0; b < BL; ++b)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[b][j][e] = 0.f;
    // One step for a number of blocks that is known when this is compiled: their
    // chains of products then run side by side (one row, 4096 x 22016: 15.3 ->
    // 14.5 us).  With more rows the copies of the code spill, and it is asked.
    auto products = [&](auto width, int i) {
      constexpr int WIDE = decltype(width)::value;
      const uint8_t* rec = mem + slot * slot_bytes;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if constexpr (AHEAD) {
          if (half == 0)
            load_x(x[1], i, 1);
          else
            load_x(x[0], i + 1 < n ? i + 1 : 0, 0);  // (behind the last: the next pass)
        } else if (half == 1) {
          load_x(x[0], i, 1);
        }
        const Half& h = x[AHEAD ? half : 0];
        const uint8_t* scale = scale0 + slot * slot_bytes + half * half_at * (int)sizeof(T);
        const uint8_t* zero = zero0 + slot * slot_bytes + half * half_at * 2;
#pragma unroll
        for (int b = 0; b < WIDE; ++b) {
          if (NT > 2 && b >= wide) break;
          const uint4 c =
              *reinterpret_cast<const uint4*>(rec + b * s.record + (half * 32 + lane) * 16);
          const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
          float sc[2];
          uint32_t z[2] = {zero_half(W::kHalf, 8, 0) * 0x00010001u,
                           zero_half(W::kHalf, 8, 1) * 0x00010001u};
          auto scales = [&](int group) {  // of the half
            load_cvt2(reinterpret_cast<const T*>(scale + b * s.record) + group * kBlockN, sc);
            if (zeros) {
              const uint32_t zz =
                  *reinterpret_cast<const uint32_t*>(zero + b * s.record + group * 2 * kBlockN);
              z[0] = __byte_perm(zz, 0u, 0x1010);
              z[1] = __byte_perm(zz, 0u, 0x3232);
            }
          };
          scales(0);
          float acc[NT][4];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            if (q == 1 && fine) scales(1);
#pragma unroll
            for (int st = 0; st < 2; ++st) {
              uint32_t A[4];
              W::fragment(cw[2 * q + st], mask, z, A);
#pragma unroll
              for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int w = 0; w < W::PARTS; ++w)
                  if (st == 0 && w == 0 && (q == 0 || fine))
                    W::first(acc[j], A, h.f[j][q].w[w][0], h.f[j][q].w[w][1]);
                  else
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
    };
    for (int i = 0; i < n; ++i) {
      if (!AHEAD) load_x(x[0], i, 0);
      mbar_wait(&s_full[warp][slot], phase, a.errflag);
      if (NT > 2 || wide == BL)
        products(std::integral_constant<int, BL>(), i);
      else if (wide == 1)
        products(std::integral_constant<int, 1>(), i);
      else if constexpr (BL == 4) {
        if (wide == 2)
          products(std::integral_constant<int, 2>(), i);
        else
          products(std::integral_constant<int, 3>(), i);
      }
      __syncwarp();  // the slot is read
      if (lane == 0 && pass * n + i + kStages < total) copy(false);
      if (++slot == kStages) {
        slot = 0;
        phase ^= 1;
      }
    }

    // ---- the warps' sums, [warp][row][column]
    if (pass > 0) __syncthreads();  // the last pass's are read
#pragma unroll
    for (int b = 0; b < BL; ++b)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sums[(warp * kRows + j * 8 + 2 * t + (e & 1)) * kPitch + b * kBlockN + g + 8 * (e >> 1)] =
              y[b][j][e];
    __syncthreads();
    const int columns = wide * kBlockN, outputs = a.rows * columns;
    auto finish = [&](int r, int col, float v) {
      const int at = first * kBlockN + col;
      if (at >= s.N) return;
      const int64_t o = (int64_t)r * s.N + at;
      if (a.residual) v += Elem<T>::to_f(static_cast<const T*>(a.residual)[o]);
      static_cast<T*>(a.out)[o] = Elem<T>::from_f(v);
    };
    for (int e = tid; e < outputs; e += kW4Threads) {
      const int r = e / columns, col = e - r * columns, at = r * kPitch + col;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += sums[w * kRows * kPitch + at];
      if (a.split == 1)
        finish(r, col, v);
      else
        sums[at] = v;
    }
    if (a.split == 1) continue;
    cluster_sync_all();
    const uint32_t base = smem_u32(sums);
    for (int e = part * kW4Threads + tid; e < outputs; e += a.split * kW4Threads) {
      const int r = e / columns, col = e - r * columns;
      float v = 0.f;
      for (int q = 0; q < a.split; ++q) v += ld_cluster(mapa(base, q) + (r * kPitch + col) * 4);
      finish(r, col, v);
    }
    cluster_sync_all();  // the sums are read: they may be overwritten, and the block may end
  }
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
// What a launch of `rows` rows takes: n-tiles of 8 rows, blocks of columns of a
// pass, thread blocks on an SM, shared memory (rings and sums).
struct W4Plan {
  int nt, wide, per_sm, smem, split, shares;
};
constexpr int kMaxSmem = 160 * 1024;  // fp32, groups of 32, zeros, 32 rows: 156 KB
W4Plan w4_plan(const W4Shape& s, int dtype, int rows, int sms) {
  W4Plan p;
  p.nt = rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 32 ? 4 : 8;
  p.wide = p.nt == 1 ? kWide<1> : p.nt == 2 ? kWide<2> : p.nt == 4 ? kWide<4> : kWide<8>;
  p.per_sm = p.nt * (dtype == CF_F32 ? 3 : 1) <= 2 ? 2 : 1;
  p.smem = kWarps * (kStages * p.wide * s.record + 8 * p.nt * (p.wide * kBlockN + 4) * 4);
  // Splitting k shortens a warp's way along it where columns are too few for the
  // SMs, and costs the exchange.  In cycles, roughly: a step's x and loop 500 and
  // 100 more for each 8 rows, a block of columns 550 and 100; an exchange 1500,
  // twice that with two blocks to an SM.  Clusters do not fill the SMs: seven
  // eighths of the places, with eight blocks half of them.  One row, us with 1, 2,
  // 4, 8: 14336 x 256 9.9, 6.5, 4.7, 3.9; 14336 x 4096 12.4, 11.4, 16.3, 21.2;
  // 4096 x 12288 8.6, 11.2.
  const int places = p.per_sm * sms;
  long long best = -1;
  for (int split = 1; split <= kMaxSplit && split <= s.units; split *= 2) {
    const int slots = split == 1 ? places : split == 8 ? places / 2 : places * 7 / 8;
    const int shares = std::max(1, std::min(s.blocks, slots / split));
    const long long blocks = (s.blocks + shares - 1) / shares;
    const long long passes = (blocks + p.wide - 1) / p.wide;
    const long long steps = ((s.units + split - 1) / split + kWarps - 1) / kWarps;
    long long cost = steps * (passes * (500 + 100 * p.nt) + blocks * (550 + 100 * p.nt));
    if (split > 1) cost += passes * (shares * split > sms ? 3000 : 1500);
    if (best < 0 || cost < best) {
      best = cost;
      p.split = split;
      p.shares = shares;
    }
  }
  return p;
}

}  // namespace

struct cf_w4_handle {
  cf_w4_config cfg;
  W4Shape s;
  int device = 0, sm_count = 0;
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
  s.half = c.dtype == CF_F16;
  s.units = (s.K + kUnitK - 1) / kUnitK;
  s.blocks = (s.N + kBlockN - 1) / kBlockN;
  s.record = kCodeBytes + s.groups() * kBlockN * (s.es + 2 * s.zeros);
  if ((int64_t)s.units * s.blocks > INT32_MAX) {  // the grid of the layout's kernel
    delete h;
    return CF_ERR_INVALID_ARG;
  }
  auto fail = [&]() {
    cudaGetLastError();
    if (h->errflag) cudaFree(h->errflag);
    delete h;
    return CF_ERR_CUDA;
  };
  if (cudaGetDevice(&h->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&h->sm_count, cudaDevAttrMultiProcessorCount, h->device) !=
          cudaSuccess)
    return fail();
  for (int rows = 8; rows <= launch_rows(c.dtype); rows *= 2)
    if (cudaFuncSetAttribute(w4_fn_of(c.dtype, rows), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMaxSmem) != cudaSuccess)
      return fail();
  if (cudaMalloc(&h->errflag, sizeof(int)) != cudaSuccess || !clear(h->errflag, sizeof(int)))
    return fail();
  *out = h;
  return CF_OK;
}

size_t cf_w4_packed_bytes(const cf_w4_handle* h) {
  return h == nullptr ? 0 : (size_t)h->s.units * h->s.blocks * h->s.record;
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
  if (!launch_pdl((const void*)&w4_pack_kernel, dim3((unsigned)(s.units * s.blocks)), kPackThreads, 0,
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
  void* args[] = {&a};
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  lc.blockDim = dim3(kW4Threads);
  lc.stream = static_cast<cudaStream_t>(stream);
  lc.attrs = attr;
  const int step = launch_rows(h->cfg.dtype);
  for (int r0 = 0; r0 < rows; r0 += step) {
    a.rows = std::min(step, rows - r0);
    a.x = static_cast<const uint8_t*>(x) + r0 * x_stride * s.es;
    a.out = static_cast<uint8_t*>(out) + (int64_t)r0 * s.N * s.es;
    a.residual = residual ? static_cast<const uint8_t*>(residual) + (int64_t)r0 * s.N * s.es
                          : nullptr;
    const W4Plan plan = w4_plan(s, h->cfg.dtype, a.rows, h->sm_count);
    a.split = plan.split;
    a.shares = plan.shares;
    attr[1].val.clusterDim.x = (unsigned)plan.split;
    lc.gridDim = dim3((unsigned)(plan.shares * plan.split));
    lc.dynamicSmemBytes = plan.smem;
    lc.numAttrs = plan.split > 1 ? 2 : 1;
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
  if (flag != 0 && !clear(h->errflag, sizeof(int))) return CF_ERR_CUDA;
  return flag != 0 ? CF_ERR_DEVICE_TIMEOUT : CF_OK;
}

void cf_w4_destroy(cf_w4_handle* h) {
  if (h == nullptr) return;
  if (h->errflag) cudaFree(h->errflag);
  delete h;
}

}  // extern "C"
