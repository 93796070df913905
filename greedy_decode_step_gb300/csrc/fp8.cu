// 8-bit rows and weights: quantising to e4m3 codes with a power-of-two scale
// per block, and reading back.
//
//   a = max |x| over the block's finite values
//   s = the smallest power of two, 2^-126 at least, with a <= 448 s (a == 0: 1)
//   c = e4m3(x / s), to nearest even; NaN for a value that is not finite
//
// A power of two costs no accuracy in a floating-point code (its steps are
// relative; only values below 2^-6 s get coarser ones) and makes x / s exact
// in float32, so a code is defined to the bit and no step divides.  s comes
// from the bits of a: with a = 1.m 2^e and 448 = 1.75 2^8, s is 2^(e - 8), one
// more where 1.m > 1.75.
//
// Both directions are bound by DRAM.  Rows (1 x 128 blocks): 32 (float32) or 16
// (bf16) lanes hold one block, 16 bytes a lane, so a block's maximum is a few
// shuffles; weights (128 x 128 blocks): one CTA holds a block in registers and
// meets once in shared memory.  Every value is read once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "dec_fp8.cuh"
#include "dec_launch.cuh"

namespace dec {
namespace {

constexpr int kQuantThreads = 256;

// Bits of |x|, zero for a value that is not finite.
__device__ __forceinline__ uint32_t finite_magnitude(float x) {
  const uint32_t b = __float_as_uint(x) & 0x7FFFFFFFu;
  return b < 0x7F800000u ? b : 0u;
}

// Biased exponent of the scale of a block whose largest finite magnitude has these bits.
__device__ __forceinline__ uint32_t scale_exponent(uint32_t top) {
  if (top == 0) return 127;
  const int e = static_cast<int>(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(max(e, 1));
}

// Two e4m3 codes, the first value in the low byte.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// x / s; an infinity becomes NaN (the conversion would hold it as 448).
__device__ __forceinline__ float scaled(float x, float inv) {
  const float v = x * inv;
  return fabsf(v) <= 448.0f ? v : __uint_as_float(0x7FFFFFFFu);
}

template <bool BF16>
struct Vec {  // 16 bytes of a source row
  static constexpr int kN = BF16 ? 8 : 4;
  float v[kN];
  __device__ __forceinline__ void load(const void* p) {
    const uint4 w = __ldg(static_cast<const uint4*>(p));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (BF16) {
        v[2 * i] = bf16lo(u[i]);
        v[2 * i + 1] = bf16hi(u[i]);
      } else {
        v[i] = __uint_as_float(u[i]);
      }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = 0.f;
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kN; ++i) m = max(m, finite_magnitude(v[i]));
    return m;
  }
  __device__ __forceinline__ void store(uint8_t* p, float inv) const {
    uint32_t w[kN / 4];
#pragma unroll
    for (int i = 0; i < kN / 4; ++i)
      w[i] = e4m3_pair(scaled(v[4 * i], inv), scaled(v[4 * i + 1], inv)) |
             (e4m3_pair(scaled(v[4 * i + 2], inv), scaled(v[4 * i + 3], inv)) << 16);
    if (kN == 8)
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[kN / 4 - 1]);
    else
      *reinterpret_cast<uint32_t*>(p) = w[0];
  }
};

template <bool BF16>
__device__ __forceinline__ const char* source(const Fp8QuantArgs& a, long long mat, long long row, int k) {
  return static_cast<const char*>(a.x) + (mat * a.sm + row * a.sr + k) * (BF16 ? 2 : 4);
}

// 1 x 128 blocks: LANES lanes per block, kUnroll blocks of a lane in flight.
template <bool BF16>
__global__ void __launch_bounds__(kQuantThreads) quant_rows_kernel(const Fp8QuantArgs a) {
  constexpr int kN = Vec<BF16>::kN, kLanes = kFp8Block / kN, kPer = kQuantThreads / kLanes, kUnroll = 4;
  pdl_wait();
  pdl_launch_dependents();
  const int KB = (a.K + kFp8Block - 1) / kFp8Block;
  const long long blocks = static_cast<long long>(a.n) * a.rows * KB;
  const int sub = threadIdx.x / kLanes, in = threadIdx.x % kLanes;
  // consecutive blocks of a CTA lie side by side in memory; the loop's bound is CTA-uniform, so that the shuffles
  // below are met by whole warps
  for (long long b0 = static_cast<long long>(blockIdx.x) * kPer * kUnroll; b0 < blocks;
       b0 += static_cast<long long>(gridDim.x) * kPer * kUnroll) {
    Vec<BF16> x[kUnroll];
    long long row[kUnroll];
    int k[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long long b = b0 + u * kPer + sub;
      row[u] = b < blocks ? b / KB : -1;
      k[u] = static_cast<int>(b - row[u] * KB) * kFp8Block + in * kN;
      if (row[u] >= 0 && k[u] < a.K) {
        const long long mat = row[u] / a.rows;
        x[u].load(source<BF16>(a, mat, row[u] - mat * a.rows, k[u]));
      } else {
        x[u].zero();
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      uint32_t top = x[u].top();
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      const uint32_t e = scale_exponent(top);
      if (row[u] < 0) continue;
      if (k[u] < a.K) x[u].store(a.codes + row[u] * a.K + k[u], __uint_as_float((254u - e) << 23));
      if (in == 0) a.scales[row[u] * KB + k[u] / kFp8Block] = __uint_as_float(e << 23);
    }
  }
}

// 128 x 128 blocks: one CTA per block.
template <bool BF16>
__global__ void __launch_bounds__(kQuantThreads) quant_tiles_kernel(const Fp8QuantArgs a) {
  constexpr int kN = Vec<BF16>::kN, kLanes = kFp8Block / kN, kRows = kQuantThreads / kLanes, kUnroll = kFp8Block / kRows;
  __shared__ uint32_t tops[kQuantThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  const int KB = (a.K + kFp8Block - 1) / kFp8Block, RB = (a.rows + kFp8Block - 1) / kFp8Block;
  const long long tiles = static_cast<long long>(a.n) * RB * KB;
  const int sub = threadIdx.x / kLanes, in = threadIdx.x % kLanes;
  for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const long long mb = tile / KB, mat = mb / RB;
    const int k = static_cast<int>(tile - mb * KB) * kFp8Block + in * kN;
    const long long r0 = (mb - mat * RB) * kFp8Block + sub;
    Vec<BF16> x[kUnroll];
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (r0 + u * kRows < a.rows && k < a.K)
        x[u].load(source<BF16>(a, mat, r0 + u * kRows, k));
      else
        x[u].zero();
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) top = max(top, x[u].top());
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) tops[threadIdx.x / 32] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kQuantThreads / 32; ++w) top = max(top, tops[w]);
    __syncthreads();
    const uint32_t e = scale_exponent(top);
    const float inv = __uint_as_float((254u - e) << 23);
    if (threadIdx.x == 0) a.scales[tile] = __uint_as_float(e << 23);
    if (k < a.K) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (r0 + u * kRows < a.rows) x[u].store(a.codes + (mat * a.rows + r0 + u * kRows) * a.K + k, inv);
    }
  }
}

// 16 codes per thread and step: one scale holds for all of them (K is a multiple of 16).
template <bool BF16>
__global__ void __launch_bounds__(kQuantThreads) dequant_kernel(const Fp8DequantArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int KB = (a.K + kFp8Block - 1) / kFp8Block, per_row = a.K / 16;
  const long long RB = (static_cast<long long>(a.rows) + a.block_rows - 1) / a.block_rows;
  const long long total = static_cast<long long>(a.n) * a.rows * per_row;
  for (long long i = static_cast<long long>(blockIdx.x) * kQuantThreads + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * kQuantThreads) {
    const long long row = i / per_row, mat = row / a.rows, r = row - mat * a.rows;
    const int k = static_cast<int>(i - row * per_row) * 16;
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(a.codes) + i);
    const float s = __ldg(a.scales + (mat * RB + r / a.block_rows) * KB + k / kFp8Block);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    float v[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t h;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(u[j / 2] >> (16 * (j & 1)))));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      v[2 * j] = f.x * s;
      v[2 * j + 1] = f.y * s;
    }
    char* dst = static_cast<char*>(a.out) + (mat * a.sm + r * a.sr + k) * (BF16 ? 2 : 4);
    if (BF16) {
      uint32_t p[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        p[j] = *reinterpret_cast<const uint32_t*>(&b);
      }
      reinterpret_cast<uint4*>(dst)[0] = make_uint4(p[0], p[1], p[2], p[3]);
      reinterpret_cast<uint4*>(dst)[1] = make_uint4(p[4], p[5], p[6], p[7]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        reinterpret_cast<float4*>(dst)[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    }
  }
}

int grid_of(long long items, int sms) {
  return static_cast<int>(std::max(1ll, std::min<long long>(items, static_cast<long long>(sms) * 8)));
}

}  // namespace

cudaError_t launch_fp8_quant(const Fp8QuantArgs& a, bool bf16, int block_rows, int sms, cudaStream_t st) {
  const long long KB = (a.K + kFp8Block - 1) / kFp8Block;
  if (block_rows == 1) {
    const long long per = 4ll * kQuantThreads * (bf16 ? 8 : 4) / kFp8Block;
    const int grid = grid_of((static_cast<long long>(a.n) * a.rows * KB + per - 1) / per, sms);
    return bf16 ? launch(quant_rows_kernel<true>, dim3(grid), dim3(kQuantThreads), 0, st, true, a)
                : launch(quant_rows_kernel<false>, dim3(grid), dim3(kQuantThreads), 0, st, true, a);
  }
  const int grid = grid_of(static_cast<long long>(a.n) * ((a.rows + kFp8Block - 1) / kFp8Block) * KB, sms);
  return bf16 ? launch(quant_tiles_kernel<true>, dim3(grid), dim3(kQuantThreads), 0, st, true, a)
              : launch(quant_tiles_kernel<false>, dim3(grid), dim3(kQuantThreads), 0, st, true, a);
}

cudaError_t launch_fp8_dequant(const Fp8DequantArgs& a, bool bf16, int sms, cudaStream_t st) {
  const long long total = static_cast<long long>(a.n) * a.rows * (a.K / 16);
  const int grid = grid_of((total + kQuantThreads - 1) / kQuantThreads, sms);
  return bf16 ? launch(dequant_kernel<true>, dim3(grid), dim3(kQuantThreads), 0, st, true, a)
              : launch(dequant_kernel<false>, dim3(grid), dim3(kQuantThreads), 0, st, true, a);
}

// The same shared-memory carveout as the kernels that follow them, so that those may start beside them.
cudaError_t allow_smem_fp8() {
  cudaError_t e;
  if ((e = prefer_max_carveout(quant_rows_kernel<false>)) != cudaSuccess) return e;
  if ((e = prefer_max_carveout(quant_rows_kernel<true>)) != cudaSuccess) return e;
  if ((e = prefer_max_carveout(quant_tiles_kernel<false>)) != cudaSuccess) return e;
  if ((e = prefer_max_carveout(quant_tiles_kernel<true>)) != cudaSuccess) return e;
  if ((e = prefer_max_carveout(dequant_kernel<false>)) != cudaSuccess) return e;
  return prefer_max_carveout(dequant_kernel<true>);
}

}  // namespace dec
