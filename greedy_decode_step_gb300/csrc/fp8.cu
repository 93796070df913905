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
struct Vec {  // 16 bytes of a source row, as they came
  static constexpr int kN = BF16 ? 8 : 4;
  uint4 w;
  __device__ __forceinline__ void load(const void* p) { w = *static_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ float value(int i) const {
    const uint32_t u = BF16 ? (i / 2 == 0 ? w.x : i / 2 == 1 ? w.y : i / 2 == 2 ? w.z : w.w)
                            : (i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w);
    return BF16 ? (i & 1 ? bf16hi(u) : bf16lo(u)) : __uint_as_float(u);
  }
  // Bits of the largest magnitude, as a float's: 0x7F800000 or more if a value is not finite.
  __device__ __forceinline__ uint32_t top() const {
    if (BF16) {
      const uint32_t k = 0x7FFF7FFFu;  // two at a time
      const uint32_t m = __vmaxu2(__vmaxu2(w.x & k, w.y & k), __vmaxu2(w.z & k, w.w & k));
      return max(m & 0xFFFF0000u, m << 16);
    }
    const uint32_t k = 0x7FFFFFFFu;
    return max(max(w.x & k, w.y & k), max(w.z & k, w.w & k));
  }
  // The same over the finite values.
  __device__ __forceinline__ uint32_t finite_top() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kN; ++i) m = max(m, finite_magnitude(value(i)));
    return m;
  }
  // ALL: every value is finite.
  template <bool ALL>
  __device__ __forceinline__ void store(uint8_t* p, float inv) const {
    auto v = [&](int i) { return ALL ? value(i) * inv : scaled(value(i), inv); };
    uint32_t c[kN / 4];
#pragma unroll
    for (int i = 0; i < kN / 4; ++i)
      c[i] = e4m3_pair(v(4 * i), v(4 * i + 1)) | (e4m3_pair(v(4 * i + 2), v(4 * i + 3)) << 16);
    if (kN == 8)
      *reinterpret_cast<uint2*>(p) = make_uint2(c[0], c[kN / 4 - 1]);
    else
      *reinterpret_cast<uint32_t*>(p) = c[0];
  }
};

// n / d for n < 2^31 by a multiplication (Granlund and Montgomery, "Division by
// invariant integers using multiplication", 1994): with 2^s >= d and
// m = floor(2^(31 + s) / d) + 1, m d exceeds 2^(31 + s) by at most 2^s.  The
// index divisions were a third of the read-back's instructions.
struct Divisor {
  uint32_t d, m, s;
  explicit Divisor(uint32_t by) : d(by), m(0), s(0) {
    while ((1ull << s) < d) ++s;
    m = static_cast<uint32_t>((1ull << (31 + s)) / d + 1);
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return s == 0 ? n : __umulhi(n, m) >> (s - 1); }
};

// Rows of one launch: flat row f0 + i of all matrices' rows laid end to end.
// Launches are cut so that every index below fits 32 bits.
struct Slice {
  uint32_t mat, row, rows;  // first matrix, first row in it, rows
  Divisor per_row, per_mat;  // items of a row, rows of a matrix
};

template <bool BF16>
__device__ __forceinline__ const char* source(const Fp8QuantArgs& a, long long mat, long long row, int k) {
  return static_cast<const char*>(a.x) + (mat * a.sm + row * a.sr + k) * (BF16 ? 2 : 4);
}

// 1 x 128 blocks: 128 / kN lanes per block, kUnroll blocks of a lane in flight.
template <bool BF16>
__global__ void __launch_bounds__(kQuantThreads) quant_rows_kernel(const Fp8QuantArgs a, const Slice s) {
  constexpr int kN = Vec<BF16>::kN, kLanes = kFp8Block / kN, kPer = kQuantThreads / kLanes, kUnroll = 4;
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t KB = (a.K + kFp8Block - 1) / kFp8Block, blocks = s.rows * KB;
  const int sub = threadIdx.x / kLanes, in = threadIdx.x % kLanes;
  // consecutive blocks of a CTA lie side by side in memory; the loop's bound is CTA-uniform, so that the shuffles
  // below are met by whole warps
  for (uint32_t b0 = blockIdx.x * (kPer * kUnroll); b0 < blocks; b0 += gridDim.x * (kPer * kUnroll)) {
    Vec<BF16> x[kUnroll];
    long long flat[kUnroll];  // row among all codes, or -1
    int k[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t b = b0 + u * kPer + sub, i = s.per_row(b);
      k[u] = static_cast<int>(b - i * KB) * kFp8Block + in * kN;
      flat[u] = -1;
      x[u].zero();
      if (b < blocks) {
        const uint32_t r = s.row + i, m = s.per_mat(r);
        flat[u] = static_cast<long long>(s.mat) * a.rows + r;
        if (k[u] < a.K) x[u].load(source<BF16>(a, s.mat + m, r - m * a.rows, k[u]));
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      uint32_t top = x[u].top();
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      const bool all = top < 0x7F800000u;
      if (__any_sync(0xffffffffu, !all)) {  // rare: once more without the infinities and NaNs
        top = x[u].finite_top();
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      }
      const uint32_t e = scale_exponent(top);
      if (flat[u] < 0) continue;
      if (k[u] < a.K) {
        uint8_t* dst = a.codes + flat[u] * a.K + k[u];
        const float inv = __uint_as_float((254u - e) << 23);
        if (all)
          x[u].template store<true>(dst, inv);
        else
          x[u].template store<false>(dst, inv);
      }
      if (in == 0) a.scales[flat[u] * KB + k[u] / kFp8Block] = __uint_as_float(e << 23);
    }
  }
}

template <bool BF16>
constexpr int kTileCtas = BF16 ? 4 : 2;  // per SM

// 128 x 128 blocks: one CTA per block, which it holds in registers as it came.
template <bool BF16>
__global__ void __launch_bounds__(kQuantThreads, kTileCtas<BF16>) quant_tiles_kernel(const Fp8QuantArgs a) {
  constexpr int kN = Vec<BF16>::kN, kLanes = kFp8Block / kN, kRows = kQuantThreads / kLanes, kUnroll = kFp8Block / kRows;
  __shared__ uint32_t tops[2][kQuantThreads / 32];
  pdl_wait();
  const int KB = (a.K + kFp8Block - 1) / kFp8Block, RB = (a.rows + kFp8Block - 1) / kFp8Block;
  const long long tiles = static_cast<long long>(a.n) * RB * KB;
  const int sub = threadIdx.x / kLanes, in = threadIdx.x % kLanes;
  int turn = 0;
  for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const long long mb = tile / KB, mat = mb / RB;
    const int k = static_cast<int>(tile - mb * KB) * kFp8Block + in * kN;
    const int r0 = static_cast<int>(mb - mat * RB) * kFp8Block + sub;
    Vec<BF16> x[kUnroll];
    const char* src = source<BF16>(a, mat, r0, k);
    const long long step = kRows * a.sr * (BF16 ? 2 : 4);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (r0 + u * kRows < a.rows && k < a.K)
        x[u].load(src + u * step);
      else
        x[u].zero();
    }
    // two sets of maxima in turn: one barrier a block
    auto meet = [&](uint32_t top) {
      top = __reduce_max_sync(0xffffffffu, top);
      if ((threadIdx.x & 31) == 0) tops[turn][threadIdx.x / 32] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kQuantThreads / 32; ++w) top = max(top, tops[turn][w]);
      turn ^= 1;
      return top;
    };
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) top = max(top, x[u].top());
    top = meet(top);
    const bool all = top < 0x7F800000u;
    if (!all) {  // rare: once more without the infinities and NaNs
      top = 0;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) top = max(top, x[u].finite_top());
      top = meet(top);
    }
    const uint32_t e = scale_exponent(top);
    const float inv = __uint_as_float((254u - e) << 23);
    if (threadIdx.x == 0) a.scales[tile] = __uint_as_float(e << 23);
    if (k < a.K) {
      uint8_t* dst = a.codes + (mat * a.rows + r0) * a.K + k;
      const long long next = static_cast<long long>(kRows) * a.K;
      if (all) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (r0 + u * kRows < a.rows) x[u].template store<true>(dst + u * next, inv);
      } else {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (r0 + u * kRows < a.rows) x[u].template store<false>(dst + u * next, inv);
      }
    }
  }
}

// 4 (float32) or 8 (bf16) codes per thread and step, so that a warp writes 512
// bytes side by side; one scale holds for all of them (K is a multiple of 16).
template <bool BF16>
__global__ void __launch_bounds__(kQuantThreads) dequant_kernel(const Fp8DequantArgs a, const Slice s) {
  constexpr int kN = BF16 ? 8 : 4, kUnroll = 4;
  pdl_wait();  // and no early start for the next launch: a GEMV may fetch this as its weights, ahead of its own wait
  const uint32_t KB = (a.K + kFp8Block - 1) / kFp8Block, per_row = a.K / kN, total = s.rows * per_row;
  const uint32_t RB = (static_cast<uint32_t>(a.rows) + a.block_rows - 1) / a.block_rows;
  for (uint32_t i0 = blockIdx.x * (kQuantThreads * kUnroll) + threadIdx.x; i0 < total;
       i0 += gridDim.x * (kQuantThreads * kUnroll)) {
    uint2 w[kUnroll];
    float scale[kUnroll];
    char* dst[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t i = i0 + u * kQuantThreads, f = s.per_row(i), r = s.row + f, m = s.per_mat(r);
      const uint32_t k = (i - f * per_row) * kN, mat = s.mat + m, row = r - m * a.rows;
      dst[u] = nullptr;
      if (i >= total) continue;
      const uint8_t* src = a.codes + (static_cast<long long>(s.mat) * a.rows + r) * a.K + k;
      w[u] = BF16 ? *reinterpret_cast<const uint2*>(src) : make_uint2(*reinterpret_cast<const uint32_t*>(src), 0u);
      const uint32_t rb = a.block_rows == 1 ? row : row / kFp8Block;
      scale[u] = a.scales[(static_cast<long long>(mat) * RB + rb) * KB + k / kFp8Block];
      dst[u] = static_cast<char*>(a.out) + (mat * a.sm + row * a.sr + k) * (BF16 ? 2 : 4);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (!dst[u]) continue;
      float v[kN];
#pragma unroll
      for (int j = 0; j < kN / 2; ++j) {
        uint32_t h;
        const uint32_t c = j < 2 ? w[u].x : w[u].y;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(c >> (16 * (j & 1)))));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        v[2 * j] = f.x * scale[u];
        v[2 * j + 1] = f.y * scale[u];
      }
      if constexpr (BF16) {
        uint32_t p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
          p[j] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(dst[u]) = make_uint4(p[0], p[1], p[2], p[3]);
      } else {
        *reinterpret_cast<float4*>(dst[u]) = make_float4(v[0], v[1], v[2], v[3]);
      }
    }
  }
}

int grid_of(long long items, int sms) {
  return static_cast<int>(std::max(1ll, std::min<long long>(items, static_cast<long long>(sms) * 8)));
}

// Calls f(slice) for row ranges of at most 2^31 / per_row rows, until one fails.
template <typename F>
cudaError_t in_slices(int n, int rows, long long per_row, F f) {
  const long long all = static_cast<long long>(n) * rows, most = std::max(1ll, (1ll << 31) / per_row - 1);
  for (long long at = 0; at < all;) {
    const Slice s{static_cast<uint32_t>(at / rows), static_cast<uint32_t>(at % rows),
                  static_cast<uint32_t>(std::min(all - at, std::min(most, (1ll << 31) - rows))),
                  Divisor(static_cast<uint32_t>(per_row)), Divisor(static_cast<uint32_t>(rows))};
    const cudaError_t e = f(s);
    if (e != cudaSuccess) return e;
    at += s.rows;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_fp8_quant(const Fp8QuantArgs& a, bool bf16, int block_rows, int sms, cudaStream_t st) {
  const long long KB = (a.K + kFp8Block - 1) / kFp8Block;
  if (block_rows == 1)
    return in_slices(a.n, a.rows, KB, [&](const Slice& s) {
      const long long per = 4ll * kQuantThreads * (bf16 ? 8 : 4) / kFp8Block;
      const int grid = grid_of((s.rows * KB + per - 1) / per, sms);
      return bf16 ? launch(quant_rows_kernel<true>, dim3(grid), dim3(kQuantThreads), 0, st, true, a, s)
                  : launch(quant_rows_kernel<false>, dim3(grid), dim3(kQuantThreads), 0, st, true, a, s);
    });
  // as many CTAs as run at once: each takes the same number of blocks, but for one
  const long long tiles = static_cast<long long>(a.n) * ((a.rows + kFp8Block - 1) / kFp8Block) * KB;
  const int grid = static_cast<int>(std::min<long long>(tiles, sms * (bf16 ? kTileCtas<true> : kTileCtas<false>)));
  return bf16 ? launch(quant_tiles_kernel<true>, dim3(grid), dim3(kQuantThreads), 0, st, true, a)
              : launch(quant_tiles_kernel<false>, dim3(grid), dim3(kQuantThreads), 0, st, true, a);
}

cudaError_t launch_fp8_dequant(const Fp8DequantArgs& a, bool bf16, int sms, cudaStream_t st) {
  const long long per_row = a.K / (bf16 ? 8 : 4);
  return in_slices(a.n, a.rows, per_row, [&](const Slice& s) {
    const int grid = grid_of((s.rows * per_row + 4 * kQuantThreads - 1) / (4 * kQuantThreads), sms);
    return bf16 ? launch(dequant_kernel<true>, dim3(grid), dim3(kQuantThreads), 0, st, true, a, s)
                : launch(dequant_kernel<false>, dim3(grid), dim3(kQuantThreads), 0, st, true, a, s);
  });
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
