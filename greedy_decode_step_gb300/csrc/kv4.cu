// The 4-bit KV cache: quantising K and V rows as they are written, and
// reading a range back.
//
// For each (row, token, head) the D values are cut into groups; with lo and
// hi a group's extremes,
//   s = half((hi - lo) / 15),  z = half(lo + 8 s),
//   c = clamp(rint((x - z) / s) + 8, 0, 15)        (c = 8 where s = 0)
// in float32 IEEE operations, s and z clamped to the half range; the code
// stands for z + s (c - 8).  A group holding an infinity or a NaN stores
// s = z = NaN, so that it reads back as NaN whole.
//
// Reading back is bound by memory (0.53 to 0.63 bytes read and 2 or 4 written
// per value): one thread takes 8 dims of a row, a 32-bit word of codes.
// Storing is bound by instructions: one thread takes 16 dims, so that a group's
// scale is worked out half as often (8 dims a thread: 199 instructions for
// every 8 values and 34 us for 84 MB of bf16 rows, 16 dims: 23 us), and
// group / 16 neighbouring lanes find the extremes by shuffles.
#include <cuda_fp16.h>

#include "dec_launch.cuh"
#include "dec_long.cuh"

namespace dec {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerThread = 8;  // rows in flight per thread, reading back
constexpr int kVals = 16;          // dims per thread, storing
constexpr int kStoreRows = 4;      // rows in flight per thread, storing

__device__ __forceinline__ __half2 as_half2(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }
__device__ __forceinline__ float half_bits_to_float(uint32_t h) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xFFFFu)));
}

// Tokens of row b, or -1 where its slots leave the cache (or the source).
__device__ __forceinline__ int row_tokens(const int32_t* pos, const int32_t* lens, int b, int T, int S_max,
                                          int src_limit, int* p0) {
  const int n = lens ? lens[b] : T;
  const int p = pos[b];
  *p0 = p;
  if (n == 0) return 0;
  if (n < 0 || n > T || p < 0 || p > S_max - n || p > src_limit - n) return -1;
  return n;
}

template <bool BF16>
struct Raw {
  static constexpr int kWords = kVals * (BF16 ? 2 : 4) / 16;
  uint4 w[kWords];
  __device__ __forceinline__ void load(const void* base, long long at) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(base) + at * (BF16 ? 2 : 4));
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = p[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (auto& u : w) u = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void get(float (&x)[kVals]) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (BF16) {
          x[8 * i + 2 * j] = bf16lo(u[j]);
          x[8 * i + 2 * j + 1] = bf16hi(u[j]);
        } else {
          x[4 * i + j] = __uint_as_float(u[j]);
        }
      }
    }
  }
  // Largest and smallest value over the LANES neighbouring lanes of a group; NaN if any is.
  template <int LANES>
  __device__ __forceinline__ void extremes(float* hi, float* lo) const {
    if constexpr (BF16) {  // two at a time
      uint32_t h = max2(max2(w[0].x, w[0].y), max2(w[0].z, w[0].w));
      uint32_t l = min2(min2(w[0].x, w[0].y), min2(w[0].z, w[0].w));
#pragma unroll
      for (int i = 1; i < kWords; ++i) {
        h = max2(h, max2(max2(w[i].x, w[i].y), max2(w[i].z, w[i].w)));
        l = min2(l, min2(min2(w[i].x, w[i].y), min2(w[i].z, w[i].w)));
      }
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) {
        h = max2(h, __shfl_xor_sync(0xffffffffu, h, o));
        l = min2(l, __shfl_xor_sync(0xffffffffu, l, o));
      }
      *hi = max1(bf16lo(h), bf16hi(h));
      *lo = min1(bf16lo(l), bf16hi(l));
    } else {
      float x[kVals];
      get(x);
      float h = x[0], l = x[0];
#pragma unroll
      for (int i = 1; i < kVals; ++i) {
        h = max1(h, x[i]);
        l = min1(l, x[i]);
      }
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) {
        h = max1(h, __shfl_xor_sync(0xffffffffu, h, o));
        l = min1(l, __shfl_xor_sync(0xffffffffu, l, o));
      }
      *hi = h;
      *lo = l;
    }
  }
  // extremes that keep a NaN
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ float max1(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
  }
  static __device__ __forceinline__ float min1(float a, float b) {
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
  }
};

// d / 15, correctly rounded: the product with RN(1/15) and one step on its
// exact remainder (Markstein's method; exhaustively equal to the division).
// Not a number where d is infinite.
__device__ __forceinline__ float div15(float d) {
  const float y = 1.f / 15.f;
  const float q = d * y;
  return fmaf(fmaf(-15.f, q, d), y, q);
}
// Eight codes as a word.  Each x is a quotient in [-8.5, 7.5) plus 1.5 * 2^23 + 8,
// whose low bits are its code: 0x4B400000 + code, of which the leading parts sum
// to a constant.
__device__ __forceinline__ uint32_t join8(const float* x) {
  uint32_t w = __float_as_uint(x[7]);
#pragma unroll
  for (int i = 6; i >= 0; --i) w = (w << 4) + __float_as_uint(x[i]);
  return w - 0x4B400000u * 0x11111111u;
}

// The group / 16 lanes of a group, 16 values each: this lane's code words, and
// the group's (s, z) pair.  (x - z) / s is the product with RN(1/s) corrected by
// its exact remainder, which rounds to the code of the true division: checked
// for every half significand at 81 numerators around each half-integer.  A
// group whose ends lie outside the codes is clamped.  (84 MB of bf16 rows: 50 us
// with two conversions per value on the transcendental pipe and a division per
// group; 39 and 34 us with a plain product, and a division wherever one of a
// warp's values came within 1e-5 of a half-integer, which happens to a seventh
// of the warps.)
template <int GROUP, bool BF16>
__device__ __forceinline__ void quantise(const Raw<BF16>& raw, uint2* words, uint32_t* pair) {
  float lo, hi;
  raw.template extremes<GROUP / kVals>(&hi, &lo);
  const bool nan_group = !(hi <= 3.402823466e38f) || !(lo >= -3.402823466e38f);
  const __half sh = __float2half_rn(fminf(div15(hi - lo), 65504.f));
  const float s = __half2float(sh);
  const __half zh = __float2half_rn(fminf(fmaxf(fmaf(8.f, s, lo), -65504.f), 65504.f));
  const float z = __half2float(zh);
  const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
  constexpr float kRound = 12582920.f;  // 1.5 * 2^23 + 8
  float x[kVals];
  raw.get(x);
  const bool inside = (hi - z) * inv < 7.49f && (lo - z) * inv > -8.49f;
#pragma unroll
  for (int i = 0; i < kVals; ++i) {
    const float d = x[i] - z, q = d * inv;
    x[i] = fmaf(fmaf(-s, q, d), inv, q);
    if (inside) x[i] += kRound;
  }
  if (!inside) {
#pragma unroll
    for (int i = 0; i < kVals; ++i) x[i] = fminf(fmaxf(x[i], -8.f), 7.f) + kRound;
  }
  words->x = nan_group ? 0x88888888u : join8(x);
  words->y = nan_group ? 0x88888888u : join8(x + 8);
  *pair = nan_group ? 0x7FFF7FFFu
                    : static_cast<uint32_t>(__half_as_ushort(sh)) | (static_cast<uint32_t>(__half_as_ushort(zh)) << 16);
}

// Grid (token chunks, Hkv * 2, B); a CTA takes kThreads / (D / kVals) *
// kStoreRows tokens of one head's K or V.
template <int D, int GROUP, bool BF16>
__global__ void __launch_bounds__(kThreads) kv4_store_kernel(const __grid_constant__ Kv4StoreArgs a) {
  constexpr int kLanes = D / kVals, kRows = kThreads / kLanes, NG = D / GROUP;
  const int b = blockIdx.z, h = blockIdx.y >> 1, which = blockIdx.y & 1;
  pdl_wait();
  pdl_launch_dependents();
  int p0;
  const int n = row_tokens(a.pos, a.lens, b, a.T, a.S_max, a.from_cache ? a.src_tokens : a.S_max, &p0);
  if (n < 0) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) atomicOr(a.err, kErrPosRange);
    return;
  }
  const int first = blockIdx.x * (kRows * kStoreRows);
  if (first >= n) return;
  const int sub = threadIdx.x % kLanes;
  const int t0 = first + threadIdx.x / kLanes;
  const long long src0 = b * a.sb + h * a.sh + kVals * sub + (a.from_cache ? p0 * a.st : 0);
  const void* src = a.src[which];
  Raw<BF16> raw[kStoreRows];
#pragma unroll
  for (int i = 0; i < kStoreRows; ++i) {
    const int t = t0 + i * kRows;
    if (t < n) raw[i].load(src, src0 + t * a.st);
    else raw[i].zero();
  }
  const size_t slot0 = (static_cast<size_t>(b) * a.Hkv + h) * a.S_max + p0;
  uint2* codes = reinterpret_cast<uint2*>(a.codes[which]);
#pragma unroll
  for (int i = 0; i < kStoreRows; ++i) {
    if (first + i * kRows >= n) break;  // the same verdict in the whole CTA
    const int t = t0 + i * kRows;
    uint2 words;
    uint32_t pair;
    quantise<GROUP, BF16>(raw[i], &words, &pair);
    if (t < n) {
      const size_t slot = slot0 + t;
      codes[slot * kLanes + sub] = words;
      if (sub % (GROUP / kVals) == 0) a.params[which][slot * NG + sub / (GROUP / kVals)] = pair;
    }
  }
}

// The reverse; the same grid.
template <int D, int GROUP, bool BF16>
__global__ void __launch_bounds__(kThreads) kv4_load_kernel(const __grid_constant__ Kv4LoadArgs a) {
  constexpr int kLanes = D / 8, kRows = kThreads / kLanes, NG = D / GROUP;
  const int b = blockIdx.z, h = blockIdx.y >> 1, which = blockIdx.y & 1;
  pdl_wait();
  pdl_launch_dependents();
  int p0;
  const int n = row_tokens(a.pos, a.lens, b, a.T, a.S_max, a.S_max, &p0);
  if (n < 0) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) atomicOr(a.err, kErrPosRange);
    return;
  }
  const int sub = threadIdx.x % kLanes;
  const int t0 = blockIdx.x * (kRows * kRowsPerThread) + threadIdx.x / kLanes;
  const size_t slot0 = (static_cast<size_t>(b) * a.Hkv + h) * a.S_max + p0;
  const uint32_t* codes = reinterpret_cast<const uint32_t*>(a.codes[which]);
  uint32_t word[kRowsPerThread], pair[kRowsPerThread];
#pragma unroll
  for (int i = 0; i < kRowsPerThread; ++i) {
    const int t = t0 + i * kRows;
    if (t < n) {
      word[i] = codes[(slot0 + t) * kLanes + sub];
      pair[i] = a.params[which][(slot0 + t) * NG + sub / (GROUP / 8)];
    }
  }
#pragma unroll
  for (int i = 0; i < kRowsPerThread; ++i) {
    const int t = t0 + i * kRows;
    if (t >= n) break;
    const float s = half_bits_to_float(pair[i]), z = half_bits_to_float(pair[i] >> 16);
    // s (c - 8) has at most 15 significant bits, so the fused step rounds once.
    // Two codes at a time through half arithmetic: 1024 + c less 1032, exactly,
    // and the odd nibbles 16 times that (a conversion per code on the
    // transcendental pipe: 20.2 us where this takes 19.4, 110 MB).
    const float s16 = s * 0.0625f;
    float x[8];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t w = word[i] >> (8 * j);
      const uint32_t lo = (w & 0x000F000Fu) | 0x64006400u, hi = (w & 0x00F000F0u) | 0x64006400u;
      const float2 even = __half22float2(__hadd2(as_half2(lo), as_half2(0xE408E408u)));
      const float2 odd = __half22float2(__hadd2(as_half2(hi), as_half2(0xE480E480u)));
      x[2 * j] = fmaf(s, even.x, z);
      x[2 * j + 4] = fmaf(s, even.y, z);
      x[2 * j + 1] = fmaf(s16, odd.x, z);
      x[2 * j + 5] = fmaf(s16, odd.y, z);
    }
    const long long at = b * a.sb + t * a.st + h * a.sh + 8 * sub;
    if constexpr (BF16) {
      uint32_t u[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[j]) : "f"(x[2 * j + 1]), "f"(x[2 * j]));
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.dst[which]) + at) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(a.dst[which]) + at);
      p[0] = make_float4(x[0], x[1], x[2], x[3]);
      p[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
  }
}

dim3 kv4_grid(int T, int per, int Hkv, int B) { return dim3((T - 1) / per + 1, Hkv * 2, B); }

// (D, group, type) -> instantiation
template <template <int, int, bool> class F, typename A>
cudaError_t dispatch(const A& a, int D, int group, bool bf16, cudaStream_t st) {
#define DEC_KV4_CASE(d, g) \
  if (D == d && group == g) return bf16 ? F<d, g, true>::run(a, st) : F<d, g, false>::run(a, st);
  DEC_KV4_CASE(64, 32)
  DEC_KV4_CASE(64, 64)
  DEC_KV4_CASE(128, 32)
  DEC_KV4_CASE(128, 64)
  DEC_KV4_CASE(128, 128)
#undef DEC_KV4_CASE
  return cudaErrorInvalidValue;
}
template <int D, int G, bool BF16>
struct Store {
  static cudaError_t run(const Kv4StoreArgs& a, cudaStream_t st) {
    const dim3 grid = kv4_grid(a.T, kThreads / (D / kVals) * kStoreRows, a.Hkv, a.B);
    return launch(kv4_store_kernel<D, G, BF16>, grid, dim3(kThreads), 0, st, true, a);
  }
};
template <int D, int G, bool BF16>
struct Load {
  static cudaError_t run(const Kv4LoadArgs& a, cudaStream_t st) {
    const dim3 grid = kv4_grid(a.T, kThreads / (D / 8) * kRowsPerThread, a.Hkv, a.B);
    return launch(kv4_load_kernel<D, G, BF16>, grid, dim3(kThreads), 0, st, true, a);
  }
};

}  // namespace

cudaError_t launch_kv4_store(const Kv4StoreArgs& a, int D, int group, bool bf16, cudaStream_t st) {
  return dispatch<Store>(a, D, group, bf16, st);
}
cudaError_t launch_kv4_load(const Kv4LoadArgs& a, int D, int group, bool bf16, cudaStream_t st) {
  return dispatch<Load>(a, D, group, bf16, st);
}

}  // namespace dec
