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
// Both kernels are bound by memory (2 or 4 bytes read and 0.53 to 0.63
// written per value, or the reverse).  One thread takes 8 dims of a row: 16
// or 32 bytes in, one 32-bit word of codes out, so that a warp's loads and
// stores are contiguous, and group / 8 neighbouring lanes find the extremes by
// shuffles.
#include <cuda_fp16.h>

#include "dec_launch.cuh"
#include "dec_long.cuh"

namespace dec {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerThread = 4;  // rows in flight per thread

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
struct Raw8 {
  uint4 w[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* base, long long at) {
    if constexpr (BF16) {
      w[0] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at));
    } else {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + at);
      w[0] = __ldg(p);
      w[1] = __ldg(p + 1);
    }
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    if constexpr (BF16) {
      const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16lo(u[i]);
        x[2 * i + 1] = bf16hi(u[i]);
      }
    } else {
      const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(u[i]);
    }
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
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Four codes less 8 (whole numbers -8 .. 7) as 16 bits, by exact float sums.
__device__ __forceinline__ uint32_t join4(float a, float b, float c, float d) {
  const float v = fmaf(d, 4096.f, fmaf(c, 256.f, fmaf(b, 16.f, a)));
  return __float_as_uint(v + (8388608.f + 34952.f)) & 0xFFFFu;  // 2^23 + 8 * 0x1111
}

// The group / 8 lanes of a group, 8 values each: this lane's code word, and
// the group's (s, z) pair.  rint((x - z) / s) goes by a product with an
// approximate 1 / s and by adding 1.5 * 2^23: the product is within 3e-6 of the
// quotient, so only one within 1e-5 of a half-integer could round otherwise,
// and a thread that meets such a one divides.  (Two conversions per value on
// the transcendental pipe and a division per group took 50 us where this
// takes 24: 84 MB of bf16 rows.)
template <int GROUP>
__device__ __forceinline__ void quantise8(const float (&x)[8], uint32_t* word, uint32_t* pair) {
  float lo = fminf(x[0], x[1]), hi = fmaxf(x[0], x[1]), zero = fmaf(x[0], 0.f, x[1] * 0.f);
#pragma unroll
  for (int i = 2; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
    zero = fmaf(x[i], 0.f, zero);  // NaN once a value is not finite
  }
#pragma unroll
  for (int o = GROUP / 16; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t peers = ((1u << (GROUP / 8)) - 1u) << (lane & ~(GROUP / 8 - 1u));
  const bool nan_group = (__ballot_sync(0xffffffffu, zero != 0.f) & peers) != 0;
  const __half sh = __float2half_rn(fminf(div15(hi - lo), 65504.f));
  const float s = __half2float(sh);
  const __half zh = __float2half_rn(fminf(fmaxf(fmaf(8.f, s, lo), -65504.f), 65504.f));
  const float z = __half2float(zh);
  const float inv = s > 0.f ? rcp_approx(s) : 0.f;
  float r[8], off = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = fminf(fmaxf((x[i] - z) * inv, -8.f), 7.f);
    r[i] = (t + 12582912.f) - 12582912.f;
    off = fmaxf(off, fabsf(t - r[i]));
  }
  if (off > 0.49999f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = rintf(fminf(fmaxf(__fdiv_rn(x[i] - z, s), -8.f), 7.f));
  }
  *word = nan_group ? 0x88888888u : join4(r[0], r[1], r[2], r[3]) | (join4(r[4], r[5], r[6], r[7]) << 16);
  *pair = nan_group ? 0x7FFF7FFFu
                    : static_cast<uint32_t>(__half_as_ushort(sh)) | (static_cast<uint32_t>(__half_as_ushort(zh)) << 16);
}

// Grid (token chunks, Hkv * 2, B); a CTA takes kThreads / (D / 8) *
// kRowsPerThread tokens of one head's K or V.
template <int D, int GROUP, bool BF16>
__global__ void __launch_bounds__(kThreads) kv4_store_kernel(const __grid_constant__ Kv4StoreArgs a) {
  constexpr int kLanes = D / 8, kRows = kThreads / kLanes, NG = D / GROUP;
  const int b = blockIdx.z, h = blockIdx.y >> 1, which = blockIdx.y & 1;
  int p0;
  const int n = row_tokens(a.pos, a.lens, b, a.T, a.S_max, a.from_cache ? a.src_tokens : a.S_max, &p0);
  if (n < 0) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) atomicOr(a.err, kErrPosRange);
    return;
  }
  const int sub = threadIdx.x % kLanes;
  const int t0 = blockIdx.x * (kRows * kRowsPerThread) + threadIdx.x / kLanes;
  if (blockIdx.x * (kRows * kRowsPerThread) >= n) return;
  const long long src0 = b * a.sb + h * a.sh + 8 * sub + (a.from_cache ? p0 * a.st : 0);
  const void* src = a.src[which];
  Raw8<BF16> raw[kRowsPerThread];
#pragma unroll
  for (int i = 0; i < kRowsPerThread; ++i) {
    const int t = t0 + i * kRows;
    if (t < n) raw[i].load(src, src0 + t * a.st);
  }
  const size_t slot0 = (static_cast<size_t>(b) * a.Hkv + h) * a.S_max + p0;
  uint32_t* codes = reinterpret_cast<uint32_t*>(a.codes[which]);
#pragma unroll
  for (int i = 0; i < kRowsPerThread; ++i) {
    const int t = t0 + i * kRows;
    if (t0 - static_cast<int>(threadIdx.x / kLanes) + i * kRows >= n) break;  // the same verdict in the whole CTA
    float x[8];
    if (t < n) {
      raw[i].get(x);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = 0.f;
    }
    uint32_t word, pair;
    quantise8<GROUP>(x, &word, &pair);
    if (t < n) {
      const size_t slot = slot0 + t;
      codes[slot * kLanes + sub] = word;
      if (sub % (GROUP / 8) == 0) a.params[which][slot * NG + sub / (GROUP / 8)] = pair;
    }
  }
}

// The reverse; the same grid.
template <int D, int GROUP, bool BF16>
__global__ void __launch_bounds__(kThreads) kv4_load_kernel(const __grid_constant__ Kv4LoadArgs a) {
  constexpr int kLanes = D / 8, kRows = kThreads / kLanes, NG = D / GROUP;
  const int b = blockIdx.z, h = blockIdx.y >> 1, which = blockIdx.y & 1;
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
      word[i] = __ldg(codes + (slot0 + t) * kLanes + sub);
      pair[i] = __ldg(a.params[which] + (slot0 + t) * NG + sub / (GROUP / 8));
    }
  }
#pragma unroll
  for (int i = 0; i < kRowsPerThread; ++i) {
    const int t = t0 + i * kRows;
    if (t >= n) break;
    const float s = half_bits_to_float(pair[i]), z = half_bits_to_float(pair[i] >> 16);
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)  // s (c - 8) has at most 15 significant bits: one rounding
      x[j] = fmaf(s, static_cast<float>(static_cast<int>((word[i] >> (4 * j)) & 15u) - 8), z);
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

template <int D>
dim3 kv4_grid(int T, int Hkv, int B) {
  constexpr int per = kThreads / (D / 8) * kRowsPerThread;
  return dim3((T + per - 1) / per, Hkv * 2, B);
}

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
    return launch(kv4_store_kernel<D, G, BF16>, kv4_grid<D>(a.T, a.Hkv, a.B), dim3(kThreads), 0, st, false, a);
  }
};
template <int D, int G, bool BF16>
struct Load {
  static cudaError_t run(const Kv4LoadArgs& a, cudaStream_t st) {
    return launch(kv4_load_kernel<D, G, BF16>, kv4_grid<D>(a.T, a.Hkv, a.B), dim3(kThreads), 0, st, false, a);
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
