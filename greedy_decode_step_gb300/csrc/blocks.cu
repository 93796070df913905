// Block-sparse decode attention, the cheap part: per-block channel bounds of
// the key cache, and the choice of each (row, KV head)'s blocks by them.
//
// A block is 64 consecutive cache slots.  With hi and lo a block's largest and
// smallest key value per dim, q . k <= sum_d max(q_d hi_d, q_d lo_d) for every
// key of the block.  A group's query heads share one choice, by the sum of
// their bounds, which folds into one dot product per block:
//   score = sum_d P_d hi_d + N_d lo_d,  P = sum_h max(q_h, 0), N = sum_h min(q_h, 0)
#include <cuda_bf16.h>

#include "dec_launch.cuh"
#include "dec_long.cuh"

namespace dec {
namespace {

// ----------------------------------------------------------------------------- bounds

constexpr int kBoundThreads = 256;

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmin2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Grid (blocks touched at most, Hkv, B).  A CTA reads its block's live slots
// once, 16 bytes per thread and row group, and folds the row groups in shared
// memory; memory bound (16 KB read, 0.5 KB written per block of D = 128).
template <int D>
__global__ void __launch_bounds__(kBoundThreads) block_bounds_kernel(const __grid_constant__ BoundsArgs a) {
  constexpr int kLanes = D / 8, kRows = kBoundThreads / kLanes, kPer = kBlockKeys / kRows;
  __shared__ uint4 fold[2][kBoundThreads / 32][kLanes];
  const int h = blockIdx.y, b = blockIdx.z;
  const int p = a.pos[b];
  if (p < 0 || p > a.S_max - a.T) {
    if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) atomicOr(a.err, kErrPosRange);
    return;
  }
  const int j = p / kBlockKeys + blockIdx.x, end = p + a.T;
  const int k0 = j * kBlockKeys;
  if (k0 >= end) return;
  const int n = min(kBlockKeys, end - k0);
  const int sub = threadIdx.x % kLanes, r0 = threadIdx.x / kLanes;
  const size_t item = static_cast<size_t>(b) * a.Hkv + h;
  const uint4* src = reinterpret_cast<const uint4*>(a.k + (item * a.S_max + k0) * D) + sub;
  uint4 w[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = min(r0 + i * kRows, n - 1);  // a row twice changes no extreme
    w[i] = __ldg(src + static_cast<size_t>(r) * kLanes);
  }
  uint4 hi = w[0], lo = w[0];
#pragma unroll
  for (int i = 1; i < kPer; ++i) {
    hi = make_uint4(max2(hi.x, w[i].x), max2(hi.y, w[i].y), max2(hi.z, w[i].z), max2(hi.w, w[i].w));
    lo = make_uint4(min2(lo.x, w[i].x), min2(lo.y, w[i].y), min2(lo.z, w[i].z), min2(lo.w, w[i].w));
  }
#pragma unroll
  for (int o = kLanes; o < 32; o <<= 1) {
    hi.x = max2(hi.x, __shfl_xor_sync(0xffffffffu, hi.x, o));
    hi.y = max2(hi.y, __shfl_xor_sync(0xffffffffu, hi.y, o));
    hi.z = max2(hi.z, __shfl_xor_sync(0xffffffffu, hi.z, o));
    hi.w = max2(hi.w, __shfl_xor_sync(0xffffffffu, hi.w, o));
    lo.x = min2(lo.x, __shfl_xor_sync(0xffffffffu, lo.x, o));
    lo.y = min2(lo.y, __shfl_xor_sync(0xffffffffu, lo.y, o));
    lo.z = min2(lo.z, __shfl_xor_sync(0xffffffffu, lo.z, o));
    lo.w = min2(lo.w, __shfl_xor_sync(0xffffffffu, lo.w, o));
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane < kLanes) {
    fold[0][warp][lane] = hi;
    fold[1][warp][lane] = lo;
  }
  __syncthreads();
  if (threadIdx.x < 2 * kLanes) {
    const int which = threadIdx.x / kLanes, s = threadIdx.x % kLanes;
    uint4 x = fold[which][0][s];
#pragma unroll
    for (int i = 1; i < kBoundThreads / 32; ++i) {
      const uint4 y = fold[which][i][s];
      x = which == 0 ? make_uint4(max2(x.x, y.x), max2(x.y, y.y), max2(x.z, y.z), max2(x.w, y.w))
                     : make_uint4(min2(x.x, y.x), min2(x.y, y.y), min2(x.z, y.z), min2(x.w, y.w));
    }
    reinterpret_cast<uint4*>(a.bounds + ((item * a.NB + j) * 2 + which) * D)[s] = x;
  }
}

// ----------------------------------------------------------------------------- selection

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;

// Largest score first; a NaN counts as -infinity.
__device__ __forceinline__ uint32_t score_key(float s) {
  return float_order_key(s == s ? s + 0.0f : -INFINITY);
}

// Sum over the CTA of one int per thread; every thread gets it.
__device__ __forceinline__ int cta_sum(int v, int* red) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  int s = 0;
#pragma unroll
  for (int i = 0; i < kSelWarps; ++i) s += red[i];
  return s;
}

// One CTA per (row, KV head).  The row's blocks 0 .. pos / 64 are scored in
// fp32; the cut is found by bisection over the order-preserving integer keys.
// An fp32 score is within E of the exact one, so blocks more than 2 E above
// the cut are in and those more than 2 E below are out whatever the rounding;
// the few between are scored again in 64 bits and ranked (ties: the lower
// block), so that the choice is that of the exact scores.
// Bound by latency and, per CTA, by reading 4 D bytes per block.
template <int D>
__global__ void __launch_bounds__(kSelThreads) select_blocks_kernel(const __grid_constant__ SelectBlocksArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int kVec = 2 * D / 8;                       // 16-byte vectors of a block's bounds
  constexpr int kPerWarp = 32 / (kVec < 32 ? kVec : 32);  // blocks a warp scores side by side
  __shared__ float w32[2 * D];
  __shared__ float err_red[kSelWarps];
  __shared__ int red[kSelWarps];
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.Hq / a.Hkv;
  const size_t item = static_cast<size_t>(b) * a.Hkv + h;
  int32_t* out = a.blocks + item * a.n_select;
  const int p = a.pos[b];
  if (p < -1 || p >= a.S_max) {
    if (h == 0 && tid == 0) atomicOr(a.err, kErrPosRange);
    return;
  }
  const int nb = p < 0 ? 0 : p / kBlockKeys + 1;
  if (nb <= a.n_select) {  // all of them
    for (int i = tid; i < a.n_select; i += kSelThreads) out[i] = i < nb ? i : -1;
    return;
  }
  float* score = reinterpret_cast<float*>(smem);                                // [nb]
  double* exact = reinterpret_cast<double*>(smem + (a.NB * 4 + 15) / 16 * 16);  // [nb], of the blocks in `list`
  int* list = reinterpret_cast<int*>(exact + a.NB);                             // blocks near the cut
  for (int d = tid; d < D; d += kSelThreads) {
    double P = 0., N = 0.;
    for (int i = 0; i < G; ++i) {
      const double q = a.q[(static_cast<size_t>(b) * a.Hq + static_cast<size_t>(h) * G + i) * D + d];
      if (q > 0.) P += q;
      else N += q;  // a NaN goes here
    }
    w32[d] = static_cast<float>(P);
    w32[D + d] = static_cast<float>(N);
  }
  __syncthreads();
  // blocks lo_free .. hi_free - 1 compete; the others are taken
  const int lo_free = min(a.n_first, nb), hi_free = max(lo_free, nb - a.n_last);
  const int want = a.n_select - (nb - (hi_free - lo_free));
  const uint4* rows = reinterpret_cast<const uint4*>(a.bounds + item * a.NB * 2 * D);
  const int part = lane / kVec, vec = lane % kVec;  // D = 64: two blocks side by side
  float w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = w32[8 * vec + i];
  float amax = 0.f;  // the largest sum of term magnitudes that this lane met
  constexpr int kBatch = 8;
  for (int j0 = lo_free + warp * kPerWarp * kBatch; j0 < hi_free; j0 += kSelWarps * kPerWarp * kBatch) {
    uint4 u[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int j = min(j0 + i * kPerWarp + part, hi_free - 1);
      u[i] = __ldg(rows + static_cast<size_t>(j) * kVec + vec);
    }
    float s[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const uint32_t x[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
      float t = 0.f, m = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        t = fmaf(w[2 * e], bf16lo(x[e]), t);
        t = fmaf(w[2 * e + 1], bf16hi(x[e]), t);
        m = fmaf(fabsf(w[2 * e]), fabsf(bf16lo(x[e])), m);
        m = fmaf(fabsf(w[2 * e + 1]), fabsf(bf16hi(x[e])), m);
      }
      s[i] = t;
      amax = fmaxf(amax, m == m ? m : INFINITY);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
#pragma unroll
      for (int o = kVec / 2; o > 0; o >>= 1) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
      const int j = j0 + i * kPerWarp + part;
      if (vec == 0 && j < hi_free) score[j] = s[i];
    }
  }
  // E: the rounding of the weights, products and sums is below 16 * 2^-24 of
  // the sum of magnitudes (8 fused steps, 5 additions, 1 rounding of w), and
  // 256 results below the normal range lose 2^-149 each.  Not finite: every
  // block counts as near the cut.
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax += __shfl_xor_sync(0xffffffffu, amax, o);
  if (lane == 0) err_red[warp] = amax;
  __syncthreads();
  float E = 0.f;
#pragma unroll
  for (int i = 0; i < kSelWarps; ++i) E = fmaxf(E, err_red[i]);
  E = fmaf(E, 1.0f / (1 << 20), 1e-41f);
  // the want-th largest score, bit by bit
  uint32_t cut = 0;
  if (want > 0) {
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t trial = cut | (1u << bit);
      int n = 0;
      for (int j = lo_free + tid; j < hi_free; j += kSelThreads) n += score_key(score[j]) >= trial ? 1 : 0;
      if (cta_sum(n, red) >= want) cut = trial;
    }
  }
  const float tau = float_from_order_key(cut);
  // above: in; near the cut: listed in block order
  int taken = 0, near = 0;  // of the blocks before the chunk
  for (int base = lo_free; base < hi_free; base += kSelThreads) {
    const int j = base + tid;
    const float s = j < hi_free ? score[j] : 0.f;
    const bool over = j < hi_free && s > tau + 2.f * E;
    const bool close = j < hi_free && !over && !(s < tau - 2.f * E);
    const unsigned mine = __ballot_sync(0xffffffffu, close);
    taken += cta_sum(over ? 1 : 0, red);
    __syncthreads();
    if (lane == 0) red[warp] = __popc(mine);
    __syncthreads();
    int before = near;
    for (int i = 0; i < kSelWarps; ++i) {
      if (i < warp) before += red[i];
      near += red[i];
    }
    if (close) list[before + __popc(mine & ((1u << lane) - 1u))] = j;
    // the score's place now says whether the block is in
    if (j < hi_free) score[j] = over ? 1.f : 0.f;
  }
  __syncthreads();
  const int rest = want - taken;  // of the near ones
  if (rest >= near) {
    for (int i = tid; i < near; i += kSelThreads) score[list[i]] = 1.f;
  } else if (rest > 0) {
    for (int i = warp; i < near; i += kSelWarps) {
      const uint16_t* r = a.bounds + (item * a.NB + list[i]) * 2 * D;
      double s = 0.;
      for (int d = lane; d < D; d += 32) {
        const double hi = __uint_as_float(static_cast<uint32_t>(r[d]) << 16);
        const double lo = __uint_as_float(static_cast<uint32_t>(r[D + d]) << 16);
        for (int e = 0; e < G; ++e) {  // the definition itself: it also holds for infinite bounds
          const double q = a.q[(static_cast<size_t>(b) * a.Hq + static_cast<size_t>(h) * G + e) * D + d];
          const double x = q * hi, y = q * lo;
          s += x > y || x != x ? x : y;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (lane == 0) exact[i] = s == s ? s : -INFINITY;
    }
    __syncthreads();
    for (int i = tid; i < near; i += kSelThreads) {
      const double s = exact[i];
      int better = 0;
      for (int e = 0; e < near; ++e) better += exact[e] > s || (exact[e] == s && e < i) ? 1 : 0;
      if (better < rest) score[list[i]] = 1.f;
    }
  }
  __syncthreads();
  // the chosen blocks in order
  int done = 0;
  for (int base = 0; base < nb; base += kSelThreads) {
    const int j = base + tid;
    const bool in = j < nb && (j < lo_free || j >= hi_free || score[j] != 0.f);
    const unsigned mine = __ballot_sync(0xffffffffu, in);
    __syncthreads();
    if (lane == 0) red[warp] = __popc(mine);
    __syncthreads();
    int before = done;
    for (int i = 0; i < kSelWarps; ++i) {
      if (i < warp) before += red[i];
      done += red[i];
    }
    if (in) out[before + __popc(mine & ((1u << lane) - 1u))] = j;
  }
}

uint32_t select_smem(int NB) { return (NB * 4 + 15) / 16 * 16 + NB * 8 + NB * 4; }

}  // namespace

cudaError_t launch_block_bounds(const BoundsArgs& a, int D, cudaStream_t st) {
  const dim3 grid((a.T + kBlockKeys - 2) / kBlockKeys + 1, a.Hkv, a.B);
  return D == 64 ? launch(block_bounds_kernel<64>, grid, dim3(kBoundThreads), 0, st, false, a)
                 : launch(block_bounds_kernel<128>, grid, dim3(kBoundThreads), 0, st, false, a);
}

cudaError_t launch_select_blocks(const SelectBlocksArgs& a, int D, cudaStream_t st) {
  const dim3 grid(a.Hkv, a.B);
  return D == 64 ? launch(select_blocks_kernel<64>, grid, dim3(kSelThreads), select_smem(a.NB), st, false, a)
                 : launch(select_blocks_kernel<128>, grid, dim3(kSelThreads), select_smem(a.NB), st, false, a);
}

cudaError_t allow_smem_blocks() {
  const int most = static_cast<int>(select_smem(kSelMaxBlocks));
  cudaError_t e = cudaFuncSetAttribute(select_blocks_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(select_blocks_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  return e;
}

}  // namespace dec
