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
  pdl_wait();
  pdl_launch_dependents();
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
    w[i] = src[static_cast<size_t>(r) * kLanes];
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

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelMaxCluster = 8;

// Larger score, larger key; a NaN counts as -infinity.
__device__ __forceinline__ uint32_t score_key(float s) {
  return float_order_key(s == s ? s + 0.0f : -INFINITY);
}

// The sums over LANES lanes of kBatch values per lane: lane i of the group
// gets the sum of value i / (LANES / kBatch).  Each step exchanges half of the
// values still held, so that the batch takes kBatch + 1 (or 2) shuffles, not
// 4 or 5 for every value.
constexpr int kBatch = 8;
template <int LANES>
__device__ __forceinline__ float batch_sum(float (&s)[kBatch]) {
  const int lane = threadIdx.x & 31;
  int width = kBatch;
#pragma unroll
  for (int o = LANES / 2; o >= LANES / kBatch; o >>= 1) {
    width >>= 1;
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < kBatch / 2; ++i) {
      if (i < width) {
        const float give = up ? s[i] : s[i + width], keep = up ? s[i + width] : s[i];
        s[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
    }
  }
#pragma unroll
  for (int o = LANES / kBatch / 2; o > 0; o >>= 1) s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
  return s[0];
}

// The want-th largest of n <= kWarpKeys keys, by a search of three trials a
// round in warp 0, whose lanes hold them in registers; it ends once a trial
// splits off exactly `want` keys (about half of log2 n + 2 rounds for unlike
// keys, 16 at most).
constexpr int kWarpKeys = 512;
__device__ __forceinline__ uint32_t kth_largest_warp(const uint32_t* key, int n, int want, uint32_t* result) {
  if (threadIdx.x < 32) {
    constexpr int kPer = kWarpKeys / 32;
    uint32_t k[kPer], most = 0, least = 0xFFFFFFFFu;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int j = threadIdx.x + 32 * i;
      k[i] = j < n ? key[j] : 0u;  // below every trial
      most = max(most, k[i]);
      least = min(least, j < n ? k[i] : 0xFFFFFFFFu);
    }
    uint32_t lo = __reduce_min_sync(0xffffffffu, least), hi = __reduce_max_sync(0xffffffffu, most);
    // at least `want` keys reach lo; fewer reach hi + 1
    while (lo < hi) {
      const uint32_t t2 = hi - (hi - lo) / 2, t1 = t2 - (t2 - lo) / 2, t3 = hi - (hi - t2) / 2;
      int c1 = 0, c2 = 0, c3 = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        c1 += k[i] >= t1 ? 1 : 0;
        c2 += k[i] >= t2 ? 1 : 0;
        c3 += k[i] >= t3 ? 1 : 0;
      }
      c1 = __reduce_add_sync(0xffffffffu, c1);
      c2 = __reduce_add_sync(0xffffffffu, c2);
      c3 = __reduce_add_sync(0xffffffffu, c3);
      const int c = c3 >= want ? c3 : c2 >= want ? c2 : c1;
      const uint32_t t = c3 >= want ? t3 : c2 >= want ? t2 : t1;
      if (c == want) {
        uint32_t m = 0xFFFFFFFFu;
#pragma unroll
        for (int i = 0; i < kPer; ++i) m = min(m, k[i] >= t ? k[i] : 0xFFFFFFFFu);
        lo = hi = __reduce_min_sync(0xffffffffu, m);
      } else if (c > want) {
        hi = c3 >= want ? hi : c2 >= want ? t3 - 1 : t2 - 1;
        lo = t;
      } else {
        hi = t1 - 1;
      }
    }
    if (threadIdx.x == 0) *result = lo;
  }
  __syncthreads();
  return *result;
}

// The same for any n: four bits per round, the warps counting the keys at or
// above 15 trial cuts, 15 passes over shared memory each.  (One row, 8 KV heads,
// the whole selection: 14.8 us for 1,024 blocks, 22.5 for 2,048, 73 for 8,192; 6.3
// for 512 by the search above.)
__device__ __forceinline__ uint32_t kth_largest_cta(const uint32_t* key, int n, int want, int (*counts)[16]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t cut = 0;
#pragma unroll 1
  for (int shift = 28; shift >= 0; shift -= 4) {
    int* c = counts[(shift >> 2) & 1];
    for (int w = warp; w < 15; w += kSelWarps) {
      const uint32_t trial = cut | (static_cast<uint32_t>(w + 1) << shift);
      int m = 0;
#pragma unroll 4
      for (int j = lane; j < n; j += 32) m += key[j] >= trial ? 1 : 0;
      m = __reduce_add_sync(0xffffffffu, m);
      if (lane == 0) c[w] = m;
    }
    __syncthreads();
    int digit = 0;  // the counts fall with the trial
#pragma unroll
    for (int i = 0; i < 15; ++i) digit += c[i] >= want ? 1 : 0;
    cut |= static_cast<uint32_t>(digit) << shift;
  }
  return cut;
}

// A cluster of CTAs per (row, KV head): all of them score the row's blocks
// 0 .. pos / 64 in fp32, in turn, into CTA 0's shared memory, and CTA 0 goes on
// alone.  The cut is found on order-preserving integer keys.  An fp32 score is
// within E of the exact one, so blocks more than 2 E above the cut are in and
// those more than 2 E below are out whatever the rounding; the few between are
// scored again in 64 bits and ranked (ties: the lower block), so that the
// choice is that of the exact scores.
// Bound by latency: the chain position, query, bounds, cut, list, each a few
// hundred nanoseconds; one SM alone takes 6 us to read 512 blocks' bounds.
template <int D>
__global__ void __launch_bounds__(kSelThreads) select_blocks_kernel(const __grid_constant__ SelectBlocksArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int kVec = 2 * D / 8;       // 16-byte vectors of a block's bounds
  constexpr int kPerWarp = 32 / kVec;   // blocks a warp scores side by side
  __shared__ float w32[2 * D];
  __shared__ float err_red[kSelMaxCluster][kSelWarps];
  __shared__ int counts[2][16];
  __shared__ int n_near, n_over;
  __shared__ uint32_t s_cut;
  const int ctas = a.cluster, rank = blockIdx.x % ctas;
  const int h = blockIdx.x / ctas, b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.Hq / a.Hkv;
  const size_t item = static_cast<size_t>(b) * a.Hkv + h;
  if (ctas > 1) cluster_arrive();  // before the others write here, CTA 0 has started
  pdl_wait();
  pdl_launch_dependents();
  const float* q = a.q + (static_cast<size_t>(b) * a.Hq + static_cast<size_t>(h) * G) * D;
  int32_t* out = a.blocks + item * a.n_select;
  const int p = a.pos[b];
  if (tid < D) {
    float P = 0.f, N = 0.f;
    for (int i = 0; i < G; i += 4) {  // four loads at once: each costs half a microsecond
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = i + e < G ? q[(i + e) * D + tid] : 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (x[e] > 0.f) P += x[e];
        else N += x[e];  // a NaN goes here
      }
    }
    w32[tid] = P;
    w32[D + tid] = N;
  }
  const bool refused = p < -1 || p >= a.S_max;
  const int nb = p < 0 ? 0 : p / kBlockKeys + 1;
  if (refused || nb <= a.n_select) {  // nothing, or all of them
    if (refused && h == 0 && rank == 0 && tid == 0) atomicOr(a.err, kErrPosRange);
    if (!refused && rank == 0)
      for (int i = tid; i < a.n_select; i += kSelThreads) out[i] = i < nb ? i : -1;
    if (ctas > 1) cluster_wait();
    return;
  }
  uint32_t* key = reinterpret_cast<uint32_t*>(smem);                            // [nb]
  double* exact = reinterpret_cast<double*>(smem + (a.NB * 4 + 15) / 16 * 16);  // [nb], of the blocks in `list`
  int* list = reinterpret_cast<int*>(exact + a.NB);                             // blocks near the cut
  // blocks lo_free .. hi_free - 1 compete; the others are taken
  const int lo_free = min(a.n_first, nb), hi_free = max(lo_free, nb - a.n_last);
  const int want = a.n_select - (nb - (hi_free - lo_free));
  const uint4* rows = reinterpret_cast<const uint4*>(a.bounds + item * a.NB * 2 * D);
  const int part = lane / kVec, vec = lane % kVec;  // D = 64: two blocks side by side
  const int step = ctas * kSelWarps * kPerWarp * kBatch;
  uint4 u[kBatch];
  auto load = [&](int j0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      u[i] = rows[static_cast<size_t>(min(j0 + i * kPerWarp + part, nb - 1)) * kVec + vec];
  };
  const int first = lo_free + (rank * kSelWarps + warp) * kPerWarp * kBatch;
  if (first < hi_free) load(first);
  if (tid == 0) n_near = n_over = 0;
  if (ctas > 1) cluster_wait();
  __syncthreads();
  float w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = w32[8 * vec + i];
  float amax = 0.f;  // the largest sum of term magnitudes that this lane met
  for (int j0 = first; j0 < hi_free; j0 += step) {
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
    if (j0 + step < hi_free) load(j0 + step);
    const float sum = batch_sum<kVec>(s);
    const int j = j0 + vec / (kVec / kBatch) * kPerWarp + part;
    if (vec % (kVec / kBatch) == 0 && j < hi_free) {
      if (ctas > 1) store_cta0(key + j, score_key(sum));
      else key[j] = score_key(sum);
    }
  }
  // E: the rounding of the weights (15 additions), products and sums (8 fused
  // steps, 5 additions) is below 32 * 2^-24 of the sum of magnitudes, and 256
  // results below the normal range lose 2^-149 each.  Not finite: every block
  // counts as near the cut.
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax += __shfl_xor_sync(0xffffffffu, amax, o);
  if (lane == 0) {
    if (ctas > 1) store_cta0(&err_red[rank][warp], __float_as_uint(amax));
    else err_red[0][warp] = amax;
  }
  if (ctas > 1) {
    cluster_arrive();
    cluster_wait();
    if (rank) return;
  }
  __syncthreads();
  float E = 0.f;
  for (int i = 0; i < ctas; ++i)
#pragma unroll
    for (int j = 0; j < kSelWarps; ++j) E = fmaxf(E, err_red[i][j]);
  E = fmaf(E, 1.0f / (1 << 19), 1e-41f);
  const int n_free = hi_free - lo_free;
  uint32_t cut = 0;
  if (want > 0)
    cut = n_free <= kWarpKeys ? kth_largest_warp(key + lo_free, n_free, want, &s_cut)
                              : kth_largest_cta(key + lo_free, n_free, want, counts);
  const float tau = float_from_order_key(cut);
  // above: in; near the cut: listed, in any order
  int over = 0;
  for (int j = lo_free + tid; j < hi_free; j += kSelThreads) {
    const float s = float_from_order_key(key[j]);
    const bool in = want > 0 && s > tau + 2.f * E;
    if (in) ++over;
    else if (want > 0 && !(s < tau - 2.f * E)) list[atomicAdd(&n_near, 1)] = j;
    key[j] = in ? 1u : 0u;  // from here on: whether the block is in
  }
  over = __reduce_add_sync(0xffffffffu, over);
  if (lane == 0 && over) atomicAdd(&n_over, over);
  __syncthreads();
  const int near = n_near, rest = want - n_over;  // of the near ones
  if (rest >= near) {
    for (int i = tid; i < near; i += kSelThreads) key[list[i]] = 1u;
  } else if (rest > 0) {
    for (int i = warp; i < near; i += kSelWarps) {
      const uint16_t* r = a.bounds + (item * a.NB + list[i]) * 2 * D;
      double s = 0.;
      for (int d = lane; d < D; d += 32) {
        const double hi = __uint_as_float(static_cast<uint32_t>(r[d]) << 16);
        const double lo = __uint_as_float(static_cast<uint32_t>(r[D + d]) << 16);
        for (int e = 0; e < G; ++e) {  // the definition itself: it also holds for infinite bounds
          const double qd = q[e * D + d];
          const double x = qd * hi, y = qd * lo;
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
      const int j = list[i];
      int better = 0;
      for (int e = 0; e < near; ++e) better += exact[e] > s || (exact[e] == s && list[e] < j) ? 1 : 0;
      if (better < rest) key[j] = 1u;
    }
  }
  // the chosen blocks in order
  int done = 0, turn = 0;
  for (int base = 0; base < nb; base += kSelThreads, turn ^= 1) {
    __syncthreads();
    const int j = base + tid;
    const bool in = j < nb && (j < lo_free || j >= hi_free || key[j] != 0u);
    const unsigned mine = __ballot_sync(0xffffffffu, in);
    if (lane == 0) counts[turn][warp] = __popc(mine);
    __syncthreads();
    int before = done;
#pragma unroll
    for (int i = 0; i < kSelWarps; ++i) {
      const int n = counts[turn][i];
      before += i < warp ? n : 0;
      done += n;
    }
    if (in) out[before + __popc(mine & ((1u << lane) - 1u))] = j;
  }
}

uint32_t select_smem(int NB) { return (NB * 4 + 15) / 16 * 16 + NB * 8 + NB * 4; }

}  // namespace

cudaError_t launch_block_bounds(const BoundsArgs& a, int D, cudaStream_t st) {
  const dim3 grid((a.T - 1 + kBlockKeys - 1) / kBlockKeys + 1, a.Hkv, a.B);
  return D == 64 ? launch(block_bounds_kernel<64>, grid, dim3(kBoundThreads), 0, st, true, a)
                 : launch(block_bounds_kernel<128>, grid, dim3(kBoundThreads), 0, st, true, a);
}

// CTAs per item: while all items' come to at most two per SM, and no more than
// leave each warp its batch of blocks.  (b = 1, 8 heads, 512 blocks: 9.6 us with
// one, 6.9 with four, 6.4 with eight; CTAs of 512 threads 9.2, 6.9 and 6.9.)  Two
// CTAs fit an SM's shared memory up to about 7,000 blocks; longer rows of so many
// items run in two waves.
int select_cluster(int items, int NB, int D, int sms) {
  const int batch = kSelWarps * (32 / (2 * D / 8)) * kBatch;
  int c = 1;
  while (c < kSelMaxCluster && 2 * c * items <= 2 * sms && c * batch < NB) c *= 2;
  return c;
}

cudaError_t launch_select_blocks(SelectBlocksArgs a, int D, int sms, cudaStream_t st) {
  a.cluster = select_cluster(a.B * a.Hkv, a.NB, D, sms);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.Hkv * a.cluster, a.B);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = select_smem(a.NB);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.cluster > 1 ? 2 : 1;
  return D == 64 ? cudaLaunchKernelEx(&cfg, select_blocks_kernel<64>, a)
                 : cudaLaunchKernelEx(&cfg, select_blocks_kernel<128>, a);
}

cudaError_t allow_smem_blocks() {
  const int most = static_cast<int>(select_smem(kSelMaxBlocks));
  cudaError_t e = cudaFuncSetAttribute(select_blocks_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(select_blocks_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  return e;
}

}  // namespace dec
