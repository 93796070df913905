// The router of a mixture-of-experts layer: logits, the k best experts of each
// token, and their weights.
//
//   z[e] = Wr[e] . y;  p = softmax over all experts of z, or sigmoid(z)
//   chosen: the k largest of p + bias, or of z without a bias (p grows with z);
//           equal ones by the lower id; NaN behind every number
//   weight: p, divided by the sum of the chosen ones' if asked, times scale
//
// A cluster of 8 CTAs per token, so that one launch serves: each CTA takes an
// eighth of the experts, a warp per two experts with the token's row in shared
// memory, and puts the logits into CTA 0, which chooses.  The sums of different
// experts run in one order, so equal rows of Wr give equal logits.  Bound by
// latency: a warp's first weights, 4096 of each expert, are on their way to L2 before
// the wait for the launch that makes y; up to 256 experts are ranked at once, by
// counting the better ones of each (64 experts: 1200 cycles where eight rounds of a
// warp's maximum took 3000).
#include <cuda_runtime.h>

#include "dec_launch.cuh"
#include "dec_long.cuh"
#include "dec_moe.cuh"

namespace dec {
namespace {

constexpr int kRouteCluster = 8;
constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = kRouteThreads / 32;

constexpr int kRouteAhead = 16;   // 16-byte pieces of a row of Wr that a lane holds
constexpr int kRouteRanked = kRouteThreads;  // experts that are ranked at once

// Eight products of bf16 weights, in four sums.
__device__ __forceinline__ void dot8(const uint4& w, const float4& a, const float4& b, float (&acc)[4]) {
  acc[0] = fmaf(bf16lo(w.x), a.x, acc[0]);
  acc[1] = fmaf(bf16hi(w.x), a.y, acc[1]);
  acc[2] = fmaf(bf16lo(w.y), a.z, acc[2]);
  acc[3] = fmaf(bf16hi(w.y), a.w, acc[3]);
  acc[0] = fmaf(bf16lo(w.z), b.x, acc[0]);
  acc[1] = fmaf(bf16hi(w.z), b.y, acc[1]);
  acc[2] = fmaf(bf16lo(w.w), b.z, acc[2]);
  acc[3] = fmaf(bf16hi(w.w), b.w, acc[3]);
}

__global__ void __cluster_dims__(kRouteCluster, 1, 1) __launch_bounds__(kRouteThreads)
    moe_route_kernel(const MoeRouteArgs a) {
  extern __shared__ __align__(16) float4 y[];  // [ceil(H / 256)][2][32]: first and second halves of 32 pieces of 8
  __shared__ float z[kMoeMaxExperts];
  __shared__ __align__(16) uint32_t key[kMoeMaxExperts];
  __shared__ uint32_t chosen[32];
  const int rank = blockIdx.x % kRouteCluster, t = blockIdx.x / kRouteCluster;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  constexpr int kStep = kRouteCluster * kRouteWarps, kSpan = kRouteAhead * 256;
  uint4 w[2][kRouteAhead];
  auto fetch = [&](uint4(&to)[kRouteAhead], int e, int h0) {
    if (e >= a.E) return;
#pragma unroll
    for (int i = 0; i < kRouteAhead; ++i) {
      const int h = h0 + (32 * i + lane) * 8;
      if (h < a.H) to[i] = __ldg(reinterpret_cast<const uint4*>(a.Wr + static_cast<size_t>(e) * a.H + h));
    }
  };
  cluster_arrive();
  const int e0 = rank * kRouteWarps + warp;
  // two experts a warp at once: ahead of the wait into L2 only, as the launch ahead may be the one that writes them
  auto ask = [&](int e) {
    if (e >= a.E) return;
    for (int h = 64 * lane; h < min(a.H, kSpan); h += 64 * 32)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(a.Wr + static_cast<size_t>(e) * a.H + h));
  };
  ask(e0);
  ask(e0 + kStep);
  pdl_wait();
  pdl_launch_dependents();
  fetch(w[0], e0, 0);
  fetch(w[1], e0 + kStep, 0);
  for (int i = threadIdx.x; i < a.H / 4; i += kRouteThreads)
    y[(i / 64) * 64 + (i & 1) * 32 + (i / 2) % 32] = __ldg(reinterpret_cast<const float4*>(a.y + static_cast<size_t>(t) * a.H) + i);
  __syncthreads();
  cluster_wait();  // CTA 0 has started: its shared memory may be written
  for (int e = e0; e < a.E; e += 2 * kStep) {
    float acc[2][4] = {};
    for (int h0 = 0; h0 < a.H; h0 += kSpan) {
      if (e != e0 || h0 > 0) {
        fetch(w[0], e, h0);
        fetch(w[1], e + kStep, h0);
      }
#pragma unroll
      for (int i = 0; i < kRouteAhead; ++i) {
        const int h = h0 + (32 * i + lane) * 8;
        if (h < a.H) {
          const float4 lo = y[h0 / 4 + 64 * i + lane], hi = y[h0 / 4 + 64 * i + 32 + lane];
          dot8(w[0][i], lo, hi, acc[0]);
          if (e + kStep < a.E) dot8(w[1][i], lo, hi, acc[1]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float sum = warp_sum((acc[i][0] + acc[i][1]) + (acc[i][2] + acc[i][3]));
      if (lane == 0 && e + i * kStep < a.E) store_cta0(z + e + i * kStep, __float_as_uint(sum));
    }
  }
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  if (rank != 0) return;

  // every warp by itself: the softmax's largest logit and its sum, where scores are needed before the choice or whole
  const bool whole = !a.sigmoid && (a.bias || !a.renormalise);
  float top = 0.f, total = 1.f;
  if (whole) {
    top = -INFINITY;
    for (int e = lane; e < a.E; e += 32) top = fmaxf(top, z[e]);
    top = warp_max(top);
    total = 0.f;
    for (int e = lane; e < a.E; e += 32) total += expf(z[e] - top);
    total = warp_sum(total);
  }
  auto score = [&](float v) { return a.sigmoid ? 1.f / (1.f + expf(-v)) : expf(v - top) / total; };
  auto order = [&](int e) {
    const float v = (a.bias ? score(z[e]) + a.bias[e] : z[e]) + 0.f;  // -0 and 0 are equal
    return v == v ? float_order_key(v) : 1u;                           // 0: none, or taken
  };
  if (a.E <= kRouteRanked) {
    key[threadIdx.x] = threadIdx.x < a.E ? order(threadIdx.x) : 0u;
    __syncthreads();
    // 1 to 8 threads an expert, side by side, count the better ones among every so many fours
    const int log = a.E <= 32 ? 3 : a.E <= 64 ? 2 : a.E <= 128 ? 1 : 0, part = threadIdx.x & ((1 << log) - 1);
    const int e = threadIdx.x >> log;
    const uint32_t mine = key[e];
    int better = 0;
#pragma unroll 4
    for (int i = 4 * part; i < a.E; i += 4 << log) {  // behind the last: 0, better than none
      const uint4 o = *reinterpret_cast<const uint4*>(key + i);
      better += (o.x > mine || (o.x == mine && i < e)) + (o.y > mine || (o.y == mine && i + 1 < e)) +
                (o.z > mine || (o.z == mine && i + 2 < e)) + (o.w > mine || (o.w == mine && i + 3 < e));
    }
    for (int o = 1; o < 1 << log; o *= 2) better += __shfl_xor_sync(0xffffffffu, better, o);
    if (part == 0 && e < a.E && better < a.k) chosen[better] = e;
    __syncthreads();
    if (warp != 0) return;
  } else {
    if (warp != 0) return;
    uint32_t best = 0, at = 0;  // of this lane's experts; it looks anew only after it lost that one
    for (int e = lane; e < a.E; e += 32) {
      const uint32_t o = order(e);
      key[e] = o;
      if (o > best) {
        best = o;
        at = e;
      }
    }
    for (int j = 0; j < a.k; ++j) {
      const uint32_t most = __reduce_max_sync(0xffffffffu, best);
      const uint32_t e = __reduce_min_sync(0xffffffffu, best == most ? at : 0xffffffffu);
      if (lane == 0) chosen[j] = e;
      if (best == most && at == e) {
        key[e] = 0;
        best = 0;
        for (int i = lane; i < a.E; i += 32)
          if (key[i] > best) {
            best = key[i];
            at = i;
          }
      }
    }
    __syncwarp();
  }
  const uint32_t mine = lane < a.k ? chosen[lane] : 0u;
  const float v = z[mine], most = warp_max(lane < a.k ? v : -INFINITY);
  float p = 0.f;
  if (lane < a.k) {
    // Renormalised, a common factor of the chosen scores cancels: it is taken so that the largest is a half at least (1
    // for a softmax), however small they are.  For a sigmoid e^-c with c = min(0, the largest logit): e^v / (1 + e^v)
    // becomes e^(v - c) / (1 + e^v).
    if (!a.renormalise || !(total == total))  // as it is, or NaN for one among all the logits
      p = score(v);
    else if (!a.sigmoid)
      p = expf(v - most);
    else
      p = v >= 0.f ? score(v) : expf(v - fminf(most, 0.f)) / (1.f + expf(v));
  }
  const float sum = a.renormalise ? warp_sum(p) : 1.f;
  if (lane < a.k) {
    a.ids[static_cast<size_t>(t) * a.k + lane] = static_cast<int>(mine);
    a.gates[static_cast<size_t>(t) * a.k + lane] = p / sum * a.scale;
  }
}

}  // namespace

cudaError_t launch_moe_route(const MoeRouteArgs& a, int T, cudaStream_t st) {
  return launch(moe_route_kernel, dim3(T * kRouteCluster), dim3(kRouteThreads), (static_cast<size_t>(a.H) + 255) / 256 * 1024, st, true, a);
}

cudaError_t allow_smem_moe_route() {
  const cudaError_t e = cudaFuncSetAttribute(moe_route_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMoeMaxDim * 4);
  return e != cudaSuccess ? e : prefer_max_carveout(moe_route_kernel);
}

}  // namespace dec
