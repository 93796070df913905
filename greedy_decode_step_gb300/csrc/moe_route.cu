// The router of a mixture-of-experts layer: logits, the k best experts of each
// token, and their weights.
//
//   z[e] = Wr[e] . y;  p = softmax over all experts of z, or sigmoid(z)
//   chosen: the k largest of p + bias, or of z without a bias (p grows with z);
//           equal ones by the lower id; NaN behind every number
//   weight: p, divided by the sum of the chosen ones' if asked, times scale
//
// A cluster of 8 CTAs per token, so that one launch serves: each CTA takes an
// eighth of the experts, a warp per expert, and puts the logits into CTA 0,
// whose first warp chooses.  The sums of different experts run in one order, so
// equal rows of Wr give equal logits.  Bound by latency: a warp's first 2048
// weights are on their way before the wait for the launch that makes y; each
// lane keeps the best of its own experts and looks anew only after it lost
// that one.
#include <cuda_runtime.h>

#include "dec_launch.cuh"
#include "dec_long.cuh"
#include "dec_moe.cuh"

namespace dec {
namespace {

constexpr int kRouteCluster = 8;
constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = kRouteThreads / 32;

constexpr int kRouteAhead = 8;  // 16-byte pieces of a row of Wr that a lane holds

// Eight products of bf16 weights, in four sums.
__device__ __forceinline__ void dot8(const uint4& w, const float* y, float (&acc)[4]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(y)), b = __ldg(reinterpret_cast<const float4*>(y + 4));
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
  __shared__ float z[kMoeMaxExperts];
  __shared__ uint32_t key[kMoeMaxExperts];
  const int rank = blockIdx.x % kRouteCluster, t = blockIdx.x / kRouteCluster;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const float* y = a.y + static_cast<size_t>(t) * a.H;
  uint4 w[kRouteAhead];
  auto fetch = [&](int e, int h0) {
#pragma unroll
    for (int i = 0; i < kRouteAhead; ++i) {
      const int h = h0 + (32 * i + lane) * 8;
      if (h < a.H) w[i] = __ldg(reinterpret_cast<const uint4*>(a.Wr + static_cast<size_t>(e) * a.H + h));
    }
  };
  const int e0 = rank * kRouteWarps + warp;
  if (e0 < a.E) fetch(e0, 0);  // no kernel writes the weights
  pdl_wait();
  pdl_launch_dependents();
  for (int e = e0; e < a.E; e += kRouteCluster * kRouteWarps) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int h0 = 0; h0 < a.H; h0 += kRouteAhead * 256) {
      if (e != e0 || h0 > 0) fetch(e, h0);
#pragma unroll
      for (int i = 0; i < kRouteAhead; ++i) {
        const int h = h0 + (32 * i + lane) * 8;
        if (h < a.H) dot8(w[i], y + h, acc);
      }
    }
    const float sum = warp_sum((acc[0] + acc[1]) + (acc[2] + acc[3]));
    if (lane == 0) store_cta0(z + e, __float_as_uint(sum));
  }
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  if (rank != 0 || warp != 0) return;

  float total = 1.f, top = 0.f;
  if (!a.sigmoid) {
    top = -INFINITY;
    for (int e = lane; e < a.E; e += 32) top = fmaxf(top, z[e]);
    top = warp_max(top);
    total = 0.f;
    for (int e = lane; e < a.E; e += 32) total += expf(z[e] - top);
    total = warp_sum(total);
  }
  auto score = [&](float v) { return a.sigmoid ? 1.f / (1.f + expf(-v)) : expf(v - top) / total; };
  uint32_t best = 0, at = 0;  // of this lane's experts
  for (int e = lane; e < a.E; e += 32) {
    const float v = (a.bias ? score(z[e]) + a.bias[e] : z[e]) + 0.f;   // -0 and 0 are equal
    const uint32_t o = v == v ? float_order_key(v) : 1u;                // 0: taken
    key[e] = o;
    if (o > best) {
      best = o;
      at = e;
    }
  }
  uint32_t mine = 0;
  for (int j = 0; j < a.k; ++j) {
    const uint32_t most = __reduce_max_sync(0xffffffffu, best);
    const uint32_t e = __reduce_min_sync(0xffffffffu, best == most ? at : 0xffffffffu);
    if (lane == j) mine = e;
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
  const float p = lane < a.k ? score(z[mine]) : 0.f;
  float sum = 1.f;
  if (a.renormalise) {
    sum = 0.f;
    for (int j = 0; j < a.k; ++j) sum += __shfl_sync(0xffffffffu, p, j);
  }
  if (lane < a.k) {
    a.ids[static_cast<size_t>(t) * a.k + lane] = static_cast<int>(mine);
    a.gates[static_cast<size_t>(t) * a.k + lane] = p / sum * a.scale;
  }
}

}  // namespace

cudaError_t launch_moe_route(const MoeRouteArgs& a, int T, cudaStream_t st) {
  return launch(moe_route_kernel, dim3(T * kRouteCluster), dim3(kRouteThreads), 0, st, true, a);
}

cudaError_t allow_smem_moe_route() {
  return prefer_max_carveout(moe_route_kernel);
}

}  // namespace dec
