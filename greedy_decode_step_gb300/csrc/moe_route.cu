// The router of a mixture-of-experts layer: logits, the k best experts of each
// token, and their weights.
//
//   z[e] = Wr[e] . y;  p = softmax over all experts of z, or sigmoid(z)
//   chosen: the k largest of p + bias, or of z without a bias (p grows with z);
//           equal ones by the lower id; NaN behind every number
//   weight: p, divided by the sum of the chosen ones' if asked, times scale
//
// A cluster of 8 CTAs per token, so that one launch serves: each CTA takes an
// eighth of the experts, a warp per expert with the token's row in shared
// memory, and puts the logits into CTA 0, whose first warp chooses.  The sums
// of different experts run in one order, so equal rows of Wr give equal
// logits.  Bound by latency: the matrix (0.3 to 2 MB) comes from L2 for all
// tokens but the first to ask.
#include <cuda_runtime.h>

#include "dec_launch.cuh"
#include "dec_long.cuh"
#include "dec_moe.cuh"

namespace dec {
namespace {

constexpr int kRouteCluster = 8;
constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = kRouteThreads / 32;

// Eight products of bf16 weights, in four sums.
__device__ __forceinline__ void dot8(const uint4& w, const float* x, float (&acc)[4]) {
  const float4 a = *reinterpret_cast<const float4*>(x), b = *reinterpret_cast<const float4*>(x + 4);
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
  extern __shared__ __align__(16) float x[];  // [H]
  __shared__ float z[kMoeMaxExperts];
  __shared__ uint32_t key[kMoeMaxExperts];
  const int rank = blockIdx.x % kRouteCluster, t = blockIdx.x / kRouteCluster;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  pdl_wait();
  pdl_launch_dependents();
  const float* y = a.y + static_cast<size_t>(t) * a.H;
  for (int i = threadIdx.x * 4; i < a.H; i += kRouteThreads * 4)
    *reinterpret_cast<float4*>(x + i) = *reinterpret_cast<const float4*>(y + i);
  __syncthreads();
  for (int e = rank * kRouteWarps + warp; e < a.E; e += kRouteCluster * kRouteWarps) {
    const uint16_t* w = a.Wr + static_cast<size_t>(e) * a.H;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int h = lane * 8; h < a.H; h += 256) dot8(__ldg(reinterpret_cast<const uint4*>(w + h)), x + h, acc);
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
  for (int e = lane; e < a.E; e += 32) {
    const float v = (a.bias ? score(z[e]) + a.bias[e] : z[e]) + 0.f;  // -0 and 0 are equal
    key[e] = v == v ? float_order_key(v) : 1u;                         // 0: taken
  }
  __syncwarp();
  float mine = 0.f, sum = 0.f;
  int id = 0;
  for (int j = 0; j < a.k; ++j) {
    uint32_t best = 0, at = 0;
    for (int e = lane; e < a.E; e += 32)
      if (key[e] > best) {
        best = key[e];
        at = e;
      }
    const uint32_t most = __reduce_max_sync(0xffffffffu, best);
    const uint32_t e = __reduce_min_sync(0xffffffffu, best == most ? at : 0xffffffffu);
    const float p = score(z[e]);
    sum += p;
    if (lane == j) {
      mine = p;
      id = static_cast<int>(e);
    }
    __syncwarp();
    if (lane == 0) key[e] = 0;
    __syncwarp();
  }
  if (lane < a.k) {
    a.ids[static_cast<size_t>(t) * a.k + lane] = id;
    a.gates[static_cast<size_t>(t) * a.k + lane] = (a.renormalise ? mine / sum : mine) * a.scale;
  }
}

}  // namespace

cudaError_t launch_moe_route(const MoeRouteArgs& a, int T, cudaStream_t st) {
  return launch(moe_route_kernel, dim3(T * kRouteCluster), dim3(kRouteThreads), static_cast<size_t>(a.H) * 4, st, true, a);
}

cudaError_t allow_smem_moe_route() {
  cudaError_t e = cudaFuncSetAttribute(moe_route_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMoeMaxDim * 4);
  return e != cudaSuccess ? e : prefer_max_carveout(moe_route_kernel);
}

}  // namespace dec
