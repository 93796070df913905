// The router of a mixture-of-experts layer: logits, the k best experts of each
// token, and their weights.
//
//   z[e] = Wr[e] . y;  p = softmax over all experts of z, or sigmoid(z)
//   chosen: the k largest of p + bias, or of z without a bias (p grows with z);
//           equal ones by the lower id; NaN behind every number
//   weight: p, divided by the sum of the chosen ones' if asked, times scale
//
// Another expert is another result, so the choice is made as 64 bits make it.
// Logits are pairs of floats: a sum that starts at 1.5 2^m, m from the largest
// weight and value, takes whole steps of 2^(m - 23), and what each product
// leaves goes to a sum of its own (four operations a product in place of one).
// With W and Y the largest magnitudes, what the up to 40 products of such a sum leave is
// 2^-15 W Y each, added up in float32, so that a logit is off by 2^-34 H W Y at most (in
// random rows of 256 to 4096 by a thousandth of that, 2^-35 to 2^-38 of a logit).  Scores
// with a bias are compared in float32 first, and in doubles where two lie too close for
// it: there are two double operations a clock and SM.
//
// A cluster of 8 CTAs per token, so that one launch serves: each CTA takes an
// eighth of the experts, a warp for one after the other with the token's row in
// shared memory, and puts the logits into CTA 0, which chooses.  The sums of
// different experts run in one order, so equal rows of Wr give equal logits.
// Bound by latency, from 128 experts on by the instructions of the sums (76 for 8
// products of a warp, 2 a cycle and SM): one token of 2560, 64 experts 4.7 us, 16
// tokens and 128 experts 8.3 (3.4 and 7.2 with float32 sums and weights fetched
// ahead of the wait).  The first weights are on their way to L2 before the wait for
// the launch that makes y; the loops are short, as unrolled over a row they wait for
// their instructions (16 tokens, 1024 experts of 4096: 162 us, 87); up to 256
// experts are ranked at once, by counting the better ones of each (64 experts: 1200
// cycles where eight rounds of a warp's maximum took 3000).
#include <cuda_runtime.h>

#include <algorithm>

#include "dec_launch.cuh"
#include "dec_long.cuh"
#include "dec_moe.cuh"

namespace dec {
namespace {

constexpr int kRouteCluster = 8;
constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = kRouteThreads / 32;

constexpr int kRouteAhead = 20;   // 16-byte pieces of rows of Wr that a lane may have in flight
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

// A product onto a sum that stays within [2^m, 2^(m + 1)): the sum takes whole steps of 2^(m - 23), its difference is
// exact, and what is left of the product, half a step at most, goes to `low`.
__device__ __forceinline__ void add_product(float w, float x, float& sum, float& low) {
  const float to = fmaf(w, x, sum);
  low += fmaf(w, x, sum - to);
  sum = to;
}
__device__ __forceinline__ void dot8(const uint4& w, const float4& a, const float4& b, float (&acc)[4], float (&low)[4]) {
  add_product(bf16lo(w.x), a.x, acc[0], low[0]);
  add_product(bf16hi(w.x), a.y, acc[1], low[1]);
  add_product(bf16lo(w.y), a.z, acc[2], low[2]);
  add_product(bf16hi(w.y), a.w, acc[3], low[3]);
  add_product(bf16lo(w.z), b.x, acc[0], low[0]);
  add_product(bf16hi(w.z), b.y, acc[1], low[1]);
  add_product(bf16lo(w.w), b.z, acc[2], low[2]);
  add_product(bf16hi(w.w), b.w, acc[3], low[3]);
}

// a + b, and what its rounding leaves (Knuth, "The Art of Computer Programming", volume 2, section 4.2.2).
__device__ __forceinline__ float two_sum(float a, float b, float& left) {
  const float s = a + b, v = s - a;
  left = (a - (s - v)) + (b - v);
  return s;
}

// Bits of the largest magnitudes of pairs of bf16 values.
__device__ __forceinline__ uint32_t top_pairs(uint32_t top, const uint4& w) {
  const uint32_t k = 0x7FFF7FFFu;
  return __vmaxu2(top, __vmaxu2(__vmaxu2(w.x & k, w.y & k), __vmaxu2(w.z & k, w.w & k)));
}

// Monotone map of a double onto 64 bits; 1 << 32 for NaN, which only 0 (none, or taken) is behind.
__device__ __forceinline__ unsigned long long double_order_key(double v) {
  if (!(v == v)) return 1ull << 32;
  const long long u = __double_as_longlong(v + 0.0);  // -0 and 0 are equal
  return u < 0 ? ~static_cast<unsigned long long>(u) : static_cast<unsigned long long>(u) | (1ull << 63);
}

__global__ void __cluster_dims__(kRouteCluster, 1, 1) __launch_bounds__(kRouteThreads)
    moe_route_kernel(const MoeRouteArgs a) {
  // y as [ceil(H / 256)][2][32]: first and second halves of 32 pieces of 8; behind it the lanes' pieces of Wr
  extern __shared__ __align__(16) float4 y[];
  __shared__ float z[kMoeMaxExperts], zlow[kMoeMaxExperts];                      // logits: z + zlow
  __shared__ __align__(16) uint32_t key[kMoeMaxExperts], low[kMoeMaxExperts];    // upper and lower half of what ranks
  __shared__ uint32_t chosen[32], tops[kRouteWarps];
  __shared__ double parts[kRouteWarps];
  const int rank = blockIdx.x % kRouteCluster, t = blockIdx.x / kRouteCluster;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  constexpr int kStep = kRouteCluster * kRouteWarps;
  const int e0 = rank * kRouteWarps + warp, span = 256 * a.ahead;
  // this warp's work: experts e0, e0 + 64, ..., each in spans of its row
  struct Place {
    int e, h;
    __device__ __forceinline__ void next(int span, int H) {
      h += span;
      if (h >= H) {
        h = 0;
        e += kStep;
      }
    }
  };
  uint4* const pieces = reinterpret_cast<uint4*>(y + (a.H + 255) / 256 * 64) + warp * a.bufs * a.ahead * 32 + lane;
  auto fetch = [&](const Place& p, int buf) {  // what a lane brings it reads itself: no barrier
    if (p.e < a.E) {
      const uint16_t *from = a.Wr + static_cast<size_t>(p.e) * a.H, *end = from + min(a.H, p.h + span);
      uint32_t to = smem_addr(pieces + buf * a.ahead * 32);
#pragma unroll 4
      for (from += p.h + 8 * lane; from < end; from += 256, to += 512)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  cluster_arrive();
  Place now{e0, 0}, ahead = now;
  // ahead of the wait into L2 only, as the launch ahead may be the one that writes them
  for (int n = 0; n < 2 && ahead.e < a.E; ++n, ahead.next(span, a.H))
    for (int h = ahead.h + 64 * lane; h < min(a.H, ahead.h + span); h += 64 * 32)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(a.Wr + static_cast<size_t>(ahead.e) * a.H + h));
  pdl_wait();
  pdl_launch_dependents();
  fetch(now, 0);
  ahead = now;
  uint32_t largest = 0;  // bits of the largest |y|
  for (int i = threadIdx.x; i < a.H / 4; i += kRouteThreads) {
    const float4 v = *(reinterpret_cast<const float4*>(a.y + static_cast<size_t>(t) * a.H) + i);
    y[(i / 64) * 64 + (i & 1) * 32 + (i / 2) % 32] = v;
    const uint32_t k = 0x7FFFFFFFu;
    largest = max(largest, max(max(__float_as_uint(v.x) & k, __float_as_uint(v.y) & k),
                               max(__float_as_uint(v.z) & k, __float_as_uint(v.w) & k)));
  }
  largest = __reduce_max_sync(0xffffffffu, largest);
  if (lane == 0) tops[warp] = largest;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kRouteWarps; ++i) largest = max(largest, tops[i]);
  const int ye = static_cast<int>(largest >> 23);  // |y| < 2^(ye - 126)
  cluster_wait();  // CTA 0 has started: its shared memory may be written
  float hi = 0.f, lo = 0.f;
  for (int buf = 0; now.e < a.E; now.next(span, a.H), buf ^= 1) {
    ahead.next(span, a.H);
    fetch(ahead, buf ^ 1);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    const int h1 = min(a.H, now.h + span);
    const uint4* const first = pieces + buf * a.ahead * 32;
    const uint4* w = first;
    const float4* x = y + now.h / 4 + lane;
    uint32_t most = 0;
#pragma unroll 4
    for (int h = now.h + 8 * lane; h < h1; h += 256, w += 32) most = top_pairs(most, *w);
    w = first;
    most = max(most >> 16, most & 0xFFFFu);
    // a product is below 2^(we + ye - 252), a sum of 40 of them below 40 / 128 of 2^m
    const int we = static_cast<int>(most >> 7), m = we + ye - 118;  // exponents with their bias of 127
    const bool plain = __any_sync(0xffffffffu, we == 255 || ye == 255 || m > 253);
    const float from = plain ? 0.f : __uint_as_float((static_cast<uint32_t>(max(m, 27)) << 23) | 0x400000u);
    float acc[4], left[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      acc[j] = from;
      left[j] = 0.f;
    }
    if (!plain) {
#pragma unroll 2
      for (int h = now.h + 8 * lane; h < h1; h += 256, w += 32, x += 64) dot8(*w, x[0], x[32], acc, left);
    } else {  // infinities, NaN, sums near the largest float: as they come
      for (int h = now.h + 8 * lane; h < h1; h += 256, w += 32, x += 64) dot8(*w, x[0], x[32], acc);
    }
    float v;  // four sums of whole steps: exact
    hi = two_sum(hi, ((acc[0] - from) + (acc[1] - from)) + ((acc[2] - from) + (acc[3] - from)), v);
    lo += v + ((left[0] + left[1]) + (left[2] + left[3]));
    if (h1 < a.H) continue;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      hi = two_sum(hi, __shfl_xor_sync(0xffffffffu, hi, o), v);
      lo = (lo + __shfl_xor_sync(0xffffffffu, lo, o)) + v;
    }
    float sum = two_sum(hi, lo, v);
    if (!(fabsf(v) < INFINITY)) {  // an infinity or NaN is its own first half
      sum = hi;
      v = 0.f;
    }
    if (lane == 0) {
      store_cta0(z + now.e, __float_as_uint(sum));
      store_cta0(zlow + now.e, __float_as_uint(v));
    }
    hi = lo = 0.f;
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
    for (int e = lane; e < a.E; e += 32) total += expf((z[e] - top) + zlow[e]);
    total = warp_sum(total);
  }
  // e^(v + l - c) / (1 + e^(v + l)) for c <= 0, c == 0 where v > 0
  auto sigmoid = [](float v, float l, float c) {
    if (v >= 0.f) {
      const float x = expf(-v);
      return 1.f / (1.f + fmaf(-x, l, x));
    }
    const float x = expf(v), x1 = fmaf(x, l, x);
    return (c == 0.f ? x1 : expf((v - c) + l)) / (1.f + x1);
  };
  auto score = [&](float v, float l) { return a.sigmoid ? sigmoid(v, l, 0.f) : expf((v - top) + l) / total; };
  // Without a bias the logits rank, both halves.  With one, p + bias in float32 where that tells the chosen ones from
  // each other and from the others, else in 64 bits.  `reach`: what two such sums may be off by together (a score a
  // few 2^-24 of the largest; a softmax's sum has up to 1024 terms).
  for (int e = threadIdx.x; e < max(a.E, kRouteRanked); e += kRouteThreads) {
    const float v = e < a.E ? (a.bias ? score(z[e], zlow[e]) + a.bias[e] : z[e]) + 0.f : 0.f;  // -0 and 0 are equal
    key[e] = e >= a.E ? 0u : v == v ? float_order_key(v) : 1u;                                 // 0: none, or taken
    low[e] = e >= a.E || a.bias ? 0u : float_order_key(zlow[e] + 0.f);
  }
  const float wide = a.sigmoid ? 0x1p-19f : 0x1p-16f / total;
  auto reach = [&](float v) { return fmaf(0x1p-21f, fabsf(v), wide); };
  auto fill64 = [&] {  // every thread of CTA 0
    double most = 0.0, sum = 1.0;
    if (!a.sigmoid) {
      // any shift near the largest logit does
      most = static_cast<double>(top);
      sum = 0.0;
      for (int e = threadIdx.x; e < a.E; e += kRouteThreads) sum += exp(static_cast<double>(z[e]) + zlow[e] - most);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) parts[warp] = sum;
      __syncthreads();
      sum = 0.0;
#pragma unroll
      for (int i = 0; i < kRouteWarps; ++i) sum += parts[i];
    }
    for (int e = threadIdx.x; e < a.E; e += kRouteThreads) {
      const double v = static_cast<double>(z[e]) + zlow[e], p = a.sigmoid ? 1.0 / (1.0 + exp(-v)) : exp(v - most) / sum;
      const unsigned long long o = double_order_key(p + static_cast<double>(a.bias[e]));
      key[e] = static_cast<uint32_t>(o >> 32);
      low[e] = static_cast<uint32_t>(o);
    }
  };
  for (bool first = a.bias != nullptr;; first = false) {
    __syncthreads();
    bool unsure = false;
    if (a.E <= kRouteRanked) {
      // 1 to 8 threads an expert, side by side, count the better ones among every so many fours
      const int log = a.E <= 32 ? 3 : a.E <= 64 ? 2 : a.E <= 128 ? 1 : 0, part = threadIdx.x & ((1 << log) - 1);
      const int e = threadIdx.x >> log;
      const uint32_t mine = key[e];
      uint32_t bound = mine;  // those from here on, up to its own place, are not told from it
      if (first && mine > 1u) {
        const float v = float_from_order_key(mine), at = v - reach(v);
        if (at == at) bound = float_order_key(at);
      }
      int better = 0, within = 0;
#pragma unroll 4
      for (int i = 4 * part; i < a.E; i += 4 << log) {  // behind the last: 0, better than none
        const uint4 o = *reinterpret_cast<const uint4*>(key + i);
        better += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
        within += (o.x >= bound) + (o.y >= bound) + (o.z >= bound) + (o.w >= bound);
      }
      for (int o = 1; o < 1 << log; o *= 2) {
        better += __shfl_xor_sync(0xffffffffu, better, o);
        within += __shfl_xor_sync(0xffffffffu, within, o);
      }
      if (e < a.E && better < a.k && within > better + 1) {
        unsure = first;
        if (!first)  // equal upper halves: the lower ones, then the lower id
          for (int i = 0; i < a.E; ++i)
            if (key[i] == mine && (low[i] > low[e] || (low[i] == low[e] && i < e))) ++better;
      }
      if (part == 0 && e < a.E && better < a.k) chosen[better] = e;
    } else if (warp == 0) {
      uint32_t best = 0, rest = 0, at = 0;  // of this lane's experts; it looks anew only after it lost that one
      auto look = [&] {
        best = rest = 0;
        for (int e = lane; e < a.E; e += 32)
          if (key[e] > best || (key[e] == best && low[e] > rest)) {
            best = key[e];
            rest = low[e];
            at = e;
          }
      };
      look();
      float before = 0.f;
      for (int j = 0; j < min(a.k + first, a.E); ++j) {
        const uint32_t most = __reduce_max_sync(0xffffffffu, best);
        const uint32_t next = __reduce_max_sync(0xffffffffu, best == most ? rest : 0u);
        const uint32_t e = __reduce_min_sync(0xffffffffu, best == most && rest == next ? at : 0xffffffffu);
        if (lane == 0) chosen[j] = e;
        const float v = float_from_order_key(most);
        unsure = unsure || (first && j > 0 && before - v <= reach(before));
        before = v;
        if (best == most && at == e) {
          key[e] = 0;
          look();
        }
      }
    }
    if (!__syncthreads_or(unsure)) break;
    fill64();
  }
  if (warp != 0) return;
  const uint32_t mine = lane < a.k ? chosen[lane] : 0u;
  const float v = z[mine], l = zlow[mine], most = warp_max(lane < a.k ? v : -INFINITY);
  float p = 0.f;
  if (lane < a.k) {
    // Renormalised, a common factor of the chosen scores cancels: it is taken so that the largest is a half at least (1
    // for a softmax), however small they are.  For a sigmoid it is e^-c with c = min(0, the largest logit).
    if (!a.renormalise || !(total == total))  // as it is, or NaN for one among all the logits
      p = score(v, l);
    else
      p = a.sigmoid ? sigmoid(v, l, fminf(most, 0.f)) : expf((v - most) + l);
  }
  const float sum = a.renormalise ? warp_sum(p) : 1.f;
  if (lane < a.k) {
    a.ids[static_cast<size_t>(t) * a.k + lane] = static_cast<int>(mine);
    a.gates[static_cast<size_t>(t) * a.k + lane] = p / sum * a.scale;
  }
}

}  // namespace

cudaError_t launch_moe_route(const MoeRouteArgs& call, int T, cudaStream_t st) {
  MoeRouteArgs a = call;
  // all of a warp's pieces in flight if they fit, else two buffers of equal spans in turn; 80 KB, so that two CTAs fit an
  // SM up to H = 4096 (15 clusters are resident with one: 16 tokens, 1024 experts of 4096 took 92 us where 87)
  const int all = (a.H + 255) / 256;
  a.bufs = all <= kRouteAhead && a.E <= kRouteCluster * kRouteWarps ? 1 : 2;
  const int spans = (all + kRouteAhead / a.bufs - 1) / (kRouteAhead / a.bufs);
  a.ahead = (all + spans - 1) / spans;
  const size_t smem = all * 1024 + static_cast<size_t>(kRouteWarps) * a.bufs * a.ahead * 512;
  return launch(moe_route_kernel, dim3(T * kRouteCluster), dim3(kRouteThreads), smem, st, true, a);
}

cudaError_t allow_smem_moe_route() {
  const cudaError_t e = cudaFuncSetAttribute(moe_route_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kMoeMaxDim * 4 + kRouteWarps * kRouteAhead * 512);
  return e != cudaSuccess ? e : prefer_max_carveout(moe_route_kernel);
}

}  // namespace dec
