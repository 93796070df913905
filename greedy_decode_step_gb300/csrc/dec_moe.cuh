// Arguments and launches of the mixture-of-experts layer: the router's choice
// and the chosen experts' gated MLPs for a decode step's few tokens.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dec_common.cuh"

namespace dec {

constexpr int kMoeMaxTokens = 16;
constexpr int kMoeMaxChoices = 16;    // experts per token
constexpr int kMoeMaxExperts = 1024;
constexpr int kMoeMaxDim = 32768;     // hidden and intermediate sizes
constexpr int kMoeMaxCtas = 320;      // CTAs of the gate/up launch: two per SM
constexpr int kMoeUnit = 64;          // gate rows (and up rows) of one tile

struct MoeRouteArgs {
  const float* y;                // [T][H]
  const uint16_t* Wr;            // bf16 [E][H]
  const float* bias;             // [E] or null
  int32_t* ids;                  // [T][k]
  float* gates;                  // [T][k]
  int H, E, k, sigmoid, renormalise;
  float scale;
  int ahead, bufs;               // pieces in flight and buffers of a warp: set by the launch
};
cudaError_t launch_moe_route(const MoeRouteArgs& a, int T, cudaStream_t st);
cudaError_t allow_smem_moe_route();

struct MoeCall {
  const float* y;                // [T][H]
  const int32_t* ids;            // [T][k], -1: none
  const float* gates;            // [T][k]
  const void *wg, *wu, *wd;      // [E][I][H], [E][I][H], [E][H][I]: bf16, or e4m3 codes with scales
  const float *sg, *su, *sd;     // [E][ceil(rows / 128)][ceil(columns / 128)], null for bf16
  const float* residual;         // [T][H] or null
  float* out;                    // [T][H]
  unsigned char* ws;
  int T, k, E, H, I;
  uint32_t* err;
};
// Workspace (byte offsets): the plan; gate and up products of every chosen
// (token, expert); the parts of tiles that a CTA took over from the one before
// it; the sums of the down launch's CTAs; the split rows of y and of the inner vectors, 1 KB per token and 64 or
// 128 values.
constexpr int kMoeRows = kMoeMaxTokens * kMoeMaxChoices;  // (token, expert) pairs
constexpr int kMoePlanBytes = 4096;
struct MoeWorkspace {
  size_t main, cut, sums, xb, hb, bytes;
};
inline MoeWorkspace moe_workspace(int T, int k, int H, int I) {
  auto up = [](size_t n) { return (n + 1023) & ~size_t(1023); };
  MoeWorkspace w;
  w.main = kMoePlanBytes;
  w.cut = w.main + up(static_cast<size_t>(T) * k * 2 * I * 4);
  w.sums = w.cut + static_cast<size_t>(kMoeMaxCtas) * kMoeMaxTokens * 2 * kMoeUnit * 4;
  w.xb = w.sums + static_cast<size_t>(kMoeMaxCtas) * kMoeMaxTokens * 128 * 4;
  w.hb = w.xb + static_cast<size_t>(T) * ((H + 63) / 64) * 1024;
  w.bytes = w.hb + static_cast<size_t>(T) * k * ((I + 63) / 64) * 1024;
  return w;
}
// 0, or 1 (*why says why) or 3 (a CUDA error)
int moe_experts(const MoeCall& c, int sms, cudaStream_t st, const char** why);
cudaError_t allow_smem_moe();

}  // namespace dec
