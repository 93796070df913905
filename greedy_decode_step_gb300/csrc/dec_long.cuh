// Arguments and launches of the long-cache operators: the 4-bit KV cache
// (store, read-back, attention) and block-sparse attention (channel bounds,
// selection, attention over listed blocks).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dec_common.cuh"

namespace dec {

constexpr int kLongMaxBatch = 1024;   // rows of one call
constexpr int kBlockKeys = 64;        // keys of a selectable block
constexpr int kLongMaxCtas = 480;     // CTAs of one attention launch (three per SM, or one)
constexpr int kSelMaxBlocks = 8192;   // blocks of a row that the selection holds in shared memory

// Cluster barrier in two halves, and a store of a word at CTA 0's copy of a
// shared-memory address.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void store_cta0(const void* p, uint32_t v) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(at) : "r"(smem_addr(p)));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

// 4-bit cache.  Per (row, KV head, slot): D/2 bytes of codes (dim 2i in the
// low nibble of byte i, dim 2i + 1 in the high one) and per group of dims a
// half pair (scale s, middle z); code c stands for z + s (c - 8).
struct Kv4StoreArgs {
  const void* src[2];            // K rows, V rows
  uint8_t* codes[2];
  uint32_t* params[2];           // (s, z) half pairs
  const int32_t* pos;            // [B] first slot
  const int32_t* lens;           // [B] tokens of each row, or null: all T
  long long sb, st, sh;          // source strides (elements) of row, token, head
  int B, T, Hkv, S_max, from_cache, src_tokens;
  uint32_t* err;
};
struct Kv4LoadArgs {
  void* dst[2];
  const uint8_t* codes[2];
  const uint32_t* params[2];
  const int32_t* pos;
  const int32_t* lens;
  long long sb, st, sh;
  int B, T, Hkv, S_max;
  uint32_t* err;
};
cudaError_t launch_kv4_store(const Kv4StoreArgs& a, int D, int group, bool bf16, cudaStream_t st);
cudaError_t launch_kv4_load(const Kv4LoadArgs& a, int D, int group, bool bf16, cudaStream_t st);

// Decode attention over the 4-bit cache (blocks null) or over listed blocks
// of a bf16 cache.
struct LongAttnArgs {
  const float* q;                // [B][Hq][D]
  float* o;                      // [B][Hq][D]
  const int32_t* pos;            // [B], -1: a row without keys
  const void* k;                 // codes [B][Hkv][S_max][D/2] or bf16 [B][Hkv][S_max][D]
  const void* v;
  const uint32_t* kp;            // (s, z) pairs [B][Hkv][S_max][D/group]
  const uint32_t* vp;
  const int32_t* blocks;         // [B][Hkv][n_select] block ids, -1: none
  int n_select;
  float* part;                   // [2 * n_cta][G * (D + 2)]
  int B, Hq, Hkv, S_max;
  int G;                         // Hq / Hkv: set by the launch
  int n_cta;                     // CTAs of the balanced launch: set by the launch
  int cluster;                   // CTAs per (row, KV head), or 1: set by the launch
  float scale_log2;              // log2(e) / sqrt(D)
  uint32_t* err;
};
cudaError_t launch_long_attn(const LongAttnArgs& a, int D, int group, int sms, cudaStream_t st);
cudaError_t allow_smem_long();

// Per-block channel bounds of a bf16 key cache: bounds[b][g][j][0] the
// largest, [1] the smallest value of each dim over the block's slots.
struct BoundsArgs {
  const uint16_t* k;
  const int32_t* pos;            // [B] first of the T slots just written
  uint16_t* bounds;              // [B][Hkv][NB][2][D]
  int B, T, Hkv, S_max, NB;
  uint32_t* err;
};
cudaError_t launch_block_bounds(const BoundsArgs& a, int D, cudaStream_t st);

struct SelectBlocksArgs {
  const float* q;                // [B][Hq][D]
  const uint16_t* bounds;
  const int32_t* pos;            // [B] last key
  int32_t* blocks;               // [B][Hkv][n_select]
  int B, Hq, Hkv, S_max, NB, n_select, n_first, n_last;
  int cluster;                   // CTAs per (row, KV head): set by the launch
  uint32_t* err;
};
cudaError_t launch_select_blocks(SelectBlocksArgs a, int D, int sms, cudaStream_t st);
cudaError_t allow_smem_blocks();

}  // namespace dec
