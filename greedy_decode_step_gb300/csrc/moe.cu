// The experts of a mixture-of-experts layer for a decode step's few tokens:
//
//   out[t] = res[t] + sum over experts e chosen by t, gate weight w:
//            Wd[e] (w silu(Wg[e] y[t]) * (Wu[e] y[t]))
//
// in two launches, gate/up and down, both bound by the stream of the chosen
// experts' weights: each is read once, whatever number of tokens chose it.
//
// The products run on the tensor cores with weight rows on the 128 lanes of an
// accumulator and the tokens on its columns (tcgen05.mma, M = 128).  fp32
// activations are kept whole by giving every token several columns: its row is
// split into parts whose products with the weights are exact and whose columns
// are added at the end.
//   * bf16 weights: three bf16 parts (24 bits);
//   * e4m3 weights: five e4m3 parts, each 2^-5 of the one before, of x / s with s
//     a power of two per token and 128 values (what is left is 2^-23 of the
//     largest of the 128); every 128 values the column sums leave tensor memory
//     to meet s and the weights' own block scale in fp32.
// The parts are made in shared memory beside the weight stream, by four warps
// that each take every fourth 128-byte chunk of K; columns cost little: 16 for
// one or two tokens, 48 (bf16) or 80 (e4m3) for 16, next to 128 weight rows.
//
// gate/up: a tile is 64 gate rows and the same 64 up rows of an expert.  How
// many experts are active is known on the device only, so a persistent grid
// lays all tiles' chunks end to end and gives every CTA an equal run of them;
// a tile cut between CTAs leaves parts, which the down launch adds, in CTA
// order, as it reads them.
// down: a tile is 128 output rows, its K axis all active experts' h one behind
// the other, split over a cluster of CTAs whose sums meet in distributed shared
// memory in rank order: results do not depend on timing.  Its first weights
// are on their way while gate/up still runs.
//
// Every wait is bounded (an error bit and an early exit instead of a hang),
// and tensor memory is released on every path.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <mutex>

#include "dec_fp8.cuh"
#include "dec_launch.cuh"
#include "dec_moe.cuh"
#include "dec_tc.cuh"

namespace dec {
namespace {

constexpr int kMoeThreads = 320;      // warp 0 copies, 1 multiplies, 2-5 take sums off, 6-9 split rows into parts
constexpr int kMoeSplitWarps = 4;
constexpr uint32_t kMoeATile = 128 * 128;
constexpr int kMoeRows = kMoeMaxTokens * kMoeMaxChoices;  // (token, expert) pairs
constexpr uint32_t kMoeSmemMax = 112 * 1024;              // both launches' CTAs share an SM
constexpr int kMoeMaxStages = 8;
constexpr int kMoeMaxSplits = 8;

template <bool F8, int NT>
struct Shape {
  static constexpr int kParts = F8 ? 5 : 3;
  static constexpr int kN = (kParts * NT + 15) / 16 * 16;   // columns of the MMA
  static constexpr int kChunk = F8 ? 128 : 64;              // values of K per 128-byte row
  static constexpr int kVals = kChunk / 32;                 // of them per lane of a splitting warp
  static constexpr uint32_t kBTile = kN * 128;
  static constexpr int kBStages = kMoeSplitWarps;
  static constexpr int kScaleSlots = kBStages + 2;
};

struct MoeArgs {
  CUtensorMap g, u, d;           // boxes of 64, 64 and 128 rows
  const float* y;
  const int32_t* ids;
  const float* gates;
  const float *sg, *su, *sd;
  const float* residual;
  float* out;
  float *main, *cut;             // workspace
  int T, k, E, H, I;
  int ctas;                      // of the gate/up launch
  int splits, stages;
  uint32_t* err;
};

// What both launches derive from the ids: the active experts in ascending
// order, the tokens of each and where their rows begin.
struct Plan {
  uint32_t chosen[kMoeMaxExperts / 2];   // 16 token bits per expert
  uint16_t expert[kMoeRows], tokens[kMoeRows], first[kMoeRows];
  float gate[kMoeRows];                  // per row (down)
  int active;
};

// Called by all threads; ends with a barrier.
__device__ __forceinline__ void make_plan(Plan& p, const MoeArgs& a, bool gates) {
  const int n = a.T * a.k;
  for (int i = threadIdx.x; i < (a.E + 1) / 2; i += kMoeThreads) p.chosen[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kMoeThreads) {
    const int e = a.ids[i];
    if (e >= 0 && e < a.E)
      atomicOr(&p.chosen[e >> 1], (1u << (i / a.k)) << (16 * (e & 1)));
    else if (e != -1 && blockIdx.x == 0)
      atomicOr(a.err, kErrPosRange);
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int active = 0, rows = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      const uint32_t m = e < a.E ? (p.chosen[e >> 1] >> (16 * (e & 1))) & 0xFFFFu : 0u;
      const uint32_t any = __ballot_sync(0xffffffffu, m != 0);
      if (any == 0) continue;
      const int c = __popc(m);
      int upto = c;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      if (m) {
        const int at = active + __popc(any & ((1u << lane) - 1));
        p.expert[at] = static_cast<uint16_t>(e);
        p.tokens[at] = static_cast<uint16_t>(m);
        p.first[at] = static_cast<uint16_t>(rows + upto - c);
      }
      active += __popc(any);
      rows += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (lane == 0) p.active = active;
  }
  __syncthreads();
  if (gates) {
    for (int i = threadIdx.x; i < p.active * kMoeMaxTokens; i += kMoeThreads) {
      const int at = i / kMoeMaxTokens, t = i % kMoeMaxTokens;
      const uint32_t m = p.tokens[at];
      if (!((m >> t) & 1u)) continue;
      float w = 0.f;  // an expert that a token lists twice counts twice
      for (int j = 0; j < a.k; ++j)
        if (a.ids[t * a.k + j] == p.expert[at]) w += a.gates[t * a.k + j];
      p.gate[p.first[at] + __popc(m & ((1u << t) - 1))] = w;
    }
    __syncthreads();
  }
}

// The runs of gate/up: W chunks over n CTAs.  A run is at least an eighth of a
// tile's K axis, so that a tile is cut into nine parts at most.
struct Runs {
  long long W;
  int n, kch, units;
  __device__ __forceinline__ Runs(const Plan& p, const MoeArgs& a, int chunk) {
    kch = (a.H + chunk - 1) / chunk;
    units = (a.I + kMoeUnit - 1) / kMoeUnit;
    const long long tiles = static_cast<long long>(p.active) * units;
    W = tiles * kch;
    n = static_cast<int>(min(static_cast<long long>(a.ctas), min(8 * tiles, W)));  // no run is empty
  }
  __device__ __forceinline__ int begin(int c) const { return c >= n ? static_cast<int>(W) : static_cast<int>(W * c / n); }
  __device__ __forceinline__ int owner(long long pos) const { return static_cast<int>(((pos + 1) * n - 1) / W); }
};

// ----------------------------------------------------------------------------- parts of an activation row

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Byte offset of this lane's 4 bytes in row `row` of a swizzled tile.
__device__ __forceinline__ uint32_t part_at(int row, int lane) {
  return row * 128 + ((((lane >> 2) ^ row) & 7) << 4) + ((lane & 3) << 2);
}

// Three bf16 parts of this lane's two values into rows t, NT + t, 2 NT + t.
template <int NT>
__device__ __forceinline__ void put_parts(unsigned char* tile, int t, int lane, const float (&x)[2]) {
  float a = x[0], b = x[1];
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    const uint32_t w = pack_bf16(a, b);
    *reinterpret_cast<uint32_t*>(tile + part_at(p * NT + t, lane)) = w;
    a -= bf16lo(w);
    b -= bf16hi(w);
  }
}

// Five e4m3 parts of this lane's four values; returns s (the same in all lanes).
// s: the largest magnitude of the 128 is at most 224 s, so that what a part
// leaves, half a step of at most 16, is at most 8 and 2^5 of it fits again.
template <int NT>
__device__ __forceinline__ float put_parts(unsigned char* tile, int t, int lane, const float (&x)[4]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = __float_as_uint(x[i]) & 0x7FFFFFFFu;
    top = max(top, b < 0x7F800000u ? b : 0u);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  const int e = min(max(static_cast<int>(top >> 23) - 7 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0), 1), 253);
  const float inv = __uint_as_float((254u - e) << 23);
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = x[i] * inv;
    if (!(fabsf(v[i]) <= 448.f)) v[i] = __uint_as_float(0x7FFFFFFFu);  // an infinity: NaN
  }
#pragma unroll
  for (int p = 0; p < 5; ++p) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(v[1]), "f"(v[0]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v[3]), "f"(v[2]));
    *reinterpret_cast<uint32_t*>(tile + part_at(p * NT + t, lane)) = lo | (static_cast<uint32_t>(hi) << 16);
    if (p < 4) {
      uint32_t h0, h1;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h0) : "h"(lo));
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h1) : "h"(hi));
      const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&h0));
      const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&h1));
      v[0] = (v[0] - f0.x) * 32.f;
      v[1] = (v[1] - f0.y) * 32.f;
      v[2] = (v[2] - f1.x) * 32.f;
      v[3] = (v[3] - f1.y) * 32.f;
    }
  }
  return __uint_as_float(static_cast<uint32_t>(e) << 23);
}

template <int NT, int PARTS>
__device__ __forceinline__ void put_zeros(unsigned char* tile, int t, int lane) {
#pragma unroll
  for (int p = 0; p < PARTS; ++p) *reinterpret_cast<uint32_t*>(tile + part_at(p * NT + t, lane)) = 0;
}

// The accumulator's columns of this thread's lane, parts added per token, the smallest first.
template <bool F8, int NT>
__device__ __forceinline__ void take_sums(uint32_t taddr, float (&s)[NT]) {
  using S = Shape<F8, NT>;
  uint32_t v[S::kN / 16][16];
#pragma unroll
  for (int c = 0; c < S::kN / 16; ++c) tmem_ld_issue(taddr + 16 * c, v[c]);
#pragma unroll
  for (int c = 0; c < S::kN / 16; ++c) tmem_ld_wait(v[c]);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float r = 0.f;
#pragma unroll
    for (int p = S::kParts - 1; p >= 0; --p) {
      const float x = __uint_as_float(v[(p * NT + t) / 16][(p * NT + t) % 16]);
      r = F8 ? fmaf(r, 0.03125f, x) : r + x;
    }
    s[t] = r;
  }
}

// ----------------------------------------------------------------------------- shared state of a CTA

template <bool F8, int NT>
struct Cta {
  using S = Shape<F8, NT>;
  uint64_t *fullA, *emptyA, *fullB, *emptyB, *accum, *drained;
  uint32_t* tmem_slot;
  volatile int* stop;
  float (*scales)[kMoeMaxTokens];  // [kScaleSlots] s of every token of a chunk
  Plan* plan;
  unsigned char *A, *B;
  int stages;

  static constexpr uint32_t kHead = 1024, kPlan = (sizeof(Plan) + 1023) / 1024 * 1024;
  static constexpr int kStages = static_cast<int>((kMoeSmemMax - 1024 - kHead - kPlan - S::kBStages * S::kBTile) / kMoeATile) <
                                         kMoeMaxStages
                                     ? static_cast<int>((kMoeSmemMax - 1024 - kHead - kPlan - S::kBStages * S::kBTile) /
                                                        kMoeATile)
                                     : kMoeMaxStages;
  static constexpr uint32_t kSmem = 1024 + kHead + kPlan + S::kBStages * S::kBTile + kStages * kMoeATile;
  static constexpr uint32_t kCols = tmem_columns(2 * S::kN);

  __device__ __forceinline__ explicit Cta(unsigned char* raw) {
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    fullA = reinterpret_cast<uint64_t*>(smem);
    emptyA = fullA + kMoeMaxStages;
    fullB = emptyA + kMoeMaxStages;
    emptyB = fullB + S::kBStages;
    accum = emptyB + S::kBStages;
    drained = accum + 2;
    tmem_slot = reinterpret_cast<uint32_t*>(drained + 2);
    stop = reinterpret_cast<volatile int*>(tmem_slot + 1);
    scales = reinterpret_cast<float(*)[kMoeMaxTokens]>(smem + 512);
    static_assert((2 * kMoeMaxStages + 2 * S::kBStages + 4) * 8 + 8 <= 512, "barriers");
    static_assert(512 + S::kScaleSlots * kMoeMaxTokens * 4 <= kHead, "scales");
    plan = reinterpret_cast<Plan*>(smem + kHead);
    A = smem + kHead + kPlan;
    B = A + kStages * kMoeATile;
  }
  // All threads; returns the accumulators' address.
  __device__ __forceinline__ uint32_t begin() {
    if (threadIdx.x == 0) {
      for (int s = 0; s < kStages; ++s) {
        mbar_init(&fullA[s], 1);
        mbar_init(&emptyA[s], 1);
      }
      for (int s = 0; s < S::kBStages; ++s) {
        mbar_init(&fullB[s], 1);
        mbar_init(&emptyB[s], 1);
      }
      for (int s = 0; s < 2; ++s) {
        mbar_init(&accum[s], 1);
        mbar_init(&drained[s], 4);
      }
      *stop = 0;
      fence_mbar_init();
    }
    if (threadIdx.x / 32 == 1) tmem_alloc(tmem_slot, kCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    return *tmem_slot;
  }
  __device__ __forceinline__ void end(uint32_t tmem) {
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x / 32 == 1) {
      tc_fence_after();
      tmem_free(tmem, kCols);
    }
  }
  // Whole warp: waits in lane 0, one answer for all.
  __device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t* err, uint32_t code) const {
    int ok = 1;
    if (threadIdx.x % 32 == 0) ok = (mbar_wait(bar, parity, stop, err, code) && !*stop) ? 1 : 0;
    return __shfl_sync(0xffffffffu, ok, 0) != 0;
  }
  // One lane: the copies of the last stages have landed (an early end must not leave them in flight).
  __device__ __forceinline__ void drain(int issued, uint32_t* err) const {
    for (int i = max(0, issued - kStages); i < issued; ++i)
      if (!tc_wait(&fullA[i % kStages], (i / kStages) & 1, err, kErrDrain)) break;
  }
  // One lane: the MMAs of chunk `it` into the accumulator at `d`; false when a wait ran out.
  __device__ __forceinline__ bool multiply(int it, uint32_t d, bool fresh, uint32_t* err) const {
    const int s = it % kStages, b = it % S::kBStages;
    if (!mbar_wait(&fullA[s], (it / kStages) & 1, stop, err, kErrWaitFull) ||
        !mbar_wait(&fullB[b], (it / S::kBStages) & 1, stop, err, kErrWaitFull) || *stop)
      return false;
    tc_fence_after();
    const uint32_t sa = smem_addr(A + s * kMoeATile), sb = smem_addr(B + b * S::kBTile);
    constexpr uint32_t idesc = tc_idesc_of(S::kN, !F8);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {  // 32 bytes of K per instruction
      const uint64_t ad = smem_desc_sw128(sa + kk * 32), bd = smem_desc_sw128(sb + kk * 32);
      const uint32_t more = !fresh || kk > 0;
      if (F8)
        tc_mma_f8(d, ad, bd, idesc, more);
      else
        tc_mma(d, ad, bd, idesc, more);
    }
    tc_commit(&emptyA[s]);
    tc_commit(&emptyB[b]);
    return true;
  }
};

// ----------------------------------------------------------------------------- gate/up

template <bool F8, int NT>
__global__ void __launch_bounds__(kMoeThreads, 1) moe_gate_up_kernel(const __grid_constant__ MoeArgs a) {
  using S = Shape<F8, NT>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Cta<F8, NT> c(smem_raw);
  const uint32_t tmem = c.begin();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  const Plan& p = *c.plan;
  make_plan(*c.plan, a, false);
  const Runs r(p, a, S::kChunk);
  const int lo = r.begin(blockIdx.x), hi = r.begin(blockIdx.x + 1);

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol = l2_policy_evict_first();
      int it = 0;
      for (int pos = lo; pos < hi && !*c.stop;) {
        const int tile = pos / r.kch, j0 = pos - tile * r.kch, n = min(r.kch - j0, hi - pos);
        const int row = (tile % r.units) * kMoeUnit, e = p.expert[tile / r.units];
        for (int j = j0; j < j0 + n; ++j, ++it) {
          const int s = it % c.kStages;
          if (it >= c.kStages && !mbar_wait(&c.emptyA[s], ((it / c.kStages) - 1) & 1, c.stop, a.err, kErrWaitEmpty))
            *c.stop = 1;
          if (*c.stop) break;
          mbar_arrive_expect_tx(&c.fullA[s], kMoeATile);
          tma_load_3d(c.A + s * kMoeATile, &a.g, j * S::kChunk, row, e, &c.fullA[s], pol);
          tma_load_3d(c.A + s * kMoeATile + kMoeATile / 2, &a.u, j * S::kChunk, row, e, &c.fullA[s], pol);
        }
        pos += n;
      }
      if (*c.stop) c.drain(it, a.err);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int it = 0, seg = 0;
      for (int pos = lo; pos < hi && !*c.stop; ++seg) {
        const int j0 = pos % r.kch, n = min(r.kch - j0, hi - pos);
        for (int j = 0; j < n; ++j, ++it) {
          // e4m3: an accumulator per chunk; bf16: per tile
          const int b = (F8 ? it : seg) & 1, turn = (F8 ? it : seg) >> 1;
          if ((F8 || j == 0) && turn > 0 &&
              !mbar_wait(&c.drained[b], (turn - 1) & 1, c.stop, a.err, kErrWaitFull))
            *c.stop = 1;
          if (*c.stop || !c.multiply(it, tmem + b * S::kN, F8 || j == 0, a.err)) {
            *c.stop = 1;
            break;
          }
          if (F8 || j + 1 == n) tc_commit(&c.accum[b]);
        }
        pos += n;
      }
    }
  } else if (warp < 6) {
    const int q = warp & 3, m = 32 * q + lane;  // TMEM lanes; row of the tile: gate below 64, up from 64 on
    const uint32_t at = tmem + (static_cast<uint32_t>(32 * q) << 16);
    const int IB = (a.I + kFp8Block - 1) / kFp8Block;
    int it = 0, seg = 0;
    bool ok = true;
    for (int pos = lo; pos < hi && ok; ++seg) {
      const int tile = pos / r.kch, j0 = pos - tile * r.kch, n = min(r.kch - j0, hi - pos);
      const int act = tile / r.units, ub = tile - act * r.units;
      const uint32_t tokens = p.tokens[act];
      float sum[NT];
      if (F8) {
#pragma unroll
        for (int t = 0; t < NT; ++t) sum[t] = 0.f;
        const float* sw = (m < kMoeUnit ? a.sg : a.su) +
                          (static_cast<size_t>(p.expert[act]) * IB + ub * kMoeUnit / kFp8Block) * r.kch;
        float next = __ldg(sw + j0);
        for (int j = j0; j < j0 + n; ++j, ++it) {
          const float w = next;
          if (j + 1 < j0 + n) next = __ldg(sw + j + 1);
          ok = c.warp_wait(&c.accum[it & 1], (it >> 1) & 1, a.err, kErrWaitFull);
          if (!ok) break;
          tc_fence_after();
          float part[NT];
          take_sums<F8, NT>(at + (it & 1) * S::kN, part);
          const float* sx = c.scales[it % S::kScaleSlots];
#pragma unroll
          for (int t = 0; t < NT; ++t) sum[t] = fmaf(part[t], w * sx[t], sum[t]);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&c.drained[it & 1]);
        }
      } else {
        ok = c.warp_wait(&c.accum[seg & 1], (seg >> 1) & 1, a.err, kErrWaitFull);
        if (ok) {
          tc_fence_after();
          take_sums<F8, NT>(at + (seg & 1) * S::kN, sum);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&c.drained[seg & 1]);
        }
      }
      if (!ok) break;
      const int i = ub * kMoeUnit + (m & (kMoeUnit - 1));
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (!((tokens >> t) & 1u)) continue;
        if (j0 > 0) {
          a.cut[(static_cast<size_t>(blockIdx.x) * kMoeMaxTokens + t) * (2 * kMoeUnit) + m] = sum[t];
        } else if (i < a.I) {
          const int row = p.first[act] + __popc(tokens & ((1u << t) - 1));
          a.main[(static_cast<size_t>(row) * 2 + (m >= kMoeUnit)) * a.I + i] = sum[t];
        }
      }
      pos += n;
    }
    if (!ok) *c.stop = 1;
  } else {
    const int mine = warp - 6;
    int it = mine;
    for (int pos = lo + mine; pos < hi; pos += kMoeSplitWarps, it += kMoeSplitWarps) {
      const int tile = pos / r.kch, j = pos - tile * r.kch;
      const uint32_t tokens = p.tokens[tile / r.units];
      const int k = j * S::kChunk + lane * S::kVals;
      float x[NT][S::kVals];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int v = 0; v < S::kVals; ++v) x[t][v] = 0.f;
        if (((tokens >> t) & 1u) && k < a.H) {
          const float* src = a.y + static_cast<size_t>(t) * a.H + k;
          if constexpr (F8) {
            const float4 f = __ldg(reinterpret_cast<const float4*>(src));
            x[t][0] = f.x, x[t][1] = f.y, x[t][2] = f.z, x[t][3] = f.w;
          } else {
            const float2 f = __ldg(reinterpret_cast<const float2*>(src));
            x[t][0] = f.x, x[t][1] = f.y;
          }
        }
      }
      const int b = it % S::kBStages;
      if (it >= S::kBStages && !c.warp_wait(&c.emptyB[b], ((it / S::kBStages) - 1) & 1, a.err, kErrWaitEmpty)) break;
      unsigned char* tileB = c.B + b * S::kBTile;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (!((tokens >> t) & 1u)) continue;
        if constexpr (F8) {
          const float s = put_parts<NT>(tileB, t, lane, x[t]);
          if (lane == 0) c.scales[it % S::kScaleSlots][t] = s;
        } else {
          put_parts<NT>(tileB, t, lane, x[t]);
        }
      }
      fence_to_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.fullB[b]);
    }
  }
  c.end(tmem);
}

// ----------------------------------------------------------------------------- down

template <bool F8, int NT>
__global__ void __launch_bounds__(kMoeThreads, 1) moe_down_kernel(const __grid_constant__ MoeArgs a) {
  using S = Shape<F8, NT>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Cta<F8, NT> c(smem_raw);
  const uint32_t tmem = c.begin();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x % a.splits, m0 = (blockIdx.x / a.splits) * 128;
  const Plan& p = *c.plan;
  // ids and gates were complete before gate/up could begin
  make_plan(*c.plan, a, true);
  const Runs r(p, a, S::kChunk);
  const int kch = (a.I + S::kChunk - 1) / S::kChunk, all = p.active * kch;
  const int lo = static_cast<int>(static_cast<long long>(split) * all / a.splits);
  const int n = static_cast<int>(static_cast<long long>(split + 1) * all / a.splits) - lo;
  float* part = reinterpret_cast<float*>(c.A);  // [NT][128] this CTA's sums, once the ring is done

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol = l2_policy_evict_first();
      int it = 0;
      for (; it < n; ++it) {
        const int s = it % c.kStages, act = (lo + it) / kch, j = lo + it - act * kch;
        if (it >= c.kStages && !mbar_wait(&c.emptyA[s], ((it / c.kStages) - 1) & 1, c.stop, a.err, kErrWaitEmpty)) *c.stop = 1;
        if (*c.stop) break;
        mbar_arrive_expect_tx(&c.fullA[s], kMoeATile);
        tma_load_3d(c.A + s * kMoeATile, &a.d, j * S::kChunk, m0, p.expert[act], &c.fullA[s], pol);
      }
      if (*c.stop) c.drain(it, a.err);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      for (int it = 0; it < n; ++it) {
        const int b = F8 ? it & 1 : 0;
        if (F8 && it >= 2 && !mbar_wait(&c.drained[b], ((it >> 1) - 1) & 1, c.stop, a.err, kErrWaitFull)) *c.stop = 1;
        if (*c.stop || !c.multiply(it, tmem + b * S::kN, F8 || it == 0, a.err)) {
          *c.stop = 1;
          break;
        }
        if (F8 || it + 1 == n) tc_commit(&c.accum[b]);
      }
    }
  } else if (warp < 6) {
    const int q = warp & 3;
    const uint32_t at = tmem + (static_cast<uint32_t>(32 * q) << 16);
    float sum[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) sum[t] = 0.f;
    bool ok = true;
    if (F8) {
      const int HB = (a.H + kFp8Block - 1) / kFp8Block;
      auto scale = [&](int it) {
        const int act = (lo + it) / kch, j = lo + it - act * kch;
        return __ldg(a.sd + (static_cast<size_t>(p.expert[act]) * HB + m0 / kFp8Block) * kch + j);
      };
      float next = n > 0 ? scale(0) : 0.f;
      for (int it = 0; it < n && ok; ++it) {
        const float w = next;
        if (it + 1 < n) next = scale(it + 1);
        ok = c.warp_wait(&c.accum[it & 1], (it >> 1) & 1, a.err, kErrWaitFull);
        if (!ok) break;
        tc_fence_after();
        float v[NT];
        take_sums<F8, NT>(at + (it & 1) * S::kN, v);
        const float* sx = c.scales[it % S::kScaleSlots];
#pragma unroll
        for (int t = 0; t < NT; ++t) sum[t] = fmaf(v[t], w * sx[t], sum[t]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.drained[it & 1]);
      }
    } else if (n > 0) {
      ok = c.warp_wait(&c.accum[0], 0, a.err, kErrWaitFull);
      tc_fence_after();
      if (ok) take_sums<F8, NT>(at, sum);
    }
    if (!ok) *c.stop = 1;
    // every product of this CTA is done, so the ring's memory is free
    if (ok) {
#pragma unroll
      for (int t = 0; t < NT; ++t) part[t * 128 + 32 * q + lane] = sum[t];
    }
  } else {
    pdl_wait();  // gate and up products
    const int mine = warp - 6;
    for (int it = mine; it < n; it += kMoeSplitWarps) {
      const int act = (lo + it) / kch, j = lo + it - act * kch;
      const uint32_t tokens = p.tokens[act];
      const int i = j * S::kChunk + lane * S::kVals, ub = i / kMoeUnit;
      const bool inside = i < a.I;
      int c0 = 0, c1 = 0;  // the CTAs that hold parts of this lane's tile
      if (inside) {
        const long long pos = (static_cast<long long>(act) * r.units + ub) * r.kch;
        c0 = r.owner(pos);
        c1 = r.owner(pos + r.kch - 1);
      }
      float x[NT][S::kVals];
      int row = p.first[act];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int v = 0; v < S::kVals; ++v) x[t][v] = 0.f;
        if (!((tokens >> t) & 1u)) continue;
        if (inside) {
          float g[S::kVals], u[S::kVals];
          auto load = [](float(&d)[S::kVals], const float* src) {
            if constexpr (F8) {
              const float4 f = *reinterpret_cast<const float4*>(src);
              d[0] = f.x, d[1] = f.y, d[2] = f.z, d[3] = f.w;
            } else {
              const float2 f = *reinterpret_cast<const float2*>(src);
              d[0] = f.x, d[1] = f.y;
            }
          };
          load(g, a.main + static_cast<size_t>(row) * 2 * a.I + i);
          load(u, a.main + (static_cast<size_t>(row) * 2 + 1) * a.I + i);
          for (int cc = c0 + 1; cc <= c1; ++cc) {
            const float* src = a.cut + (static_cast<size_t>(cc) * kMoeMaxTokens + t) * (2 * kMoeUnit) + (i & (kMoeUnit - 1));
            float dg[S::kVals], du[S::kVals];
            load(dg, src);
            load(du, src + kMoeUnit);
#pragma unroll
            for (int v = 0; v < S::kVals; ++v) {
              g[v] += dg[v];
              u[v] += du[v];
            }
          }
          const float w = p.gate[row];
#pragma unroll
          for (int v = 0; v < S::kVals; ++v) x[t][v] = g[v] / (1.f + expf(-g[v])) * u[v] * w;
        }
        ++row;
      }
      const int b = it % S::kBStages;
      if (it >= S::kBStages && !c.warp_wait(&c.emptyB[b], ((it / S::kBStages) - 1) & 1, a.err, kErrWaitEmpty)) break;
      unsigned char* tileB = c.B + b * S::kBTile;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (!((tokens >> t) & 1u)) {  // a token that did not choose the expert
          put_zeros<NT, S::kParts>(tileB, t, lane);
          if (F8 && lane == 0) c.scales[it % S::kScaleSlots][t] = 0.f;
        } else if constexpr (F8) {
          const float s = put_parts<NT>(tileB, t, lane, x[t]);
          if (lane == 0) c.scales[it % S::kScaleSlots][t] = s;
        } else {
          put_parts<NT>(tileB, t, lane, x[t]);
        }
      }
      fence_to_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.fullB[b]);
    }
  }
  __syncwarp();
  pdl_wait();  // the result may be what an earlier kernel reads or writes
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  {
    const uint32_t local = smem_addr(part);
    const int total = a.T * 128, per = (total + a.splits - 1) / a.splits, end = min(total, (split + 1) * per);
    for (int o = split * per + static_cast<int>(threadIdx.x); o < end; o += kMoeThreads) {
      const int t = o >> 7, m = m0 + (o & 127);
      float x[kMoeMaxSplits];
#pragma unroll
      for (int k = 0; k < kMoeMaxSplits; ++k) {
        x[k] = 0.f;
        if (k < a.splits) {
          uint32_t remote;
          asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local + 4u * o), "r"(k));
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x[k]) : "r"(remote));
        }
      }
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < kMoeMaxSplits; ++k) sum += x[k];
      const size_t to = static_cast<size_t>(t) * a.H + m;
      if (m < a.H) a.out[to] = (a.residual ? a.residual[to] : 0.f) + sum;
    }
  }
  __syncwarp();
  // no CTA leaves while others may still read its shared memory
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  c.end(tmem);
}

// ----------------------------------------------------------------------------- host side

template <bool F8, int NT>
int down_clusters(int size) {
  static std::mutex mu;
  static int cache[kMoeMaxSplits + 1] = {};
  std::lock_guard<std::mutex> lock(mu);
  if (cache[size] == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(size * 64);
    cfg.blockDim = dim3(kMoeThreads);
    cfg.dynamicSmemBytes = Cta<F8, NT>::kSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(size);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, moe_down_kernel<F8, NT>, &cfg) != cudaSuccess || n == 0) {
      (void)cudaGetLastError();
      n = -1;
    }
    cache[size] = n;
  }
  return cache[size];
}

template <bool F8, int NT>
cudaError_t run_experts(MoeArgs& a, cudaStream_t st) {
  cudaError_t e = launch(moe_gate_up_kernel<F8, NT>, dim3(a.ctas), dim3(kMoeThreads), Cta<F8, NT>::kSmem, st, true, a);
  if (e != cudaSuccess) return e;
  // K splits of a tile of the down product: as many as run at once
  const int tiles = (a.H + 127) / 128;
  a.splits = 1;
  while (a.splits * 2 <= kMoeMaxSplits && down_clusters<F8, NT>(a.splits * 2) >= tiles) a.splits *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles * a.splits);
  cfg.blockDim = dim3(kMoeThreads);
  cfg.dynamicSmemBytes = Cta<F8, NT>::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(a.splits);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, moe_down_kernel<F8, NT>, a);
}

template <bool F8, int NT>
cudaError_t allow_one() {
  cudaError_t e = allow_smem(moe_gate_up_kernel<F8, NT>);
  return e != cudaSuccess ? e : allow_smem(moe_down_kernel<F8, NT>);
}

}  // namespace

int moe_experts(const MoeCall& c, int sms, cudaStream_t st, const char** why) {
  *why = nullptr;
  const bool f8 = c.sg != nullptr;
  const int bytes = f8 ? 1 : 2;
  static thread_local MoeArgs a;
  std::memset(&a, 0, sizeof(a));
  if (!make_tmap_mats(&a.g, c.wg, bytes, c.H, c.I, c.E, kMoeUnit) ||
      !make_tmap_mats(&a.u, c.wu, bytes, c.H, c.I, c.E, kMoeUnit) ||
      !make_tmap_mats(&a.d, c.wd, bytes, c.I, c.H, c.E, 128)) {
    *why = "a tensor map could not be made";
    return 1;
  }
  a.y = c.y;
  a.ids = c.ids;
  a.gates = c.gates;
  a.sg = c.sg;
  a.su = c.su;
  a.sd = c.sd;
  a.residual = c.residual;
  a.out = c.out;
  a.main = c.ws;
  a.cut = c.ws + ((moe_main_floats(c.T, c.k, c.I) + 63) & ~size_t(63));
  a.T = c.T;
  a.k = c.k;
  a.E = c.E;
  a.H = c.H;
  a.I = c.I;
  a.ctas = std::min(sms, kMoeMaxCtas);
  a.err = c.err;
  const int nt = c.T <= 2 ? 2 : (c.T <= 8 ? 8 : 16);
  cudaError_t e = f8 ? (nt == 2 ? run_experts<true, 2>(a, st) : nt == 8 ? run_experts<true, 8>(a, st) : run_experts<true, 16>(a, st))
                     : (nt == 2 ? run_experts<false, 2>(a, st)
                                : nt == 8 ? run_experts<false, 8>(a, st) : run_experts<false, 16>(a, st));
  if (e != cudaSuccess) {
    *why = cudaGetErrorString(e);
    return 3;
  }
  return 0;
}

cudaError_t allow_smem_moe() {
  cudaError_t e;
  if ((e = allow_one<false, 2>()) != cudaSuccess) return e;
  if ((e = allow_one<false, 8>()) != cudaSuccess) return e;
  if ((e = allow_one<false, 16>()) != cudaSuccess) return e;
  if ((e = allow_one<true, 2>()) != cudaSuccess) return e;
  if ((e = allow_one<true, 8>()) != cudaSuccess) return e;
  return allow_one<true, 16>();
}

}  // namespace dec
