// The experts of a mixture-of-experts layer for a decode step's few tokens:
//
//   out[t] = res[t] + sum over experts e chosen by t, gate weight w:
//            Wd[e] (w silu(Wg[e] y[t]) * (Wu[e] y[t]))
//
// Bound by the stream of the chosen experts' weights: each is read once,
// whatever number of tokens chose it.  Two launches (gate/up and down) stream
// them, a short one adds the parts of the result; from three tokens on, a short
// one ahead of each makes the activations' operand.
//
// The products run on the tensor cores with weight rows on the 128 lanes of an
// accumulator and the tokens on its columns (tcgen05.mma, M = 128).  fp32
// activations are kept whole by giving every token several columns: its row is
// split into parts whose products with the weights are exact and whose columns
// are added at the end.
//   * bf16 weights: three bf16 parts (24 bits);
//   * e4m3 weights: five e4m3 parts, each 2^-5 of the one before, of x / s with s
//     a power of two per token and 128 values (what is left is 2^-23 of the
//     largest of the 128).
// After every 128 bytes of K the column sums leave tensor memory and are added
// in fp32 registers, times s and the weights' own block scale: the tensor core
// cuts every product at the last place of its running sum, and one accumulator
// over a whole row of 2560 was off by 1.8e-6 where this is by 1e-7.
//
// The parts are 1 KB blocks per token and chunk: eight swizzled rows of 128
// bytes, the parts in the first three or five.  A chunk's operand is the blocks
// of the tokens that chose the expert, N = 8 per token, so its cost follows their
// number.  For one or two tokens four warps of every CTA make them beside the
// stream; for more they are made once (moe_prep_kernel for y, moe_act_kernel for
// the inner vectors) and brought by bulk copies.  (With 16 tokens four warps
// took 1.1 us a chunk, three times what its weights take; with one token the two
// launches cost 44 us a layer where this takes 37.)
//
// gate/up: a tile is 64 gate rows and the same 64 up rows of an expert.  How
// many experts are active is known on the device only, so a persistent grid
// lays all tiles' chunks end to end and gives every CTA an equal run of them;
// a tile cut between CTAs leaves parts, which moe_act_kernel adds in CTA order.
// down: a tile is 128 output rows, its K axis all active experts' inner vectors
// one behind the other, split over as many CTAs as run at once; their sums are
// added in split order by moe_sum_kernel, so results do not depend on timing.
// (Clusters that add through distributed shared memory hold 120 CTAs where 300
// run: 74 us for the down half of 16 tokens, 8 of 128 8-bit experts, against 48.
// The last of a tile's CTAs to arrive adding all 25 parts took 9 us at the end of
// 16 tokens, three times the launch that spreads it.)  The first weights are on
// their way while gate/up still runs.
//
// Every wait on an mbarrier is bounded: an error bit and an early end instead of a
// hang, in which one thread waits, bounded as well, for the copies and products
// that are still on their way before shared and tensor memory are given up.  (The
// allocation of tensor memory has no limit of its own: CTAs hold no more than leaves
// room for all of an SM.)
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "dec_fp8.cuh"
#include "dec_launch.cuh"
#include "dec_moe.cuh"
#include "dec_tc.cuh"

namespace dec {
namespace {

// warps 0 and 6 copy weights, 1 multiplies, 2-5 take sums off, 7 copies activations (7-10 split them)
constexpr int kMoeThreads = 256, kMoeThreadsOwn = 352;
constexpr int kMoeOwnWarps = 4;
constexpr int kMoeFlat = 256;         // threads of the two short launches
constexpr uint32_t kMoeATile = 128 * 128;
constexpr uint32_t kMoeBlock = 1024;  // one token's parts of one chunk
constexpr int kMoeMaxStages = 8;
constexpr int kMoeTurns = 8;          // chunks whose activations may be in shared memory at once
constexpr int kMoeMaxSplits = 32;

template <bool F8>
struct Parts {
  static constexpr int kParts = F8 ? 5 : 3;
  static constexpr int kChunk = F8 ? 128 : 64;              // values of K per 128-byte row
  static constexpr int kVals = kChunk / 32;                 // of them per lane of a warp
  static constexpr uint32_t kScaleAt = kParts * 128;        // e4m3: s behind the parts
  static constexpr uint32_t kCopy = kParts * 128 + (F8 ? 16 : 0);
};

// What all launches derive from the ids (made by moe_prep_kernel): the active
// experts in ascending order, the tokens of each, and one row per (expert,
// token) pair.
struct Plan {
  int active, rows;
  uint16_t expert[kMoeRows], count[kMoeRows], first[kMoeRows];  // per active expert
  uint16_t token[kMoeRows], act[kMoeRows];                      // per row
  float gate[kMoeRows];
};
static_assert(sizeof(Plan) <= kMoePlanBytes, "the plan's place in the workspace");

struct MoeArgs {
  CUtensorMap g, u, d;           // boxes of 64 rows
  const float* y;
  const int32_t* ids;
  const float* gates;
  const float *sg, *su, *sd;
  const float* residual;
  float* out;
  Plan* plan;                    // workspace
  float *main, *cut, *sums;
  unsigned char *xb, *hb;
  int T, k, E, H, I;
  int ctas;                      // of the gate/up launch
  int splits;
  uint32_t* err;
};

// The runs of gate/up: W chunks over n CTAs.  A run is at least an eighth of a
// tile's K axis, so that a tile is cut into nine parts at most.
struct Runs {
  long long W;
  int n, kch, units;
  __device__ __forceinline__ Runs(int active, const MoeArgs& a, int chunk) {
    kch = (a.H + chunk - 1) / chunk;
    units = (a.I + kMoeUnit - 1) / kMoeUnit;
    const long long tiles = static_cast<long long>(active) * units;
    W = tiles * kch;
    n = static_cast<int>(min(static_cast<long long>(a.ctas), min(8 * tiles, W)));  // no run is empty
  }
  __device__ __forceinline__ int begin(int c) const { return c >= n ? static_cast<int>(W) : static_cast<int>(W * c / n); }
  // The CTA whose run holds chunk `pos`; in 32 bits where they do, a quarter of the instructions.
  __device__ __forceinline__ int owner(long long pos) const {
    const unsigned long long x = static_cast<unsigned long long>(pos + 1) * n - 1;
    if (static_cast<unsigned long long>(W) * n <= 0xFFFFFFFFull) return static_cast<int>(static_cast<uint32_t>(x) / static_cast<uint32_t>(W));
    return static_cast<int>(x / static_cast<unsigned long long>(W));
  }
};

// ----------------------------------------------------------------------------- parts of an activation row

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Byte offset of this lane's 4 bytes in row `row` < 8 of a swizzled block.
__device__ __forceinline__ uint32_t part_at(int row, int lane) {
  return row * 128 + (((lane >> 2) ^ row) << 4) + ((lane & 3) << 2);
}

// A warp's two (bf16 parts) or four (e4m3 parts) values per lane into a block.
__device__ __forceinline__ void put_parts(unsigned char* block, int lane, const float (&x)[2]) {
  float a = x[0], b = x[1];
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    const uint32_t w = pack_bf16(a, b);
    *reinterpret_cast<uint32_t*>(block + part_at(p, lane)) = w;
    a -= bf16lo(w);
    b -= bf16hi(w);
  }
}

// s: the largest magnitude of the 128 is at most 224 s, so that what a part
// leaves, half a step of at most 16, is at most 8 and 2^5 of it fits again.
__device__ __forceinline__ void put_parts(unsigned char* block, int lane, const float (&x)[4]) {
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
    *reinterpret_cast<uint32_t*>(block + part_at(p, lane)) = lo | (static_cast<uint32_t>(hi) << 16);
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
  if (lane == 0) *reinterpret_cast<float*>(block + Parts<true>::kScaleAt) = __uint_as_float(static_cast<uint32_t>(e) << 23);
}

// A lane's consecutive values.
__device__ __forceinline__ void load_vals(float (&x)[2], const float* src) {
  const float2 f = *reinterpret_cast<const float2*>(src);
  x[0] = f.x, x[1] = f.y;
}
__device__ __forceinline__ void load_vals(float (&x)[4], const float* src) {
  const float4 f = *reinterpret_cast<const float4*>(src);
  x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
}

// ----------------------------------------------------------------------------- plan and parts of y

// One CTA.
__device__ __forceinline__ void make_plan(Plan& p, const MoeArgs& a) {
  __shared__ uint32_t chosen[kMoeMaxExperts / 2];                       // 16 token bits per expert
  __shared__ uint16_t act_of[kMoeMaxExperts], first_of[kMoeMaxExperts];  // of active experts
  __shared__ int32_t ids[kMoeRows];
  __shared__ float gates[kMoeRows];
  const int n = a.T * a.k, i = threadIdx.x;
  for (int w = i; w < (a.E + 1) / 2; w += kMoeFlat) chosen[w] = 0;
  static_assert(kMoeRows <= kMoeFlat, "a thread per choice");
  if (i < n) {
    ids[i] = a.ids[i];
    gates[i] = a.gates[i];
  }
  __syncthreads();
  const int mine = i < n ? ids[i] : -1, t = i / a.k;
  const bool valid = mine >= 0 && mine < a.E;
  if (valid)
    atomicOr(&chosen[mine >> 1], (1u << t) << (16 * (mine & 1)));
  else if (mine != -1)
    atomicOr(a.err, kErrPosRange);
  __syncthreads();
  if (i < 32) {
    int active = 0, rows = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + i;
      const uint32_t m = e < a.E ? (chosen[e >> 1] >> (16 * (e & 1))) & 0xFFFFu : 0u;
      const uint32_t any = __ballot_sync(0xffffffffu, m != 0);
      if (any == 0) continue;
      const int c = __popc(m);
      int upto = c;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (i >= o) upto += v;
      }
      if (m) {
        const int at = active + __popc(any & ((1u << i) - 1)), first = rows + upto - c;
        p.expert[at] = static_cast<uint16_t>(e);
        p.count[at] = static_cast<uint16_t>(c);
        p.first[at] = static_cast<uint16_t>(first);
        act_of[e] = static_cast<uint16_t>(at);
        first_of[e] = static_cast<uint16_t>(first);
      }
      active += __popc(any);
      rows += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (i == 0) {
      p.active = active;
      p.rows = rows;
    }
  }
  __syncthreads();
  if (!valid) return;
  const uint32_t m = (chosen[mine >> 1] >> (16 * (mine & 1))) & 0xFFFFu;
  float w = 0.f;  // an expert that a token lists twice counts twice
  for (int j = t * a.k; j < (t + 1) * a.k; ++j)
    if (ids[j] == mine) {
      if (j < i) return;  // an earlier listing makes the row
      w += gates[j];
    }
  const int row = first_of[mine] + __popc(m & ((1u << t) - 1));
  p.token[row] = static_cast<uint16_t>(t);
  p.act[row] = act_of[mine];
  p.gate[row] = w;
}

// The plan of at most two tokens, by one warp of every CTA that needs it, experts in the order of their first listing.
__device__ __forceinline__ void make_small_plan(Plan& p, const MoeArgs& a, bool report) {
  const int lane = threadIdx.x & 31, n = a.T * a.k;
  static_assert(2 * kMoeMaxChoices <= 32, "a lane per choice");
  const int e = lane < n ? a.ids[lane] : -1;
  const float g = lane < n ? a.gates[lane] : 0.f;
  const bool valid = e >= 0 && e < a.E;
  if (report && !valid && e != -1) atomicOr(a.err, kErrPosRange);
  const uint32_t same = __match_any_sync(0xffffffffu, valid ? e : -1 - lane);
  const uint32_t first_token = a.k < 32 ? (1u << a.k) - 1 : 0xffffffffu;
  const bool leads = valid && lane == __ffs(same) - 1;
  const int count = ((same & first_token) != 0) + ((same & ~first_token) != 0);
  const uint32_t leaders = __ballot_sync(0xffffffffu, leads), pairs = __ballot_sync(0xffffffffu, leads && count == 2);
  float w0 = 0.f, w1 = 0.f;  // an expert that a token lists twice counts twice
  for (int j = 0; j < n; ++j) {
    const float gj = __shfl_sync(0xffffffffu, g, j);
    if ((same >> j) & 1u) (j < a.k ? w0 : w1) += gj;
  }
  if (leads) {
    const uint32_t before = (1u << lane) - 1;
    const int at = __popc(leaders & before);
    int row = at + __popc(pairs & before);
    p.expert[at] = static_cast<uint16_t>(e);
    p.count[at] = static_cast<uint16_t>(count);
    p.first[at] = static_cast<uint16_t>(row);
    if (same & first_token) {
      p.token[row] = 0;
      p.gate[row++] = w0;
    }
    if (same & ~first_token) {
      p.token[row] = 1;
      p.gate[row] = w1;
    }
  }
  if (lane == 0) p.active = __popc(leaders);
}

// Block 0: the plan.  Warps of the others: one block of parts each, chunk j of token t at j T + t.
template <bool F8>
__global__ void __launch_bounds__(kMoeFlat) moe_prep_kernel(const __grid_constant__ MoeArgs a) {
  using P = Parts<F8>;
  pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.x == 0) {
    make_plan(*a.plan, a);
    return;
  }
  const int lane = threadIdx.x & 31, i = (blockIdx.x - 1) * (kMoeFlat / 32) + threadIdx.x / 32;
  const int j = i / a.T, t = i - j * a.T, k = j * P::kChunk + lane * P::kVals;
  if (j * P::kChunk >= a.H) return;
  float x[P::kVals];
#pragma unroll
  for (int v = 0; v < P::kVals; ++v) x[v] = 0.f;
  if (k < a.H) load_vals(x, a.y + static_cast<size_t>(t) * a.H + k);
  put_parts(a.xb + static_cast<size_t>(i) * kMoeBlock, lane, x);
}

// w silu(g) u of this lane's values of chunk j in row `row`, which is token `rank` of active expert `act`: the products of
// gate/up, and the parts of a tile that CTAs c0 + 1 .. c1 took over.
template <bool F8>
struct Inner {
  using P = Parts<F8>;
  int i, c0, c1, row, rank;
  bool inside;
  __device__ __forceinline__ Inner(const MoeArgs& a, const Runs& r, int act, int row_, int rank_, int j)
      : i(j * P::kChunk + static_cast<int>(threadIdx.x & 31) * P::kVals), c0(0), c1(0), row(row_), rank(rank_) {
    inside = i < a.I;
    if (inside) {
      const long long pos = (static_cast<long long>(act) * r.units + i / kMoeUnit) * r.kch;
      c0 = r.owner(pos);
      c1 = r.owner(pos + r.kch - 1);
    }
  }
  __device__ __forceinline__ void get(const MoeArgs& a, float w, float (&x)[P::kVals]) const {
#pragma unroll
    for (int v = 0; v < P::kVals; ++v) x[v] = 0.f;
    if (!inside) return;
    // the products and the first part, which is the only one as a rule, in flight together
    float g[P::kVals], u[P::kVals], dg[P::kVals], du[P::kVals];
    const size_t part = kMoeMaxTokens * 2 * kMoeUnit;
    const float* src = a.cut + (static_cast<size_t>(c0 + 1) * kMoeMaxTokens + rank) * (2 * kMoeUnit) + (i & (kMoeUnit - 1));
    load_vals(g, a.main + static_cast<size_t>(row) * 2 * a.I + i);
    load_vals(u, a.main + (static_cast<size_t>(row) * 2 + 1) * a.I + i);
    if (c1 > c0) {
      load_vals(dg, src);
      load_vals(du, src + kMoeUnit);
    }
    for (int c = c0 + 1; c <= c1; ++c) {
      if (c > c0 + 1) {
        src += part;
        load_vals(dg, src);
        load_vals(du, src + kMoeUnit);
      }
#pragma unroll
      for (int v = 0; v < P::kVals; ++v) {
        g[v] += dg[v];
        u[v] += du[v];
      }
    }
#pragma unroll
    for (int v = 0; v < P::kVals; ++v) x[v] = g[v] / (1.f + expf(-g[v])) * u[v] * w;
  }
};

// The inner vectors' blocks, one warp per row and chunk, in the order that the down launch reads them: expert, chunk,
// token.  The plan was complete before gate/up could begin, and that began before this launch could.
template <bool F8>
__global__ void __launch_bounds__(kMoeFlat) moe_act_kernel(const __grid_constant__ MoeArgs a) {
  using P = Parts<F8>;
  pdl_launch_dependents();  // the next launch reads nothing of this one's before its own wait
  const Plan& p = *a.plan;
  const int lane = threadIdx.x & 31, id = blockIdx.x * (kMoeFlat / 32) + threadIdx.x / 32;
  const int kch = (a.I + P::kChunk - 1) / P::kChunk, row = id / kch, j = id - row * kch;
  const bool live = row < p.rows;
  const int act = live ? p.act[row] : 0, first = live ? p.first[act] : 0, count = live ? p.count[act] : 0;
  const float w = live ? p.gate[row] : 0.f;
  const Runs r(p.active, a, P::kChunk);
  const Inner<F8> inner(a, r, act, row, row - first, live ? j : kch);
  pdl_wait();
  if (!live) return;
  float x[P::kVals];
  inner.get(a, w, x);
  put_parts(a.hb + (static_cast<size_t>(first) * kch + static_cast<size_t>(j) * count + row - first) * kMoeBlock, lane, x);
}

// The result: the sums of a tile's CTAs in split order, on top of the residual.
__global__ void __launch_bounds__(128) moe_sum_kernel(const __grid_constant__ MoeArgs a) {
  const int per = a.H / 4, id = blockIdx.x * 128 + threadIdx.x, t = id / per, m = 4 * (id - t * per);
  pdl_wait();
  pdl_launch_dependents();
  if (t >= a.T) return;
  const size_t to = static_cast<size_t>(t) * a.H + m;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f), res = sum;
  if (a.residual) res = *reinterpret_cast<const float4*>(a.residual + to);
  // [tile][split][T][128]
  const float* src = a.sums + (static_cast<size_t>(m / 128) * a.splits * a.T + t) * 128 + m % 128;
  for (int s0 = 0; s0 < a.splits; s0 += 16) {
    float4 x[16];
#pragma unroll
    for (int s = 0; s < 16; ++s)
      if (s0 + s < a.splits) x[s] = *reinterpret_cast<const float4*>(src + static_cast<size_t>(s0 + s) * a.T * 128);
#pragma unroll
    for (int s = 0; s < 16; ++s)
      if (s0 + s < a.splits) sum = make_float4(sum.x + x[s].x, sum.y + x[s].y, sum.z + x[s].z, sum.w + x[s].w);
  }
  *reinterpret_cast<float4*>(a.out + to) = make_float4(res.x + sum.x, res.y + sum.y, res.z + sum.z, res.w + sum.w);
}

// ----------------------------------------------------------------------------- a CTA of the two streaming launches

// Where the chunks' activations lie: a ring of 2 KB slots, a chunk of n tokens
// in (n + 1) / 2 of them side by side (the ring's end is passed over where they
// would not fit).  Every role keeps its own copy of this and steps it alike.
template <int SLOTS>
struct Ring {
  int head = 0;
  __device__ __forceinline__ int take(int n, int* used) {
    const int want = (n + 1) >> 1;
    const bool wraps = head + want > SLOTS;
    const int skip = wraps ? SLOTS - head : 0, at = wraps ? 0 : head;
    head = at + want;
    *used = want + skip;
    return at;
  }
};

// NT: the most tokens of a call, 2, 8 or 16.  Two CTAs fit an SM, of one launch
// or of two: a thread takes about 55 ns to issue a copy, so three warps of each
// share them, and with one CTA per SM the same stream was 10 % slower.
template <bool F8, int NT>
struct Cta {
  using P = Parts<F8>;
  static constexpr bool kOwn = NT == 2;  // makes its own plan and blocks
  static constexpr int kThreads = kOwn ? kMoeThreadsOwn : kMoeThreads;
  static constexpr int kSlots = NT <= 2 ? 8 : 16;
  static constexpr uint32_t kSlot = 2 * kMoeBlock;
  uint64_t *fullA, *emptyA, *fullB, *emptyB, *accum, *drained;
  uint32_t* tmem_slot;
  volatile int* stop;  // a wait ran out: every role ends
  volatile int* ends;  // chunks whose weights' halves and activations were asked for, and that were multiplied
  Plan* plan;
  float* total;        // [NT][128] sums of the down launch
  unsigned char *A, *B;
  uint32_t tmem;

  static constexpr uint32_t kHead = 1024, kPlan = kMoePlanBytes, kTotal = NT * 512;
  static constexpr int kStages = static_cast<int>((112 * 1024 - 1024 - kHead - kPlan - kTotal - kSlots * kSlot) / kMoeATile);
  static_assert(kStages >= 4 && kStages <= kMoeMaxStages && kSlots >= NT / 2, "shared memory");
  static constexpr uint32_t kSmem = 1024 + kHead + kPlan + kTotal + kSlots * kSlot + kStages * kMoeATile;
  static constexpr int kAccs = NT <= 8 ? 4 : 2;             // accumulators in turn: two CTAs' fit tensor memory
  static constexpr uint32_t kAcc = 8 * NT;                  // columns of one
  static constexpr uint32_t kCols = tmem_columns(kAccs * kAcc);
  static constexpr int kGroup = NT < 4 ? NT : 4;            // tokens whose sums are loaded together

  // All threads.
  __device__ __forceinline__ explicit Cta(unsigned char* raw) {
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    fullA = reinterpret_cast<uint64_t*>(smem);
    emptyA = fullA + kMoeMaxStages;
    fullB = emptyA + kMoeMaxStages;
    emptyB = fullB + kMoeTurns;
    accum = emptyB + kMoeTurns;
    drained = accum + kAccs;
    tmem_slot = reinterpret_cast<uint32_t*>(drained + kAccs);
    stop = reinterpret_cast<volatile int*>(tmem_slot + 1);
    ends = stop + 1;
    static_assert((2 * kMoeMaxStages + 2 * kMoeTurns + 2 * kAccs) * 8 + 24 <= kHead, "barriers");
    A = smem + kHead;
    B = A + kStages * kMoeATile;
    plan = reinterpret_cast<Plan*>(B + kSlots * kSlot);
    total = reinterpret_cast<float*>(reinterpret_cast<unsigned char*>(plan) + kPlan);
    if (threadIdx.x == 0) {
      for (int s = 0; s < kStages; ++s) {
        mbar_init(&fullA[s], 2);
        mbar_init(&emptyA[s], 1);
      }
      for (int s = 0; s < kMoeTurns; ++s) {
        mbar_init(&fullB[s], 1);
        mbar_init(&emptyB[s], 4);
      }
      for (int s = 0; s < kAccs; ++s) {
        mbar_init(&accum[s], 1);
        mbar_init(&drained[s], 4);
      }
      *stop = 0;
      for (int i = 0; i < 4; ++i) ends[i] = 0;
      fence_mbar_init();
    }
    if (threadIdx.x / 32 == 1) tmem_alloc(tmem_slot, kCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    tmem = *tmem_slot;
  }
  // All threads.
  __device__ __forceinline__ void take_plan(const Plan* from) {
    const uint32_t* src = reinterpret_cast<const uint32_t*>(from);
    for (int i = threadIdx.x; i < static_cast<int>(sizeof(Plan) / 4); i += kThreads)
      reinterpret_cast<uint32_t*>(plan)[i] = src[i];
    __syncthreads();
  }
  __device__ __forceinline__ void get_plan(const MoeArgs& a, bool report) {
    if (!kOwn) return take_plan(a.plan);
    if (threadIdx.x < 32) make_small_plan(*plan, a, report);
    __syncthreads();
  }
  // Whole warp, of those that split rows: room for chunk `it` (NT = 2: one slot each); null when a wait ran out.
  __device__ __forceinline__ unsigned char* own_slot(int it, uint32_t* err) const {
    if (it >= kMoeTurns && !warp_wait(&emptyB[it % kMoeTurns], ((it / kMoeTurns) - 1) & 1, stop, err, kErrWaitEmpty)) {
      *stop = 1;
      return nullptr;
    }
    return B + it % kMoeTurns * kSlot;
  }
  __device__ __forceinline__ void own_done(int it) const {
    fence_to_async();
    __syncwarp();
    if (threadIdx.x % 32 == 0) mbar_arrive(&fullB[it % kMoeTurns]);
  }
  __device__ __forceinline__ void end(uint32_t* err) {
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x / 32 == 1) {
      if (*stop) {  // after an early end: copies and products that are still on their way
        if (threadIdx.x % 32 == 0) {
          // a chunk with one half asked for: the other's arrival is made good, so that its phase ends with that half
          for (int i = min(ends[0], ends[1]); i < max(ends[0], ends[1]); ++i) mbar_arrive(&fullA[i % kStages]);
          drain_ring(fullA, kStages, max(ends[0], ends[1]), err);
          if (!kOwn) drain_ring(fullB, kMoeTurns, ends[2], err);
          drain_ring(emptyA, kStages, ends[3], err);
        }
        __syncwarp();
      }
      tc_fence_after();
      tmem_free(tmem, kCols);
    }
  }
  // Whole warp, of either weight warp: a free stage for chunk `it`; false when a wait ran out.
  __device__ __forceinline__ bool claim(int it, uint32_t* err) const {
    const int s = it % kStages;
    if (it >= kStages && !warp_wait(&emptyA[s], ((it / kStages) - 1) & 1, stop, err, kErrWaitEmpty)) {
      *stop = 1;
      return false;
    }
    return true;
  }
  // One lane: half (64 rows) of chunk `it`'s weights from (x, y, z) of a map.
  __device__ __forceinline__ void bring(int it, int half, const CUtensorMap* map, int x, int y, int z, uint64_t pol) const {
    uint64_t* bar = &fullA[it % kStages];
    mbar_arrive_expect_tx(bar, kMoeATile / 2);
    tma_load_3d(A + it % kStages * kMoeATile + half * (kMoeATile / 2), map, x, y, z, bar, pol);
  }
  // Whole warp: waits until chunk `it`'s activations may be brought; `sizes` holds the slots of the chunks in turn, one
  // byte each, `tail` is the oldest that holds some, `room` the free slots.  False when a wait ran out.
  __device__ __forceinline__ bool make_room(int it, int used, uint64_t& sizes, int& tail, int& room, uint32_t* err) const {
    while (room < used || it - tail >= kMoeTurns) {
      if (!warp_wait(&emptyB[tail % kMoeTurns], (tail / kMoeTurns) & 1, stop, err, kErrWaitEmpty)) {
        *stop = 1;
        return false;
      }
      room += static_cast<int>((sizes >> (8 * (tail % kMoeTurns))) & 0xFF);
      ++tail;
    }
    room -= used;
    const int at = 8 * (it % kMoeTurns);
    sizes = (sizes & ~(0xFFull << at)) | (static_cast<uint64_t>(used) << at);
    return true;
  }
  // Whole warp: the MMAs of chunk `it` with n tokens in slot b; false when a wait ran out.
  __device__ __forceinline__ bool multiply(int it, int n, int b, uint32_t* err) const {
    const int s = it % kStages, acc = it % kAccs;
    if (!warp_wait(&fullA[s], (it / kStages) & 1, stop, err, kErrWaitFull) ||
        !warp_wait(&fullB[it % kMoeTurns], (it / kMoeTurns) & 1, stop, err, kErrWaitFull) ||
        (it >= kAccs && !warp_wait(&drained[acc], ((it / kAccs) - 1) & 1, stop, err, kErrWaitFull))) {
      *stop = 1;
      return false;
    }
    tc_fence_after();
    const uint32_t sa = smem_addr(A + s * kMoeATile), sb = smem_addr(B + b * kSlot), d = tmem + acc * kAcc;
    const uint32_t idesc = tc_idesc_of(8 * ((n + 1) & ~1), !F8);  // columns of a missing last token hold anything
    if (elect_one()) {
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {  // 32 bytes of K per instruction
        const uint64_t ad = smem_desc_sw128(sa + kk * 32), bd = smem_desc_sw128(sb + kk * 32);
        if (F8)
          tc_mma_f8(d, ad, bd, idesc, kk > 0);
        else
          tc_mma(d, ad, bd, idesc, kk > 0);
      }
      tc_commit(&emptyA[s]);
      tc_commit(&accum[acc]);
    }
    __syncwarp();
    return true;
  }
  // Whole warp: adds chunk `it`'s sums of n tokens in slot b, weights' scale w (1 for bf16); false when a wait ran out.
  __device__ __forceinline__ bool add(int it, int n, int b, float w, float (&sum)[NT], uint32_t* err) const {
    const int acc = it % kAccs;
    if (!warp_wait(&accum[acc], (it / kAccs) & 1, stop, err, kErrWaitFull)) {
      *stop = 1;
      return false;
    }
    tc_fence_after();
    const uint32_t at = tmem + (static_cast<uint32_t>(threadIdx.x & 96) << 16) + acc * kAcc;
    const unsigned char* blocks = B + b * kSlot;
#pragma unroll
    for (int t0 = 0; t0 < NT; t0 += kGroup) {
      if (t0 >= n) break;
      uint32_t v[kGroup / 2][16];
#pragma unroll
      for (int h = 0; h < kGroup / 2; ++h)
        if (h == 0 || t0 + 2 * h < n) tmem_ld_issue(at + 8 * (t0 + 2 * h), v[h]);
#pragma unroll
      for (int h = 0; h < kGroup / 2; ++h)
        if (h == 0 || t0 + 2 * h < n) tmem_ld_wait(v[h]);
#pragma unroll
      for (int t = 0; t < kGroup; ++t) {
        if (t0 + t >= n) break;
        float x = 0.f;  // the smallest part first
#pragma unroll
        for (int p = P::kParts - 1; p >= 0; --p) {
          const float part = __uint_as_float(v[t / 2][8 * (t & 1) + p]);
          x = F8 ? fmaf(x, 0.03125f, part) : x + part;
        }
        if (F8)
          sum[t0 + t] = fmaf(x, w * *reinterpret_cast<const float*>(blocks + (t0 + t) * kMoeBlock + P::kScaleAt), sum[t0 + t]);
        else
          sum[t0 + t] += x;
      }
    }
    tc_fence_before();
    __syncwarp();
    if (threadIdx.x % 32 == 0) {
      mbar_arrive(&drained[acc]);
      mbar_arrive(&emptyB[it % kMoeTurns]);
    }
    return true;
  }
};

// ----------------------------------------------------------------------------- gate/up

template <bool F8, int NT>
__global__ void __launch_bounds__(Cta<F8, NT>::kThreads, 2) moe_gate_up_kernel(const __grid_constant__ MoeArgs a) {
  using P = Parts<F8>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Cta<F8, NT> c(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  c.get_plan(a, blockIdx.x == 0);
  const Plan& p = *c.plan;
  const Runs r(p.active, a, P::kChunk);
  const int lo = r.begin(blockIdx.x), hi = r.begin(blockIdx.x + 1);

  using Slots = Ring<Cta<F8, NT>::kSlots>;
  if (warp == 0 || warp == 6) {
    const int half = warp == 6;
    const uint64_t pol = l2_policy_evict_first();
    const CUtensorMap* map = half ? &a.u : &a.g;
    int it = 0;
    bool ok = true;
    for (int pos = lo; pos < hi && ok;) {
      const int tile = pos / r.kch, j0 = pos - tile * r.kch, n = min(r.kch - j0, hi - pos);
      const int row = (tile % r.units) * kMoeUnit, e = p.expert[tile / r.units];
      for (int j = j0; j < j0 + n; ++j, ++it) {
        ok = c.claim(it, a.err);
        if (!ok) break;
        if (elect_one()) c.bring(it, half, map, j * P::kChunk, row, e, pol);
        __syncwarp();
      }
      pos += n;
    }
    if (lane == 0) c.ends[half] = it;
  } else if (c.kOwn && warp >= 7) {
    const int mine = warp - 7;
    for (int it = mine, pos = lo + mine; pos < hi; it += kMoeOwnWarps, pos += kMoeOwnWarps) {
      const int tile = pos / r.kch, act = tile / r.units, first = p.first[act], count = p.count[act];
      const int k = (pos - tile * r.kch) * P::kChunk + lane * P::kVals;
      float x[2][P::kVals];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int v = 0; v < P::kVals; ++v) x[t][v] = 0.f;
        if (t < count && k < a.H) load_vals(x[t], a.y + static_cast<size_t>(p.token[first + t]) * a.H + k);
      }
      unsigned char* slot = c.own_slot(it, a.err);
      if (!slot) break;
      put_parts(slot, lane, x[0]);
      if (count == 2) put_parts(slot + kMoeBlock, lane, x[1]);
      c.own_done(it);
    }
  } else if (warp == 7) {
    const uint64_t pol = l2_policy_evict_last();
    Slots ring;
    uint64_t sizes = 0;
    int it = 0, tail = 0, room = c.kSlots, used;
    bool ok = true;
    for (int pos = lo; pos < hi && ok;) {
      const int tile = pos / r.kch, j0 = pos - tile * r.kch, n = min(r.kch - j0, hi - pos);
      const int act = tile / r.units, count = p.count[act], t = lane < count ? p.token[p.first[act] + lane] : 0;
      for (int j = j0; j < j0 + n; ++j, ++it) {
        const int at = ring.take(count, &used);
        ok = c.make_room(it, used, sizes, tail, room, a.err);
        if (!ok) break;
        uint64_t* bar = &c.fullB[it % kMoeTurns];
        if (lane == 0) mbar_arrive_expect_tx(bar, count * P::kCopy);
        __syncwarp();
        if (lane < count)
          bulk_copy_g2s(c.B + at * c.kSlot + lane * kMoeBlock, a.xb + (static_cast<size_t>(j) * a.T + t) * kMoeBlock, P::kCopy,
                        bar, pol);
      }
      pos += n;
    }
    if (lane == 0) c.ends[2] = it;
  } else if (warp == 1) {
    Slots ring;
    int it = 0, used;
    bool ok = true;
    for (int pos = lo; pos < hi && ok;) {
      const int tile = pos / r.kch, n = min((tile + 1) * r.kch, hi) - pos, count = p.count[tile / r.units];
      for (int j = 0; j < n && ok; ++j, ++it) ok = c.multiply(it, count, ring.take(count, &used), a.err);
      pos += n;
    }
    if (lane == 0) c.ends[3] = it - !ok;
  } else {
    const int m = (32 * warp + lane) & 127;  // TMEM lane; row of the tile: gate below 64, up from 64 on
    const int IB = (a.I + kFp8Block - 1) / kFp8Block;
    Slots ring;
    int it = 0, used;
    bool ok = true;
    for (int pos = lo; pos < hi && ok;) {
      const int tile = pos / r.kch, j0 = pos - tile * r.kch, n = min(r.kch - j0, hi - pos);
      const int act = tile / r.units, ub = tile - act * r.units, count = p.count[act];
      float sum[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) sum[t] = 0.f;
      const float* sw = nullptr;
      float next = 1.f;
      if (F8) {
        sw = (m < kMoeUnit ? a.sg : a.su) + (static_cast<size_t>(p.expert[act]) * IB + ub * kMoeUnit / kFp8Block) * r.kch;
        next = sw[j0];
      }
      for (int j = j0; j < j0 + n && ok; ++j, ++it) {
        const float w = next;
        if (F8 && j + 1 < j0 + n) next = sw[j + 1];
        ok = c.add(it, count, ring.take(count, &used), w, sum, a.err);
      }
      if (!ok) break;
      const int i = ub * kMoeUnit + (m & (kMoeUnit - 1));
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (t >= count) break;
        if (j0 > 0)
          a.cut[(static_cast<size_t>(blockIdx.x) * kMoeMaxTokens + t) * (2 * kMoeUnit) + m] = sum[t];
        else if (i < a.I)
          a.main[(static_cast<size_t>(p.first[act] + t) * 2 + (m >= kMoeUnit)) * a.I + i] = sum[t];
      }
      pos += n;
    }
  }
  c.end(a.err);
}

// ----------------------------------------------------------------------------- down

template <bool F8, int NT>
__global__ void __launch_bounds__(Cta<F8, NT>::kThreads, 2) moe_down_kernel(const __grid_constant__ MoeArgs a) {
  using P = Parts<F8>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Cta<F8, NT> c(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x % a.splits, tile = blockIdx.x / a.splits, m0 = tile * 128;
  // the plan (or what it is made of) was complete before gate/up could begin, and that began before this launch could
  c.get_plan(a, false);
  pdl_launch_dependents();
  const Plan& p = *c.plan;
  const int kch = (a.I + P::kChunk - 1) / P::kChunk, all = p.active * kch;
  const int lo = static_cast<int>(static_cast<long long>(split) * all / a.splits);
  const int hi = static_cast<int>(static_cast<long long>(split + 1) * all / a.splits);

  using Slots = Ring<Cta<F8, NT>::kSlots>;
  if (warp == 0 || warp == 6) {
    const int half = warp == 6;
    const uint64_t pol = l2_policy_evict_first();
    int act = lo / kch, j = lo - act * kch, it = 0;
    for (; it < hi - lo; ++it) {
      if (!c.claim(it, a.err)) break;
      // rows behind the last are filled with zeros
      if (elect_one()) c.bring(it, half, &a.d, j * P::kChunk, m0 + half * 64, p.expert[act], pol);
      __syncwarp();
      if (++j == kch) {
        j = 0;
        ++act;
      }
    }
    if (lane == 0) c.ends[half] = it;
  } else if (c.kOwn && warp >= 7) {
    const Runs r(p.active, a, P::kChunk);
    const int mine = warp - 7;
    // the next chunk's places are worked out while this one's values come
    auto place = [&](int it) {
      const int act = min(lo + it, all - 1) / kch, j = lo + it - act * kch;
      return Inner<F8>(a, r, act, p.first[act], 0, j);
    };
    // without a chunk (with no expert at all there is none) there is no place: j behind the last
    Inner<F8> at = hi > lo ? place(mine) : Inner<F8>(a, r, 0, 0, 0, kch);
    pdl_wait();  // gate and up products
    for (int it = mine; it < hi - lo; it += kMoeOwnWarps) {
      const int act = (lo + it) / kch, count = p.count[act];
      Inner<F8> two = at;
      ++two.row;
      ++two.rank;
      float x[2][P::kVals];
      const float w = p.gate[at.row];
      at.get(a, w, x[0]);
      if (count == 2) two.get(a, p.gate[two.row], x[1]);
      if (it + kMoeOwnWarps < hi - lo) at = place(it + kMoeOwnWarps);
      unsigned char* slot = c.own_slot(it, a.err);
      if (!slot) break;
      put_parts(slot, lane, x[0]);
      if (count == 2) put_parts(slot + kMoeBlock, lane, x[1]);
      c.own_done(it);
    }
  } else if (warp == 7) {
    pdl_wait();  // the inner vectors
    const uint64_t pol = l2_policy_evict_last();
    Slots ring;
    uint64_t sizes = 0;
    int it = 0, tail = 0, room = c.kSlots, used;
    bool ok = true;
    for (int pos = lo; pos < hi && ok;) {
      const int act = pos / kch, j0 = pos - act * kch, n = min(kch - j0, hi - pos), count = p.count[act];
      const unsigned char* src = a.hb + (static_cast<size_t>(p.first[act]) * kch + static_cast<size_t>(j0) * count) * kMoeBlock;
      for (int j = 0; j < n; ++j, ++it, src += count * kMoeBlock) {
        const int at = ring.take(count, &used);
        ok = c.make_room(it, used, sizes, tail, room, a.err);
        if (!ok) break;
        if (elect_one()) {  // a chunk's blocks lie side by side
          const uint32_t bytes = (count - 1) * kMoeBlock + P::kCopy;
          mbar_arrive_expect_tx(&c.fullB[it % kMoeTurns], bytes);
          bulk_copy_g2s(c.B + at * c.kSlot, src, bytes, &c.fullB[it % kMoeTurns], pol);
        }
        __syncwarp();
      }
      pos += n;
    }
    if (lane == 0) c.ends[2] = it;
  } else if (warp == 1) {
    Slots ring;
    int it = 0, used;
    bool ok = true;
    for (int pos = lo; pos < hi && ok;) {
      const int act = pos / kch, n = min((act + 1) * kch, hi) - pos, count = p.count[act];
      for (int j = 0; j < n && ok; ++j, ++it) ok = c.multiply(it, count, ring.take(count, &used), a.err);
      pos += n;
    }
    if (lane == 0) c.ends[3] = it - !ok;
  } else {
    const int m = (32 * warp + lane) & 127, HB = (a.H + kFp8Block - 1) / kFp8Block;
#pragma unroll
    for (int t = 0; t < NT; ++t) c.total[t * 128 + m] = 0.f;
    Slots ring;
    int it = 0, used;
    bool ok = true;
    for (int pos = lo; pos < hi && ok;) {
      const int act = pos / kch, j0 = pos - act * kch, n = min(kch - j0, hi - pos), count = p.count[act];
      float sum[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) sum[t] = 0.f;
      const float* sw = nullptr;
      float next = 1.f;
      if (F8) {
        sw = a.sd + (static_cast<size_t>(p.expert[act]) * HB + m0 / kFp8Block) * kch;
        next = sw[j0];
      }
      for (int j = j0; j < j0 + n && ok; ++j, ++it) {
        const float w = next;
        if (F8 && j + 1 < j0 + n) next = sw[j + 1];
        ok = c.add(it, count, ring.take(count, &used), w, sum, a.err);
      }
      // this thread's column of its tokens' sums
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (t >= count) break;
        c.total[p.token[p.first[act] + t] * 128 + m] += sum[t];
      }
      pos += n;
    }
  }
  __syncwarp();
  pdl_wait();  // every thread: the launches before are complete before this one is
  __syncthreads();
  // [tile][split][T][128]
  const int n4 = a.T * 32;
  float4* mine = reinterpret_cast<float4*>(a.sums) + (static_cast<size_t>(tile) * a.splits + split) * n4;
  for (int i = threadIdx.x; i < n4; i += c.kThreads) mine[i] = reinterpret_cast<const float4*>(c.total)[i];
  c.end(a.err);
}

// ----------------------------------------------------------------------------- host side

template <bool F8, int NT>
cudaError_t run_experts(MoeArgs& a, cudaStream_t st) {
  using P = Parts<F8>;
  using C = Cta<F8, NT>;
  constexpr int kWarps = kMoeFlat / 32;
  const int blocks = a.T * ((a.H + P::kChunk - 1) / P::kChunk), rows = a.T * a.k * ((a.I + P::kChunk - 1) / P::kChunk);
  cudaError_t e = cudaSuccess;
  if (!C::kOwn) e = launch(moe_prep_kernel<F8>, dim3(1 + (blocks + kWarps - 1) / kWarps), dim3(kMoeFlat), 0, st, true, a);
  if (e == cudaSuccess) e = launch(moe_gate_up_kernel<F8, NT>, dim3(a.ctas), dim3(C::kThreads), C::kSmem, st, true, a);
  if (!C::kOwn && e == cudaSuccess)
    e = launch(moe_act_kernel<F8>, dim3((rows + kWarps - 1) / kWarps), dim3(kMoeFlat), 0, st, true, a);
  if (e != cudaSuccess) return e;
  // K splits of a tile of the down product: as many CTAs as run at once, each with two chunks if all choices differ
  const int tiles = (a.H + 127) / 128;
  a.splits = std::max(1, std::min({a.ctas / tiles, kMoeMaxSplits, rows / 2}));
  e = launch(moe_down_kernel<F8, NT>, dim3(tiles * a.splits), dim3(C::kThreads), C::kSmem, st, true, a);
  if (e != cudaSuccess) return e;
  return launch(moe_sum_kernel, dim3((a.T * (a.H / 4) + 127) / 128), dim3(128), 0, st, true, a);
}

template <bool F8, int NT>
cudaError_t allow_one() {
  cudaError_t e = prefer_max_carveout(moe_prep_kernel<F8>);
  if (e == cudaSuccess) e = prefer_max_carveout(moe_act_kernel<F8>);
  if (e == cudaSuccess) e = prefer_max_carveout(moe_sum_kernel);
  if (e == cudaSuccess) e = allow_smem(moe_gate_up_kernel<F8, NT>);
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
      !make_tmap_mats(&a.d, c.wd, bytes, c.I, c.H, c.E, kMoeUnit)) {
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
  const MoeWorkspace w = moe_workspace(c.T, c.k, c.H, c.I);
  a.plan = reinterpret_cast<Plan*>(c.ws);
  a.main = reinterpret_cast<float*>(c.ws + w.main);
  a.cut = reinterpret_cast<float*>(c.ws + w.cut);
  a.sums = reinterpret_cast<float*>(c.ws + w.sums);
  a.xb = c.ws + w.xb;
  a.hb = c.ws + w.hb;
  a.T = c.T;
  a.k = c.k;
  a.E = c.E;
  a.H = c.H;
  a.I = c.I;
  a.ctas = std::min(2 * sms, kMoeMaxCtas);
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
