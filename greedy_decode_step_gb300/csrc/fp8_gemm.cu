// Matrix product of 8-bit rows and weights with a scale per block of 128, on
// the 5th-generation tensor cores:
//
//   out[m][n] = res[m][n] + sum_kb sx[m][kb] sw[n / 128][kb] P_kb[m][n],
//   P_kb[m][n] = sum over the 128 values of block kb of xc[m][k] wc[n][k]
//
// Products of e4m3 codes are exact; the tensor core adds a block's 128 of them
// in fp32 (tcgen05.mma kind::f8f6f4, K = 32 per instruction), and the block's
// sum leaves tensor memory to meet its two scales in fp32 registers.  The
// scales are any floats, so they cannot ride along in the instruction (its
// block-scaled form takes powers of two per 32 values).  While the epilogue
// warps add block kb, the tensor core fills the other of two accumulators with
// block kb + 1.
//
// Two forms of one pipeline (a TMA producer lane, an MMA lane, epilogue warps):
//
// * narrow: few rows.  The 128 lanes of an accumulator are weight rows, its
//   BN columns the rows of x, so a decode step's few rows waste no tensor
//   time.  Bound by the weight stream: K is split over a cluster of CTAs
//   until the GPU is full, and the splits are added through distributed shared
//   memory in rank order.
// * wide: many rows.  The lanes are 128 rows of x, 256 columns of weight rows,
//   so that a thread's scale is one register per block and half tile: 128
//   FMAs and 4 TMEM loads per thread and block, next to 685 cycles of the tensor
//   core.  Persistent CTAs, so the store of one tile runs beside the
//   products of the next.
//
// Every wait on an mbarrier is bounded: an error bit and an early end instead of a
// hang, in which one thread waits, bounded as well, for the copies and products
// that are still on their way before shared and tensor memory are given up.
// Cluster barriers and the allocation of tensor memory have no limit of their own:
// a cluster's CTAs are resident together, every role comes to its end, and a kernel
// holds no more tensor memory than leaves room for all CTAs of an SM.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <mutex>

#include "dec_fp8.cuh"
#include "dec_launch.cuh"
#include "dec_long.cuh"
#include "dec_tc.cuh"

namespace dec {
namespace {

constexpr int kF8BM = 128;                    // accumulator lanes
constexpr int kF8BK = kFp8Block;              // K per stage: one scale block, one 128-byte swizzle row
constexpr uint32_t kF8Tile = kF8BM * kF8BK;   // 16 KB: 128 rows of a stage
constexpr uint32_t kF8Head = 1024;            // barriers
constexpr int kNarrowGroup = 8;               // blocks whose scales are fetched together
constexpr int kNarrowAccs = 4;                // accumulators in turn
constexpr uint32_t kNarrowHead = kF8Head + 2 * kNarrowGroup * 32 * 4;  // barriers, and two groups' scales per row of x

// ----------------------------------------------------------------------------- narrow: weight rows on the lanes

constexpr int kNarrowThreads = 192;
constexpr int kNarrowMaxStages = 12;
constexpr int kNarrowMaxSplits = 8;

constexpr uint32_t kNarrowSmemMax = 112 * 1024;  // two CTAs per SM

template <int BN>
constexpr int narrow_stages() {
  constexpr int fit = static_cast<int>((kNarrowSmemMax - 1024 - kNarrowHead) / (kF8Tile + BN * kF8BK));
  return fit < kNarrowMaxStages ? fit : kNarrowMaxStages;
}
template <int BN>
constexpr uint32_t narrow_smem() {
  return 1024 + kNarrowHead + narrow_stages<BN>() * (kF8Tile + BN * kF8BK);
}

struct NarrowArgs {
  CUtensorMap wmap, xmap;  // box 128 rows of wc, BN rows of xc
  const float *sx, *sw, *residual;
  float* out;
  long long ldr, ldo;
  int M, N, KB, n_tiles, splits;
  uint32_t* err;
};

template <int BN>
__global__ void __launch_bounds__(kNarrowThreads, 1) fp8_narrow_kernel(const __grid_constant__ NarrowArgs a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);
  uint64_t* empty = full + kNarrowMaxStages;
  uint64_t* accum = empty + kNarrowMaxStages;  // an accumulator holds a block
  uint64_t* drained = accum + kNarrowAccs;     // it has been read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + kNarrowAccs);
  volatile int* stop = reinterpret_cast<volatile int*>(tmem_slot + 1);  // a wait ran out: every role ends
  volatile int* ends = stop + 1;                                        // stages asked for, and multiplied
  float(*scales)[BN] = reinterpret_cast<float(*)[BN]>(smem + kF8Head);  // [2 groups x blocks]
  static_assert(kF8Head + 2 * kNarrowGroup * BN * 4 <= kNarrowHead, "scales");
  unsigned char* tiles = smem + kNarrowHead;
  constexpr uint32_t kXTile = BN * kF8BK, kStage = kF8Tile + kXTile;
  constexpr int kStages = narrow_stages<BN>();
  constexpr uint32_t kCols = tmem_columns(kNarrowAccs * BN);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x % a.splits, tile = blockIdx.x / a.splits;
  const int m0 = (tile / a.n_tiles) * kF8BM;  // weight rows
  const int r0 = (tile % a.n_tiles) * BN;     // rows of x
  const int kb0 = static_cast<int>(static_cast<long long>(split) * a.KB / a.splits);
  const int nkb = static_cast<int>(static_cast<long long>(split + 1) * a.KB / a.splits) - kb0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kNarrowAccs; ++s) {
      mbar_init(&accum[s], 1);
      mbar_init(&drained[s], 4);
    }
    *stop = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    const uint64_t wpol = l2_policy_evict_first(), xpol = l2_policy_evict_last();
    auto bring_w = [&](int i) {
      tma_load_3d(tiles + i % kStages * kStage, &a.wmap, (kb0 + i) * kF8BK, m0, 0, &full[i % kStages], wpol);
    };
    auto bring_x = [&](int i) {
      tma_load_3d(tiles + i % kStages * kStage + kF8Tile, &a.xmap, (kb0 + i) * kF8BK, r0, 0, &full[i % kStages], xpol);
    };
    // Ahead of the wait the first weights are asked into L2 only: whichever launch made them, theirs are the bytes that the
    // copies behind the wait bring.  (Copies issued here would read what the launch ahead has not written yet, or not
    // made visible: only the wait does that.)
    const int pre = min(nkb, kStages);
    if (elect_one())
      for (int i = 0; i < pre; ++i) tma_prefetch_3d(&a.wmap, (kb0 + i) * kF8BK, m0, 0, wpol);
    __syncwarp();
    pdl_wait();
    pdl_launch_dependents();
    int it = 0;
    bool ok = true;
    for (; it < nkb; ++it) {
      ok = it < kStages || warp_wait(&empty[it % kStages], ((it / kStages) - 1) & 1, stop, a.err, kErrWaitEmpty);
      if (!ok) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(&full[it % kStages], kStage);
        bring_w(it);
        bring_x(it);
      }
      __syncwarp();
    }
    if (!ok) *stop = 1;
    if (lane == 0) ends[0] = it;
  } else if (warp == 1) {
    constexpr uint32_t idesc = tc_idesc_of(BN, false);
    bool ok = true;
    int i = 0;
    for (; i < nkb; ++i) {
      const int s = i % kStages, b = i % kNarrowAccs;
      ok = warp_wait(&full[s], (i / kStages) & 1, stop, a.err, kErrWaitFull) &&
           (i < kNarrowAccs || warp_wait(&drained[b], ((i / kNarrowAccs) - 1) & 1, stop, a.err, kErrWaitFull));
      if (!ok) break;
      tc_fence_after();
      const uint32_t sa = smem_addr(tiles + s * kStage);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kF8BK / 32; ++kk)
          tc_mma_f8(tmem + b * BN, smem_desc_sw128(sa + kk * 32), smem_desc_sw128(sa + kF8Tile + kk * 32), idesc, kk > 0);
        tc_commit(&empty[s]);
        tc_commit(&accum[b]);
      }
      __syncwarp();
    }
    if (!ok) *stop = 1;
    if (lane == 0) ends[1] = i;
  } else {
    pdl_wait();
    const int q = warp & 3, t = threadIdx.x - 64;
    const int m = m0 + 32 * q + lane;
    const uint32_t at = tmem + (static_cast<uint32_t>(32 * q) << 16);
    float acc[BN];
#pragma unroll
    for (int j = 0; j < BN; ++j) acc[j] = 0.f;
    // the 128 threads bring the products of a group's scales, the next group's while this one is added
    constexpr int kEach = kNarrowGroup * BN / 128;
    const float* sw = a.sw + static_cast<long long>(m0 / kFp8Block) * a.KB + kb0;
    float next[kEach];
    auto fetch = [&](int first) {
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        const int i = first + (t + 128 * e) / BN, r = r0 + t % BN;
        next[e] = i < nkb && r < a.M ? a.sx[static_cast<long long>(r) * a.KB + kb0 + i] * sw[i] : 0.f;
      }
    };
    fetch(0);
    bool ok = nkb > 0;
    for (int i = 0; i < nkb; ++i) {
      const int b = i % kNarrowAccs, turn = i / kNarrowGroup & 1;
      if (i % kNarrowGroup == 0) {
#pragma unroll
        for (int e = 0; e < kEach; ++e) scales[turn * kNarrowGroup + (t + 128 * e) / BN][t % BN] = next[e];
        fetch(i + kNarrowGroup);
        asm volatile("bar.sync 1, 128;" ::: "memory");
      }
      const float* scale = scales[turn * kNarrowGroup + i % kNarrowGroup];
      ok = warp_wait(&accum[b], (i / kNarrowAccs) & 1, stop, a.err, kErrWaitFull);
      if (!ok) *stop = 1;
      tc_fence_after();
      if (ok) {
#pragma unroll
        for (int c = 0; c < BN; c += 16) {
          uint32_t v[16];
          tmem_ld_issue(at + b * BN + c, v);
          tmem_ld_wait(v);
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[c + j] = fmaf(__uint_as_float(v[j]), scale[c + j], acc[c + j]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&drained[b]);
    }
    if (a.splits == 1) {
      if (ok && m < a.N) {
#pragma unroll
        for (int j = 0; j < BN; ++j) {
          const int r = r0 + j;
          if (r < a.M) a.out[r * a.ldo + m] = acc[j] + (a.residual ? a.residual[r * a.ldr + m] : 0.f);
        }
      }
    } else {
      // the ring is done: every block's products have been committed
      float* part = reinterpret_cast<float*>(tiles);
#pragma unroll
      for (int j = 0; j < BN; ++j) part[j * kF8BM + 32 * q + lane] = acc[j];
    }
  }
  __syncwarp();
  if (a.splits > 1) {
    pdl_wait();  // every thread writes the result here
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    const uint32_t local = smem_addr(tiles);
    const int rows = min(BN, a.M - r0), total = rows * kF8BM, per = (total + a.splits - 1) / a.splits;
    const int end = min(total, (split + 1) * per);
    for (int o = split * per + static_cast<int>(threadIdx.x); o < end; o += kNarrowThreads) {
      const int r = r0 + o / kF8BM, m = m0 + o % kF8BM;
      float x[kNarrowMaxSplits];
#pragma unroll
      for (int k = 0; k < kNarrowMaxSplits; ++k) {
        x[k] = 0.f;
        if (k < a.splits) {
          uint32_t remote;
          asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local + 4u * o), "r"(k));
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x[k]) : "r"(remote));
        }
      }
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < kNarrowMaxSplits; ++k) sum += x[k];
      if (m < a.N) a.out[r * a.ldo + m] = sum + (a.residual ? a.residual[r * a.ldr + m] : 0.f);
    }
    __syncwarp();
    // no CTA leaves while others may still read its shared memory
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    if (*stop) {  // after an early end: copies and products that are still on their way
      if (lane == 0) {
        drain_ring(full, kStages, ends[0], a.err);
        drain_ring(empty, kStages, ends[1], a.err);
      }
      __syncwarp();
    }
    tc_fence_after();
    tmem_free(tmem, kCols);
  }
}

// ----------------------------------------------------------------------------- wide: rows of x on the lanes

constexpr int kWideThreads = 384;   // warp 0 copies, 1 and 2 multiply, 4-11 scale and store
constexpr int kWideMaxStages = 6;
// Tiles of BN weight rows, 64, 128, 192 or 256, by 128 rows of x; PAIR: by 256,
// 128 in each of two CTAs (cta_group::2) that hold half of the weight rows each.
// A pair reads two thirds of the bytes from L2 and shared memory per product,
// and the tensor core takes 512 cycles a block where it takes 685 alone.
//
// How results leave: as they are, by tensor copies; the same on top of a residual
// that tensor copies bring into the staging rows while the tile is multiplied;
// or row by row, where rows of either are not whole 16 bytes.  (Each in a kernel
// of its own: with all in one the loop over blocks took 7 % longer, 8191 x 2560 x
// 19456 in 406 us where 378.)
enum Out { kPlain, kAdd, kRows };

template <int BN, bool PAIR, Out OUT>
struct Wide {
  static constexpr int kBRows = PAIR ? BN / 2 : BN;  // weight rows of a CTA
  static constexpr uint32_t kStage = kF8Tile + kBRows * kF8BK;
  static constexpr int kBufs = !PAIR ? 2 : OUT == kAdd ? 4 : 3;  // 32 rows of 32 results per warp, on their way out
  static constexpr uint32_t kOut = 8 * kBufs * 32 * 128;
  static constexpr int kFit = static_cast<int>((kSmemMax - 1024 - kF8Head - kOut) / kStage);
  static constexpr int kStages = kFit < kWideMaxStages ? kFit : kWideMaxStages;  // 3 at 256, 4 as a pair (3 with a residual)
  static constexpr uint32_t kSmem = 1024 + kF8Head + kStages * kStage + kOut;
  static constexpr int kChunks = BN / 64;  // of 32 columns, per epilogue warp
};

struct WideArgs {
  CUtensorMap wmap, xmap;  // box BN rows of wc, 128 rows of xc
  CUtensorMap omap, rmap;  // of the result, if `bulk`, and of the residual for kAdd
  const float *sx, *sw, *residual;
  float* out;
  long long ldr, ldo;
  int M, N, KB, NB, m_tiles, tiles;
  int bulk;    // rows of the result are whole 16 bytes: tensor copies store them
  uint32_t* err;
};

template <int BN, bool PAIR, Out OUT>
__global__ void __launch_bounds__(kWideThreads, 1) fp8_wide_kernel(const __grid_constant__ WideArgs a) {
  using W = Wide<BN, PAIR, OUT>;
  constexpr int kWideStages = W::kStages, kChunks = W::kChunks, kCtas = PAIR ? 2 : 1;
  constexpr uint32_t kWideStage = W::kStage, kCols = tmem_columns(2 * BN);
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // done: a stage's products are in its accumulator, and the stage may be filled anew
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);
  uint64_t* done = full + kWideStages;
  uint64_t* drained = done + kWideStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 2);
  volatile int* stop = reinterpret_cast<volatile int*>(tmem_slot + 1);  // a wait ran out: every role ends
  volatile int* ends = stop + 1;  // stages that each CTA asked for, and the last that each issuing warp multiplied
  uint64_t* came = reinterpret_cast<uint64_t*>(smem + kF8Head / 2);     // kAdd: a warp's staging rows hold the residual
  static_assert((2 * kWideMaxStages + 5) * 8 <= kF8Head / 2 && 8 * W::kBufs * 8 <= kF8Head / 2, "barriers");
  unsigned char* tiles = smem + kF8Head;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = PAIR ? blockIdx.x & 1 : 0, first = blockIdx.x / kCtas, step = gridDim.x / kCtas;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kWideStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&done[s], 1);
    }
    for (int s = 0; s < 2; ++s) mbar_init(&drained[s], 8 * kCtas);
    if (OUT == kAdd)
      for (int s = 0; s < 8 * W::kBufs; ++s) mbar_init(&came[s], 1);
    *stop = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    if (PAIR)
      tmem_alloc_pair(tmem_slot, kCols);
    else
      tmem_alloc(tmem_slot, kCols);
  }
  tc_fence_before();
  if (PAIR) {  // the other CTA's barriers are set up, too
    cluster_arrive();
    cluster_wait();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto leave = [&] {  // every thread, at its end
    __syncwarp();
    tc_fence_before();
    if (PAIR) {  // neither CTA leaves while the other may reach into it
      if (*stop && lane == 0) store_other(const_cast<int*>(stop), 1);
      cluster_arrive();
      cluster_wait();
    }
    asm volatile("bar.sync 1, %0;" ::"n"(kWideThreads) : "memory");
  };
  // 128 threads x 40 + 256 x 232 registers = the 384 x 168 of the launch.  What runs with fewer or more stands in its
  // own branch to the end of the kernel, so that no value has to be held in one place by both.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0) {
      const uint64_t keep = l2_policy_evict_last();
      // a pair's copies complete on the even CTA's barrier
      auto bring = [&](const CUtensorMap* map, int it, uint32_t at, int kb, int row) {
        const int s = it % kWideStages;
        unsigned char* to = tiles + s * kWideStage + at;
        if (PAIR)
          tma_load_3d_pair(to, map, kb * kF8BK, row, 0, in_even(&full[s]), keep);
        else
          tma_load_3d(to, map, kb * kF8BK, row, 0, &full[s], keep);
      };
      // the first weights into L2 ahead of the wait, as in the narrow form
      const int pre = first < a.tiles ? min(a.KB, kWideStages) : 0;
      if (elect_one())
        for (int i = 0; i < pre; ++i) tma_prefetch_3d(&a.wmap, i * kF8BK, first / a.m_tiles * BN + rank * W::kBRows, 0, keep);
      __syncwarp();
      pdl_wait();
      pdl_launch_dependents();
      int it = 0;
      bool ok = true;
      for (int tile = first; tile < a.tiles && ok; tile += step) {
        const int m0 = (tile % a.m_tiles * kCtas + rank) * kF8BM, n0 = (tile / a.m_tiles) * BN + rank * W::kBRows;
        for (int kb = 0; kb < a.KB; ++kb, ++it) {
          if (it >= kWideStages)
            ok = warp_wait(&done[it % kWideStages], ((it / kWideStages) - 1) & 1, stop, a.err, kErrWaitEmpty);
          if (!ok) break;
          if (elect_one()) {
            if (rank == 0) mbar_arrive_expect_tx(&full[it % kWideStages], kCtas * kWideStage);
            bring(&a.xmap, it, 0, kb, m0);
            bring(&a.wmap, it, kF8Tile, kb, n0);
          }
          __syncwarp();
        }
      }
      if (!ok) *stop = 1;
      if (lane == 0) {
        if (PAIR)
          store_cta0(const_cast<int*>(ends + rank), it);
        else
          ends[0] = it;
      }
    } else if ((warp == 1 || warp == 2) && rank == 0) {
      // every second block each, so that one waits for its next while the other's products are being issued
      constexpr uint32_t idesc = PAIR ? tc_idesc_pair(BN) : tc_idesc_of(BN, false);
      const int b = warp - 1;
      const int mine = (a.tiles - first + step - 1) / step;
      bool ok = true;
      int it = b;
      for (; it < mine * a.KB; it += 2) {
        const int s = it % kWideStages;
        // The accumulator first: once block it - 2 has been read, every block before it, the one that held this stage
        // among them, is done.  Of an odd number of stages a warp sees every second phase only, and asked too early
        // the parity would answer for the phase before the last.
        ok = (it < 2 || warp_wait(&drained[b], ((it >> 1) - 1) & 1, stop, a.err, kErrWaitFull)) &&
             warp_wait(&full[s], (it / kWideStages) & 1, stop, a.err, kErrWaitFull);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sa = smem_addr(tiles + s * kWideStage);
        if (elect_one()) {
  #pragma unroll
          for (int kk = 0; kk < kF8BK / 32; ++kk) {
            const uint64_t ad = smem_desc_sw128(sa + kk * 32), bd = smem_desc_sw128(sa + kF8Tile + kk * 32);
            if (PAIR)
              tc_mma_f8_pair(tmem + b * BN, ad, bd, idesc, kk > 0);
            else
              tc_mma_f8(tmem + b * BN, ad, bd, idesc, kk > 0);
          }
          if (PAIR)
            tc_commit_pair(&done[s]);
          else
            tc_commit(&done[s]);
        }
        __syncwarp();
      }
      if (!ok) *stop = 1;
      if (lane == 0) ends[2 + b] = it - 2;  // below 0: none
    }
    leave();
    if (*stop) {  // after an early end of either CTA: copies and products that are still on their way
      if (warp == 1 && lane == 0 && rank == 0) {
        drain_ring(full, kWideStages, PAIR ? max(ends[0], ends[1]) : ends[0], a.err);
        for (int b = 0; b < 2; ++b)
          if (ends[2 + b] >= 0) tc_wait(&done[ends[2 + b] % kWideStages], (ends[2 + b] / kWideStages) & 1, a.err, kErrDrain);
      }
      __syncwarp();
      if (PAIR) cluster_arrive();
      if (PAIR) cluster_wait();
    }
    if (warp == 1) {
      tc_fence_after();
      if (PAIR)
        tmem_free_pair(tmem, kCols);
      else
        tmem_free(tmem, kCols);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    const int q = warp & 3, half = (warp - 4) >> 2;  // TMEM lanes 32 q .., columns BN / 2 half ..
    unsigned char* stages = tiles + kWideStages * kWideStage + (warp - 4) * W::kBufs * 32 * 128;
    const uint32_t at = tmem + (static_cast<uint32_t>(32 * q) << 16) + half * (BN / 2);
    auto release = [&](int b) {  // this warp has read accumulator b
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR)
          mbar_arrive_cluster(in_even(&drained[b]));
        else
          mbar_arrive(&drained[b]);
      }
    };
    int it = 0, turn = 0, m0, n0, cut;
    came += (warp - 4) * W::kBufs;
    uint32_t phases = 0, coming = 0;  // a bit per buffer: the phase to wait for, a copy on its way
    auto bring = [&](int c) {         // chunk c of the residual of the tile at (m0, n0), into a buffer that is free
      const int buf = c % W::kBufs;
      coming |= 1u << buf;
      if (lane == 0) {
        mbar_arrive_expect_tx(&came[buf], 32 * 128);
        tma_load_2d(stages + buf * 32 * 128, &a.rmap, n0 + 32 * c, m0, &came[buf], l2_policy_evict_first());
      }
    };
    const float *sx, *sw, *sv;
    float x0, w0, v0, x1, w1, v1;
    auto open = [&](int tile) {  // its place, and the scales of its first two blocks
      m0 = (tile % a.m_tiles * kCtas + rank) * kF8BM + 32 * q;
      n0 = (tile / a.m_tiles) * BN + BN / 2 * half;
      // the columns of a warp lie in one block of weight rows, at BN = 192 in two
      const int nb = n0 / kFp8Block;
      cut = BN == 192 ? (nb + 1) * kFp8Block - n0 : BN;
      sx = a.sx + static_cast<long long>(min(m0 + lane, a.M - 1)) * a.KB;
      sw = a.sw + static_cast<long long>(min(nb, a.NB - 1)) * a.KB;
      sv = a.sw + static_cast<long long>(min(nb + 1, a.NB - 1)) * a.KB;
      const int one = a.KB > 1;
      x0 = *sx, w0 = *sw, v0 = BN == 192 ? *sv : 0.f;
      x1 = sx[one], w1 = sw[one], v1 = BN == 192 ? sv[one] : 0.f;
    };
    pdl_wait();  // the rows' scales and the residual
    open(first);
    for (int tile = first; tile < a.tiles; tile += step) {
      float acc[BN / 2];
#pragma unroll
      for (int j = 0; j < BN / 2; ++j) acc[j] = 0.f;
      if (OUT == kAdd && m0 < a.M) {
        tma_store_wait_read<0>();  // the tile before has left the buffers
#pragma unroll
        for (int c = 0; c < kChunks && c < W::kBufs; ++c)
          if (n0 + 32 * c < a.N) bring(c);
      }
      if (OUT == kRows && a.residual && m0 + lane < a.M) {  // a lane's row of the residual is in L2 by the time it is added
        const float* res = a.residual + static_cast<long long>(m0 + lane) * a.ldr + n0;
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          if (n0 + 32 * c < a.N) asm volatile("prefetch.global.L2 [%0];" ::"l"(res + 32 * c));
      }
      bool ok = true;
      for (int kb = 0; kb < a.KB; ++kb, ++it) {
        const int b = it & 1;
        const float s = x0 * w0, s2 = x0 * v0;
        x0 = x1;
        w0 = w1;
        v0 = v1;
        if (kb + 2 < a.KB) {
          x1 = sx[kb + 2];
          w1 = sw[kb + 2];
          if (BN == 192) v1 = sv[kb + 2];
        }
        ok = warp_wait(&done[it % kWideStages], (it / kWideStages) & 1, stop, a.err, kErrWaitFull);
        if (!ok) break;
        tc_fence_after();
        // 64 columns asked for at once, added while the next 32 come
        uint32_t v[2][32];
        tmem_ld_issue32(at + b * BN, v[0]);
        tmem_ld_wait32(v[0]);
        if (kChunks == 1) release(b);
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          if (c + 1 < kChunks) tmem_ld_issue32(at + b * BN + 32 * (c + 1), v[(c + 1) & 1]);
          const float f = BN == 192 && 32 * c >= cut ? s2 : s;
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[32 * c + j] = fmaf(__uint_as_float(v[c & 1][j]), f, acc[32 * c + j]);
          if (c + 1 < kChunks) tmem_ld_wait32(v[(c + 1) & 1]);
          if (c + 2 == kChunks) release(b);
        }
      }
      if (!ok) {
        *stop = 1;
        break;
      }
      const int out_m = m0, out_n = n0;
      // 32 columns at a time through shared memory (rows of 128 bytes, their 16-byte pieces swizzled), so that whole
      // lines leave: by a tensor copy, which runs beside the next tile, or by a warp a row
      auto mine = [&](unsigned char* stage, int j) { return reinterpret_cast<float4*>(stage + lane * 128 + ((j ^ (lane & 7)) << 4)); };
      auto send = [&](unsigned char* stage, int n) {  // by the lane that waits for it
        fence_to_async();
        __syncwarp();
        if (lane == 0) tma_store_2d(&a.omap, stage, n, out_m);
      };
      if (OUT == kAdd) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          const int n = out_n + 32 * c, buf = c % W::kBufs;
          if (ok && n < a.N && out_m < a.M) {  // warp-uniform
            unsigned char* stage = stages + buf * 32 * 128;
            ok = warp_wait(&came[buf], phases >> buf & 1, stop, a.err, kErrWaitFull);
            if (ok) {
              phases ^= 1u << buf;
              coming &= ~(1u << buf);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float4 r = *mine(stage, j);
                *mine(stage, j) = make_float4(acc[32 * c + 4 * j] + r.x, acc[32 * c + 4 * j + 1] + r.y,
                                              acc[32 * c + 4 * j + 2] + r.z, acc[32 * c + 4 * j + 3] + r.w);
              }
              send(stage, n);
              if (c + W::kBufs < kChunks && n + 32 * W::kBufs < a.N) {
                tma_store_wait_read<0>();
                bring(c + W::kBufs);
              }
            }
          }
        }
        if (!ok) {
          *stop = 1;
          break;
        }
        open(min(tile + step, a.tiles - 1));
        continue;
      }
      open(min(tile + step, a.tiles - 1));  // the next tile's scales come while this one's results leave
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int n = out_n + 32 * c;
        if (n < a.N && out_m < a.M) {  // warp-uniform
          unsigned char* stage = stages + turn % W::kBufs * 32 * 128;
          ++turn;
          if (OUT == kPlain || a.bulk) tma_store_wait_read<W::kBufs - 1>();  // what this buffer held has left
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *mine(stage, j) = make_float4(acc[32 * c + 4 * j], acc[32 * c + 4 * j + 1], acc[32 * c + 4 * j + 2], acc[32 * c + 4 * j + 3]);
          if (OUT == kRows) {  // a lane a column, 8 rows at once
            __syncwarp();
            const int rows = min(32, a.M - out_m);
            const bool in = n + lane < a.N;
            float* dst = a.out + static_cast<long long>(out_m) * a.ldo + n + lane;
            const float* res = a.residual ? a.residual + static_cast<long long>(out_m) * a.ldr + n + lane : nullptr;
            unsigned char* from = stage + 4 * (lane & 3);
#pragma unroll 1
            for (int r8 = 0; r8 < rows; r8 += 8, from += 8 * 128) {
              float v[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                v[k] = 0.f;
                if (res && in && r8 + k < rows) v[k] = *res;
                if (res) res += a.ldr;
              }
#pragma unroll
              for (int k = 0; k < 8; ++k)
                v[k] += *reinterpret_cast<const float*>(from + k * 128 + (((lane >> 2) ^ k) << 4));
              if (a.bulk) {
#pragma unroll
                for (int k = 0; k < 8; ++k) *reinterpret_cast<float*>(from + k * 128 + (((lane >> 2) ^ k) << 4)) = v[k];
              } else {
#pragma unroll
                for (int k = 0; k < 8; ++k, dst += a.ldo)
                  if (in && r8 + k < rows) *dst = v[k];
              }
            }
          }
          if (OUT == kPlain || a.bulk) send(stage, n);
        }
      }
    }
    if (OUT == kAdd && lane == 0)  // after an early end only: its own copies
      for (int buf = 0; buf < W::kBufs; ++buf)
        if (coming >> buf & 1) tc_wait(&came[buf], phases >> buf & 1, a.err, kErrDrain);
    if (OUT != kRows || a.bulk) tma_store_wait_read<0>();  // its memory is in use until then
    leave();
    if (PAIR && *stop) {  // as above
      cluster_arrive();
      cluster_wait();
    }
  }
}

// ----------------------------------------------------------------------------- host side

// Clusters of `size` CTAs that run at once on the current device, 0 if the
// query fails; what it answered is kept per device.  It counts one CTA per SM
// wherever tensor memory is used; two fit here.
template <int BN>
int narrow_clusters(int size) {
  constexpr int kDevices = 64;
  static std::mutex mu;
  static int cache[kDevices][kNarrowMaxSplits + 1] = {};
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  const bool keep = dev >= 0 && dev < kDevices;
  std::lock_guard<std::mutex> lock(mu);
  if (keep && cache[dev][size] != 0) return cache[dev][size];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(size * 64);
  cfg.blockDim = dim3(kNarrowThreads);
  cfg.dynamicSmemBytes = narrow_smem<BN>();
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(size);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, fp8_narrow_kernel<BN>, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;
  }
  if (keep) cache[dev][size] = 2 * n;
  return 2 * n;
}

// K splits: double while every split keeps two blocks and all clusters run at
// once (76 clusters of 4, four more than fit, took 13.2 us where 2 take 8).
template <int BN>
int narrow_splits(long long tiles, int KB, int sms) {
  int splits = 1;
  while (splits * 2 <= kNarrowMaxSplits && tiles * splits * 2 <= 2ll * sms && KB / (splits * 2) >= 2 &&
         narrow_clusters<BN>(splits * 2) >= tiles)
    splits *= 2;
  return splits;
}

// Which form is quickest, by what each took per wave of CTAs and block of K
// (us, fitted to M = 16 .. 8192 with K = 2560 and 8960, within 10 %):
//   narrow, 16 or 32 rows, two CTAs per SM:          5 + waves (0.37 or 0.45 KB / splits)
//   wide, tiles of 64, 128, 192, 256 columns, pairs: 4 + waves (0.8, 1.6, 1.9, 2.2, 3.1 +
//                                                               0.214, 0.27, 0.36, 0.456, 0.39 KB)
// e.g. 64 x 9728 x 2560: 10.9 narrow, 9.0 wide 64; 512 x 1536 x 8960: 31 narrow,
// 20.6 wide 64, 38 wide 256; 509 x 6144 x 2560: 17.6, 13.0, 16.0, 15.9 wide 128,
// 192, 256 and pairs; 8192 x 9728 x 2560: 225, 200, 182, 175.
// Tiles of 192 and 256 columns hold two thirds and half of a residual's chunks ahead
// where pairs hold all: 4096 x 9728 x 528 in 72 us, 61 as pairs; 2050 x 9728 x 272 in
// 37, 32; 4096 x 2560 x 9728 in 97 (192), 117 as pairs.
enum Form { kNarrow16, kNarrow32, kWide64, kWide128, kWide192, kWide256, kPairs };
Form best_form(const Fp8GemmCall& c, int sms) {
  const int KB = (c.K + kF8BK - 1) / kF8BK;
  auto up = [](long long a, long long b) { return (a + b - 1) / b; };
  Form best = kPairs;
  double least = 1e30;
  auto offer = [&](Form f, double us) {
    if (us < least) {
      least = us;
      best = f;
    }
  };
  const long long n128 = up(c.N, kF8BM), t16 = up(c.M, 16) * n128, t32 = up(c.M, 32) * n128, m128 = up(c.M, kF8BM);
  const int s16 = narrow_splits<16>(t16, KB, sms), s32 = narrow_splits<32>(t32, KB, sms);
  offer(kNarrow16, 5.0 + up(t16 * s16, 2 * sms) * 0.37 * up(KB, s16));
  if (c.M > 16) offer(kNarrow32, 5.0 + up(t32 * s32, 2 * sms) * 0.45 * up(KB, s32));
  const Form wide[4] = {kWide64, kWide128, kWide192, kWide256};
  const double tile[4] = {0.8, 1.6, 1.9, 2.2}, block[4] = {0.214, 0.27, 0.36, 0.456};
  const double wait[4] = {0.0, 0.0, 1.0, 2.0};  // for a residual, from the second wave on
  for (int i = 0; i < 4; ++i) {
    const long long waves = up(m128 * up(c.N, 64 * (i + 1)), sms);
    offer(wide[i], 4.0 + waves * (tile[i] + block[i] * KB) + (c.residual ? (waves - 1) * wait[i] : 0.0));
  }
  offer(kPairs, 4.0 + up(up(c.M, 2 * kF8BM) * up(c.N, 256), sms / 2) * (3.1 + 0.39 * KB));
  return best;
}

template <int BN>
cudaError_t launch_narrow(const Fp8GemmCall& c, int sms, cudaStream_t st, const char** why) {
  static thread_local NarrowArgs a;
  std::memset(&a, 0, sizeof(a));
  if (!make_tmap_mats(&a.wmap, c.wc, 1, c.K, c.N, 1, kF8BM) || !make_tmap_mats(&a.xmap, c.xc, 1, c.K, c.M, 1, BN)) {
    *why = "a tensor map could not be made";
    return cudaErrorInvalidValue;
  }
  a.sx = c.sx;
  a.sw = c.sw;
  a.residual = c.residual;
  a.out = c.out;
  a.ldr = c.ldr;
  a.ldo = c.ldo;
  a.M = c.M;
  a.N = c.N;
  a.KB = (c.K + kF8BK - 1) / kF8BK;
  a.n_tiles = (c.M + BN - 1) / BN;
  a.err = c.err;
  const long long tiles = static_cast<long long>(a.n_tiles) * ((c.N + kF8BM - 1) / kF8BM);
  const int splits = narrow_splits<BN>(tiles, a.KB, sms);
  a.splits = splits;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * splits));
  cfg.blockDim = dim3(kNarrowThreads);
  cfg.dynamicSmemBytes = narrow_smem<BN>();
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, fp8_narrow_kernel<BN>, a);
}

template <int BN, bool PAIR, Out OUT>
cudaError_t start_wide(const WideArgs& a, int sms, cudaStream_t st) {
  constexpr int kCtas = PAIR ? 2 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(std::min(a.tiles, sms / kCtas) * kCtas);
  cfg.blockDim = dim3(kWideThreads);
  cfg.dynamicSmemBytes = Wide<BN, PAIR, OUT>::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCtas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, fp8_wide_kernel<BN, PAIR, OUT>, a);
}

template <int BN, bool PAIR>
cudaError_t launch_wide(const Fp8GemmCall& c, int sms, cudaStream_t st, const char** why) {
  static thread_local WideArgs a;
  std::memset(&a, 0, sizeof(a));
  if (!make_tmap_mats(&a.wmap, c.wc, 1, c.K, c.N, 1, Wide<BN, PAIR, kPlain>::kBRows) || !make_tmap_mats(&a.xmap, c.xc, 1, c.K, c.M, 1, kF8BM)) {
    *why = "a tensor map could not be made";
    return cudaErrorInvalidValue;
  }
  a.sx = c.sx;
  a.sw = c.sw;
  a.residual = c.residual;
  a.out = c.out;
  a.ldr = c.ldr;
  a.ldo = c.ldo;
  a.M = c.M;
  a.N = c.N;
  a.KB = (c.K + kF8BK - 1) / kF8BK;
  a.NB = (c.N + kFp8Block - 1) / kFp8Block;
  constexpr int kTileRows = kF8BM * (PAIR ? 2 : 1);
  a.m_tiles = (c.M + kTileRows - 1) / kTileRows;
  a.tiles = a.m_tiles * ((c.N + BN - 1) / BN);
  a.err = c.err;
  auto rows16 = [](const void* p, long long ld) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 4 == 0; };
  a.bulk = rows16(c.out, c.ldo) && c.ldo < (1ll << 36) && c.N % 4 == 0;  // a tensor copy cuts a row off at whole 16 bytes only
  const bool add = a.bulk && c.residual && rows16(c.residual, c.ldr) && c.ldr >= c.N && c.ldr < (1ll << 36);
  if ((a.bulk && !make_tmap_out(&a.omap, c.out, c.N, c.M, c.ldo)) ||
      (add && !make_tmap_out(&a.rmap, const_cast<float*>(c.residual), c.N, c.M, c.ldr))) {
    *why = "a tensor map could not be made";
    return cudaErrorInvalidValue;
  }
  if (add) return start_wide<BN, PAIR, kAdd>(a, sms, st);
  return a.bulk && !c.residual ? start_wide<BN, PAIR, kPlain>(a, sms, st) : start_wide<BN, PAIR, kRows>(a, sms, st);
}

template <int BN, bool PAIR>
cudaError_t allow_wide() {
  cudaError_t e = allow_smem(fp8_wide_kernel<BN, PAIR, kPlain>);
  if (e == cudaSuccess) e = allow_smem(fp8_wide_kernel<BN, PAIR, kAdd>);
  return e != cudaSuccess ? e : allow_smem(fp8_wide_kernel<BN, PAIR, kRows>);
}

}  // namespace

int fp8_gemm(const Fp8GemmCall& call, int sms, cudaStream_t st, const char** why) {
  *why = nullptr;
  Fp8GemmCall c = call;
  if (c.M == 1) c.ldo = c.ldr = (static_cast<long long>(c.N) + 3) / 4 * 4;  // one row's strides mean nothing
  cudaError_t e;
  switch (best_form(c, sms)) {
    case kNarrow16: e = launch_narrow<16>(c, sms, st, why); break;
    case kNarrow32: e = launch_narrow<32>(c, sms, st, why); break;
    case kWide64: e = launch_wide<64, false>(c, sms, st, why); break;
    case kWide128: e = launch_wide<128, false>(c, sms, st, why); break;
    case kWide192: e = launch_wide<192, false>(c, sms, st, why); break;
    case kWide256: e = launch_wide<256, false>(c, sms, st, why); break;
    default: e = launch_wide<256, true>(c, sms, st, why); break;
  }
  if (*why) return 1;
  if (e != cudaSuccess) {
    *why = cudaGetErrorString(e);
    return 3;
  }
  return 0;
}

cudaError_t allow_smem_fp8_gemm() {
  cudaError_t e;
  if ((e = allow_smem(fp8_narrow_kernel<16>)) != cudaSuccess) return e;
  if ((e = allow_smem(fp8_narrow_kernel<32>)) != cudaSuccess) return e;
  if ((e = allow_wide<64, false>()) != cudaSuccess) return e;
  if ((e = allow_wide<128, false>()) != cudaSuccess) return e;
  if ((e = allow_wide<192, false>()) != cudaSuccess) return e;
  if ((e = allow_wide<256, false>()) != cudaSuccess) return e;
  return allow_wide<256, true>();
}

}  // namespace dec
