// Decode attention over a long cache: a cache held in 4 bits, or the listed
// 64-key blocks of a bf16 cache.
//
//   o[h] = sum_j softmax_j(q[h] . k_j / sqrt(D)) v_j
//
// One pass over the keys with a running maximum and sum.  The keys of all
// (row, KV head) items are cut into units (32 keys of the 4-bit cache, 16 of
// the bf16 one), laid end to end, and every CTA takes an equal run of them; its
// warps take the run's units in turn.  Each warp has a ring of its own in shared
// memory that it fills with cp.async, so no warp waits for another inside an
// item.  At an item's end the warps' states are merged; an item cut between
// CTAs leaves one partial per CTA, which a second, small launch joins (it starts
// by programmatic launch while the first one runs).  Few and short items go to
// thread-block clusters instead, one launch.
//
// Tensor cores (mma.sync m16n8k16): a decode step has few query rows per KV
// head, so the keys take the M side and the N side holds 4 query heads twice,
// the value's upper part and its remainder in neighbouring columns.  For up to
// 4 heads per group one instruction so does the work of both parts, and each
// lane holds the score of one head: S^T = K Q^T (keys x heads),
// O^T = V^T P^T (dims x heads), P^T transposed in registers (movmatrix).
//
// 4-bit operands.  A nibble pair masked out of a word and joined to 1024 in each
// half is 1024 + c, less 1032 exactly c - 8; the next nibble pair gives
// 16 (c - 8).  The 16 is taken out of the query operand, or of the result.
// Codes have to be centred: a sum of uncentred ones runs far above its result,
// and the tensor core cuts each product at the last place of the running sum
// (1.1e-6 of the result with uncentred keys, 0.4e-6 so; 3e-5 with uncentred
// values).  The scores' group sums are scaled in fp32 by s.  For the values a
// key's s multiplies its probability, held as two halves: the product's upper
// half, and its exact error plus the lower half's product.  A power of two C
// per warp and group keeps s C below 1 and exact; a unit whose scales spread too
// far for one C is taken in several passes, each over the keys that one serves.
// The z parts are products of their own, with the (s, z) words as the other operand.
#include <cuda_fp16.h>

#include <algorithm>

#include "dec_launch.cuh"
#include "dec_long.cuh"

namespace dec {
namespace {

constexpr int kMaxG = 16;             // query heads per KV head

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(live ? BYTES : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// every copy of this thread, of groups that are not committed too
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// D += A (16x16 half, row) * B (16x8 half, col), fp32 accumulate; and from zero
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                   uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// D = A (16x8 half, row) * B (8x8 half, col)
__device__ __forceinline__ void mma_f16_1688_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, {%7, %7, %7, %7};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(b0), "f"(0.f));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t add_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// a b - c
__device__ __forceinline__ uint32_t fms_f16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("{\n .reg .b32 n;\n neg.f16x2 n, %3;\n fma.rn.f16x2 %0, %1, %2, n;\n}" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// The codes of nibbles 0 and 4 of w (bits 0 and 16 on) as c - 8, those of
// nibbles 1 and 5 as 16 (c - 8), exactly: 1024 + c less 1032.  magic is 1024 in
// both halves, held in a register so that masking and joining is one operation.
__device__ __forceinline__ uint32_t centred_lo(uint32_t w, uint32_t magic) {
  uint32_t d;
  asm("lop3.b32 %0, %1, 0x000F000F, %2, 0xEA;" : "=r"(d) : "r"(w), "r"(magic));
  return add_f16x2(d, 0xE408E408u);
}
__device__ __forceinline__ uint32_t centred_hi(uint32_t w, uint32_t magic) {
  uint32_t d;
  asm("lop3.b32 %0, %1, 0x00F000F0, %2, 0xEA;" : "=r"(d) : "r"(w), "r"(magic));
  return add_f16x2(d, 0xE480E480u);
}
// 8x8 transpose of 16-bit values across the warp
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float half_lo(uint32_t w) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(w & 0xFFFFu)));
}
__device__ __forceinline__ float half_hi(uint32_t w) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(w >> 16)));
}
// The leading 11 significant bits of x: exact in half while |x| is at least
// 2^-14 and below 2^16; the conversion rounds smaller ones (to 2^-25).
__device__ __forceinline__ float top11(float x) { return __uint_as_float(__float_as_uint(x) & 0xFFFFE000u); }

// ----------------------------------------------------------------------------- formats

// 4-bit cache: a unit of 32 keys, rows of D/2 bytes.
template <int D_, int GROUP>
struct Kv4 {
  static constexpr bool kQuant = true;
  static constexpr int D = D_, NG = D / GROUP, kUnit = 32;
  static constexpr int kRow = D / 2, kChunks = kRow / 16, kQWords = D / 32 * 4;  // 16-byte chunks: 32 dims each
  static constexpr int kKOff = 0, kVOff = kUnit * kRow, kKpOff = 2 * kUnit * kRow, kVpOff = kKpOff + kUnit * NG * 4;
  static constexpr int kStage = kVpOff + kUnit * NG * 4;
  // chunk j of row r: the eight rows of an ldmatrix phase fall on distinct banks
  static __host__ __device__ constexpr uint32_t at(int r, int j) {
    return static_cast<uint32_t>(r * kRow + ((j ^ (kChunks == 4 ? (r >> 1) & 3 : (r >> 2) & 1)) << 4));
  }
};

// bf16 cache: a unit of 16 keys, rows of 2 D bytes.
template <int D_>
struct Bf16 {
  static constexpr bool kQuant = false;
  static constexpr int D = D_, NG = 1, kUnit = 16;
  static constexpr int kRow = 2 * D, kChunks = kRow / 16, kQWords = D / 16 * 4;
  static constexpr int kKOff = 0, kVOff = kUnit * kRow, kStage = 2 * kUnit * kRow;
  static __host__ __device__ constexpr uint32_t at(int r, int j) {
    return static_cast<uint32_t>(r * kRow + ((j ^ (r & 7)) << 4));
  }
};

// ----------------------------------------------------------------------------- plan

// x / d for x >= 0, d >= 1 by a float quotient and its correction: a division of
// integers is 20 instructions, and at a launch's start each costs some 15 cycles.
__device__ __forceinline__ int quot(int x, int d) {
  int q = static_cast<int>(__fdividef(static_cast<float>(x), static_cast<float>(d)));
  int r = x - q * d;
  while (r < 0) --q, r += d;
  while (r >= d) ++q, r -= d;
  return q;
}

// Units of all items end to end: row b's Hkv items hold pre[b] .. pre[b + 1].
// Every item opens with kOpen units without keys, about what changing over to
// an item costs a CTA (merging the warps' states, the next query), so that a run
// that meets many items holds fewer keys (8 ragged rows to 32k keys 39.4 us with
// none, 36.6 with 12 or 16; 64 listed blocks each 26.0 and 25.0).  The T units
// are cut into n runs of q or q + 1, one per CTA; n is such that
// each warp of a CTA gets a unit before the next CTA does.
constexpr int kOpen = 16;
struct Runs {
  int n, q, longer;  // runs 0 .. longer - 1 hold q + 1 units
  __device__ __forceinline__ Runs(int n_cta, int T, int warps) {
    n = min(n_cta, (T + warps - 1) / warps);
    q = n ? quot(T, n) : 0;
    longer = T - q * n;
  }
  __device__ __forceinline__ int start(int c) const { return c * q + min(c, longer); }
  // the run that holds unit x
  __device__ __forceinline__ int of(int x) const {
    const int head = longer * (q + 1);
    return x < head ? x / (q + 1) : longer + (x - head) / q;
  }
};

// Keys of a row whose last one is at p; -1: a position outside the cache.
__device__ __forceinline__ int row_keys(const LongAttnArgs& a, int p) { return p < -1 || p >= a.S_max ? -1 : p + 1; }

// Units of an item of `len` keys.  Listed blocks: of any item, so that the plan
// and the lists' loads need not wait for the positions (units without keys are
// passed over).
template <class F>
__device__ __forceinline__ int row_units(const LongAttnArgs& a, int len) {
  if constexpr (F::kQuant) return len < 0 ? 0 : (len + F::kUnit - 1) / F::kUnit;
  else return a.n_select * (kBlockKeys / F::kUnit);
}
// ... and with the opening, as the balanced runs count them.
template <class F>
__device__ __forceinline__ int row_places(const LongAttnArgs& a, int len) {
  const int n = row_units<F>(a, len);
  return n ? n + kOpen : 0;
}

// pre[0 .. B], and each row's keys in len, by one warp.
template <class F>
__device__ __forceinline__ void prefix_rows(const LongAttnArgs& a, int* pre, int* len, bool report) {
  const int lane = threadIdx.x & 31;
  int carry = 0;
  if (lane == 0) pre[0] = 0;
  for (int base = 0; base < a.B; base += 32) {
    const int b = base + lane;
    int v = 0;
    if (b < a.B) {
      len[b] = row_keys(a, a.pos[b]);
      v = row_places<F>(a, len[b]) * a.Hkv;
      if (report && len[b] < 0) atomicOr(a.err, kErrPosRange);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (b < a.B) pre[b + 1] = carry + v;
    carry += __shfl_sync(0xffffffffu, v, 31);
  }
}

// A value that all lanes hold, known to the compiler as such: what depends on it
// takes the uniform registers and branches that need no reconvergence (3 % at
// 8 rows to 32k keys).
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

struct Item {
  int b, h;        // row, KV head
  int start, end;  // its units, behind the opening
  int len;         // keys of the row, -1: refused
};

// The item that holds unit t, the same for the whole warp.
template <class F>
__device__ __forceinline__ Item item_at(const LongAttnArgs& a, const int* pre, const int* len, int t) {
  int lo = 0;
  if (a.B <= 32) {  // one look by the warp
    const int lane = threadIdx.x & 31;
    lo = __popc(__ballot_sync(0xffffffffu, lane < a.B && pre[lane] <= t)) - 1;
  } else {
    int hi = a.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
  }
  Item it;
  it.b = lo;
  const int per = row_places<F>(a, len[lo]);
  it.h = quot(t - pre[lo], per);
  it.end = pre[lo] + (it.h + 1) * per;
  it.start = it.end - per + kOpen;
  it.len = len[lo];
  return it;
}

// ----------------------------------------------------------------------------- query operand

// Heads 4 nt .. 4 nt + 3 of a group (q in shared memory) as B fragments, by one
// warp.  Lane (g, c)
// holds column g: head g / 2, its upper part (g even) or the remainder.
//  * 4-bit: per chunk j four half pairs that meet the nibble pairs (0, 4),
//    (1, 5), (2, 6), (3, 7) of word c, dims 32 j + 8 c + nibble, the odd
//    nibbles' (16 times larger) with a factor 1/16.  The head is scaled by a
//    power of two to [2^14, 2^15); f takes it back.  zq: for the (s, z) pair of
//    group c, (0, Q) with Q the group's mean of q so scaled.  Two parts leave
//    2^-24 there: of the head's largest element 2^-34 for a dim's q, and 2^-38
//    times the group's size for the sum over a group.
//  * bf16: per 16 dims two pairs, as the instruction lays them out, and two
//    more whose upper-part columns hold a third part (24 bits in all; the
//    remainder columns are zero).
template <class F>
__device__ __forceinline__ void stage_query(const float* q, int G, int nt, float scale_log2, uint32_t* words, float* f,
                                            uint32_t* zq) {
  constexpr int D = F::D;
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int head = 4 * nt + (g >> 1);
  const bool rest = g & 1;
  if constexpr (F::kQuant) {
    constexpr int NJ = D / 32, NG = F::NG;
    float v[NJ][8];
    float mx = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
      if (head < G) {
        const float4* p = reinterpret_cast<const float4*>(q + head * D + 32 * j + 8 * c);
        x = p[0];
        y = p[1];
      }
      v[j][0] = x.x, v[j][1] = x.y, v[j][2] = x.z, v[j][3] = x.w;
      v[j][4] = y.x, v[j][5] = y.y, v[j][6] = y.z, v[j][7] = y.w;
#pragma unroll
      for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(v[j][i]));
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const int ex = static_cast<int>(__float_as_uint(mx) >> 23) - 127;
    const int e = mx > 0.f ? min(max(14 - ex, -100), 100) : 0;
    const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    float mine = 0.f;
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
      float s = 0.f;
#pragma unroll
      for (int j = gr * NJ / NG; j < (gr + 1) * NJ / NG; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) s += v[j][i];
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      if (gr == c) mine = s;
    }
    mine *= up * (1.f / (D / NG));
    const float top = top11(mine), part = rest ? mine - top : top;
    zq[nt * 32 + lane] = pack_f16(0.f, part);
    if (c == 0 && !rest) f[head] = __uint_as_float(static_cast<uint32_t>(127 - e) << 23) * scale_log2;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float k = (i & 1) ? up * 0.0625f : up;
        const float x0 = v[j][i] * k, x1 = v[j][i + 4] * k;
        const float h0 = top11(x0), h1 = top11(x1);
        w[i] = rest ? pack_f16(x0 - h0, x1 - h1) : pack_f16(h0, h1);
      }
      *reinterpret_cast<uint4*>(words + ((nt * NJ + j) * 32 + lane) * 4) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
    constexpr int NJ = D / 16;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float2 x = make_float2(0.f, 0.f);
        if (head < G) x = *reinterpret_cast<const float2*>(q + head * D + 16 * j + 8 * i + 2 * c);
        const uint32_t hi = pack_bf16(x.x, x.y);
        const float x0 = x.x - bf16lo(hi), x1 = x.y - bf16hi(hi);
        const uint32_t mid = pack_bf16(x0, x1);
        w[i] = rest ? mid : hi;
        w[2 + i] = rest ? 0u : pack_bf16(x0 - bf16lo(mid), x1 - bf16hi(mid));
      }
      *reinterpret_cast<uint4*>(words + ((nt * NJ + j) * 32 + lane) * 4) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (c == 0 && !rest) f[head] = scale_log2;
  }
}

// ----------------------------------------------------------------------------- one unit

// A warp's running state.  Lane (g, c) of n-tile nt serves head 4 nt + c: m
// the reference score (log2 units; the same in the eight lanes of a head), mu
// the value subtracted (0 while m is -inf; kUp less for the 4-bit cache), l
// this lane's share of the sum, o[nt][..][e] rows of O^T, columns (upper part,
// remainder) of the head.  zs: sum_j p_j times the words of key j's (s, z) pairs, row g the
// g-th half word, so that row 2 i + 1 is the z sum of group i.
template <class F, int NT>
struct State {
  // m follows a larger score only once it leads by kSlack, so that the sums are
  // rescaled seldom; probabilities are at most 2^(kUp + kSlack), with the 4-bit
  // cache the top of the half range
  static constexpr float kUp = F::kQuant ? 11.f : 0.f, kSlack = 4.f;
  float o[NT][F::D / 16][4];
  float m[NT], mu[NT], l[NT];
  float zs[NT];
  // 4-bit: the window of scales (below) of this lane's group (lane & 3), 0 at first.
  // Where registers suffice it is held as its ends, half bits << 16, and every
  // group's factor as two halves
  static constexpr bool kHeld = NT < 4;
  int window;                       // not kHeld
  uint32_t lo, width, c2[F::NG];    // kHeld
};

template <class F, int NT>
__device__ __forceinline__ void state_init(State<F, NT>& st) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < F::D / 16; ++i) st.o[nt][i][0] = st.o[nt][i][1] = st.o[nt][i][2] = st.o[nt][i][3] = 0.f;
    st.zs[nt] = 0.f;
    st.m[nt] = -INFINITY;
    st.mu[nt] = -State<F, NT>::kUp;
    st.l[nt] = 0.f;
  }
#pragma unroll
  for (int gr = 0; gr < F::NG; ++gr) st.c2[gr] = 0x3C003C00u;
  st.window = 0;
  st.lo = 0u;
  st.width = 0x10000u;
}

// NG (s, z) pairs of key r
template <int NG>
__device__ __forceinline__ void load_pairs(const unsigned char* base, int r, uint32_t (&w)[NG]) {
  if constexpr (NG == 4) {
    const uint4 u = *reinterpret_cast<const uint4*>(base + r * 16);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  } else if constexpr (NG == 2) {
    const uint2 u = *reinterpret_cast<const uint2*>(base + r * 8);
    w[0] = u.x, w[1] = u.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(base + r * 4);
  }
}

// New maxima: the state's sums go over to them, and to new factors of the groups,
// `ratio` times the ones before.  All 32 lanes; x: this lane's largest score per
// n-tile.
template <class F, int NT>
__device__ __forceinline__ void raise(State<F, NT>& st, const float (&x)[NT], const float (&ratio)[F::NG]) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float mx = x[nt];
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
    mx = fmaxf(mx, st.m[nt]);
    const float mu = mx == -INFINITY ? 0.f : mx;
    const float corr = ex2(st.m[nt] - mu);
    st.m[nt] = mx;
    st.mu[nt] = mu - State<F, NT>::kUp;
    st.l[nt] *= corr;
    st.zs[nt] *= corr;
#pragma unroll
    for (int i = 0; i < F::D / 16; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) st.o[nt][i][e] *= corr * ratio[i / (F::D / 16 / F::NG)];
  }
}

// Windows of scales.  Window e, 1 .. 31, holds s in [2^(e-27), 2^(e-15)), and C =
// 2^(15-e) takes them to [2^-12, 1), exactly (a half has 14 bits down to its
// subnormals).  Probabilities are held, in both of their halves, to 2^-36 of the
// largest one; at the window's lower end 2^-24 is left of that, as float32 sums
// leave.  (Windows of 2^6 leave 2^-30, but keys whose values spread by 2^10 took
// 124 us in their passes where alike ones take 36.)  Window 0, at first, holds
// zero alone: the scale of a constant group, such as dims that only pad a head.
constexpr int kWindow = 12;
__device__ __forceinline__ uint32_t window_lo(int e) {  // half bits
  return e > kWindow ? static_cast<uint32_t>(e - kWindow) << 10 : 1u << max(e + 9 - kWindow, 0);
}
// 1 / c of a power of two
__device__ __forceinline__ float inverse(float c) { return __uint_as_float(0x7F000000u - __float_as_uint(c)); }
__device__ __forceinline__ uint32_t window_factor(int e) {  // C as half bits; 1 in window 0
  return e == 0 ? 0x3C00u : e < 30 ? static_cast<uint32_t>(30 - e) << 10 : 0x400u >> (e - 29);
}
template <class F, int NT>
__device__ __forceinline__ int window_of(const State<F, NT>& st) {
  if constexpr (State<F, NT>::kHeld) return static_cast<int>((st.lo + st.width) >> 26);
  else return st.window;
}
template <class F, int NT>
__device__ __forceinline__ void window_ends(const State<F, NT>& st, uint32_t* lo, uint32_t* width) {
  if constexpr (State<F, NT>::kHeld) {
    *lo = st.lo;
    *width = st.width;
  } else {
    *lo = st.window ? window_lo(st.window) << 16 : 0u;
    *width = (st.window ? static_cast<uint32_t>(st.window) << 26 : 0x10000u) - *lo;
  }
}
// Group gr's factor as two halves.  All 32 lanes.
template <class F, int NT>
__device__ __forceinline__ uint32_t group_factor(const State<F, NT>& st, int gr) {
  if constexpr (State<F, NT>::kHeld) return st.c2[gr];
  else return __shfl_sync(0xffffffffu, window_factor(st.window) * 0x10001u, gr);
}

// Each lane's group goes over to window e; the sums have to be taken times
// `ratio`.  All 32 lanes.
template <class F, int NT>
__device__ __forceinline__ void move_windows(State<F, NT>& st, int e, float (&ratio)[F::NG]) {
  const int was = window_of(st);
  const uint32_t both = window_factor(e) | static_cast<uint32_t>(127 + (was ? was : 15) - (e ? e : 15)) << 23;
  if constexpr (State<F, NT>::kHeld) {
    st.lo = e ? window_lo(e) << 16 : 0u;
    st.width = (e ? static_cast<uint32_t>(e) << 26 : 0x10000u) - st.lo;
  } else {
    st.window = e;
  }
#pragma unroll
  for (int gr = 0; gr < F::NG; ++gr) {
    const uint32_t w = __shfl_sync(0xffffffffu, both, gr);
    ratio[gr] = __uint_as_float(w & 0x7F800000u);
    if constexpr (State<F, NT>::kHeld) st.c2[gr] = __byte_perm(w, w, 0x1010);
  }
}

// The pair of key r, of this lane's group.  vw: this lane's pairs of keys 8 i + g.
__device__ __forceinline__ uint32_t pair_of(const uint32_t (&vw)[4], int r) {
  const uint32_t mine = r < 16 ? (r < 8 ? vw[0] : vw[1]) : r < 24 ? vw[2] : vw[3];
  return __shfl_sync(0xffffffffu, mine, 4 * (r & 7) + (threadIdx.x & 3));
}

// Of a unit whose scales do not all fit one window per group: the window of this
// lane's group with the first live key's scale in its middle (where that is zero,
// `next`), and the live keys, as bits, whose scales lie in the windows of all
// groups.  Seldom run, so that it is a call.  (Such a unit in one pass, its
// products in fp32 under a power of two of their own: the code beside the loop
// costs the units that do not need it more, 16 rows of 8k keys 18.9 us where this
// takes 17.9.)
__device__ __noinline__ uint2 first_and_alike(uint4 pairs, uint32_t live, int next) {
  const uint32_t vw[4] = {pairs.x, pairs.y, pairs.z, pairs.w};
  const uint32_t s = pair_of(vw, __ffs(live) - 1) & 0x7FFFu;
  if (s) next = s < 0x400u ? 1 : min(static_cast<int>(s >> 10) + 1 + kWindow / 2, 31);
  uint32_t served = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = vw[i] & 0x7FFFu;
    const bool in = x == 0u || x >= 0x7C00u || (x >= window_lo(next) && x < static_cast<uint32_t>(next) << 10);
    uint32_t b = __ballot_sync(0xffffffffu, in);  // bits 4 g + c; all groups of key g to bit g
    b &= b >> 1;
    b = b & b >> 2 & 0x11111111u;
    b = (b | b >> 3) & 0x03030303u;
    b = (b | b >> 6) & 0x000F000Fu;
    served |= ((b | b >> 12) & 0xFFu) << (8 * i);
  }
  return make_uint2(served & live, static_cast<uint32_t>(next));
}

// A unit with a scale outside its group's window (a zero outside window 0 too).  The windows
// move to serve all its `live` keys where the scales of each group span no more
// than a window, or else the first one and those like it.  Returns the keys that
// are served, as bits.  vw as above, dead keys with a live one's.  All 32 lanes.
template <class F, int NT>
__device__ __forceinline__ uint32_t fit_windows(State<F, NT>& st, const uint32_t (&vw)[4], uint32_t live,
                                                float (&ratio)[F::NG]) {
  uint32_t most = 0u, less = ~0u;  // the largest scale; the smallest but zero, less 1
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t s = vw[i] << 16 & 0x7FFF0000u;
    most = max(most, s < 0x7C000000u ? s : 0u);  // an infinity or a NaN needs no window
    less = min(less, s - 0x10000u);
  }
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    less = min(less, __shfl_xor_sync(0xffffffffu, less, o));
  }
  const uint32_t least = (less >> 16) + 1u;
  const int now = window_of(st), own = most ? static_cast<int>(most >> 26) + 1 : now;
  int next = own <= now && least >= window_lo(now) ? now : own;
  uint32_t served = live;
  if (!__all_sync(0xffffffffu, least >= window_lo(next))) {
    const uint2 r = first_and_alike(make_uint4(vw[0], vw[1], vw[2], vw[3]), live, next);
    served = r.x;
    next = static_cast<int>(r.y);
  }
  move_windows(st, next, ratio);
  return served;
}

// Half words (row g) of the (s, z) pairs of keys 8 i + 2 c and + 1, i = 0 .. 3.
template <int NG>
__device__ __forceinline__ void load_pairs_trans(const unsigned char* base, uint32_t addr, uint32_t (&w)[4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  if constexpr (NG == 4) {
    ldsm_x4_trans(w, addr + lane * 16);
  } else {
    const unsigned short* h = reinterpret_cast<const unsigned short*>(base);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = (8 * i + 2 * c) * 2 * NG + (g < 2 * NG ? g : 0);
      w[i] = static_cast<uint32_t>(h[at]) | (static_cast<uint32_t>(h[at + 2 * NG]) << 16);
    }
  }
}

// 32 keys of the 4-bit cache, of which those in `live` count.  Returns those that
// are left for another pass.
template <class F, int NT>
__device__ __forceinline__ uint32_t unit_kv4(const unsigned char* stage, uint32_t stage_addr, uint32_t live,
                                             const uint32_t* words, const float (&fs)[NT], const uint32_t (&zq)[NT],
                                             State<F, NT>& st) {
  constexpr int NJ = F::D / 32, NG = F::NG, PER = NJ / NG;  // chunks per group
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int lrow = (lane & 7) + (lane & 8), lchunk = lane >> 4;
  uint32_t magic;
  asm volatile("mov.b32 %0, 0x64006400;" : "=r"(magic));
  // the lane's own pair (group c) of keys 8 i + g
  uint32_t kw[4], vw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = ((8 * i + g) * NG + (c < NG ? c : 0)) * 4;
    kw[i] = *reinterpret_cast<const uint32_t*>(stage + F::kKpOff + at);
    vw[i] = *reinterpret_cast<const uint32_t*>(stage + F::kVpOff + at);
    if (NG < 4 && c >= NG) kw[i] = 0;
  }
  float s[NT][4];
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    uint32_t p0[NG], p1[NG];
    load_pairs<NG>(stage + F::kKpOff, 16 * hh + g, p0);
    load_pairs<NG>(stage + F::kKpOff, 16 * hh + g + 8, p1);
    float acc[NT][NG][4], zp[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) mma_f16_1688_zero(zp[nt], kw[2 * hh], kw[2 * hh + 1], zq[nt]);
#pragma unroll
    for (int jj = 0; jj < NJ; jj += 2) {
      uint32_t r[4];
      ldsm_x4(r, stage_addr + F::kKOff + F::at(16 * hh + lrow, jj + lchunk));
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int j = jj + t, gr = j / PER;
        const uint32_t w0 = r[2 * t], w1 = r[2 * t + 1], x0 = w0 >> 8, x1 = w1 >> 8;
        const uint32_t e0 = centred_lo(w0, magic), e1 = centred_lo(w1, magic);
        const uint32_t e2 = centred_hi(w0, magic), e3 = centred_hi(w1, magic);
        const uint32_t f0 = centred_lo(x0, magic), f1 = centred_lo(x1, magic);
        const uint32_t f2 = centred_hi(x0, magic), f3 = centred_hi(x1, magic);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint4 b = *reinterpret_cast<const uint4*>(words + ((nt * NJ + j) * 32 + lane) * 4);
          if (j % PER == 0) mma_f16_16816_zero(acc[nt][gr], e0, e1, e2, e3, b.x, b.y);
          else mma_f16_16816(acc[nt][gr], e0, e1, e2, e3, b.x, b.y);
          mma_f16_16816(acc[nt][gr], f0, f1, f2, f3, b.z, b.w);
        }
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float a0 = (zp[nt][0] + zp[nt][1]) * (F::D / NG), a1 = (zp[nt][2] + zp[nt][3]) * (F::D / NG);
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        a0 = fmaf(half_lo(p0[gr]), acc[nt][gr][0] + acc[nt][gr][1], a0);
        a1 = fmaf(half_lo(p1[gr]), acc[nt][gr][2] + acc[nt][gr][3], a1);
      }
      s[nt][2 * hh] = a0 * fs[nt];
      s[nt][2 * hh + 1] = a1 * fs[nt];
    }
  }
  uint32_t left = 0u;
  auto drop = [&](uint32_t keys) {  // those without a bit
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!(keys >> (8 * i + g) & 1u)) s[nt][i] = -INFINITY;
  };
  if (live != ~0u) {
    drop(live);
    const uint32_t first = pair_of(vw, __ffs(live) - 1);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!(live >> (8 * i + g) & 1u)) vw[i] = first;
  }
  // a larger score than before, or a scale outside its window, anywhere in the warp?
  float mx[NT];
  uint32_t off = 0u, lo, width;
  window_ends(st, &lo, &width);
#pragma unroll
  for (int i = 0; i < 4; ++i) off = max(off, (vw[i] << 16) - lo);
  bool more = off >= width;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    mx[nt] = fmaxf(fmaxf(s[nt][0], s[nt][1]), fmaxf(s[nt][2], s[nt][3]));
    more |= mx[nt] > st.m[nt] + State<F, NT>::kSlack;
  }
  if (__any_sync(0xffffffffu, more)) {
    float ratio[NG];
    const uint32_t served = fit_windows(st, vw, live, ratio);
    raise<F, NT>(st, mx, ratio);
    if (served != live) {
      drop(served);
      left = live & ~served;
    }
  }
  uint32_t vt[4];
  load_pairs_trans<NG>(stage + F::kVpOff, stage_addr + F::kVpOff, vt);
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    // probabilities of keys g and g + 8 (times 2^kUp) as upper halves and remainders
    uint32_t top[NT], rem[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float q0 = ex2(s[nt][2 * hh] - st.mu[nt]), q1 = ex2(s[nt][2 * hh + 1] - st.mu[nt]);
      st.l[nt] += q0 + q1;
      top[nt] = pack_f16(q0, q1);
      rem[nt] = pack_f16(q0 - half_lo(top[nt]), q1 - half_hi(top[nt]));
      // joined in fp32: the tensor core cuts each product at the last place of the
      // running sum, and these sums are long (4e-6 of the result at 33k keys, 1e-6 so)
      float z[4];
      mma_f16_16816_zero(z, vt[2 * hh], 0u, vt[2 * hh + 1], 0u, transpose8(__byte_perm(top[nt], rem[nt], 0x5410)),
                         transpose8(__byte_perm(top[nt], rem[nt], 0x7632)));
      st.zs[nt] += z[0] + z[1];
    }
    uint32_t p0[NG], p1[NG];
    load_pairs<NG>(stage + F::kVpOff, 16 * hh + g, p0);
    load_pairs<NG>(stage + F::kVpOff, 16 * hh + g + 8, p1);
#pragma unroll
    for (int jj = 0; jj < NJ; jj += 2) {
      uint32_t r[4], b0[NT], b1[NT];
      ldsm_x4_trans(r, stage_addr + F::kVOff + F::at(16 * hh + lrow, jj + lchunk));
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int j = jj + t, gr = j / PER;
        if (j % PER == 0) {
          // times the keys' scales: the product's upper half, its exact error, and the remainder's share
          const uint32_t sc = mul_f16x2(__byte_perm(p0[gr], p1[gr], 0x5410), group_factor(st, gr));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint32_t x = mul_f16x2(top[nt], sc);
            const uint32_t y = fma_f16x2(rem[nt], sc, fms_f16x2(top[nt], sc, x));
            b0[nt] = transpose8(__byte_perm(x, y, 0x5410));
            b1[nt] = transpose8(__byte_perm(x, y, 0x7632));
          }
        }
        const uint32_t w0 = r[2 * t], w1 = r[2 * t + 1], y0 = w0 >> 8, y1 = w1 >> 8;
        const uint32_t e0 = centred_lo(w0, magic), e1 = centred_hi(w0, magic);
        const uint32_t e2 = centred_lo(w1, magic), e3 = centred_hi(w1, magic);
        const uint32_t f0 = centred_lo(y0, magic), f1 = centred_hi(y0, magic);
        const uint32_t f2 = centred_lo(y1, magic), f3 = centred_hi(y1, magic);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16_16816(st.o[nt][2 * j], e0, e1, e2, e3, b0[nt], b1[nt]);
          mma_f16_16816(st.o[nt][2 * j + 1], f0, f1, f2, f3, b0[nt], b1[nt]);
        }
      }
    }
  }
  return left;
}

// 16 keys of a bf16 cache, of which the first nk count.
template <class F, int NT>
__device__ __forceinline__ void unit_bf16(uint32_t stage_addr, int nk, const uint32_t* words, const float (&fs)[NT],
                                          State<F, NT>& st) {
  constexpr int NJ = F::D / 16;
  const int lane = threadIdx.x & 31, g = lane >> 2;
  float acc[NT][2][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[nt][0][e] = acc[nt][1][e] = 0.f;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    uint32_t r[4];
    ldsm_x4(r, stage_addr + F::kKOff + F::at(lane & 15, 2 * j + (lane >> 4)));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint4 b = *reinterpret_cast<const uint4*>(words + ((nt * NJ + j) * 32 + lane) * 4);
      mma_bf16_16816(acc[nt][0], r, b.x, b.y);
      mma_bf16_16816(acc[nt][1], r, b.z, b.w);
    }
  }
  float s[NT][2], mx[NT];
  bool more = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const float f = fs[nt];
    s[nt][0] = ((acc[nt][0][0] + acc[nt][1][0]) + (acc[nt][0][1] + acc[nt][1][1])) * f;
    s[nt][1] = ((acc[nt][0][2] + acc[nt][1][2]) + (acc[nt][0][3] + acc[nt][1][3])) * f;
    if (g >= nk) s[nt][0] = -INFINITY;
    if (g + 8 >= nk) s[nt][1] = -INFINITY;
    mx[nt] = fmaxf(s[nt][0], s[nt][1]);
    more |= mx[nt] > st.m[nt] + State<F, NT>::kSlack;
  }
  if (__any_sync(0xffffffffu, more)) raise<F, NT>(st, mx, {1.f});
  uint32_t b0[NT], b1[NT], c0[NT], c1[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const float x0 = ex2(s[nt][0] - st.mu[nt]), x1 = ex2(s[nt][1] - st.mu[nt]);
    st.l[nt] += x0 + x1;
    const uint32_t h = pack_bf16(x0, x1);
    const float y0 = x0 - bf16lo(h), y1 = x1 - bf16hi(h);
    const uint32_t l = pack_bf16(y0, y1);
    const uint32_t t = pack_bf16(y0 - bf16lo(l), y1 - bf16hi(l));
    b0[nt] = transpose8(__byte_perm(h, l, 0x5410));
    b1[nt] = transpose8(__byte_perm(h, l, 0x7632));
    c0[nt] = transpose8(t & 0xFFFFu);  // the third part, in the upper parts' columns
    c1[nt] = transpose8(t >> 16);
  }
  const int vrow = (lane & 7) + ((lane >> 4) << 3), vchunk = (lane >> 3) & 1;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    uint32_t r[4];
    ldsm_x4_trans(r, stage_addr + F::kVOff + F::at(vrow, 2 * j + vchunk));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      mma_bf16_16816(st.o[nt][j], r, b0[nt], b1[nt]);
      mma_bf16_16816(st.o[nt][j], r, c0[nt], c1[nt]);
    }
  }
}

// ----------------------------------------------------------------------------- kernel

// Shape of a launch: warps of a CTA, units in flight per warp, CTAs of an SM.
// Four-warp CTAs wait less at an item's end and share the SM more evenly than
// larger ones (the 4-bit cache, 8 ragged rows to 32k keys: 12 warps as 3 x 4 with
// 3 units each 42.5 us, 16 as 2 x 8 with 2 45.6, 16 in one CTA 61.2).  In a
// cluster all warps of an SM work on one item.
template <class F, int NT, bool CL>
struct Shape {
  static constexpr bool kSmall = F::kQuant && NT == 1 && !CL;
  static constexpr int kW = kSmall ? 4 : 8, kStages = kSmall ? 3 : 2, kPerSm = kSmall ? 3 : 1;
};

// CL: a cluster of a.cluster CTAs per (row, KV head), each with an equal run of
// its units, joined in CTA 0's shared memory: no partials, no second launch.
template <class F, int kW, int STAGES>
struct Smem {
  static __host__ __device__ uint32_t ring(int B, int G, int NT) { return qraw(B, G, NT) + G * F::D * 4; }
  static __host__ __device__ uint32_t qraw(int B, int G, int NT) { return obuf(B, NT) + kW * G * (F::D + 4) * 4; }
  // the plan of the 4-bit cache's balanced runs comes first
  static __host__ __device__ uint32_t words(int B) { return F::kQuant ? ((2 * B + 1) * 4 + 127) / 128 * 128 : 0; }
  static __host__ __device__ uint32_t f(int B, int NT) { return words(B) + NT * F::kQWords * 32 * 4; }
  static __host__ __device__ uint32_t zq(int B, int NT) { return f(B, NT) + kMaxG * 4; }
  static __host__ __device__ uint32_t ms(int B, int NT) { return zq(B, NT) + 4 * 32 * 4; }
  static __host__ __device__ uint32_t ls(int B, int NT) { return ms(B, NT) + kW * kMaxG * 4; }
  static __host__ __device__ uint32_t obuf(int B, int NT) { return ls(B, NT) + kW * kMaxG * 4; }
  static __host__ __device__ uint32_t join(int B, int G, int NT) {
    return (ring(B, G, NT) + 127) / 128 * 128 + kW * STAGES * F::kStage;
  }
  static __host__ __device__ uint32_t bytes(int B, int G, int NT, int cluster) {
    return join(B, G, NT) + (cluster > 1 ? cluster * G * (F::D + 2) * 4 : 0);
  }
};

template <class F, int NT, bool CL>
__global__ void __launch_bounds__(32 * Shape<F, NT, CL>::kW, Shape<F, NT, CL>::kPerSm)
    long_attn_kernel(const __grid_constant__ LongAttnArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int kW = Shape<F, NT, CL>::kW, kThreads = 32 * kW, STAGES = Shape<F, NT, CL>::kStages;
  using L = Smem<F, kW, STAGES>;
  constexpr int D = F::D;
  const int G = a.G;
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  int* pre = reinterpret_cast<int*>(smem);
  int* len = pre + a.B + 1;
  uint32_t* words = reinterpret_cast<uint32_t*>(smem + L::words(a.B));
  float* f_smem = reinterpret_cast<float*>(smem + L::f(a.B, NT));
  uint32_t* zq_smem = reinterpret_cast<uint32_t*>(smem + L::zq(a.B, NT));
  float* ms = reinterpret_cast<float*>(smem + L::ms(a.B, NT));
  float* ls = reinterpret_cast<float*>(smem + L::ls(a.B, NT));
  float* obuf = reinterpret_cast<float*>(smem + L::obuf(a.B, NT));
  unsigned char* ring = smem + (L::ring(a.B, G, NT) + 127) / 128 * 128 + warp * (STAGES * F::kStage);
  const uint32_t ring_addr = smem_addr(ring);

  // what needs no memory, while the launch before may still run
  int cta = blockIdx.x, T = 0;
  Item only{};  // CL: the cluster's item
  if constexpr (CL) {
    cluster_arrive();  // CTA 0 has started before anybody writes to it
    const int item = quot(blockIdx.x, a.cluster);
    cta = blockIdx.x - item * a.cluster;
    only.b = quot(item, a.Hkv);
    only.h = item - only.b * a.Hkv;
  }
  if constexpr (!F::kQuant) T = CL ? row_units<F>(a, 0) : a.B * a.Hkv * row_places<F>(a, 0);
  Runs runs(CL ? a.cluster : a.n_cta, T, kW);
  // an item's query rows, without a commit of their own
  float* qraw = reinterpret_cast<float*>(smem + L::qraw(a.B, G, NT));
  auto fetch_query = [&](const Item& it) {
    const float* q = a.q + (static_cast<size_t>(it.b) * a.Hq + static_cast<size_t>(it.h) * G) * D;
    for (int e = tid * 4; e < G * D; e += kThreads * 4) cp_async16(smem_addr(qraw + e), q + e, true);
  };
  pdl_wait();
  pdl_launch_dependents();
  if constexpr (CL) {
    fetch_query(only);
    only.len = row_keys(a, a.pos[only.b]);
    if (only.len < 0 && only.h == 0 && cta == 0 && tid == 0) atomicOr(a.err, kErrPosRange);
    only.end = row_units<F>(a, only.len);
  } else if constexpr (F::kQuant) {
    if (warp == 0) prefix_rows<F>(a, pre, len, cta == 0);
    __syncthreads();
  } else if (cta == 0) {
    for (int b = tid; b < a.B; b += kThreads)
      if (row_keys(a, a.pos[b]) < 0) atomicOr(a.err, kErrPosRange);
  }
  if constexpr (F::kQuant) {  // units by the positions
    T = CL ? only.end : pre[a.B];
    runs = Runs(CL ? a.cluster : a.n_cta, T, kW);
  }
  if (!CL && cta >= runs.n) return;  // the same verdict in every thread
  const int t0 = cta < runs.n ? runs.start(cta) : T, t1 = cta < runs.n ? runs.start(cta + 1) : T;
  auto locate = [&](int t) {
    if constexpr (CL) {
      return only;
    } else if constexpr (!F::kQuant) {
      const int per = row_places<F>(a, 0), item = quot(t, per);
      Item it;
      it.b = quot(item, a.Hkv);
      it.h = item - it.b * a.Hkv;
      it.end = (item + 1) * per;
      it.start = it.end - per + kOpen;
      it.len = row_keys(a, a.pos[it.b]);
      return it;
    } else {
      return item_at<F>(a, pre, len, t);
    }
  };

  // ---- loads: this warp's units t0 + warp + kW k, in order.  A lane copies
  // the 16-byte pieces lane, lane + 32, .. of a unit, at fixed places in shared
  // memory (the swizzle has a period of 32 pieces)
  static_assert(F::at(0, 0) == 0 && 32 % F::kChunks == 0, "lane-fixed pieces");
  constexpr int kPieces = F::kUnit * F::kChunks / 32;
  const uint32_t lane_at = F::at(lane / F::kChunks, lane % F::kChunks);
  int list_k = 0;                 // listed blocks: units list_k .. list_k + 31 of this warp have their ids in the lanes
  int ids = 0, ids_next = 0;
  auto fetch_ids = [&](int k) {   // lane i: the block of unit k + i of this warp
    const int t = t0 + warp + kW * (k + lane);
    if (t >= t1) return -1;
    const int per = row_places<F>(a, 0);
    const int item = CL ? only.b * a.Hkv + only.h : quot(t, per), u = CL ? t : t - item * per - kOpen;
    if (u < 0) return -1;
    return a.blocks[static_cast<size_t>(item) * a.n_select + static_cast<unsigned>(u) / (kBlockKeys / F::kUnit)];
  };
  if constexpr (!F::kQuant) {
    ids = fetch_ids(0);
    ids_next = fetch_ids(32);
  }
  Item li = locate(t0);  // the item being loaded
  const unsigned char *k_src = nullptr, *v_src = nullptr;  // 4-bit: this lane's first piece of slot 0 of the item
  const uint32_t *kp_src = nullptr, *vp_src = nullptr;
  auto item_sources = [&]() {
    const size_t row = (static_cast<size_t>(li.b) * a.Hkv + li.h) * a.S_max;
    k_src = static_cast<const unsigned char*>(a.k) + row * F::kRow + lane * 16;
    v_src = static_cast<const unsigned char*>(a.v) + row * F::kRow + lane * 16;
    kp_src = a.kp + (row + lane) * F::NG;
    vp_src = a.vp + (row + lane) * F::NG;
  };
  if constexpr (F::kQuant) item_sources();
  // issues unit k of this warp into a slot; returns its keys (bf16 only)
  auto issue = [&](int k, int slot) -> int {
    const int t = t0 + warp + kW * k;
    int nk = 0;
    if constexpr (!F::kQuant) {
      if (k - list_k == 32) {
        list_k += 32;
        ids = ids_next;
        ids_next = fetch_ids(list_k + 32);
      }
    }
    if (t < t1) {
      if (t >= li.end) {
        li = locate(t);
        if constexpr (F::kQuant) item_sources();
      }
      const uint32_t dst = ring_addr + slot * F::kStage + lane_at;
      if (t < li.start) {  // the opening
      } else if constexpr (F::kQuant) {
        const int k0 = (t - li.start) * F::kUnit;
        const unsigned char* ks = k_src + static_cast<size_t>(k0) * F::kRow;
        const unsigned char* vs = v_src + static_cast<size_t>(k0) * F::kRow;
        const uint32_t* kps = kp_src + static_cast<size_t>(k0) * F::NG;
        const uint32_t* vps = vp_src + static_cast<size_t>(k0) * F::NG;
        const uint32_t pdst = ring_addr + slot * F::kStage + lane * F::NG * 4;
        nk = li.len - k0;
        if (nk >= F::kUnit) {
#pragma unroll
          for (int i = 0; i < kPieces; ++i) {
            cp_async16(dst + F::kKOff + 512 * i, ks + 512 * i, true);
            cp_async16(dst + F::kVOff + 512 * i, vs + 512 * i, true);
          }
          cp_async_small<F::NG * 4>(pdst + F::kKpOff, kps, true);
          cp_async_small<F::NG * 4>(pdst + F::kVpOff, vps, true);
        } else {  // zeros behind the last key; their sources lie inside the unit's live part
#pragma unroll
          for (int i = 0; i < kPieces; ++i) {
            const bool live = lane / F::kChunks + 32 / F::kChunks * i < nk;
            const size_t off = live ? 512 * i : 0;
            cp_async16(dst + F::kKOff + 512 * i, (live ? ks : ks - lane * 16) + off, live);
            cp_async16(dst + F::kVOff + 512 * i, (live ? vs : vs - lane * 16) + off, live);
          }
          const bool live = lane < nk;
          cp_async_small<F::NG * 4>(pdst + F::kKpOff, live ? kps : kps - lane * F::NG, live);
          cp_async_small<F::NG * 4>(pdst + F::kVpOff, live ? vps : vps - lane * F::NG, live);
        }
      } else {
        const int id = __shfl_sync(0xffffffffu, ids, k - list_k);
        const bool bad = id < -1 || id > (a.S_max - 1) / kBlockKeys;
        if (bad && lane == 0) atomicOr(a.err, kErrPosRange);
        const int k0 =
            bad || id < 0 ? max(li.len, 0) : id * kBlockKeys + ((t - li.start) & (kBlockKeys / F::kUnit - 1)) * F::kUnit;
        nk = max(0, min(F::kUnit, li.len - k0));
        if (nk > 0) {
          const size_t row = (static_cast<size_t>(li.b) * a.Hkv + li.h) * a.S_max + k0;
          const unsigned char* ks = static_cast<const unsigned char*>(a.k) + row * F::kRow + lane * 16;
          const unsigned char* vs = static_cast<const unsigned char*>(a.v) + row * F::kRow + lane * 16;
#pragma unroll
          for (int i = 0; i < kPieces; ++i) {
            const bool live = lane / F::kChunks + 32 / F::kChunks * i < nk;
            const size_t off = live ? 512 * i : 0;
            const uint32_t at = ring_addr + slot * F::kStage +
                                F::at(lane / F::kChunks + 32 / F::kChunks * i, lane % F::kChunks);
            cp_async16(at + F::kKOff, (live ? ks : ks - lane * 16) + off, live);
            cp_async16(at + F::kVOff, (live ? vs : vs - lane * 16) + off, live);
          }
        }
      }
    }
    cp_async_commit();
    return nk;
  };
  if (!CL && t0 < t1) fetch_query(li);  // ahead of the stream: behind it they would wait for it
  cp_async_commit();
  int ring_nk[STAGES];  // bf16: keys of the units in flight
  ring_nk[0] = issue(0, 0);

  // ---- items of this run
  cp_async_wait<1>();
  __syncthreads();
  int k = 0, slot = 0;
  for (int t = t0; t < t1;) {
    const Item it = locate(t);
    const int seg_end = min(t1, it.end);
    if (seg_end <= it.start) break;  // the run ends in an opening
    if (warp < NT)
      stage_query<F>(qraw, G, warp, a.scale_log2, words, f_smem, zq_smem);
    __syncthreads();
    if (t == t0) {
#pragma unroll
      for (int i = 1; i < STAGES; ++i) ring_nk[i] = issue(i, i);
    }
    if (seg_end < t1) fetch_query(locate(seg_end));  // the next item's, with the next commit
    float fs[NT];
    uint32_t zq[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      fs[nt] = f_smem[4 * nt + (lane & 3)];
      zq[nt] = zq_smem[nt * 32 + lane];
    }
    State<F, NT> st;
    state_init(st);
    for (; t0 + warp + kW * k < seg_end; ++k) {
      cp_async_wait<STAGES - 1>();
      __syncwarp();
      if constexpr (F::kQuant) {
        const int u = t0 + warp + kW * k - it.start;
        const int at = slot * F::kStage;
        if (u >= 0) {
          const int nk = it.len - u * F::kUnit;
          uint32_t live = nk < 32 ? (1u << nk) - 1u : ~0u;
          do live = unit_kv4<F, NT>(ring + at, ring_addr + at, live, words, fs, zq, st);
          while (live);
        }
        __syncwarp();
        issue(k + STAGES, slot);
      } else {
        int nk = ring_nk[0];
#pragma unroll
        for (int i = 1; i < STAGES; ++i) nk = slot == i ? ring_nk[i] : nk;
        if (nk > 0) unit_bf16<F, NT>(ring_addr + slot * F::kStage, nk, words, fs, st);
        __syncwarp();
        nk = issue(k + STAGES, slot);
#pragma unroll
        for (int i = 0; i < STAGES; ++i)
          if (slot == i) ring_nk[i] = nk;
      }
      slot = slot + 1 == STAGES ? 0 : slot + 1;
    }
    // the next query has to be in; a warp without a unit here has not committed it
    if (seg_end < t1) cp_async_wait_all();
    // the warps' states, each relative to its own maximum
    const int g = lane >> 2, c = lane & 3;
    float units[F::NG];
    if constexpr (F::kQuant) {
#pragma unroll
      for (int gr = 0; gr < F::NG; ++gr) units[gr] = inverse(half_lo(group_factor(st, gr)));
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int h = 4 * nt + c;
      float l = st.l[nt], zs[F::NG];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
      for (int gr = 0; gr < F::NG; ++gr)
        zs[gr] = __shfl_sync(0xffffffffu, st.zs[nt], 4 * (2 * gr + 1) + c);
      if (g == 0) {
        ms[warp * kMaxG + h] = st.m[nt];
        ls[warp * kMaxG + h] = l;
      }
      if (h < G) {
        float* to = obuf + (warp * G + h) * (D + 4);
        if constexpr (F::kQuant) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const int gr = i / 2 / (D / 32 / F::NG);
            const float z = zs[gr], u0 = units[gr], u1 = u0 * 0.0625f;
            *reinterpret_cast<float2*>(to + 32 * (i >> 1) + 4 * g + 2 * (i & 1)) =
                make_float2(fmaf(st.o[nt][i][0] + st.o[nt][i][1], u0, z), fmaf(st.o[nt][i][2] + st.o[nt][i][3], u1, z));
          }
        } else {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            to[16 * i + g] = st.o[nt][i][0] + st.o[nt][i][1];
            to[16 * i + g + 8] = st.o[nt][i][2] + st.o[nt][i][3];
          }
        }
      }
    }
    __syncthreads();
    const bool whole = it.start >= t0 && it.end <= t1;
    float* join = reinterpret_cast<float*>(smem + L::join(a.B, G, NT)) + cta * G * (D + 2);
    float* part = a.part + static_cast<size_t>(2 * cta + (it.start <= t0 ? 0 : 1)) * (G * (D + 2));
    if constexpr (CL) cluster_wait();
    float* out = a.o + (static_cast<size_t>(it.b) * a.Hq + static_cast<size_t>(it.h) * G) * D;
    for (int e = tid; e < G * D; e += kThreads) {
      const int h = e / D, d = e - h * D;
      float M = -INFINITY, sum = 0.f, l = 0.f;
#pragma unroll
      for (int w = 0; w < kW; ++w) M = fmaxf(M, ms[w * kMaxG + h]);
      const float mu = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int w = 0; w < kW; ++w) {
        const float x = ex2(ms[w * kMaxG + h] - mu);
        l = fmaf(x, ls[w * kMaxG + h], l);
        sum = fmaf(x, obuf[(w * G + h) * (D + 4) + d], sum);
      }
      if (whole) {
        if (it.len >= 0) out[e] = l == 0.f ? 0.f : sum / l;
      } else if constexpr (CL) {
        store_cta0(join + e, __float_as_uint(sum));
        if (d == 0) {
          store_cta0(join + G * D + h, __float_as_uint(M));
          store_cta0(join + G * D + G + h, __float_as_uint(l));
        }
      } else {
        part[e] = sum;
        if (d == 0) {
          part[G * D + h] = M;
          part[G * D + G + h] = l;
        }
      }
    }
    __syncthreads();
    t = seg_end;
  }
  cp_async_wait_all();
  if constexpr (CL) {
    if (t0 >= t1) cluster_wait();
    cluster_arrive();
    cluster_wait();
    if (cta > 0 || runs.n == 1) return;
    float* out = a.o + (static_cast<size_t>(only.b) * a.Hq + static_cast<size_t>(only.h) * G) * D;
    const float* join = reinterpret_cast<const float*>(smem + L::join(a.B, G, NT));
    for (int e = tid; e < G * D; e += kThreads) {
      const int h = e / D;
      float M = -INFINITY, sum = 0.f, l = 0.f;
      for (int i = 0; i < runs.n; ++i) M = fmaxf(M, join[i * G * (D + 2) + G * D + h]);
      const float mu = M == -INFINITY ? 0.f : M;
      for (int i = 0; i < runs.n; ++i) {
        const float* p = join + i * G * (D + 2);
        const float x = ex2(p[G * D + h] - mu);
        l = fmaf(x, p[G * D + G + h], l);
        sum = fmaf(x, p[e], sum);
      }
      if (only.len >= 0) out[e] = l == 0.f ? 0.f : sum / l;
    }
  }
}


// Joins the partials of the items that are cut between CTAs, and writes the
// zeros of rows without keys.  Grid (Hq, B), one thread per dim.  Everything
// that the positions decide is done before the wait for the attention launch
// (plan and partial addresses behind it cost 2.5 us at 16 partials).
template <class F, int NT>
__global__ void __launch_bounds__(F::D) long_merge_kernel(const __grid_constant__ LongAttnArgs a) {
  extern __shared__ __align__(16) int pre[];
  constexpr int D = F::D;
  const int G = a.G, head = blockIdx.x, b = blockIdx.y, d = threadIdx.x;
  int* at = pre + 2 * a.B + 1;  // [n_cta] partials of this item, in floats
  float* ml = reinterpret_cast<float*>(at + a.n_cta);  // [2 n_cta] their maxima and sums
  if (threadIdx.x < 32) prefix_rows<F>(a, pre, pre + a.B + 1, false);
  __syncthreads();
  const int places = (pre[b + 1] - pre[b]) / a.Hkv;
  const int g = head / G, h = head - g * G, stride = G * (D + 2);
  int parts = 0;
  if (places > 0) {
    const Runs runs(a.n_cta, pre[a.B], Shape<F, NT, false>::kW);
    const int start = pre[b] + g * places + kOpen;
    const int c0 = runs.of(start);
    parts = runs.of(start - kOpen + places - 1) - c0 + 1;
    if (parts > 1)
      for (int i = d; i < parts; i += D) at[i] = (2 * (c0 + i) + (start <= runs.start(c0 + i) ? 0 : 1)) * stride;
  }
  const int len = pre[a.B + 1 + b];
  __syncthreads();
  pdl_wait();
  float* out = a.o + (static_cast<size_t>(b) * a.Hq + head) * D + d;
  if (len < 0) return;  // refused
  if (places == 0) {
    *out = 0.f;
    return;
  }
  if (parts == 1) return;  // written by its CTA
  constexpr int kBatch = 16;
  float x[kBatch];
  auto load = [&](int base) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) x[i] = base + i < parts ? __ldcg(a.part + at[base + i] + h * D + d) : 0.f;
  };
  load(0);
  for (int i = d; i < 2 * parts; i += D) ml[i] = __ldcg(a.part + at[i >> 1] + G * D + (i & 1 ? G : 0) + h);
  __syncthreads();
  float M = -INFINITY, L = 0.f, sum = 0.f;
  for (int i = 0; i < parts; ++i) M = fmaxf(M, ml[2 * i]);
  const float mu = M == -INFINITY ? 0.f : M;
  for (int base = 0; base < parts; base += kBatch) {
    if (base) load(base);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (base + i < parts) {
        const float w = ex2(ml[2 * (base + i)] - mu);
        L = fmaf(w, ml[2 * (base + i) + 1], L);
        sum = fmaf(w, x[i], sum);
      }
    }
  }
  *out = L == 0.f ? 0.f : sum / L;
}

// CTAs per (row, KV head): up to 8, while the clusters take at most two thirds
// of the SMs (16 clusters of 8 wait for one another at 128 of 152: 9.3 us where
// 64 CTAs take 7.4), or 1: the balanced runs with their partials and second
// launch, about 3 us more, but all SMs.  A unit takes a warp about 1 us, NT times
// that for wide groups, so the clusters win while a warp of theirs has at most
// 5 / NT units more than one of the balanced runs.  Measured, clusters against runs (b rows, query/KV heads, keys):
// 1 32/8 4k 6.6 / 8.6 us, 16k 12.8 / 15.9, 32k 21.1 / 19.6; 8 12/3 8k 12.5 / 15.1,
// 16k 20.6 / 20.7, 32k 35.8 / 29.7; 1 16/1 2k 9.9 / 9.7, 4k 11.9 / 10.2; 64 listed
// blocks 7.7 / 9.9, 256 17.6 / 18.5.
template <class F, int NT>
int cluster_size(const LongAttnArgs& a, int sms) {
  using S = Shape<F, NT, true>;
  const int items = a.B * a.Hkv;
  const long long units = F::kQuant ? (a.S_max + F::kUnit - 1) / F::kUnit : a.n_select * (kBlockKeys / F::kUnit);
  int c = 1;
  while (c < 8 && 2 * c * items <= 2 * sms / 3 &&
         Smem<F, S::kW, S::kStages>::bytes(a.B, a.Hq / a.Hkv, NT, 2 * c) <= kSmemMax)
    c *= 2;
  return (units * sms - units * items * c) * NT <= 5ll * S::kW * sms * c ? c : 1;
}

template <class F, int NT>
cudaError_t run(LongAttnArgs a, int sms, cudaStream_t st) {
  const int G = a.Hq / a.Hkv;
  a.G = G;
  a.cluster = cluster_size<F, NT>(a, sms);
  if (a.cluster > 1) {
    using S = Shape<F, NT, true>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.B * a.Hkv * a.cluster);
    cfg.blockDim = dim3(32 * S::kW);
    cfg.dynamicSmemBytes = Smem<F, S::kW, S::kStages>::bytes(a.B, G, NT, a.cluster);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, long_attn_kernel<F, NT, true>, a);
  }
  using S = Shape<F, NT, false>;
  a.n_cta = std::min(kLongMaxCtas, S::kPerSm * sms);
  cudaError_t e = launch(long_attn_kernel<F, NT, false>, dim3(a.n_cta), dim3(32 * S::kW),
                         Smem<F, S::kW, S::kStages>::bytes(a.B, G, NT, 1), st, true, a);
  if (e != cudaSuccess) return e;
  return launch(long_merge_kernel<F, NT>, dim3(a.Hq, a.B), dim3(F::D), (2 * a.B + 1 + 3 * a.n_cta) * 4, st, true, a);
}
template <class F>
cudaError_t run_format(const LongAttnArgs& a, int sms, cudaStream_t st) {
  const int G = a.Hq / a.Hkv;
  if (G <= 4) return run<F, 1>(a, sms, st);
  if (G <= 8) return run<F, 2>(a, sms, st);
  return run<F, 4>(a, sms, st);
}
template <class F, int NT>
cudaError_t allow() {
  cudaError_t e = allow_smem(long_attn_kernel<F, NT, false>);
  if (e == cudaSuccess) e = allow_smem(long_attn_kernel<F, NT, true>);
  return e;
}
template <class F>
cudaError_t allow_format() {
  cudaError_t e = allow<F, 1>();
  if (e == cudaSuccess) e = allow<F, 2>();
  if (e == cudaSuccess) e = allow<F, 4>();
  return e;
}

}  // namespace

cudaError_t launch_long_attn(const LongAttnArgs& a, int D, int group, int sms, cudaStream_t st) {
  if (a.blocks) return D == 64 ? run_format<Bf16<64>>(a, sms, st) : run_format<Bf16<128>>(a, sms, st);
  if (D == 64) return group == 32 ? run_format<Kv4<64, 32>>(a, sms, st) : run_format<Kv4<64, 64>>(a, sms, st);
  if (group == 32) return run_format<Kv4<128, 32>>(a, sms, st);
  if (group == 64) return run_format<Kv4<128, 64>>(a, sms, st);
  return run_format<Kv4<128, 128>>(a, sms, st);
}

cudaError_t allow_smem_long() {
  cudaError_t e = allow_format<Kv4<64, 32>>();
  if (e == cudaSuccess) e = allow_format<Kv4<64, 64>>();
  if (e == cudaSuccess) e = allow_format<Kv4<128, 32>>();
  if (e == cudaSuccess) e = allow_format<Kv4<128, 64>>();
  if (e == cudaSuccess) e = allow_format<Kv4<128, 128>>();
  if (e == cudaSuccess) e = allow_format<Bf16<64>>();
  if (e == cudaSuccess) e = allow_format<Bf16<128>>();
  return e;
}

}  // namespace dec
