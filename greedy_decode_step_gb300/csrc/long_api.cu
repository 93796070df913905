// C-ABI of the long-cache operators: argument checks and launches.
// Declarations and contracts are in include/libdec.h.
#include <cmath>

#include "dec_host.cuh"
#include "dec_launch.cuh"
#include "dec_long.cuh"
#include "libdec.h"

using namespace dec;

namespace {

#define DEC_CHECK(cond, code, ...)                   \
  do {                                               \
    if (!(cond)) return host_fail(code, __VA_ARGS__); \
  } while (0)
#define DEC_TRY(expr)            \
  do {                           \
    int r_ = (expr);             \
    if (r_ != DEC_OK) return r_; \
  } while (0)
#define DEC_LAUNCHED(expr, what)                                                                    \
  do {                                                                                              \
    cudaError_t e_ = (expr);                                                                        \
    if (e_ != cudaSuccess) return host_fail(DEC_ECUDA, "%s: %s", what, cudaGetErrorString(e_));      \
  } while (0)

bool aligned(const void* p, uintptr_t n) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
#define DEC_PTR(p) DEC_CHECK(aligned(p, 16), DEC_EINVAL, "%s must be a non-null 16-byte aligned pointer", #p)
#define DEC_INTS(p) DEC_CHECK(aligned(p, 4), DEC_EINVAL, "%s must be a non-null 4-byte aligned pointer", #p)

int check_heads(int Hkv, int D) {
  DEC_CHECK(Hkv >= 1 && Hkv <= 4096, DEC_EUNSUPPORTED, "Hkv = %d outside 1..4096", Hkv);
  DEC_CHECK(D == 64 || D == 128, DEC_EUNSUPPORTED, "head_dim %d: supported 64 and 128", D);
  return DEC_OK;
}

// Sizes shared by every call: a cache of B rows, Hkv heads, S_max slots.
int check_cache(int B, int Hkv, int D, int S_max) {
  DEC_CHECK(B >= 1 && B <= kLongMaxBatch, DEC_EUNSUPPORTED, "batch %d outside 1..%d", B, kLongMaxBatch);
  DEC_TRY(check_heads(Hkv, D));
  DEC_CHECK(S_max >= 1, DEC_EINVAL, "S_max must be >= 1");
  // positions, and a CTA's tokens behind the last, stay in an int
  DEC_CHECK(static_cast<long long>(B) * Hkv * S_max <= (1ll << 31) - 1024, DEC_EUNSUPPORTED,
            "a cache of %lld (row, head, slot) entries: at most 2^31 - 1024", static_cast<long long>(B) * Hkv * S_max);
  return DEC_OK;
}

int check_queries(int Hq, int Hkv) {
  DEC_CHECK(Hq >= 1 && Hq % Hkv == 0, DEC_EINVAL, "Hq=%d must be a positive multiple of Hkv=%d", Hq, Hkv);
  DEC_CHECK(Hq / Hkv <= 16, DEC_EUNSUPPORTED, "Hq/Hkv = %d above 16", Hq / Hkv);
  return DEC_OK;
}

int check_group(int D, int group) {
  DEC_CHECK((group == 32 || group == 64 || group == 128) && group <= D, DEC_EUNSUPPORTED,
            "group %d: supported 32, 64 and 128, at most head_dim", group);
  return DEC_OK;
}

int check_tokens(int T) {
  DEC_CHECK(T <= (1 << 30), DEC_EUNSUPPORTED, "T = %d tokens of a row: at most 2^30", T);
  return DEC_OK;
}

// Strides (elements) of rows given as views: whole 16-byte vectors, no overlap check.
int check_strides(long long sb, long long st, long long sh, int bf16) {
  const int per = bf16 ? 8 : 4;
  DEC_CHECK(sb >= 0 && st >= 0 && sh >= 0 && sb % per == 0 && st % per == 0 && sh % per == 0, DEC_EINVAL,
            "row, token and head strides must be non-negative multiples of 16 bytes");
  return DEC_OK;
}

int check_workspace(const void* ws, size_t have, size_t need) {
  DEC_CHECK(aligned(ws, 256), DEC_EINVAL, "workspace must be non-null and 256-byte aligned");
  DEC_CHECK(have >= need, DEC_EINVAL, "attention workspace has %zu bytes, needs %zu", have, need);
  return DEC_OK;
}

// Two partials per CTA at most: its first and its last item.
size_t part_bytes(int Hq, int Hkv, int D) {
  return 2ull * kLongMaxCtas * (Hq / Hkv) * (D + 2) * sizeof(float);
}

float softmax_scale(int D) { return static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(D))); }

}  // namespace

extern "C" {

int dec_kv4_store(const void* k, const void* v, int bf16, int64_t stride_row, int64_t stride_token,
                  int64_t stride_head, int from_cache, int src_tokens, const int32_t* pos, const int32_t* lens, int T,
                  void* k_codes, void* k_params, void* v_codes, void* v_params, int B, int Hkv, int D, int group,
                  int S_max, void* stream) {
  DEC_TRY(check_cache(B, Hkv, D, S_max));
  DEC_TRY(check_group(D, group));
  DEC_CHECK(T >= 0 && src_tokens >= 0, DEC_EINVAL, "T and src_tokens must be >= 0");
  DEC_TRY(check_tokens(T));
  DEC_CHECK(T <= src_tokens, DEC_EINVAL, "T = %d tokens, but the source has %d", T, src_tokens);
  if (T == 0) return DEC_OK;
  DEC_PTR(k);
  DEC_PTR(v);
  DEC_TRY(check_strides(stride_row, stride_token, stride_head, bf16));
  DEC_INTS(pos);
  if (lens) DEC_INTS(lens);
  DEC_PTR(k_codes);
  DEC_PTR(k_params);
  DEC_PTR(v_codes);
  DEC_PTR(v_params);
  DEC_CHECK(k_codes != v_codes && k_params != v_params, DEC_EINVAL, "K and V need caches of their own");
  Kv4StoreArgs a{};
  int sms;
  DEC_TRY(host_device(&sms, &a.err));
  a.src[0] = k;
  a.src[1] = v;
  a.codes[0] = static_cast<uint8_t*>(k_codes);
  a.codes[1] = static_cast<uint8_t*>(v_codes);
  a.params[0] = static_cast<uint32_t*>(k_params);
  a.params[1] = static_cast<uint32_t*>(v_params);
  a.pos = pos;
  a.lens = lens;
  a.sb = stride_row;
  a.st = stride_token;
  a.sh = stride_head;
  a.B = B;
  a.T = T;
  a.Hkv = Hkv;
  a.S_max = S_max;
  a.from_cache = from_cache != 0;
  a.src_tokens = src_tokens;
  DEC_LAUNCHED(launch_kv4_store(a, D, group, bf16 != 0, static_cast<cudaStream_t>(stream)), "4-bit cache store");
  return DEC_OK;
}

int dec_kv4_load(const void* k_codes, const void* k_params, const void* v_codes, const void* v_params,
                 const int32_t* pos, const int32_t* lens, int T, void* k_out, void* v_out, int bf16,
                 int64_t stride_row, int64_t stride_token, int64_t stride_head, int B, int Hkv, int D, int group,
                 int S_max, void* stream) {
  DEC_TRY(check_cache(B, Hkv, D, S_max));
  DEC_TRY(check_group(D, group));
  DEC_CHECK(T >= 0, DEC_EINVAL, "T must be >= 0");
  DEC_TRY(check_tokens(T));
  if (T == 0) return DEC_OK;
  DEC_PTR(k_codes);
  DEC_PTR(k_params);
  DEC_PTR(v_codes);
  DEC_PTR(v_params);
  DEC_INTS(pos);
  if (lens) DEC_INTS(lens);
  DEC_PTR(k_out);
  DEC_PTR(v_out);
  DEC_CHECK(k_out != v_out, DEC_EINVAL, "k_out and v_out must differ");
  DEC_TRY(check_strides(stride_row, stride_token, stride_head, bf16));
  DEC_CHECK((B == 1 || stride_row) && (T == 1 || stride_token) && (Hkv == 1 || stride_head), DEC_EINVAL,
            "rows read back may not share memory (a stride of zero)");
  Kv4LoadArgs a{};
  int sms;
  DEC_TRY(host_device(&sms, &a.err));
  a.dst[0] = k_out;
  a.dst[1] = v_out;
  a.codes[0] = static_cast<const uint8_t*>(k_codes);
  a.codes[1] = static_cast<const uint8_t*>(v_codes);
  a.params[0] = static_cast<const uint32_t*>(k_params);
  a.params[1] = static_cast<const uint32_t*>(v_params);
  a.pos = pos;
  a.lens = lens;
  a.sb = stride_row;
  a.st = stride_token;
  a.sh = stride_head;
  a.B = B;
  a.T = T;
  a.Hkv = Hkv;
  a.S_max = S_max;
  DEC_LAUNCHED(launch_kv4_load(a, D, group, bf16 != 0, static_cast<cudaStream_t>(stream)), "4-bit cache read-back");
  return DEC_OK;
}

size_t dec_long_attn_workspace_size(int Hq, int Hkv, int D) {
  if (check_heads(Hkv, D) != DEC_OK || check_queries(Hq, Hkv) != DEC_OK) return 0;
  return part_bytes(Hq, Hkv, D);
}

int dec_kv4_decode_attn(const float* q, const void* k_codes, const void* k_params, const void* v_codes,
                        const void* v_params, const int32_t* pos, float* o, void* ws, size_t ws_bytes, int B, int Hq,
                        int Hkv, int D, int group, int S_max, void* stream) {
  DEC_TRY(check_cache(B, Hkv, D, S_max));
  DEC_TRY(check_queries(Hq, Hkv));
  DEC_TRY(check_group(D, group));
  DEC_PTR(q);
  DEC_PTR(k_codes);
  DEC_PTR(k_params);
  DEC_PTR(v_codes);
  DEC_PTR(v_params);
  DEC_INTS(pos);
  DEC_PTR(o);
  DEC_TRY(check_workspace(ws, ws_bytes, part_bytes(Hq, Hkv, D)));
  LongAttnArgs a{};
  int sms;
  DEC_TRY(host_device(&sms, &a.err));
  a.q = q;
  a.o = o;
  a.pos = pos;
  a.k = k_codes;
  a.v = v_codes;
  a.kp = static_cast<const uint32_t*>(k_params);
  a.vp = static_cast<const uint32_t*>(v_params);
  a.part = static_cast<float*>(ws);
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.S_max = S_max;
  a.scale_log2 = softmax_scale(D);
  DEC_LAUNCHED(launch_long_attn(a, D, group, sms, static_cast<cudaStream_t>(stream)), "attention over the 4-bit cache");
  return DEC_OK;
}

int dec_block_bounds(const void* k_cache, const int32_t* pos, int T, void* bounds, int B, int Hkv, int D, int S_max,
                     void* stream) {
  DEC_TRY(check_cache(B, Hkv, D, S_max));
  DEC_CHECK(T >= 0 && T <= S_max, DEC_EINVAL, "T = %d tokens outside 0..S_max = %d", T, S_max);
  if (T == 0) return DEC_OK;
  DEC_PTR(k_cache);
  DEC_INTS(pos);
  DEC_PTR(bounds);
  BoundsArgs a{};
  int sms;
  DEC_TRY(host_device(&sms, &a.err));
  a.k = static_cast<const uint16_t*>(k_cache);
  a.pos = pos;
  a.bounds = static_cast<uint16_t*>(bounds);
  a.B = B;
  a.T = T;
  a.Hkv = Hkv;
  a.S_max = S_max;
  a.NB = (S_max + kBlockKeys - 1) / kBlockKeys;
  DEC_LAUNCHED(launch_block_bounds(a, D, static_cast<cudaStream_t>(stream)), "block bounds");
  return DEC_OK;
}

int dec_select_blocks(const float* q, const void* bounds, const int32_t* pos, int32_t* blocks, int n_select,
                      int n_first, int n_last, int B, int Hq, int Hkv, int D, int S_max, void* stream) {
  DEC_TRY(check_cache(B, Hkv, D, S_max));
  DEC_TRY(check_queries(Hq, Hkv));
  const int NB = (S_max - 1) / kBlockKeys + 1;
  DEC_CHECK(NB <= kSelMaxBlocks, DEC_EUNSUPPORTED, "S_max = %d: the selection takes up to %d slots", S_max,
            kSelMaxBlocks * kBlockKeys);
  DEC_CHECK(n_select >= 1 && n_select <= kSelMaxBlocks, DEC_EINVAL, "n_select = %d outside 1..%d", n_select,
            kSelMaxBlocks);
  DEC_CHECK(n_first >= 0 && n_last >= 0 && n_first <= n_select && n_last <= n_select - n_first, DEC_EINVAL,
            "n_first = %d and n_last = %d must be >= 0 and fit n_select = %d", n_first, n_last, n_select);
  DEC_PTR(q);
  DEC_PTR(bounds);
  DEC_INTS(pos);
  DEC_INTS(blocks);
  SelectBlocksArgs a{};
  int sms;
  DEC_TRY(host_device(&sms, &a.err));
  a.q = q;
  a.bounds = static_cast<const uint16_t*>(bounds);
  a.pos = pos;
  a.blocks = blocks;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.S_max = S_max;
  a.NB = NB;
  a.n_select = n_select;
  a.n_first = n_first;
  a.n_last = n_last;
  DEC_LAUNCHED(launch_select_blocks(a, D, sms, static_cast<cudaStream_t>(stream)), "block selection");
  return DEC_OK;
}

int dec_block_decode_attn(const float* q, const void* k_cache, const void* v_cache, const int32_t* pos,
                          const int32_t* blocks, int n_select, float* o, void* ws, size_t ws_bytes, int B, int Hq,
                          int Hkv, int D, int S_max, void* stream) {
  DEC_TRY(check_cache(B, Hkv, D, S_max));
  DEC_TRY(check_queries(Hq, Hkv));
  DEC_CHECK(n_select >= 1, DEC_EINVAL, "n_select must be >= 1");
  DEC_CHECK(static_cast<long long>(B) * Hkv * (n_select * 4ll + 16) < (1ll << 30), DEC_EUNSUPPORTED,
            "%lld listed blocks and their heads: about 2^28 at most", static_cast<long long>(B) * Hkv * n_select);
  DEC_PTR(q);
  DEC_PTR(k_cache);
  DEC_PTR(v_cache);
  DEC_INTS(pos);
  DEC_INTS(blocks);
  DEC_PTR(o);
  DEC_TRY(check_workspace(ws, ws_bytes, part_bytes(Hq, Hkv, D)));
  LongAttnArgs a{};
  int sms;
  DEC_TRY(host_device(&sms, &a.err));
  a.q = q;
  a.o = o;
  a.pos = pos;
  a.k = k_cache;
  a.v = v_cache;
  a.blocks = blocks;
  a.n_select = n_select;
  a.part = static_cast<float*>(ws);
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.S_max = S_max;
  a.scale_log2 = softmax_scale(D);
  DEC_LAUNCHED(launch_long_attn(a, D, 0, sms, static_cast<cudaStream_t>(stream)), "attention over listed blocks");
  return DEC_OK;
}

}  // extern "C"
