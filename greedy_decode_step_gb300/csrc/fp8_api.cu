// C-ABI of the 8-bit weight operators and the mixture-of-experts layer:
// argument checks and launches.  Declarations and contracts are in
// include/libdec.h.
#include <algorithm>
#include <cmath>

#include "dec_fp8.cuh"
#include "dec_host.cuh"
#include "dec_launch.cuh"
#include "dec_moe.cuh"
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
#define DEC_WORDS(p) DEC_CHECK(aligned(p, 4), DEC_EINVAL, "%s must be a non-null 4-byte aligned pointer", #p)

// Matrices of rows of 8-bit codes.
int check_codes(int n, int rows, int K) {
  DEC_CHECK(n >= 0 && rows >= 0, DEC_EINVAL, "matrices and rows must be >= 0 (got %d and %d)", n, rows);
  DEC_CHECK(n <= kFp8MaxDim && rows <= kFp8MaxDim, DEC_EUNSUPPORTED, "%d matrices of %d rows: at most 2^24 each", n, rows);
  DEC_CHECK(K >= 16 && K % 16 == 0, DEC_EUNSUPPORTED, "rows of %d codes: a positive multiple of 16", K);
  DEC_CHECK(K <= kFp8MaxDim, DEC_EUNSUPPORTED, "rows of %d codes: at most 2^24", K);
  return DEC_OK;
}

int check_blocks(int block_rows) {
  DEC_CHECK(block_rows == 1 || block_rows == kFp8Block, DEC_EUNSUPPORTED, "blocks of %d rows: supported 1 and 128",
            block_rows);
  return DEC_OK;
}

// Strides (elements) of float rows given as views.
int check_strides(long long sm, long long sr, int bf16) {
  const int per = bf16 ? 8 : 4;
  DEC_CHECK(sm >= 0 && sr >= 0 && sm % per == 0 && sr % per == 0, DEC_EINVAL,
            "matrix and row strides must be non-negative multiples of 16 bytes");
  return DEC_OK;
}

// Whether no two of n x rows rows of K elements, at matrix and row strides sm and sr, have an element in common.
bool rows_apart(int n, long long sm, int rows, long long sr, int K) {
  if (n > 1 && sm < K) return false;
  if (rows > 1 && sr < K) return false;
  if (n == 1 || rows == 1) return true;
  // rows whose places differ by i of the larger stride and by j of the other, in opposite directions
  using Wide = __int128;
  const bool mats = sm >= sr;
  const Wide far = mats ? sm : sr, near = mats ? sr : sm, nf = mats ? n : rows, nn = mats ? rows : n;
  for (Wide i = 1; i < nf && i * far < (nn - 1) * near + K; ++i) {
    const Wide j = std::min(i * far / near, nn - 1), left = i * far - j * near;
    if (left < K || (j + 1 < nn && near - left < K)) return false;
  }
  return true;
}

int check_moe(int T, int E, int H) {
  DEC_CHECK(T >= 0, DEC_EINVAL, "T must be >= 0");
  DEC_CHECK(T <= kMoeMaxTokens, DEC_EUNSUPPORTED, "%d tokens: at most %d", T, kMoeMaxTokens);
  DEC_CHECK(E >= 1 && E <= kMoeMaxExperts, DEC_EUNSUPPORTED, "%d experts outside 1..%d", E, kMoeMaxExperts);
  DEC_CHECK(H >= 8 && H % 8 == 0 && H <= kMoeMaxDim, DEC_EUNSUPPORTED, "H = %d: a positive multiple of 8 up to %d", H,
            kMoeMaxDim);
  return DEC_OK;
}

int check_choices(int k, int E) {
  DEC_CHECK(k >= 1 && k <= kMoeMaxChoices, DEC_EUNSUPPORTED, "%d experts per token outside 1..%d", k, kMoeMaxChoices);
  DEC_CHECK(k <= E, DEC_EINVAL, "%d experts per token, but there are %d", k, E);
  return DEC_OK;
}

int check_inner(int I, bool fp8, int H) {
  DEC_CHECK(I >= 8 && I % 8 == 0 && I <= kMoeMaxDim, DEC_EUNSUPPORTED, "I = %d: a positive multiple of 8 up to %d", I,
            kMoeMaxDim);
  DEC_CHECK(!fp8 || (H % 16 == 0 && I % 16 == 0), DEC_EUNSUPPORTED, "H = %d, I = %d: multiples of 16 for 8-bit weights", H,
            I);
  return DEC_OK;
}

}  // namespace

extern "C" {

int dec_fp8_quant(const void* x, int bf16, int64_t stride_mat, int64_t stride_row, void* codes, float* scales, int n,
                  int rows, int K, int block_rows, void* stream) {
  DEC_TRY(check_codes(n, rows, K));
  DEC_TRY(check_blocks(block_rows));
  if (n == 0 || rows == 0) return DEC_OK;
  DEC_PTR(x);
  DEC_TRY(check_strides(stride_mat, stride_row, bf16));
  DEC_PTR(codes);
  DEC_WORDS(scales);
  int sms;
  uint32_t* err;
  DEC_TRY(host_device(&sms, &err));
  Fp8QuantArgs a{};
  a.x = x;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  a.sm = stride_mat;
  a.sr = stride_row;
  a.n = n;
  a.rows = rows;
  a.K = K;
  DEC_LAUNCHED(launch_fp8_quant(a, bf16 != 0, block_rows, sms, static_cast<cudaStream_t>(stream)), "8-bit quantiser");
  return DEC_OK;
}

int dec_fp8_dequant(const void* codes, const float* scales, void* out, int bf16, int64_t stride_mat, int64_t stride_row,
                    int n, int rows, int K, int block_rows, void* stream) {
  DEC_TRY(check_codes(n, rows, K));
  DEC_TRY(check_blocks(block_rows));
  if (n == 0 || rows == 0) return DEC_OK;
  DEC_PTR(codes);
  DEC_WORDS(scales);
  DEC_PTR(out);
  DEC_TRY(check_strides(stride_mat, stride_row, bf16));
  DEC_CHECK(rows_apart(n, stride_mat, rows, stride_row, K), DEC_EINVAL,
            "rows read back may not share memory: of %d x %d rows of %d, %lld and %lld apart, some do", n, rows, K,
            static_cast<long long>(stride_mat), static_cast<long long>(stride_row));
  int sms;
  uint32_t* err;
  DEC_TRY(host_device(&sms, &err));
  Fp8DequantArgs a{};
  a.out = out;
  a.codes = static_cast<const uint8_t*>(codes);
  a.scales = scales;
  a.sm = stride_mat;
  a.sr = stride_row;
  a.n = n;
  a.rows = rows;
  a.K = K;
  a.block_rows = block_rows;
  DEC_LAUNCHED(launch_fp8_dequant(a, bf16 != 0, sms, static_cast<cudaStream_t>(stream)), "8-bit read-back");
  return DEC_OK;
}

int dec_fp8_gemm(const void* x_codes, const float* x_scales, const void* w_codes, const float* w_scales,
                 const float* residual, int64_t stride_residual, float* out, int64_t stride_out, int M, int N, int K,
                 void* stream) {
  DEC_TRY(check_codes(1, M, K));
  DEC_CHECK(N >= 1, DEC_EINVAL, "N must be >= 1");
  DEC_CHECK(N <= kFp8MaxDim, DEC_EUNSUPPORTED, "N = %d: at most 2^24", N);
  DEC_CHECK(static_cast<long long>(M) * N <= 1ll << 40, DEC_EUNSUPPORTED, "%d x %d results: at most 2^40", M, N);
  if (M == 0) return DEC_OK;
  DEC_PTR(x_codes);
  DEC_WORDS(x_scales);
  DEC_PTR(w_codes);
  DEC_WORDS(w_scales);
  if (residual) DEC_WORDS(residual);
  DEC_WORDS(out);
  DEC_CHECK(stride_out >= 0 && (M == 1 || stride_out >= N), DEC_EINVAL, "rows of the result are %lld apart: N = %d at least",
            static_cast<long long>(stride_out), N);
  DEC_CHECK(!residual || stride_residual >= 0, DEC_EINVAL, "the residual's stride must be >= 0");
  Fp8GemmCall c{};
  int sms;
  DEC_TRY(host_device(&sms, &c.err));
  c.xc = static_cast<const uint8_t*>(x_codes);
  c.sx = x_scales;
  c.wc = static_cast<const uint8_t*>(w_codes);
  c.sw = w_scales;
  c.residual = residual;
  c.out = out;
  c.ldr = stride_residual;
  c.ldo = stride_out;
  c.M = M;
  c.N = N;
  c.K = K;
  const char* why;
  const int rc = fp8_gemm(c, sms, static_cast<cudaStream_t>(stream), &why);
  DEC_CHECK(rc == 0, rc == 1 ? DEC_EUNSUPPORTED : DEC_ECUDA, "8-bit product: %s", why);
  return DEC_OK;
}

int dec_moe_route(const float* y, const void* Wr, const float* bias, int sigmoid, int renormalise, float scale,
                  int32_t* ids, float* weights, int T, int H, int E, int k, void* stream) {
  DEC_TRY(check_moe(T, E, H));
  DEC_TRY(check_choices(k, E));
  DEC_CHECK(std::isfinite(scale), DEC_EINVAL, "scale must be finite");
  if (T == 0) return DEC_OK;
  DEC_PTR(y);
  DEC_PTR(Wr);
  if (bias) DEC_WORDS(bias);
  DEC_WORDS(ids);
  DEC_WORDS(weights);
  int sms;
  uint32_t* err;
  DEC_TRY(host_device(&sms, &err));
  MoeRouteArgs a{};
  a.y = y;
  a.Wr = static_cast<const uint16_t*>(Wr);
  a.bias = bias;
  a.ids = ids;
  a.gates = weights;
  a.H = H;
  a.E = E;
  a.k = k;
  a.sigmoid = sigmoid != 0;
  a.renormalise = renormalise != 0;
  a.scale = scale;
  DEC_LAUNCHED(launch_moe_route(a, T, static_cast<cudaStream_t>(stream)), "expert choice");
  return DEC_OK;
}

size_t dec_moe_workspace_size(int T, int k, int H, int I) {
  if (check_moe(T, kMoeMaxExperts, H) != DEC_OK || check_choices(k, kMoeMaxExperts) != DEC_OK ||
      check_inner(I, false, H) != DEC_OK)
    return 0;
  return moe_workspace(T, k, H, I).bytes;
}

int dec_moe_experts(const float* y, const int32_t* ids, const float* weights, const void* Wg, const void* Wu, const void* Wd,
                    const float* Sg, const float* Su, const float* Sd, const float* residual, float* out, void* ws,
                    size_t ws_bytes, int T, int k, int E, int H, int I, void* stream) {
  DEC_TRY(check_moe(T, E, H));
  DEC_TRY(check_choices(k, kMoeMaxExperts));
  const bool fp8 = Sg || Su || Sd;
  DEC_TRY(check_inner(I, fp8, H));
  if (T == 0) return DEC_OK;
  DEC_PTR(y);
  DEC_WORDS(ids);
  DEC_WORDS(weights);
  DEC_PTR(Wg);
  DEC_PTR(Wu);
  DEC_PTR(Wd);
  if (fp8) {
    DEC_WORDS(Sg);
    DEC_WORDS(Su);
    DEC_WORDS(Sd);
  }
  if (residual) DEC_PTR(residual);
  DEC_PTR(out);
  DEC_CHECK(aligned(ws, 256), DEC_EINVAL, "workspace must be non-null and 256-byte aligned");
  const size_t need = moe_workspace(T, k, H, I).bytes;
  DEC_CHECK(ws_bytes >= need, DEC_EINVAL, "experts' workspace has %zu bytes, needs %zu", ws_bytes, need);
  MoeCall c{};
  int sms;
  DEC_TRY(host_device(&sms, &c.err));
  c.y = y;
  c.ids = ids;
  c.gates = weights;
  c.wg = Wg;
  c.wu = Wu;
  c.wd = Wd;
  c.sg = Sg;
  c.su = Su;
  c.sd = Sd;
  c.residual = residual;
  c.out = out;
  c.ws = static_cast<unsigned char*>(ws);
  c.T = T;
  c.k = k;
  c.E = E;
  c.H = H;
  c.I = I;
  const char* why;
  const int rc = moe_experts(c, sms, static_cast<cudaStream_t>(stream), &why);
  DEC_CHECK(rc == 0, rc == 1 ? DEC_EUNSUPPORTED : DEC_ECUDA, "experts: %s", why);
  return DEC_OK;
}

}  // extern "C"
