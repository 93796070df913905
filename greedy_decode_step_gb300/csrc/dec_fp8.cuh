// Arguments and launches of the 8-bit weight operators: e4m3 codes with a
// float scale per block of 128 values (rows) or 128 x 128 values (weights).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dec_common.cuh"

namespace dec {

constexpr int kFp8Block = 128;
constexpr int kFp8MaxDim = 1 << 24;  // rows, values of a row, matrices

struct Fp8QuantArgs {
  const void* x;                 // float32 or bf16 [n][rows][K], strided
  uint8_t* codes;                // [n][rows][K]
  float* scales;                 // [n][ceil(rows / R)][ceil(K / 128)]
  long long sm, sr;              // source strides (elements) of matrix and row
  int n, rows, K;
};
struct Fp8DequantArgs {
  void* out;
  const uint8_t* codes;
  const float* scales;
  long long sm, sr;
  int n, rows, K, block_rows;
};
cudaError_t launch_fp8_quant(const Fp8QuantArgs& a, bool bf16, int block_rows, int sms, cudaStream_t st);
cudaError_t launch_fp8_dequant(const Fp8DequantArgs& a, bool bf16, int sms, cudaStream_t st);
cudaError_t allow_smem_fp8();

// out[m][n] = residual[m][n] + sum over K blocks of sx[m][kb] sw[n / 128][kb] (xc[m] . wc[n]) in the block
struct Fp8GemmCall {
  const uint8_t* xc;             // [M][K]
  const float* sx;               // [M][KB]
  const uint8_t* wc;             // [N][K]
  const float* sw;               // [NB][KB]
  const float* residual;         // [M][N] at ldr, or null
  float* out;                    // [M][N] at ldo
  long long ldr, ldo;
  int M, N, K;
  uint32_t* err;
};
// 0, or 1 (*why says why) or 3 (a CUDA error)
int fp8_gemm(const Fp8GemmCall& c, int sms, cudaStream_t st, const char** why);
cudaError_t allow_smem_fp8_gemm();

}  // namespace dec
