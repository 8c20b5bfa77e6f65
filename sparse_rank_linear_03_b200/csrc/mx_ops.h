// Host-side internals of the microscaled operators: operands and kernel launchers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "hsl.h"

namespace hsl {

// Launches of a chain of kernels.  A chained kernel may start as soon as every CTA of the one before has
// called pdl_trigger, so that its launch and set-up overlap that kernel's end; it touches
// global memory after pdl_wait only, when that kernel has ended and can be seen.
// The first kernel of a call is never chained: what came before it on the stream is not ours.
template <typename... P, typename... A>
cudaError_t launch_chained(void (*fn)(P...), bool chained, dim3 grid, unsigned block, size_t smem, cudaStream_t s,
                           const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = chained ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, fn, P(args)...);
}

// One factor of a product, stored as [i][k] (or [k][i] when trans).
struct MxOperand {
  enum Kind : int32_t { kF32, kBF16, kE2M1, kInt8 };
  const void* p;
  const uint8_t* scales;  // e2m1, int8
  int64_t pitch;          // elements (f32, bf16) or bytes of codes per stored row
  int64_t spitch;         // scale bytes per stored row
  int32_t kind;
  int32_t trans;
  int32_t vec;            // f32: rows start on 16 bytes
};

hsl_status mx_quantize_run(const void* X, hsl_dtype dtype, int64_t rows, int64_t cols, bool int8,
                           void* codes, void* scales, cudaStream_t s);
hsl_status mx_dequantize_run(const void* codes, const void* scales, int64_t rows, int64_t cols,
                             bool int8, void* X, hsl_dtype dtype, cudaStream_t s);
// C[M][N] (row pitch N) = add + A Bᵀ in fp32; `part` holds mx_simt_workspace bytes; chained: behind another
// kernel of the same call
size_t mx_simt_workspace(int64_t M, int64_t N, int64_t K);
hsl_status mx_simt_run(const MxOperand& A, const MxOperand& B, int64_t M, int64_t N, int64_t K,
                       const void* add, void* C, hsl_dtype cdt, void* part, bool chained, cudaStream_t s);
// C = add + Σ of `ranges` partial results in part [range][count], chained
hsl_status mx_simt_sum_run(const float* part, int ranges, int64_t count, const float* add, float* C, cudaStream_t s);

// Tensor-core products (mx_gemm.cu, mx_grad.cu), bf16: X, dY, U, V on 16 bytes (mx_gemm_supported)
bool mx_gemm_supported(const void* X);
size_t mx_gemm_apply_workspace(bool trans, int64_t T, int64_t m, int64_t n);
hsl_status mx_gemm_apply_run(bool trans, const MxOperand& D, int64_t m, int64_t n, const void* X,
                             const void* add, void* Y, int64_t T, void* ws, cudaStream_t s);
size_t mx_gemm_grad_workspace(int64_t T, int64_t m, int64_t n, int64_t r);
hsl_status mx_gemm_grad_run(const MxOperand& X, int64_t T, int64_t n, const void* dY, int64_t m,
                            const void* U, const void* V, int64_t r, const void* add, void* dU, void* dV,
                            void* dX, void* ws, cudaStream_t s);
cudaError_t mx_gemm_error_word(uint32_t** p);
cudaError_t mx_grad_error_word(uint32_t** p);
// A few tokens (mx_decode.cu), any alignment of X.  bf16: as many as mx_decode_fits says.
// To 8 tokens, the columns of one register MMA: 28672 × 8192 at 8 tokens 41 µs, the tensor-core kernel 76; 11008 × 4096
// 18.5 against 22.6.  With two MMAs per block, at 16 tokens, a call alone took 99 and 28 µs, the tensor-core kernel 80
// and 24.5.
// f32 to 32: 4096 × 4096 at 32 tokens 76 µs, the tiled product 88; at 64 tokens 141 and 94 µs; 512 × 4096 at 32
// tokens 16 and 18, at 64 27 and 20 µs.
constexpr int64_t kMxDecodeMax = 8, kMxDecodeF32Max = 32;
bool mx_decode_fits(int64_t T, int64_t m, int64_t n);
cudaError_t mx_decode_error_word(uint32_t** p);
size_t mx_decode_workspace(int64_t T, int64_t n);
hsl_status mx_decode_run(const MxOperand& D, int64_t m, int64_t n, const void* X, const void* add, void* Y,
                         int64_t T, void* ws, cudaStream_t s);
hsl_status mx_decode_f32_run(const MxOperand& D, int64_t m, int64_t n, const void* X, const void* add,
                             void* Y, int64_t T, void* ws, cudaStream_t s);
size_t mx_decode_f32_workspace(int64_t T, int64_t m, int64_t n);
// Both factors in e2m1 blocks (mx_matmul.cu): Y[T][m] = A Bᵀ (+ add)
bool mx_matmul_supported();
hsl_status mx_matmul_run(const MxOperand& A, int64_t T, const MxOperand& B, int64_t m, int64_t n,
                         const void* add, void* Y, hsl_dtype dtype, cudaStream_t s);
cudaError_t mx_matmul_error_word(uint32_t** p);

}  // namespace hsl
