// Products whose operands may be microscaled, on the CUDA cores in fp32: the path of
// f32 data (and of the calls that no faster kernel takes).
//
//   C[i][j] = add[i][j] + Σ_k A(i, k) B(j, k)
//
// Each operand is fp32, bf16, e2m1 blocks or int8 blocks, stored as [i][k] or
// transposed as [k][i]; it is widened exactly to fp32 on its way to shared memory.
// A CTA owns a 64 × 64 tile (16 sums per thread).  The sums are kept in two levels,
// folded every 64 terms, so that the rounding error of a long sum grows with the
// root of 64 terms and of K/64 folds rather than of K.
// Bound by the fp32 FMA rate and, at small sizes, by the latency of a K loop.
#include "common.cuh"
#include "internal.h"
#include "mx.cuh"
#include "mx_ops.h"

namespace hsl {
namespace {

constexpr int S_BM = 64, S_BN = 64, S_BK = 16;

__device__ __forceinline__ float operand_at(const MxOperand& o, int64_t i, int64_t k) {
  const int64_t r = o.trans ? k : i, c = o.trans ? i : k;
  switch (o.kind) {
    case MxOperand::kF32: return static_cast<const float*>(o.p)[r * o.pitch + c];
    case MxOperand::kBF16:
      return __bfloat162float(static_cast<const __nv_bfloat16*>(o.p)[r * o.pitch + c]);
    case MxOperand::kE2M1:
      return mx::value<false>(static_cast<const uint8_t*>(o.p) + r * o.pitch, o.scales + r * o.spitch, c);
    default:
      return mx::value<true>(static_cast<const uint8_t*>(o.p) + r * o.pitch, o.scales + r * o.spitch, c);
  }
}

template <typename TO>
__global__ void __launch_bounds__(256)
    k_mx_simt(MxOperand A, MxOperand B, int64_t M, int64_t N, int64_t K, const TO* add,
              TO* C, int64_t ldc) {
  __shared__ float sa[S_BK][S_BM + 4], sb[S_BK][S_BN + 4];
  const int64_t i0 = int64_t(blockIdx.x) * S_BM, j0 = int64_t(blockIdx.y) * S_BN;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {}, part[4][4] = {};
  for (int64_t k0 = 0; k0 < K; k0 += S_BK) {
    for (int e = threadIdx.x; e < S_BM * S_BK; e += 256) {
      // neighbouring threads take neighbouring elements of the stored rows
      const int ka = A.trans ? e / S_BM : e % S_BK, ia = A.trans ? e % S_BM : e / S_BK;
      sa[ka][ia] = (i0 + ia < M && k0 + ka < K) ? operand_at(A, i0 + ia, k0 + ka) : 0.f;
      const int kb = B.trans ? e / S_BN : e % S_BK, jb = B.trans ? e % S_BN : e / S_BK;
      sb[kb][jb] = (j0 + jb < N && k0 + kb < K) ? operand_at(B, j0 + jb, k0 + kb) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < S_BK; ++k) {
      float a[4], b[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        a[q] = sa[k][ty * 4 + q];
        b[q] = sb[k][tx * 4 + q];
      }
#pragma unroll
      for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int q = 0; q < 4; ++q) part[p][q] = fmaf(a[p], b[q], part[p][q]);
    }
    __syncthreads();
    if ((k0 & 63) == 48 || k0 + S_BK >= K) {
#pragma unroll
      for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          acc[p][q] += part[p][q];
          part[p][q] = 0.f;
        }
    }
  }
#pragma unroll
  for (int p = 0; p < 4; ++p)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t i = i0 + ty * 4 + p, j = j0 + tx * 4 + q;
      if (i < M && j < N) {
        float v = acc[p][q];
        if (add) v += VT<TO>::f(add[i * ldc + j]);
        C[i * ldc + j] = VT<TO>::from_f(v);
      }
    }
}

}  // namespace

hsl_status mx_simt_run(const MxOperand& A, const MxOperand& B, int64_t M, int64_t N, int64_t K,
                       const void* add, void* C, hsl_dtype cdt, cudaStream_t s) {
  if (M <= 0 || N <= 0) return HSL_OK;
  // rows past 65535 column tiles: the column tiles are taken in launches of that many
  for (int64_t j0 = 0; j0 < N; j0 += int64_t(65535) * S_BN) {
    const int64_t nj = N - j0 < int64_t(65535) * S_BN ? N - j0 : int64_t(65535) * S_BN;
    MxOperand b = B;
    if (j0) b = mx_operand_from(B, j0);
    const dim3 grid(unsigned((M + S_BM - 1) / S_BM), unsigned((nj + S_BN - 1) / S_BN));
    note_launch();
    if (cdt == HSL_F32)
      k_mx_simt<float><<<grid, 256, 0, s>>>(A, b, M, nj, K, add ? static_cast<const float*>(add) + j0 : nullptr,
                                            static_cast<float*>(C) + j0, N);
    else
      k_mx_simt<__nv_bfloat16><<<grid, 256, 0, s>>>(
          A, b, M, nj, K, add ? static_cast<const __nv_bfloat16*>(add) + j0 : nullptr,
          static_cast<__nv_bfloat16*>(C) + j0, N);
    if (hsl_status e = cuda_fail(cudaGetLastError(), "fp32 product launch")) return e;
  }
  return HSL_OK;
}

}  // namespace hsl
