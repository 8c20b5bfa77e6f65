// Products whose operands may be microscaled, on the CUDA cores in fp32: the path of
// f32 data (and of the calls that no faster kernel takes).
//
//   C[i][j] = add[i][j] + Σ_k A(i, k) B(j, k)
//
// Each operand is fp32, bf16, e2m1 blocks or int8 blocks, stored as [i][k] or
// transposed as [k][i]; it is widened exactly to fp32 on its way to shared memory.
// A CTA owns a 64 × 64 tile (16 sums per thread) of a range of K; few tiles and a long K
// (the gradients of a small layer) are cut into ranges for all SMs, whose sums are
// added up in order by a second kernel.  The next 16 k are loaded while 16 are worked on.
// The sums are kept in two levels, folded every 64 terms, so that the rounding error
// of a long sum grows with the root of 64 terms and of K/64 folds rather than of K.
// Bound by the fp32 FMA rate and, at small sizes, by the latency of a K loop (64 × 4096 × 4096,
// gradient of the input: 250 µs in one range of K, 99 in eleven).
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "mx.cuh"
#include "mx_ops.h"

namespace hsl {
namespace {

constexpr int S_BM = 64, S_BN = 64, S_BK = 16;
constexpr int kAny = -1;

template <int KIND>
__device__ __forceinline__ int kind_at(const MxOperand& o) { return KIND == kAny ? o.kind : KIND >> 1; }
template <int KIND>
__device__ __forceinline__ bool is_trans(const MxOperand& o) {
  return KIND == kAny ? o.trans != 0 : (KIND & 1) != 0;
}

// Four neighbouring values of a stored row, as they are stored (loaded well before they are used).
struct Raw {
  uint32_t w[4];
  uint32_t e;
};
// Columns c .. c + 3 (c a multiple of 4) of stored row r, zeros from column `cols` on.
template <int KIND>
__device__ __forceinline__ Raw load4(const MxOperand& o, int64_t r, int64_t c, int64_t cols) {
  Raw v = {{0, 0, 0, 0}, 0};
  if (c >= cols) return v;
  const int kind = kind_at<KIND>(o);
  if (kind == MxOperand::kF32) {  // (Z and G of the factor gradients are the call's own: no read-only loads)
    const uint32_t* p = static_cast<const uint32_t*>(o.p) + r * o.pitch + c;
    if (o.vec && c + 4 <= cols) {
      const uint4 q = ld_chained16(p);
      v.w[0] = q.x; v.w[1] = q.y; v.w[2] = q.z; v.w[3] = q.w;
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (c + q < cols) v.w[q] = ld_chained4(p + q);
    }
  } else if (kind == MxOperand::kBF16) {
    const uint16_t* p = static_cast<const uint16_t*>(o.p) + r * o.pitch + c;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (c + q < cols) v.w[q] = uint32_t(__ldg(p + q)) << 16;
  } else {
    const uint8_t* p = static_cast<const uint8_t*>(o.p) + r * o.pitch;
    v.w[0] = kind == MxOperand::kE2M1 ? uint32_t(__ldg(reinterpret_cast<const uint16_t*>(p + c / 2)))
                                      : __ldg(reinterpret_cast<const uint32_t*>(p + c));
    v.e = __ldg(o.scales + r * o.spitch + (c >> 5));
    // (values past the row's end are padding codes: zero)
    const int64_t left = cols - c;
    if (left < 4) v.w[0] &= (1u << (int(left) * (kind == MxOperand::kE2M1 ? 4 : 8))) - 1;
  }
  return v;
}
template <int KIND>
__device__ __forceinline__ float4 widen4(const MxOperand& o, const Raw& v) {
  const int kind = kind_at<KIND>(o);
  if (kind == MxOperand::kE2M1) {
    const float s = mx::scale_f32(v.e);
    return make_float4(mx::e2m1_f32(v.w[0] & 15u) * s, mx::e2m1_f32((v.w[0] >> 4) & 15u) * s,
                       mx::e2m1_f32((v.w[0] >> 8) & 15u) * s, mx::e2m1_f32((v.w[0] >> 12) & 15u) * s);
  }
  if (kind == MxOperand::kInt8) {
    const float s = mx::scale_f32(v.e);
    return make_float4(float(int8_t(v.w[0])) * 0.015625f * s, float(int8_t(v.w[0] >> 8)) * 0.015625f * s,
                       float(int8_t(v.w[0] >> 16)) * 0.015625f * s, float(int8_t(v.w[0] >> 24)) * 0.015625f * s);
  }
  return make_float4(__uint_as_float(v.w[0]), __uint_as_float(v.w[1]), __uint_as_float(v.w[2]),
                     __uint_as_float(v.w[3]));
}

// One operand of a 64 × 16 step: thread t brings four neighbouring values of a stored row.
template <int KIND>
struct Side {
  int row, col;  // of the tile as it is stored: [64 i][16 k], or [16 k][64 i]
  bool trans;
  Raw raw;
  __device__ __forceinline__ explicit Side(const MxOperand& o) {
    trans = is_trans<KIND>(o);
    row = trans ? threadIdx.x / 16 : threadIdx.x / 4;
    col = trans ? threadIdx.x % 16 * 4 : threadIdx.x % 4 * 4;
  }
  __device__ __forceinline__ void load(const MxOperand& o, int64_t i0, int64_t rows, int64_t k0, int64_t kend) {
    const int64_t r = (trans ? k0 : i0) + row, c = (trans ? i0 : k0) + col;
    raw = r < (trans ? kend : rows) ? load4<KIND>(o, r, c, trans ? rows : kend) : Raw{{0, 0, 0, 0}, 0};
  }
  __device__ __forceinline__ void store(const MxOperand& o, float (*t)[68]) const {
    const float4 v = widen4<KIND>(o, raw);
    if (trans) {
      *reinterpret_cast<float4*>(&t[row][col]) = v;
    } else {
      t[col][row] = v.x;
      t[col + 1][row] = v.y;
      t[col + 2][row] = v.z;
      t[col + 3][row] = v.w;
    }
  }
};

// kPart: the fp32 sums of K range blockIdx.z go to part [range][M][N].
template <int KA, int KB, typename TO, bool kPart>
__global__ void __launch_bounds__(256)
    k_mx_simt(const MxOperand A, const MxOperand B, int64_t M, int64_t N, int64_t K, int64_t krange, const TO* add,
              TO* C, float* __restrict__ part) {
  __shared__ __align__(16) float sa[S_BK][68], sb[S_BK][68];
  pdl_trigger();
  pdl_wait();
  const unsigned tm = unsigned((M + S_BM - 1) / S_BM);
  const int64_t i0 = int64_t(blockIdx.x % tm) * S_BM, j0 = int64_t(blockIdx.x / tm) * S_BN;
  const int64_t kbeg = int64_t(blockIdx.z) * krange, kend = min(K, kbeg + krange);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {}, sum[4][4] = {};
  Side<KA> a_side(A);
  Side<KB> b_side(B);
  a_side.load(A, i0, M, kbeg, kend);
  b_side.load(B, j0, N, kbeg, kend);
  int folded = 0;
  for (int64_t k0 = kbeg; k0 < kend; k0 += S_BK) {
    __syncthreads();
    a_side.store(A, sa);
    b_side.store(B, sb);
    __syncthreads();
    if (k0 + S_BK < kend) {
      a_side.load(A, i0, M, k0 + S_BK, kend);
      b_side.load(B, j0, N, k0 + S_BK, kend);
    }
#pragma unroll
    for (int k = 0; k < S_BK; ++k) {
      const float4 a4 = *reinterpret_cast<const float4*>(&sa[k][ty * 4]);
      const float4 b4 = *reinterpret_cast<const float4*>(&sb[k][tx * 4]);
      const float a[4] = {a4.x, a4.y, a4.z, a4.w}, b[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
      for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int q = 0; q < 4; ++q) sum[p][q] = fmaf(a[p], b[q], sum[p][q]);
    }
    if (++folded == 4 || k0 + S_BK >= kend) {
      folded = 0;
#pragma unroll
      for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          acc[p][q] += sum[p][q];
          sum[p][q] = 0.f;
        }
    }
  }
#pragma unroll
  for (int p = 0; p < 4; ++p)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t i = i0 + ty * 4 + p, j = j0 + tx * 4 + q;
      if (i >= M || j >= N) continue;
      const int64_t at = i * N + j;
      if (kPart) {
        part[int64_t(blockIdx.z) * M * N + at] = acc[p][q];
      } else {
        float v = acc[p][q];
        if (add) v += VT<TO>::f(add[at]);
        C[at] = VT<TO>::from_f(v);
      }
    }
}

template <typename TO>
__global__ void __launch_bounds__(256)
    k_mx_simt_sum(const float* __restrict__ part, int ranges, int64_t count, const TO* add, TO* C) {
  pdl_trigger();
  pdl_wait();
  const int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (e >= count) return;
  float v = 0.f;
  for (int s0 = 0; s0 < ranges; s0 += 8) {  // eight loads on their way at a time
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (s0 + j < ranges) q[j] = __ldcs(part + int64_t(s0 + j) * count + e);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (s0 + j < ranges) v += q[j];
  }
  if (add) v += VT<TO>::f(add[e]);
  C[e] = VT<TO>::from_f(v);
}

// Ranges of K: five CTAs per SM (they wait for loads most of the time) where the tiles alone are fewer,
// at least 64 k each.
int ranges_of(int64_t M, int64_t N, int64_t K) {
  const int64_t tiles = (M + S_BM - 1) / S_BM * ((N + S_BN - 1) / S_BN);
  return int(std::max<int64_t>(1, std::min<int64_t>(740 / std::max<int64_t>(tiles, 1), K / 64)));
}

template <int KA, int KB, typename TO>
hsl_status run(const MxOperand& A, const MxOperand& B, int64_t M, int64_t N, int64_t K, const TO* add, TO* C,
               float* part, bool chained, cudaStream_t s) {
  const int ranges = part ? ranges_of(M, N, K) : 1;
  const int64_t krange = ranges > 1 ? ((K + ranges - 1) / ranges + S_BK - 1) / S_BK * S_BK : K;
  const int64_t nz = ranges > 1 ? (K + krange - 1) / krange : 1;
  // (tiles in one dimension: the others end at 65535)
  const dim3 grid(unsigned((M + S_BM - 1) / S_BM * ((N + S_BN - 1) / S_BN)), 1, unsigned(nz));
  note_launch();
  if (nz == 1) {
    return cuda_fail(launch_chained(k_mx_simt<KA, KB, TO, false>, chained, grid, 256, 0, s, A, B, M, N, K, K, add, C,
                                    nullptr), "fp32 product launch");
  }
  if (hsl_status e = cuda_fail(launch_chained(k_mx_simt<KA, KB, TO, true>, chained, grid, 256, 0, s, A, B, M, N, K,
                                              krange, add, C, part), "fp32 product launch"))
    return e;
  note_launch();
  return cuda_fail(launch_chained(k_mx_simt_sum<TO>, true, dim3(unsigned((M * N + 255) / 256)), 256, 0, s, part,
                                  int(nz), M * N, add, C), "split sum launch");
}

constexpr int kind_of(int kind, bool trans) { return kind * 2 + (trans ? 1 : 0); }
constexpr int F = kind_of(MxOperand::kF32, false), FT = kind_of(MxOperand::kF32, true);
constexpr int E = kind_of(MxOperand::kE2M1, false), ET = kind_of(MxOperand::kE2M1, true);
constexpr int I = kind_of(MxOperand::kInt8, false), IT = kind_of(MxOperand::kInt8, true);

}  // namespace

size_t mx_simt_workspace(int64_t M, int64_t N, int64_t K) {
  const int r = ranges_of(M, N, K);
  return r > 1 ? size_t(r) * size_t(M * N) * 4 : 0;
}

hsl_status mx_simt_sum_run(const float* part, int ranges, int64_t count, const float* add, float* C, cudaStream_t s) {
  note_launch();
  return cuda_fail(launch_chained(k_mx_simt_sum<float>, true, dim3(unsigned((count + 255) / 256)), 256, 0, s, part, ranges,
                                  count, add, C), "split sum launch");
}

hsl_status mx_simt_run(const MxOperand& A, const MxOperand& B, int64_t M, int64_t N, int64_t K,
                       const void* add, void* C, hsl_dtype cdt, void* part, bool chained, cudaStream_t s) {
  if (M <= 0 || N <= 0) return HSL_OK;
  float* w = mx_simt_workspace(M, N, K) ? static_cast<float*>(part) : nullptr;
  const int ka = kind_of(A.kind, A.trans != 0), kb = kind_of(B.kind, B.trans != 0);
  if (cdt == HSL_F32) {
    const float* a = static_cast<const float*>(add);
    float* c = static_cast<float*>(C);
    if (ka == F && kb == E) return run<F, E, float>(A, B, M, N, K, a, c, w, chained, s);
    if (ka == F && kb == ET) return run<F, ET, float>(A, B, M, N, K, a, c, w, chained, s);
    if (ka == I && kb == FT) return run<I, FT, float>(A, B, M, N, K, a, c, w, chained, s);
    if (ka == F && kb == FT) return run<F, FT, float>(A, B, M, N, K, a, c, w, chained, s);
    if (ka == FT && kb == FT) return run<FT, FT, float>(A, B, M, N, K, a, c, w, chained, s);
    if (ka == IT && kb == FT) return run<IT, FT, float>(A, B, M, N, K, a, c, w, chained, s);
    if (ka == F && kb == F) return run<F, F, float>(A, B, M, N, K, a, c, w, chained, s);
    return run<kAny, kAny, float>(A, B, M, N, K, a, c, w, chained, s);
  }
  // bf16 that the tensor-core kernels do not take (pointers off 16 bytes)
  return run<kAny, kAny, __nv_bfloat16>(A, B, M, N, K, static_cast<const __nv_bfloat16*>(add),
                                        static_cast<__nv_bfloat16*>(C), w, chained, s);
}

}  // namespace hsl
