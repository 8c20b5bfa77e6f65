// Y = X Dᵀ and its input gradient dX = dY D on the tensor cores, D in e2m1 blocks (bf16).
#include "mx_gemm.cuh"

namespace hsl {
namespace {

template <int V>
__global__ void __launch_bounds__(256)
    k_mx_reduce(const float* __restrict__ part, int splits, int64_t count, const __nv_bfloat16* add,
                __nv_bfloat16* C) {
  pdl_wait();
  const int64_t e = (int64_t(blockIdx.x) * 256 + threadIdx.x) * V;
  if (e >= count) return;
  float v[V];
  sum_splits<V>(part, splits, count, e, v);
  if (add) {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] += __bfloat162float(add[e + j]);
  }
  store_bf<V>(C + e, v);
}

hsl_status reduce_run(const float* part, int splits, int64_t count, const __nv_bfloat16* add, __nv_bfloat16* C,
                      cudaStream_t s) {
  note_launch();
  if (count % 4 == 0 && reinterpret_cast<uintptr_t>(C) % 8 == 0)
    return cuda_fail(launch_chained(k_mx_reduce<4>, true, dim3(blocks_of(count / 4)), 256, 0, s, part, splits, count,
                                    add, C), "split sum launch");
  return cuda_fail(launch_chained(k_mx_reduce<1>, true, dim3(blocks_of(count)), 256, 0, s, part, splits, count, add, C),
                   "split sum launch");
}
}  // namespace

size_t mx_gemm_apply_workspace(bool trans, int64_t T, int64_t m, int64_t n) {
  const int64_t M = trans ? n : m, K = trans ? m : n;
  const GemmShape sh = shape_of(trans ? A_E2M1_M : A_E2M1_K, M, T, K, false, 1, true);
  size_t b = 0;
  if (K % 8) b += up16(T * round_up(K, 8) * 2);
  if (sh.splits > 1) b += up16(int64_t(sh.splits) * T * M * 4);
  return b;
}

bool mx_gemm_supported(const void* X) {
  return reinterpret_cast<uintptr_t>(X) % 16 == 0 && tmap_available();
}

hsl_status mx_gemm_apply_run(bool trans, const MxOperand& D, int64_t m, int64_t n, const void* X,
                             const void* add, void* Y, int64_t T, void* ws, cudaStream_t s) {
  const int64_t M = trans ? n : m, K = trans ? m : n;
  const GemmShape sh = shape_of(trans ? A_E2M1_M : A_E2M1_K, M, T, K, false, 1, true);
  unsigned char* w = static_cast<unsigned char*>(ws);
  int64_t kp = K;
  if (K % 8) {
    kp = round_up(K, 8);
    if (hsl_status e = pad_rows(X, T, K, kp, w, s)) return e;
    X = w;
    w += up16(T * kp * 2);
  }
  GemmMaps maps;
  memset(&maps, 0, sizeof(maps));
  GemmArgs g = {};
  g.scales = D.scales;
  g.spitch = D.spitch;
  g.arows = int(m);
  g.nb = int(mx::blocks(n));
  g.M = int(M);
  g.N = int(T);
  g.nk = int((K + G_BK - 1) / G_BK);
  g.BN = sh.BN;
  g.stages = sh.stages;
  g.codes = sh.codes;
  g.splits = sh.splits;
  g.add = static_cast<const __nv_bfloat16*>(add);
  g.C = static_cast<__nv_bfloat16*>(Y);
  g.part = reinterpret_cast<float*>(w);
  if (!make_tmap_2d(&maps.b[0], kBF, 2, X, T, K, kp, 64, sh.BN, kSW) ||
      !block_maps(&maps, trans ? A_E2M1_M : A_E2M1_K, sh.MH, D, m))
    return map_failed();
  if (sh.splits > 1) {
    if (hsl_status e = trans ? launch_gemm<A_E2M1_M, false, 1, OUT_T_PART>(sh.MH, maps, g, K % 8 != 0, s)
                             : launch_gemm<A_E2M1_K, false, 1, OUT_T_PART>(sh.MH, maps, g, K % 8 != 0, s))
      return e;
    return reduce_run(g.part, sh.splits, T * M, g.add, g.C, s);
  }
  if (!out_maps(&maps, &g, T, M, sh.MH)) return map_failed();
  return trans ? launch_gemm<A_E2M1_M, false, 1, OUT_T>(sh.MH, maps, g, K % 8 != 0, s)
               : launch_gemm<A_E2M1_K, false, 1, OUT_T>(sh.MH, maps, g, K % 8 != 0, s);
}

cudaError_t mx_gemm_error_word(uint32_t** p) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_mx_gemm_err);
}

}  // namespace hsl
