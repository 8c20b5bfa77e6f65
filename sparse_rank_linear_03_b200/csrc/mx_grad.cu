// Gradients of the factors of x → U (Vᵀ x), bf16, from the input kept in int8 blocks:
//
//   Z = X V, G = dY U;   dU = dYᵀ Z, dV = Xᵀ G, dX = G Vᵀ (+ add)
//
// Five skinny products in two launches (first Z and G, then the three that use them),
// each launch one grid whose CTAs take tiles of one product or another: alone, most of
// them have fewer tiles than SMs or leave a last round half empty (28672 × 8192, rank
// 256, 4096 tokens: 317 µs as five launches, 260 so).  The second launch takes two thirds of
// that: two terms per product, and 96 KB from L2 per 256 × 256 × 64 step.  Z and G are summed over their
// splits into bf16 pairs (hi + lo, 16 significant bits), which the second
// products take as two terms.
#include "mx_gemm.cuh"

namespace hsl {
namespace {

// Each branch is the tile of one product (mx_gemm_tile.cuh).
template <int MG>
__global__ void __launch_bounds__(G_THREADS, 1)
    k_mx_grad_first(const __grid_constant__ GemmMaps gm, const __grid_constant__ GemmMaps zm,
                    const __grid_constant__ GemmArgs ga, const __grid_constant__ GemmArgs za, int ng) {
  constexpr bool BMN = true;
  constexpr int TERMS = 1, OUT = OUT_R;
  if (int(blockIdx.x) < ng) {
    constexpr int AK = A_BF16_K, MH = MG;
    const GemmMaps& maps = gm;
    const GemmArgs& g = ga;
    const int block = blockIdx.x;
#include "mx_gemm_tile.cuh"
  } else {
    constexpr int AK = A_INT8_K, MH = 1;
    const GemmMaps& maps = zm;
    const GemmArgs& g = za;
    const int block = blockIdx.x - ng;
#include "mx_gemm_tile.cuh"
  }
}
template <int MU, int MX>
__global__ void __launch_bounds__(G_THREADS, 1)
    k_mx_grad_second(const __grid_constant__ GemmMaps um, const __grid_constant__ GemmMaps vm,
                     const __grid_constant__ GemmMaps xm, const __grid_constant__ GemmArgs ua,
                     const __grid_constant__ GemmArgs va, const __grid_constant__ GemmArgs xa, int nu, int nv) {
  constexpr int TERMS = 2;
  if (int(blockIdx.x) < nu) {
    constexpr bool BMN = true;
    constexpr int AK = A_BF16_M, MH = MU, OUT = OUT_R;
    const GemmMaps& maps = um;
    const GemmArgs& g = ua;
    const int block = blockIdx.x;
#include "mx_gemm_tile.cuh"
  } else if (int(blockIdx.x) < nu + nv) {
    constexpr bool BMN = true;
    constexpr int AK = A_INT8_M, MH = 1, OUT = OUT_R;
    const GemmMaps& maps = vm;
    const GemmArgs& g = va;
    const int block = blockIdx.x - nu;
#include "mx_gemm_tile.cuh"
  } else {
    constexpr bool BMN = false;
    constexpr int AK = A_BF16_K, MH = MX, OUT = OUT_T;
    const GemmMaps& maps = xm;
    const GemmArgs& g = xa;
    const int block = blockIdx.x - nu - nv;
#include "mx_gemm_tile.cuh"
  }
}

// A sum over splits, and where it goes: a bf16 pair with rows padded to `pitch`, or bf16.
struct SumJob {
  const float* part;
  int splits, n, pitch;
  int64_t rows;
  __nv_bfloat16 *hi, *lo;  // lo: nullptr for a plain result (pitch = n)
};
template <int V>
__device__ __forceinline__ void sum_job(const SumJob& j, int64_t e) {
  if (e >= j.rows * j.pitch) return;
  const int64_t row = e / j.pitch;
  const int c = int(e - row * j.pitch);
  float v[V];
#pragma unroll
  for (int q = 0; q < V; ++q) v[q] = 0.f;
  if (c < j.n) sum_splits<V>(j.part, j.splits, j.rows * j.n, row * j.n + c, v);  // (V = 4: n = pitch)
  if (j.lo) {
    float low[V];
#pragma unroll
    for (int q = 0; q < V; ++q) {
      // (an infinity has no low part; a finite sum keeps a finite high part)
      float hi = __bfloat162float(__float2bfloat16_rn(v[q]));
      if (isinf(hi)) hi = __bfloat162float(__float2bfloat16_rz(v[q]));
      low[q] = isinf(hi) ? 0.f : v[q] - hi;
      v[q] = hi;
    }
    store_bf<V>(j.lo + e, low);
  }
  store_bf<V>(j.hi + e, v);
}
template <int V>
__global__ void __launch_bounds__(256)
    k_mx_grad_sum(const SumJob a, const SumJob b, int na) {
  pdl_trigger();
  pdl_wait();
  if (int(blockIdx.x) < na) sum_job<V>(a, (int64_t(blockIdx.x) * 256 + threadIdx.x) * V);
  else sum_job<V>(b, (int64_t(blockIdx.x - na) * 256 + threadIdx.x) * V);
}
hsl_status sum_run(const SumJob& a, const SumJob& b, bool vec, cudaStream_t s) {
  const int v = vec ? 4 : 1;
  const unsigned na = blocks_of(a.rows * a.pitch / v), nb = blocks_of(b.rows * b.pitch / v);
  if (na + nb == 0) return HSL_OK;
  note_launch();
  return cuda_fail(launch_chained(vec ? k_mx_grad_sum<4> : k_mx_grad_sum<1>, true, dim3(na + nb), 256, 0, s, a, b,
                                  int(na)), "split sum launch");
}

struct GradPlan {
  int64_t rp, mp;  // padded pitches of r- and m-wide rows
  GemmShape z, g, u, v, x;
  size_t off_dy, off_u, off_v, off_zh, off_zl, off_gh, off_gl, off_pa, off_pb, total;
};
GradPlan grad_plan(int64_t T, int64_t m, int64_t n, int64_t r) {
  GradPlan p;
  p.rp = round_up(r, 8);
  p.mp = round_up(m, 8);
  const int bn = int(round_up(r, 16));
  auto tiles = [](int64_t rows, int mh) { return (rows + 128 * mh - 1) / (128 * mh); };
  const int64_t nkg = (m + 63) / 64, nkz = (n + 63) / 64, nkt = (T + 63) / 64;

  // First launch: the SMs are shared out by work, K split accordingly, at least 4 K-blocks a
  // piece.
  p.z.MH = 1;
  p.z.BN = p.g.BN = bn;
  const int64_t tz = tiles(T, 1), cz = tz * nkz * kblock_cycles(A_INT8_K, 1, 1, bn);
  int64_t best = INT64_MAX;
  for (int mh = 1; mh <= 2; ++mh) {
    const int64_t tg = tiles(T, mh), per = kblock_cycles(A_BF16_K, 1, mh, bn), cg = tg * nkg * per;
    auto pieces = [&](int64_t work, int64_t t, int64_t nk) {
      return std::max<int64_t>(1, std::min<int64_t>(148 * work / (cg + cz) / t, nk / 4));
    };
    int64_t sg = pieces(cg, tg, nkg), sz = pieces(cz, tz, nkz);
    // (a product of little work has a piece per tile all the same: a few CTAs above 148 would be a round of their own)
    if (tg * sg + tz * sz > 148 && tz * sz < 148) sg = std::max<int64_t>(1, std::min(sg, (148 - tz * sz) / tg));
    if (tg * sg + tz * sz > 148 && tg * sg < 148) sz = std::max<int64_t>(1, std::min(sz, (148 - tg * sg) / tz));
    const int64_t time = std::max((nkg + sg - 1) / sg * per, (nkz + sz - 1) / sz * (cz / (tz * nkz))) +
                         (cg + cz) / 148;
    if (time < best) {
      best = time;
      p.g.MH = mh;
      p.g.splits = int(sg);
      p.z.splits = int(sz);
    }
  }
  fit_rings(&p.g, A_BF16_K, true, 1);
  fit_rings(&p.z, A_INT8_K, true, 1);

  // Second launch: K (the tokens) is split only where that saves more than the launch that adds
  // the pieces up, about 6000 cycles, and the pieces' traffic.
  p.v.MH = 1;
  p.u.BN = p.v.BN = bn;
  p.x = shape_of(A_BF16_K, n, T, r, false, 2, false);
  p.u.MH = tiles(m, 2) * kblock_cycles(A_BF16_M, 2, 2, bn) < tiles(m, 1) * kblock_cycles(A_BF16_M, 2, 1, bn) &&
                   tiles(m, 2) >= 74 && rings_fit(A_BF16_M, true, 2, 2, bn, 2)
               ? 2
               : 1;
  auto split_t = [&](int ak, int mh, int64_t rows) {
    const int64_t t = tiles(rows, mh), per = kblock_cycles(ak, 2, mh, bn);
    const int64_t s = std::max<int64_t>(1, std::min<int64_t>(74 / t, nkt / 4));
    return (nkt - (nkt + s - 1) / s) * per > 6000 + s * rows * r * 8 / 3500 ? int(s) : 1;
  };
  p.u.splits = split_t(A_BF16_M, p.u.MH, m);
  p.v.splits = split_t(A_INT8_M, 1, n);
  fit_rings(&p.u, A_BF16_M, true, 2);
  fit_rings(&p.v, A_INT8_M, true, 2);

  size_t o = 0;
  auto take = [&](int64_t bytes) {
    const size_t at = o;
    o += size_t(up16(bytes));
    return at;
  };
  p.off_dy = take(m % 8 ? T * p.mp * 2 : 0);
  p.off_u = take(r % 8 ? m * p.rp * 2 : 0);
  p.off_v = take(r % 8 ? n * p.rp * 2 : 0);
  p.off_zh = take(T * p.rp * 2);
  p.off_zl = take(T * p.rp * 2);
  p.off_gh = take(T * p.rp * 2);
  p.off_gl = take(T * p.rp * 2);
  // partial sums of G, then of dU; of Z, then of dV
  p.off_pa = take(std::max(p.g.splits * T * r * 4, p.u.splits > 1 ? p.u.splits * m * r * 4 : 0));
  p.off_pb = take(std::max(p.z.splits * T * r * 4, p.v.splits > 1 ? p.v.splits * n * r * 4 : 0));
  p.total = o;
  return p;
}

template <int MG>
hsl_status launch_first(const GemmMaps& gm, const GemmArgs& g, const GemmMaps& zm, const GemmArgs& z,
                        bool chained, cudaStream_t s) {
  void (*fn)(const GemmMaps, const GemmMaps, const GemmArgs, const GemmArgs, int) = k_mx_grad_first<MG>;
  const int bytes = std::max(tile_smem(A_BF16_K, true, 1, MG, false, g), tile_smem(A_INT8_K, true, 1, 1, false, z));
  if (cudaError_t e = allow_dyn_smem(reinterpret_cast<const void*>(fn), bytes))
    return cuda_fail(e, "factor gradient smem attribute");
  const int64_t ng = tile_count(MG, g), nz = tile_count(1, z);
  note_launch();
  return cuda_fail(launch_chained(fn, chained, dim3(unsigned(ng + nz)), G_THREADS, size_t(bytes), s, gm, zm, g, z,
                                  int(ng)), "factor gradient launch");
}
template <int MU, int MX>
hsl_status launch_second(const GemmMaps& um, const GemmArgs& u, const GemmMaps& vm, const GemmArgs& v,
                         const GemmMaps& xm, const GemmArgs& x, bool with_x, cudaStream_t s) {
  void (*fn)(const GemmMaps, const GemmMaps, const GemmMaps, const GemmArgs, const GemmArgs, const GemmArgs, int,
             int) = k_mx_grad_second<MU, MX>;
  int bytes = std::max(tile_smem(A_BF16_M, true, 2, MU, false, u), tile_smem(A_INT8_M, true, 2, 1, false, v));
  if (with_x) bytes = std::max(bytes, tile_smem(A_BF16_K, false, 2, MX, true, x));
  if (cudaError_t e = allow_dyn_smem(reinterpret_cast<const void*>(fn), bytes))
    return cuda_fail(e, "factor gradient smem attribute");
  const int64_t nu = tile_count(MU, u), nv = tile_count(1, v), nx = with_x ? tile_count(MX, x) : 0;
  note_launch();
  return cuda_fail(launch_chained(fn, true, dim3(unsigned(nu + nv + nx)), G_THREADS, size_t(bytes), s, um, vm, xm, u, v,
                                  x, int(nu), int(nv)), "factor gradient launch");
}

}  // namespace

size_t mx_gemm_grad_workspace(int64_t T, int64_t m, int64_t n, int64_t r) {
  return grad_plan(T, m, n, r).total;
}

hsl_status mx_gemm_grad_run(const MxOperand& X, int64_t T, int64_t n, const void* dY, int64_t m,
                            const void* U, const void* V, int64_t r, const void* add, void* dU, void* dV,
                            void* dX, void* ws, cudaStream_t s) {
  const GradPlan p = grad_plan(T, m, n, r);
  unsigned char* w = static_cast<unsigned char*>(ws);
  if (m % 8) {
    if (hsl_status e = pad_rows(dY, T, m, p.mp, w + p.off_dy, s)) return e;
    dY = w + p.off_dy;
  }
  if (r % 8) {
    if (hsl_status e = pad_rows(U, m, r, p.rp, w + p.off_u, s)) return e;
    if (hsl_status e = pad_rows(V, n, r, p.rp, w + p.off_v, s)) return e;
    U = w + p.off_u;
    V = w + p.off_v;
  }
  __nv_bfloat16* zh = reinterpret_cast<__nv_bfloat16*>(w + p.off_zh);
  __nv_bfloat16* zl = reinterpret_cast<__nv_bfloat16*>(w + p.off_zl);
  __nv_bfloat16* gh = reinterpret_cast<__nv_bfloat16*>(w + p.off_gh);
  __nv_bfloat16* gl = reinterpret_cast<__nv_bfloat16*>(w + p.off_gl);
  float* pa = reinterpret_cast<float*>(w + p.off_pa);
  float* pb = reinterpret_cast<float*>(w + p.off_pb);

  auto args = [&](const GemmShape& sh, int64_t M, int64_t N, int64_t K) {
    GemmArgs g = {};
    g.scales = X.scales;
    g.spitch = X.spitch;
    g.arows = int(T);
    g.nb = int(mx::blocks(n));
    g.M = int(M);
    g.N = int(N);
    g.nk = int((K + G_BK - 1) / G_BK);
    g.BN = sh.BN;
    g.stages = sh.stages;
    g.codes = sh.codes;
    g.splits = sh.splits;
    return g;
  };
  GemmMaps m0, m1, m2;
  memset(&m0, 0, sizeof(m0));
  memset(&m1, 0, sizeof(m1));
  memset(&m2, 0, sizeof(m2));
  GemmArgs g = args(p.g, T, r, m), z = args(p.z, T, r, n);
  g.part = pa;
  z.part = pb;
  if (!make_tmap_2d(&m0.a, kBF, 2, dY, T, m, p.mp, 64, 128, kSW) ||
      !make_tmap_2d(&m0.b0, kBF, 2, U, m, r, p.rp, 64, 64, kSW) ||
      !make_tmap_2d(&m1.b0, kBF, 2, V, n, r, p.rp, 64, 64, kSW) || !block_maps(&m1, A_INT8_K, 1, X, T))
    return map_failed();
  const bool padded = m % 8 || r % 8;
  if (hsl_status e = p.g.MH == 2 ? launch_first<2>(m0, g, m1, z, padded, s) : launch_first<1>(m0, g, m1, z, padded, s))
    return e;
  const SumJob sg = {pa, p.g.splits, int(r), int(p.rp), T, gh, gl}, sz = {pb, p.z.splits, int(r), int(p.rp), T, zh, zl};
  if (hsl_status e = sum_run(sg, sz, r % 8 == 0, s)) return e;

  GemmArgs u = args(p.u, m, r, T), v = args(p.v, n, r, T), x = args(p.x, n, T, r);
  auto result = [&](GemmArgs* a, void* out, float* part) {
    a->C = static_cast<__nv_bfloat16*>(out);
    a->cstore = (r % 8 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0) ? 1 : 0;
    a->part = a->splits > 1 ? part : nullptr;
  };
  result(&u, dU, pa);
  result(&v, dV, pb);
  memset(&m0, 0, sizeof(m0));
  memset(&m1, 0, sizeof(m1));
  if (!make_tmap_2d(&m0.a, kBF, 2, dY, T, m, p.mp, 64, 64, kSW) ||
      !make_tmap_2d(&m0.b0, kBF, 2, zh, T, r, p.rp, 64, 64, kSW) ||
      !make_tmap_2d(&m0.b1, kBF, 2, zl, T, r, p.rp, 64, 64, kSW) ||
      !make_tmap_2d(&m1.b0, kBF, 2, gh, T, r, p.rp, 64, 64, kSW) ||
      !make_tmap_2d(&m1.b1, kBF, 2, gl, T, r, p.rp, 64, 64, kSW) || !block_maps(&m1, A_INT8_M, 1, X, T))
    return map_failed();
  if (dX) {  // rows of V are the M side, tokens the N side
    x.add = static_cast<const __nv_bfloat16*>(add);
    x.C = static_cast<__nv_bfloat16*>(dX);
    if (!make_tmap_2d(&m2.a, kBF, 2, V, n, r, p.rp, 64, 128, kSW) ||
        !make_tmap_2d(&m2.b0, kBF, 2, gh, T, r, p.rp, 64, p.x.BN, kSW) ||
        !make_tmap_2d(&m2.b1, kBF, 2, gl, T, r, p.rp, 64, p.x.BN, kSW) || !out_maps(&m2, &x, T, n, p.x.MH))
      return map_failed();
  }
  const bool wx = dX != nullptr;
  hsl_status e;
  if (p.u.MH == 2)
    e = p.x.MH == 2 ? launch_second<2, 2>(m0, u, m1, v, m2, x, wx, s) : launch_second<2, 1>(m0, u, m1, v, m2, x, wx, s);
  else
    e = p.x.MH == 2 ? launch_second<1, 2>(m0, u, m1, v, m2, x, wx, s) : launch_second<1, 1>(m0, u, m1, v, m2, x, wx, s);
  if (e) return e;
  const SumJob su = {pa, p.u.splits, int(r), int(r), p.u.splits > 1 ? m : 0, static_cast<__nv_bfloat16*>(dU), nullptr};
  const SumJob sv = {pb, p.v.splits, int(r), int(r), p.v.splits > 1 ? n : 0, static_cast<__nv_bfloat16*>(dV), nullptr};
  const bool vec = r % 4 == 0 && reinterpret_cast<uintptr_t>(dU) % 8 == 0 && reinterpret_cast<uintptr_t>(dV) % 8 == 0;
  return sum_run(su, sv, vec, s);
}

cudaError_t mx_grad_error_word(uint32_t** p) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_mx_gemm_err);
}

}  // namespace hsl
