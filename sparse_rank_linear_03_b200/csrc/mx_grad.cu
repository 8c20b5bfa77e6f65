// Gradients of the factors of x → U (Vᵀ x), bf16, from the input kept in int8 blocks:
//
//   Z = X V, G = dY U;   dU = dYᵀ Z, dV = Xᵀ G, dX = G Vᵀ (+ add)
//
// Five skinny products in two launches (first Z and G, then the three that use them),
// each launch one grid whose CTAs take tiles of one product or another: alone, most of
// them have fewer tiles than SMs or leave a last round half empty.  Z and G are fp32 sums over their
// splits and stay so: three bf16 parts, which the second products take as three terms.  Sums over tokens and features
// leave the tensor unit every 16 or 24 of its steps (kFold in mx_gemm_tile.cuh; sums over r are 48 steps at
// most); that and the three parts bring the results from 2^−16 of their size to the error of fp32 sums.  What they cost, against two parts
// and sums that stay in the tensor unit: 28672 × 8192, rank 256, 4096 tokens 382 µs (269), where tiles
// become 128 columns instead of 256 and the second launch brings 80 KB from L2 per 256 × 128 × 64 step, 7 TB/s in
// all; 8192 × 8192, rank 128, 4096 tokens 154 (136); 4096 × 4096, rank 128, 500 tokens 28.7 (26.7) µs.
#include "mx_gemm.cuh"

namespace hsl {
namespace {

// Z and G are fp32 sums and stay so: hi + mid + lo, three bf16 whose bits together are the 24 of an fp32 value
// (below 2^−109 the last of them pass the end of bf16's range: each part is off by 2^−134 at most).
constexpr int Z_TERMS = 3;

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
  constexpr int TERMS = Z_TERMS;
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

// A sum over splits, and where it goes: Z_TERMS bf16 matrices, `apart` elements from one to the next, with rows
// padded to `pitch`; or one (apart = 0, pitch = n).
struct SumJob {
  const float* part;
  int splits, n, pitch;
  int64_t rows, apart;
  __nv_bfloat16* out;
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
  if (j.apart) {
#pragma unroll
    for (int t = 0; t < Z_TERMS - 1; ++t) {
      // (an infinity has no low parts; a finite sum keeps a finite high part)
      float hi[V];
#pragma unroll
      for (int q = 0; q < V; ++q) {
        hi[q] = __bfloat162float(__float2bfloat16_rn(v[q]));
        if (isinf(hi[q])) hi[q] = __bfloat162float(__float2bfloat16_rz(v[q]));
        v[q] = isinf(hi[q]) ? 0.f : v[q] - hi[q];
      }
      store_bf<V>(j.out + t * j.apart + e, hi);
    }
    e += (Z_TERMS - 1) * j.apart;
  }
  store_bf<V>(j.out + e, v);
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
  int64_t zpart;   // elements of one part of Z or G
  size_t off_dy, off_u, off_v, off_z, off_g, off_pa, off_pb, total;
};
GradPlan grad_plan(int64_t T, int64_t m, int64_t n, int64_t r) {
  GradPlan p;
  p.rp = round_up(r, 8);
  p.mp = round_up(m, 8);
  // columns of a tile: two sets of accumulators of up to 2 × 128 in TMEM
  const int64_t ntn = (r + 127) / 128;
  const int bn = int(round_up((r + ntn - 1) / ntn, 16));
  auto tiles = [&](int64_t rows, int mh) { return (rows + 128 * mh - 1) / (128 * mh) * ntn; };
  const int64_t nkg = (m + 63) / 64, nkz = (n + 63) / 64, nkt = (T + 63) / 64;

  // Cycles of a launch with na pieces of la cycles and behind them nb of lb.
  auto span = [](int64_t na, int64_t la, int64_t nb, int64_t lb) {
    if (na + nb <= 148) return std::max(la, lb);
    return std::max((na * la + nb * lb) / 148, la) + (na <= 148 ? lb : la + lb) / 2;
  };
  // First launch: pieces of G, at least 4 K-blocks each, in one round of CTAs, and pieces of Z beside and behind
  // them: shares of the SMs by work, or a whole round of G with Z in smaller pieces that take the SMs as
  // they come free, whichever is done earlier (28672 × 8192, rank 256, 4096 tokens: 64 CTAs of G and 64 of Z
  // leave most SMs idle while G's end, 128 and 192 keep them busy).
  p.z.MH = 1;
  p.z.BN = p.g.BN = bn;
  const int64_t tz = tiles(T, 1), perz = kblock_cycles(A_INT8_K, 1, 1, bn);
  int64_t best = INT64_MAX;
  for (int mh = 1; mh <= 2; ++mh) {
    const int64_t tg = tiles(T, mh), perg = kblock_cycles(A_BF16_K, 1, mh, bn);
    const int64_t cg = tg * nkg * perg, cz = tz * nkz * perz, topg = std::max<int64_t>(1, nkg / 4),
                  topz = std::max<int64_t>(1, nkz / 4);
    auto consider = [&](int64_t sg, int64_t sz) {
      sg = std::max<int64_t>(1, std::min(sg, topg));
      sz = std::max<int64_t>(1, std::min(sz, topz));
      const int64_t ng = tg * sg, nz = tz * sz;  // a piece takes its K-blocks and about 3000 cycles
      const int64_t lg = (nkg + sg - 1) / sg * perg + 3000, lz = (nkz + sz - 1) / sz * perz + 3000;
      const int64_t time = span(ng, lg, nz, lz) + (sg + sz) * T * r * 8 / 3500;  // and its sums' way through HBM
      if (time >= best) return;
      best = time;
      p.g.MH = mh;
      p.g.splits = int(sg);
      p.z.splits = int(sz);
    };
    const int64_t share = std::max<int64_t>(1, 148 * cg / (cg + cz) / tg);
    consider(share, (148 - std::min<int64_t>(148, tg * share)) / tz);
    consider((148 - std::min<int64_t>(148, tz)) / tg, 1);
    for (int64_t sz = 1; sz <= 8; sz *= 2) consider(148 / tg, sz);
  }
  fit_rings(&p.g, A_BF16_K, true, 1);
  fit_rings(&p.z, A_INT8_K, true, 1);

  // Second launch: K (the tokens) is split only where that saves more than the launch that adds
  // the pieces up, about 6000 cycles, and the pieces' traffic.
  p.v.MH = 1;
  p.u.BN = p.v.BN = bn;
  p.x = shape_of(A_BF16_K, n, T, r, false, Z_TERMS, false);
  p.u.MH = tiles(m, 2) * kblock_cycles(A_BF16_M, Z_TERMS, 2, bn) <
                       tiles(m, 1) * kblock_cycles(A_BF16_M, Z_TERMS, 1, bn) &&
                   tiles(m, 2) >= 74 && rings_fit(A_BF16_M, true, Z_TERMS, 2, bn, 2)
               ? 2
               : 1;
  // (two CTAs above 148 cost as much as a whole round: 1500 tokens, 4096 × 11008, rank 64, dU in two pieces: 60 µs, 36 in one)
  const int64_t tu = tiles(m, p.u.MH), tv = tiles(n, 1), top = std::max<int64_t>(1, nkt / 4);
  const int64_t peru = kblock_cycles(A_BF16_M, Z_TERMS, p.u.MH, bn), perv = kblock_cycles(A_INT8_M, Z_TERMS, 1, bn);
  best = INT64_MAX;
  auto split_t = [&](int64_t su, int64_t sv) {
    su = std::max<int64_t>(1, std::min(su, top));
    sv = std::max<int64_t>(1, std::min(sv, top));
    const int64_t moved = (su > 1 ? su * m : 0) + (sv > 1 ? sv * n : 0);
    const int64_t time = span(tu * su, (nkt + su - 1) / su * peru + 3000, tv * sv, (nkt + sv - 1) / sv * perv + 3000) +
                         (moved ? 6000 + moved * r * 8 / 3500 : 0);
    if (time >= best) return;
    best = time;
    p.u.splits = int(su);
    p.v.splits = int(sv);
  };
  const int64_t share = 148 * tu * peru / (tu * peru + tv * perv) / tu;
  split_t(1, 1);
  split_t(share, (148 - std::min<int64_t>(148, tu * std::max<int64_t>(1, share))) / tv);
  split_t(1, (148 - std::min<int64_t>(148, tu)) / tv);
  split_t((148 - std::min<int64_t>(148, tv)) / tu, 1);
  fit_rings(&p.u, A_BF16_M, true, Z_TERMS);
  fit_rings(&p.v, A_INT8_M, true, Z_TERMS);

  size_t o = 0;
  auto take = [&](int64_t bytes) {
    const size_t at = o;
    o += size_t(up16(bytes));
    return at;
  };
  p.off_dy = take(m % 8 ? T * p.mp * 2 : 0);
  p.off_u = take(r % 8 ? m * p.rp * 2 : 0);
  p.off_v = take(r % 8 ? n * p.rp * 2 : 0);
  p.zpart = up16(T * p.rp * 2) / 2;
  p.off_z = take(Z_TERMS * p.zpart * 2);
  p.off_g = take(Z_TERMS * p.zpart * 2);
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
  int bytes = std::max(tile_smem(A_BF16_M, true, Z_TERMS, MU, false, u), tile_smem(A_INT8_M, true, Z_TERMS, 1, false, v));
  if (with_x) bytes = std::max(bytes, tile_smem(A_BF16_K, false, Z_TERMS, MX, true, x));
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
  __nv_bfloat16* zp = reinterpret_cast<__nv_bfloat16*>(w + p.off_z);
  __nv_bfloat16* gp = reinterpret_cast<__nv_bfloat16*>(w + p.off_g);
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
      !make_tmap_2d(&m0.b[0], kBF, 2, U, m, r, p.rp, 64, 64, kSW) ||
      !make_tmap_2d(&m1.b[0], kBF, 2, V, n, r, p.rp, 64, 64, kSW) || !block_maps(&m1, A_INT8_K, 1, X, T))
    return map_failed();
  const bool padded = m % 8 || r % 8;
  if (hsl_status e = p.g.MH == 2 ? launch_first<2>(m0, g, m1, z, padded, s) : launch_first<1>(m0, g, m1, z, padded, s))
    return e;
  const SumJob sg = {pa, p.g.splits, int(r), int(p.rp), T, p.zpart, gp};
  const SumJob sz = {pb, p.z.splits, int(r), int(p.rp), T, p.zpart, zp};
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
  if (!make_tmap_2d(&m0.a, kBF, 2, dY, T, m, p.mp, 64, 64, kSW) || !block_maps(&m1, A_INT8_M, 1, X, T))
    return map_failed();
  if (dX) {  // rows of V are the M side, tokens the N side
    x.add = static_cast<const __nv_bfloat16*>(add);
    x.C = static_cast<__nv_bfloat16*>(dX);
    if (!make_tmap_2d(&m2.a, kBF, 2, V, n, r, p.rp, 64, 128, kSW) || !out_maps(&m2, &x, T, n, p.x.MH))
      return map_failed();
  }
  for (int t = 0; t < Z_TERMS; ++t)
    if (!make_tmap_2d(&m0.b[t], kBF, 2, zp + t * p.zpart, T, r, p.rp, 64, 64, kSW) ||
        !make_tmap_2d(&m1.b[t], kBF, 2, gp + t * p.zpart, T, r, p.rp, 64, 64, kSW) ||
        (dX && !make_tmap_2d(&m2.b[t], kBF, 2, gp + t * p.zpart, T, r, p.rp, 64, p.x.BN, kSW)))
      return map_failed();
  const bool wx = dX != nullptr;
  hsl_status e;
  if (p.u.MH == 2)
    e = p.x.MH == 2 ? launch_second<2, 2>(m0, u, m1, v, m2, x, wx, s) : launch_second<2, 1>(m0, u, m1, v, m2, x, wx, s);
  else
    e = p.x.MH == 2 ? launch_second<1, 2>(m0, u, m1, v, m2, x, wx, s) : launch_second<1, 1>(m0, u, m1, v, m2, x, wx, s);
  if (e) return e;
  const SumJob su = {pa, p.u.splits, int(r), int(r), p.u.splits > 1 ? m : 0, 0, static_cast<__nv_bfloat16*>(dU)};
  const SumJob sv = {pb, p.v.splits, int(r), int(r), p.v.splits > 1 ? n : 0, 0, static_cast<__nv_bfloat16*>(dV)};
  const bool vec = r % 4 == 0 && reinterpret_cast<uintptr_t>(dU) % 8 == 0 && reinterpret_cast<uintptr_t>(dV) % 8 == 0;
  return sum_run(su, sv, vec, s);
}

cudaError_t mx_grad_error_word(uint32_t** p) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_mx_gemm_err);
}

}  // namespace hsl
