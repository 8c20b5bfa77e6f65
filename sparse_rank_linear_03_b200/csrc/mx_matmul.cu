// Product of two matrices in e2m1 blocks on the block-scaled 4-bit MMA.
//
//   C[t][i] = add[t][i] + Σ_j A[t][j] B[i][j]
//
// tcgen05.mma kind::mxf4 takes both operands as packed 4-bit floats and multiplies
// each 32-term piece of a dot product by the two blocks' powers of two, with fp32
// sums: the definition itself, no widening.  With 256 tokens or more the tokens are the M
// side of the MMA and the features its N side: a TMEM lane then holds neighbouring
// values of an output row, which go out in 16-byte pieces (1000 × 1023, 300 tokens: 8.2 µs, 16.7 the
// other way round).  With fewer, the features are the M side, so that no accumulator row is
// idle (28672 × 8192: 35 µs at 16 tokens and 45 at 200, 55 and 53 the other way round).
//
//   warp 0 lane 0   TMA of the code tiles: 128·MH rows of the M side, BN of the N side, 256
//                   values (128 bytes) each, 128-byte swizzle
//   warp 10 lane 0  TMA of the scale bytes, 16 per row: two K-blocks at a time
//   warps 2-5       put a K-block's scales where the MMA reads them: TMEM lane
//                   r mod 32 of every quarter, column r / 32, four scales per
//                   column; each warp fills its quarter (tcgen05.st)
//   warp 1 lane 0   four MMAs of K = 64 per K-block and accumulator; the scale
//                   pair is selected by the instruction descriptor
//   warps 2-9       epilogue: tcgen05.ld, add, round, store
//
// Bound by shared memory: at 4 bits a 128 × 256 × 256 step takes the MMA 512 cycles and brings
// 48 KB, so the tile is 256 × 192 (two accumulators sharing the N side's tile): 56 KB per
// 768 cycles, and each MMA reads its operands again.  The two accumulators take 384
// TMEM columns, the scales of the stages the rest.  28672 × 8192 at 4096 tokens: 377 µs,
// 5.1 PFLOP/s (450 µs in a row of calls, where the power limit slows the clock).  Every wait is bounded.
#include <cuda.h>

#include <algorithm>
#include <cstring>

#include "common.cuh"
#include "internal.h"
#include "mx.cuh"
#include "mx_ops.h"
#include "tc.cuh"

namespace hsl {
namespace {

__device__ uint32_t g_mx_matmul_err;

constexpr int F_THREADS = 352;
constexpr int F_MAX_STAGES = 6;
constexpr int F_SRING = 3;                 // scale tiles (two K-blocks each) in flight
constexpr int F_SMEM_BUDGET = 216 * 1024;  // code stages and scale tiles

struct MmMaps {
  CUtensorMap b, bs;  // M side: codes box {128 B, 128}, scales box {16 B, 128}
  CUtensorMap a, as;  // N side: codes box {128 B, BN}, scales box {16 B, BN}
  CUtensorMap c;      // box {64, 128} (kRows) or {128·MH, BN}
};
struct MmArgs {
  int M, N, nk, nb;  // rows of the M side, of the N side, K-blocks of 256, blocks per row
  int BN, stages, cstore;
  const void* add;
  void* C;
};

__device__ __forceinline__ bool f_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (tc::mbar_try(bar, parity)) return true;
  if (*abort_flag) return false;
  if (tc::mbar_wait(bar, parity, &g_mx_matmul_err)) return true;
  *abort_flag = 1;
  return false;
}

// D (+)= A B, both e2m1 with ue8m0 scales of 32-value blocks in TMEM.
__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc,
                                         uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
          d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
// Instruction descriptor, kind::mxf4: e2m1 × e2m1, ue8m0 scales; `sf` (0 or 2) is the byte
// of the scale words at which this MMA's pair of scales starts.
__device__ __forceinline__ uint32_t idesc_mxf4(int M, int N, uint32_t sf) {
  return (sf << 4) | (1u << 7) | (1u << 10) | (uint32_t(N >> 3) << 17) | (1u << 23) |
         (uint32_t(M >> 4) << 24) | (sf << 29);
}

// How C is stored: [N][M], or [M][N] (tokens on the M side) in tiles, or, where rows do not start on 16 bytes
// or are fp32, row by row by way of shared memory.
enum MmOut { kCols, kTiles, kEach };
template <typename TO, int MH, MmOut kOut>
__global__ void __launch_bounds__(F_THREADS, 1)
    k_mx_matmul(const __grid_constant__ MmMaps maps, const MmArgs g) {
  constexpr bool kRows = kOut != kCols;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  // (an offset, not a rounded integer: the compiler still knows that this is shared memory)
  unsigned char* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ uint64_t full[F_MAX_STAGES], empty[F_MAX_STAGES], sfull[F_SRING], sempty[F_SRING], accf;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ntn = (g.N + g.BN - 1) / g.BN;
  // the tokens run fastest: CTAs at work at the same time share the weights' tiles in L2
  const int ntm = (g.M + 128 * MH - 1) / (128 * MH);
  const int i0 = (kRows ? blockIdx.x % ntm : blockIdx.x / ntn) * (128 * MH);
  const int j0 = (kRows ? blockIdx.x / ntm : blockIdx.x % ntn) * g.BN;
  constexpr int kM = MH * 128;
  const int kStage = kM * 128 + g.BN * 128;
  const int kScale = (kM + g.BN) * 16;
  unsigned char* sring = smem + g.stages * kStage;
  // TMEM: accumulators, then per stage the scales of M (4 columns per 128 rows and
  // group of four blocks) and of N
  const int ncols = (g.BN + 31) / 32;
  const int npitch = (ncols + 3) / 4 * 4;  // scale addresses on four columns
  const int sf_cols = MH * 8 + 2 * npitch;
  const uint32_t sf0 = uint32_t(MH * g.BN);

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < g.stages; ++s) {
      tc::mbar_init(&full[s], 1 + 4);  // the code copies and the four scale warps
      tc::mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < F_SRING; ++s) {
      tc::mbar_init(&sfull[s], 1);
      tc::mbar_init(&sempty[s], 4);
    }
    tc::mbar_init(&accf, 1);
    tc::fence_mbar_init();
    tc::prefetch_tmap(&maps.a);
    tc::prefetch_tmap(&maps.b);
    tc::prefetch_tmap(&maps.as);
    tc::prefetch_tmap(&maps.bs);
  }
  if (warp == 1) {
    tc::tmem_alloc(&tmem_slot, 512);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = tmem_slot;
  volatile int* abrt = &abort_flag;

  if (warp == 0) {
    if (lane == 0) {
      int s = 0, issued = 0;
      uint32_t ph = 1;
      for (int kb = 0; kb < g.nk; ++kb) {
        if (!f_wait(&empty[s], ph, abrt)) break;
        unsigned char* p = smem + s * kStage;
        tc::mbar_expect_tx(&full[s], kStage);
#pragma unroll
        for (int h = 0; h < MH; ++h)
          tc::tma_load_2d(p + h * 16384, &maps.b, kb * 128, i0 + h * 128, &full[s]);
        tc::tma_load_2d(p + kM * 128, &maps.a, kb * 128, j0, &full[s]);
        ++issued;
        if (++s == g.stages) {
          s = 0;
          ph ^= 1;
        }
      }
      if (*abrt)  // copies in flight land before the shared memory is given up
        for (int q = 0; q < g.stages && q < issued; ++q)
          tc::mbar_wait(&full[q], uint32_t((issued - 1 - q) / g.stages) & 1, &g_mx_matmul_err);
    }
    __syncwarp();
  } else if (warp == 10) {
    if (lane == 0) {
      int s = 0, issued = 0;
      uint32_t ph = 1;
      for (int kp = 0; kp < (g.nk + 1) / 2; ++kp) {
        if (!f_wait(&sempty[s], ph, abrt)) break;
        unsigned char* p = sring + s * kScale;
        tc::mbar_expect_tx(&sfull[s], kScale);
#pragma unroll
        for (int h = 0; h < MH; ++h)
          tc::tma_load_2d(p + h * 2048, &maps.bs, kp * 16, i0 + h * 128, &sfull[s]);
        tc::tma_load_2d(p + kM * 16, &maps.as, kp * 16, j0, &sfull[s]);
        ++issued;
        if (++s == F_SRING) {
          s = 0;
          ph ^= 1;
        }
      }
      if (*abrt)
        for (int q = 0; q < F_SRING && q < issued; ++q)
          tc::mbar_wait(&sfull[q], uint32_t((issued - 1 - q) / F_SRING) & 1, &g_mx_matmul_err);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (tc::elect_one()) {
      const uint32_t id0 = idesc_mxf4(128, g.BN, 0), id2 = idesc_mxf4(128, g.BN, 2);
      int s = 0;
      uint32_t ph = 0;
      for (int kb = 0; kb < g.nk; ++kb) {
        if (!f_wait(&full[s], ph, abrt)) break;
        tc::tc_fence_after();
        unsigned char* p = smem + s * kStage;
        const uint64_t nd = tc::desc_sw128(p + kM * 128);
        const uint32_t sfm = tmem + sf0 + uint32_t(s * sf_cols), sfn = sfm + MH * 8;
#pragma unroll
        for (int h = 0; h < MH; ++h) {
          const uint64_t md = tc::desc_sw128(p + h * 16384);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            mma_mxf4(tmem + h * g.BN, tc::desc_advance(md, q * 32), tc::desc_advance(nd, q * 32),
                     (q & 1) ? id2 : id0, sfm + h * 8 + (q >> 1) * 4, sfn + (q >> 1) * npitch,
                     (kb > 0 || q > 0) ? 1u : 0u);
        }
        tc::mma_commit(&empty[s]);
        if (++s == g.stages) {
          s = 0;
          ph ^= 1;
        }
      }
      tc::mma_commit(&accf);
    }
    __syncwarp();
  } else {
    const int tid = threadIdx.x - 64;
    if (warp < 6) {
      const uint32_t quarter = tmem + (uint32_t((warp & 3) * 32) << 16) + sf0;
      int s = 0, sr = 0;
      uint32_t ph = 1, sph = 0;
      bool live = true;
      for (int kp = 0; live && kp < (g.nk + 1) / 2; ++kp) {
        if (!(live = f_wait(&sfull[sr], sph, abrt))) break;
        const uint4* src = reinterpret_cast<const uint4*>(sring + sr * kScale);
        uint4 wm[4 * MH], wn[8];
#pragma unroll
        for (int q = 0; q < 4 * MH; ++q) wm[q] = src[q * 32 + lane];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (q < ncols) wn[q] = src[kM + min(q * 32 + lane, g.BN - 1)];
        tc::fence_async_smem();  // the loads are done before a copy may overwrite what they read
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sempty[sr]);
        if (++sr == F_SRING) {
          sr = 0;
          sph ^= 1;
        }
        const int left = g.nb - kp * 16;  // blocks of the row from here on; padding bytes count as 0
        if (left < 16) {
          const uint32_t mk[4] = {
              left >= 4 ? ~0u : (1u << (8 * max(left, 0))) - 1,
              left >= 8 ? ~0u : left <= 4 ? 0u : (1u << (8 * (left - 4))) - 1,
              left >= 12 ? ~0u : left <= 8 ? 0u : (1u << (8 * (left - 8))) - 1,
              left <= 12 ? 0u : (1u << (8 * (left - 12))) - 1};
#pragma unroll
          for (int q = 0; q < 4 * MH; ++q) {
            wm[q].x &= mk[0]; wm[q].y &= mk[1]; wm[q].z &= mk[2]; wm[q].w &= mk[3];
          }
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            wn[q].x &= mk[0]; wn[q].y &= mk[1]; wn[q].z &= mk[2]; wn[q].w &= mk[3];
          }
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          if (kp * 2 + b >= g.nk) break;
          if (!(live = f_wait(&empty[s], ph, abrt))) break;
          tc::tc_fence_after();
          const uint32_t dst = quarter + uint32_t(s * sf_cols);
#pragma unroll
          for (int q = 0; q < 4 * MH; ++q) {
            const uint32_t c = dst + (q >> 2) * 8 + (q & 3);
            tc::tmem_st1(c, b ? wm[q].z : wm[q].x);
            tc::tmem_st1(c + 4, b ? wm[q].w : wm[q].y);
          }
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (q < ncols) {
              tc::tmem_st1(dst + MH * 8 + q, b ? wn[q].z : wn[q].x);
              tc::tmem_st1(dst + MH * 8 + npitch + q, b ? wn[q].w : wn[q].y);
            }
          tc::tmem_st_wait();
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&full[s]);
          if (++s == g.stages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
    }
    __syncwarp();
    const bool ok = tc::mbar_wait(&accf, 0, &g_mx_matmul_err) && !*abrt;
    __nv_bfloat16* stg = reinterpret_cast<__nv_bfloat16*>(smem);
    if (ok) {
      tc::tc_fence_after();
      const int grp = warp >= 6 ? 1 : 0;
      const int L = ((warp & 3) << 5) | lane;
      const int R = (MH == 2 ? grp * 128 : 0) + L;
      const int i = i0 + R;
      const uint32_t tb =
          tmem + (uint32_t((warp & 3) * 32) << 16) + (MH == 2 ? uint32_t(grp * g.BN) : 0u);
      const int c_lo = MH == 2 ? 0 : (grp ? (ncols + 1) / 2 : 0);
      const int c_hi = MH == 2 ? ncols : (grp ? ncols : (ncols + 1) / 2);
      const TO* add = static_cast<const TO*>(g.add);
      TO* C = static_cast<TO*>(g.C);
#pragma unroll 1
      for (int c = c_lo; c < c_hi; ++c) {
        const int c0 = c * 32;
        float v[32];
        tc::tmem_ld32(tb + c0, v);
        const int jn = min(32, min(g.BN - c0, g.N - j0 - c0));
        if (kRows) {
          const int64_t at = int64_t(i) * g.N + j0 + c0;
          if (kOut == kTiles && add && i < g.M) {
            if (jn == 32) {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const uint4 w = *reinterpret_cast<const uint4*>(add + at + q * 8);
                v[8 * q] += bf_lo(w.x); v[8 * q + 1] += bf_hi(w.x);
                v[8 * q + 2] += bf_lo(w.y); v[8 * q + 3] += bf_hi(w.y);
                v[8 * q + 4] += bf_lo(w.z); v[8 * q + 5] += bf_hi(w.z);
                v[8 * q + 6] += bf_lo(w.w); v[8 * q + 7] += bf_hi(w.w);
              }
            } else {
#pragma unroll
              for (int q = 0; q < 32; ++q)
                if (q < jn) v[q] += VT<TO>::f(add[at + q]);
            }
          }
          if (kOut == kTiles) {
            // 64-column tiles of 128 rows in the 128-byte swizzle
            unsigned char* row = smem + ((R >> 7) * (g.BN >> 6) + (c >> 1)) * 16384 + (R & 127) * 128;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t w[4];
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[8 * q + 2 * z], v[8 * q + 2 * z + 1]);
                w[z] = *reinterpret_cast<const uint32_t*>(&h);
              }
              *reinterpret_cast<uint4*>(row + ((((c & 1) * 4 + q) ^ (R & 7)) << 4)) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
            // a lane has a row: through shared memory, fp32, an odd number of words per row, so that rows can be
            // stored (and add read) along their length (4096 × 7298 × 9440: 201 µs, 481 with a row per lane)
            float* row = reinterpret_cast<float*>(smem) + R * (g.BN + 1) + c0;
#pragma unroll
            for (int q = 0; q < 32; ++q)
              if (c0 + q < g.BN) row[q] = v[q];
          }
        } else {
          const int64_t at = int64_t(j0 + c0) * g.M + i;
          if (add && i < g.M) {
#pragma unroll
            for (int q = 0; q < 32; ++q)
              if (q < jn) v[q] += VT<TO>::f(add[at + int64_t(q) * g.M]);
          }
          if (g.cstore) {
#pragma unroll
            for (int q = 0; q < 32; ++q)
              if (c0 + q < g.BN) stg[(c0 + q) * kM + R] = __float2bfloat16_rn(v[q]);
          } else if (i < g.M) {
#pragma unroll
            for (int q = 0; q < 32; ++q)
              if (q < jn) C[at + int64_t(q) * g.M] = VT<TO>::from_f(v[q]);
          }
        }
      }
    } else {
      *abrt = 1;
    }
    if (kOut == kEach) {
      asm volatile("barrier.sync 1, 256;" ::: "memory");  // the eight epilogue warps, always
      const int cols = min(g.BN, g.N - j0);
      const TO* add = static_cast<const TO*>(g.add);
      TO* C = static_cast<TO*>(g.C);
      if (ok && !*abrt)
        for (int r = warp - 2; r < kM && i0 + r < g.M; r += 8) {
          const float* row = reinterpret_cast<const float*>(smem) + r * (g.BN + 1);
          const int64_t at = int64_t(i0 + r) * g.N + j0;
#pragma unroll 4
          for (int q = lane; q < cols; q += 32)
            C[at + q] = VT<TO>::from_f(add ? row[q] + VT<TO>::f(add[at + q]) : row[q]);
        }
    }
    if (kOut == kTiles || (kOut == kCols && g.cstore)) {
      tc::fence_async_smem();
      asm volatile("barrier.sync 1, 256;" ::: "memory");  // the eight epilogue warps, always
      if (tid == 0 && ok && !*abrt) {
        if (kRows) {
          for (int h = 0; h < MH; ++h)
            for (int q = 0; q < g.BN / 64; ++q)
              if (i0 + h * 128 < g.M && j0 + q * 64 < g.N)
                tc::tma_store_2d(&maps.c, smem + (h * (g.BN >> 6) + q) * 16384, j0 + q * 64, i0 + h * 128);
        } else {
          tc::tma_store_2d(&maps.c, stg, i0, j0);
        }
        tc::bulk_commit();
        tc::bulk_wait_read_all();
      }
    }
  }
  tc::tc_fence_before();
  tc::cta_sync();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <typename TO, int MH, MmOut kOut>
hsl_status launch_mm(const MmMaps& maps, const MmArgs& g, cudaStream_t s) {
  void (*fn)(const MmMaps, const MmArgs) = k_mx_matmul<TO, MH, kOut>;
  const int stage = (MH * 128 + g.BN) * 128, scale = (MH * 128 + g.BN) * 16;
  const int tile = kOut == kEach ? MH * 128 * (g.BN + 1) * 4 : MH * 128 * g.BN * 2;  // the epilogue's
  const int bytes = std::max(g.stages * stage + F_SRING * scale, tile) + 1024;
  if (cudaError_t e = allow_dyn_smem(reinterpret_cast<const void*>(fn), bytes))
    return cuda_fail(e, "4-bit product smem attribute");
  const int64_t tiles = int64_t((g.M + 128 * MH - 1) / (128 * MH)) * ((g.N + g.BN - 1) / g.BN);
  note_launch();
  fn<<<unsigned(tiles), F_THREADS, size_t(bytes), s>>>(maps, g);
  return cuda_fail(cudaGetLastError(), "4-bit product launch");
}

}  // namespace

bool mx_matmul_supported() { return tmap_available(); }

hsl_status mx_matmul_run(const MxOperand& A, int64_t T, const MxOperand& B, int64_t m, int64_t n,
                         const void* add, void* Y, hsl_dtype dtype, cudaStream_t s) {
  const bool rows = T >= 256;
  const MxOperand &ms = rows ? A : B, &ns = rows ? B : A;
  const int64_t M = rows ? T : m, N = rows ? m : T;
  const bool aligned = dtype == HSL_BF16 && m % 8 == 0 && reinterpret_cast<uintptr_t>(Y) % 16 == 0 &&
                       (!add || reinterpret_cast<uintptr_t>(add) % 16 == 0);
  // Two accumulators of up to 192 columns where that still gives every SM a tile, else one of up
  // to 256.  Rows of C are stored in tiles of 64 columns.
  int mh = 2;
  int64_t ntn = (N + 191) / 192;
  if ((M + 255) / 256 * ntn < 148) {
    mh = 1;
    ntn = (N + 255) / 256;
    // with few tiles, narrower ones for more SMs
    if (rows) ntn = std::min((N + 63) / 64, std::max<int64_t>(ntn, 148 / ((M + 127) / 128)));
  }
  MmArgs g = {};
  g.M = int(M);
  g.N = int(N);
  g.nb = int(mx::blocks(n));
  g.nk = (g.nb + 7) / 8;
  g.BN = int(round_up((N + ntn - 1) / ntn, rows ? 64 : 16));
  const int srows = mh * 128 + g.BN;
  const int sf_cols = mh * 8 + 2 * ((g.BN + 127) / 128 * 4);
  g.stages = std::min(F_MAX_STAGES, (F_SMEM_BUDGET - F_SRING * srows * 16) / (srows * 128));
  // the last column read of an accumulator may lie up to 16 past BN: inside the scales' columns
  g.stages = std::min(g.stages, (512 - mh * g.BN) / sf_cols);
  g.add = add;
  g.C = Y;
  g.cstore = aligned ? 1 : 0;
  MmMaps maps;
  memset(&maps, 0, sizeof(maps));
  const auto U8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const auto SW = CU_TENSOR_MAP_SWIZZLE_128B;
  const auto NO = CU_TENSOR_MAP_SWIZZLE_NONE;
  bool ok = make_tmap_2d(&maps.b, U8, 1, ms.p, M, ms.pitch, ms.pitch, 128, 128, SW) &&
            make_tmap_2d(&maps.a, U8, 1, ns.p, N, ns.pitch, ns.pitch, 128, g.BN, SW) &&
            make_tmap_2d(&maps.bs, U8, 1, ms.scales, M, ms.spitch, ms.spitch, 16, 128, NO) &&
            make_tmap_2d(&maps.as, U8, 1, ns.scales, N, ns.spitch, ns.spitch, 16, g.BN, NO);
  if (ok && g.cstore)
    ok = rows ? make_tmap_2d(&maps.c, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, Y, T, m, m, 64, 128, SW)
              : make_tmap_2d(&maps.c, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, Y, T, m, m, 128 * mh, g.BN, NO);
  if (!ok) {
    set_message("tensor map encoding failed");
    return HSL_ERR_CUDA;
  }
  using bf = __nv_bfloat16;
  if (!rows) {
    if (dtype == HSL_F32) return mh == 2 ? launch_mm<float, 2, kCols>(maps, g, s) : launch_mm<float, 1, kCols>(maps, g, s);
    return mh == 2 ? launch_mm<bf, 2, kCols>(maps, g, s) : launch_mm<bf, 1, kCols>(maps, g, s);
  }
  if (dtype == HSL_F32) return mh == 2 ? launch_mm<float, 2, kEach>(maps, g, s) : launch_mm<float, 1, kEach>(maps, g, s);
  if (aligned) return mh == 2 ? launch_mm<bf, 2, kTiles>(maps, g, s) : launch_mm<bf, 1, kTiles>(maps, g, s);
  return mh == 2 ? launch_mm<bf, 2, kEach>(maps, g, s) : launch_mm<bf, 1, kEach>(maps, g, s);
}

cudaError_t mx_matmul_error_word(uint32_t** p) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_mx_matmul_err);
}

}  // namespace hsl
