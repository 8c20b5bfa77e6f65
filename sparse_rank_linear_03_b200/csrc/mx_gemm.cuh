// Products on the tensor cores with one factor held in microscaled blocks.
//
//   C = A · (B0 + B1 + B2)ᵀ (+ add),   A [M][K], B [N][K], fp32 sums in TMEM
//
// A is the large factor: a 4-bit weight matrix, an 8-bit checkpoint, or a bf16
// matrix, each either stored as [M][K] or used transposed from [K][M].  B is a bf16
// matrix (tokens, factors), stored as [N][K] or [K][N], or an fp32 matrix held as three bf16
// parts.  The same tile serves the forward product (M = features,
// N = tokens), its input gradient (the same matrix, transposed) and the skinny
// products of the factors' gradients (N = r).
//
// Blocks are widened to bf16 on their way into shared memory.  That is exact: an
// e2m1 value has 2 significant bits and an int8 value 7, the block's scale is a
// power of two, and bf16 has 8 significant bits and fp32's exponents (values
// down to 2^−133 are bf16 subnormals).  So the products differ from the definition
// by the rounding of the fp32 sums only.
//
// Both storage orders use the same shared-memory tile: rows of 64 values (128
// bytes) in the 128-byte swizzle.  For [M][K] a tile row is a row of A and the 64
// values run along K; for [K][M] a tile row is a k and the 64 values run along M,
// which the MMA reads as an M-major operand.  Widening is the same either way: a
// thread turns the one or two blocks of its tile row into 128 bytes.
//
//   warp 0 lane 0   TMA of the B tile(s), and of A when it is bf16
//   warp 1 lane 0   tcgen05.mma, M = 128 per accumulator, N up to 256, K = 16
//   warp 18 lane 0  TMA of the code tiles, into a ring of their own
//   warps 2-17      widen A's blocks, two groups of eight taking turns at the K-blocks;
//                   then the epilogue: tcgen05.ld, add, round, store
//
// MH = 2 gives the CTA two 128-row accumulators that share every B tile.  Bound by shared memory: a K-block
// of 256 × 208 × 64 takes the MMAs 832 cycles, 1090 as measured, in which widened A (32 KB)
// and B (26 KB) are written once and B is read once per accumulator.  11008 × 4096 at 2048
// tokens: 144 µs, 1.28 PFLOP/s; the input gradient of 4096 × 11008 137 µs (172 and 162 µs in seconds
// of calls, where the power limit slows the clock).  Every wait is bounded.
#pragma once

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

__device__ uint32_t g_mx_gemm_err;

constexpr int G_BK = 64;
constexpr int G_THREADS = 608;   // 19 warps: copies, MMA, 2 × 8 widening (all 16 in the epilogue), code copies
constexpr int G_MAX_STAGES = 8;
constexpr int G_SMEM_BUDGET = 224 * 1024;  // stages and code tiles; barriers and alignment take 2 KB more

enum AKind { A_BF16_K, A_BF16_M, A_E2M1_K, A_E2M1_M, A_INT8_K, A_INT8_M };
enum OutKind { OUT_T, OUT_R, OUT_T_PART };  // C[n][m]; C[m][n], or its fp32 partials (g.part); partials of C[n][m]

constexpr bool a_is_blocks(int a) { return a >= A_E2M1_K; }
constexpr bool a_is_mmajor(int a) { return a == A_BF16_M || a == A_E2M1_M || a == A_INT8_M; }
constexpr bool a_is_int8(int a) { return a == A_INT8_K || a == A_INT8_M; }

struct GemmMaps {
  CUtensorMap a;   // bf16 A: box {64, 128} (K-major) or {64, 64}
  CUtensorMap b[3];  // B, or its parts: box {64, BN} (K-major) or {64, 64}
  CUtensorMap c;   // OUT_T: box {128·MH, BN}
  CUtensorMap add; // like c
  CUtensorMap q;   // codes: box {CodeTile::kInner bytes, CodeTile::kRows}
  CUtensorMap qs;  // scales of [K][M] blocks: box {16 bytes, 64}
};
struct GemmArgs {
  const uint8_t* scales;  // [M][K] blocks: read 16 at a time per row
  int64_t spitch;
  int arows, nb;          // stored rows of A, blocks per row
  int M, N, nk;      // nk: K-blocks of 64
  int BN, stages, splits;
  int codes;         // code tiles in flight
  int cstore;        // OUT_T: tiled store possible
  int addt;          // OUT_T: add comes as a tile as well
  const __nv_bfloat16* add;
  __nv_bfloat16* C;
  float* part;       // [splits][N][M] or [splits][M][N]; OUT_R: nullptr where C is written
};

__device__ __forceinline__ bool g_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (tc::mbar_try(bar, parity)) return true;
  if (*abort_flag) return false;
  if (tc::mbar_wait(bar, parity, &g_mx_gemm_err)) return true;
  *abort_flag = 1;
  return false;
}

// M- or N-major operand in the 128-byte swizzle: 64 values along the row, 8 k per
// 1024-byte atom; the next 64 values of the row dimension 8192 bytes on.
__device__ __forceinline__ uint64_t desc_mn_sw128(const void* tile) {
  const uint64_t addr = tc::smem_u32(tile);
  uint64_t d = 0;
  d |= (addr >> 4) & 0x3FFFull;
  d |= uint64_t(8192 >> 4) << 16;  // leading byte offset: the next 64 values
  d |= uint64_t(1024 >> 4) << 32;  // stride byte offset: the next 8 k
  d |= uint64_t(1) << 46;
  d |= uint64_t(2) << 61;          // SWIZZLE_128B
  return d;
}

// ---- widening -----------------------------------------------------------------
using mx::e2m1_scale;
using mx::int8_scale;
using mx::widen_e2m1;
using mx::widen_int8;

// The code tile of a K-block in shared memory, as copied: kBoxes boxes of kRows rows of
// kInner bytes in the swizzle of that width, so that the threads of a warp, a row
// each, read their 16-byte chunks without bank conflicts.
template <int AK, int MH>
struct CodeTile {
  static constexpr int kElem = a_is_int8(AK) ? 2 : 1;  // half-bytes per value
  static constexpr int kRowBytes = (a_is_mmajor(AK) ? 128 * MH : 64) * kElem / 2;
  static constexpr int kRows = a_is_mmajor(AK) ? 64 : 128 * MH;
  static constexpr int kInner = kRowBytes < 128 ? kRowBytes : 128;
  static constexpr int kBoxes = kRowBytes / kInner;
  static constexpr int kCodes = kRows * kRowBytes;
  static constexpr int kScales = a_is_mmajor(AK) ? 64 * 16 : 0;
  static constexpr int kBytes = a_is_blocks(AK) ? kCodes + kScales : 0;
  // address of 16-byte chunk c of row r
  __device__ static __forceinline__ uint32_t at(int r, int c) {
    constexpr int per = kInner / 16;
    const int box = c / per, in = c % per;
    const int x = kInner == 128 ? r & 7 : kInner == 64 ? (r >> 1) & 3 : (r >> 2) & 1;
    return uint32_t(box * kRows * kInner + r * kInner + ((in ^ x) << 4));
  }
};

// The codes and scale of one block of 32.
template <bool kInt8>
struct Block {
  uint4 c[kInt8 ? 2 : 1];
  uint32_t e;
};
__device__ __forceinline__ void sts128(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
// Writes the block's 32 bf16 to chunks 4·half .. 4·half + 3 of a tile row.  `row` is the address of
// the row's chunk 0 as the swizzle places it: chunk c lies at row ^ (c << 4).
template <bool kInt8>
__device__ __forceinline__ void widen(const Block<kInt8>& b, uint32_t row, int half) {
  if (kInt8) {
    const uint32_t s = int8_scale(b.e);
    const uint32_t w[8] = {b.c[0].x, b.c[0].y, b.c[0].z, b.c[0].w,
                           b.c[kInt8 ? 1 : 0].x, b.c[kInt8 ? 1 : 0].y, b.c[kInt8 ? 1 : 0].z,
                           b.c[kInt8 ? 1 : 0].w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint2 lo = widen_int8(w[2 * q], s), hi = widen_int8(w[2 * q + 1], s);
      sts128(row ^ ((half * 4 + q) << 4), make_uint4(lo.x, lo.y, hi.x, hi.y));
    }
  } else {
    const uint32_t s = e2m1_scale(b.e);
    const uint32_t w[4] = {b.c[0].x, b.c[0].y, b.c[0].z, b.c[0].w};
#pragma unroll
    for (int q = 0; q < 4; ++q) sts128(row ^ ((half * 4 + q) << 4), widen_e2m1(w[q], s));
  }
}

template <int AK, bool BMN, int TERMS, int MH, int OUT>
__global__ void __launch_bounds__(G_THREADS, 1)
    k_mx_gemm(const __grid_constant__ GemmMaps maps, const __grid_constant__ GemmArgs g) {
  const int block = blockIdx.x;
#include "mx_gemm_tile.cuh"
}

// Σ over the splits' partials in split order; four values per thread where rows and pointers allow it
// (V = 4), else one.
template <int V>
__device__ __forceinline__ void sum_splits(const float* part, int splits, int64_t stride, int64_t at, float (&v)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = 0.f;
  for (int s0 = 0; s0 < splits; s0 += 8) {  // eight loads on their way at a time
    float4 q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (s0 + j >= splits) continue;
      const float* p = part + int64_t(s0 + j) * stride + at;
      if (V == 4) q[j] = __ldcs(reinterpret_cast<const float4*>(p));
      else q[j].x = __ldcs(p);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (s0 + j >= splits) continue;
      v[0] += q[j].x;
      if (V == 4) {
        v[1 % V] += q[j].y; v[2 % V] += q[j].z; v[3 % V] += q[j].w;
      }
    }
  }
}
template <int V>
__device__ __forceinline__ void store_bf(__nv_bfloat16* p, const float (&v)[V]) {
  if (V == 4) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1 % V]), b = __floats2bfloat162_rn(v[2 % V], v[3 % V]);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    p[0] = __float2bfloat16_rn(v[0]);
  }
}
// Rows of n bf16 to rows of `pitch` (a multiple of 8, so that a tile copy can read them): a thread per 16-byte
// piece of the result, made from the two aligned pieces around its source where these lie inside src
// (4089 rows of 9441: 161 µs value by value).  `per`: CTAs per row.
__global__ void __launch_bounds__(256)
    k_mx_pad_rows(const uint16_t* __restrict__ src, const uint16_t* end, unsigned per, int n, int pitch,
                  uint16_t* __restrict__ dst) {
  pdl_trigger();
  const int64_t row = blockIdx.x / per;
  const int c = int((blockIdx.x % per) * blockDim.x + threadIdx.x) * 8;
  if (c >= pitch) return;
  const uint16_t* p = src + row * n + c;
  const uint32_t sh = uint32_t(reinterpret_cast<uintptr_t>(p) & 15);
  const char* low = reinterpret_cast<const char*>(p) - sh;
  uint32_t w[8] = {};
  if (c + 8 <= n && low >= reinterpret_cast<const char*>(src) &&
      low + (sh ? 32 : 16) <= reinterpret_cast<const char*>(end)) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(low));
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    if (sh) {
      const uint4 b = __ldg(reinterpret_cast<const uint4*>(low) + 1);
      w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    }
    mx::shift_bytes<4>(w, sh);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j < n) w[j >> 1] |= uint32_t(__ldg(p + j)) << ((j & 1) * 16);
  }
  *reinterpret_cast<uint4*>(dst + row * pitch + c) = make_uint4(w[0], w[1], w[2], w[3]);
}

unsigned blocks_of(int64_t count) { return unsigned((count + 255) / 256); }

// ---- host ---------------------------------------------------------------------
struct GemmShape {
  int BN, MH, splits, stages, codes;
};

int code_bytes(int ak, int mh) {
  if (!a_is_blocks(ak)) return 0;
  return 128 * mh * (a_is_int8(ak) ? 64 : 32) + (a_is_mmajor(ak) ? 1024 : 0);
}
int stage_bytes(bool bmn, int terms, int mh, int bn) {
  return mh * 16384 + terms * (bmn ? (bn + 63) / 64 * 8192 : bn * 128);
}

// Stages and code tiles of a tile shape.  Code tiles are small and come from farther away than
// anything else: four of them in flight at least, then as many stages as fit (two at
// least: three terms leave room for them only with narrow tiles), then more code
// tiles, an even number.
void fit_rings(GemmShape* s, int ak, bool bmn, int terms) {
  const int code = code_bytes(ak, s->MH), stage = stage_bytes(bmn, terms, s->MH, s->BN);
  s->codes = code ? 4 : 0;
  s->stages = std::min(G_MAX_STAGES, (G_SMEM_BUDGET - s->codes * code) / stage);
  if (code) s->codes = std::min(G_MAX_STAGES, (G_SMEM_BUDGET - s->stages * stage) / code) & ~1;
}
bool rings_fit(int ak, bool bmn, int terms, int mh, int bn, int stages) {
  return stages * stage_bytes(bmn, terms, mh, bn) + (a_is_blocks(ak) ? 4 : 0) * code_bytes(ak, mh) <=
         G_SMEM_BUDGET;
}
// Cycles of a K-block as measured: widening 256 rows 1040, 128 rows 720 (its chain of waits does not
// shrink with the rows); copies and MMAs 5 per column and accumulator pair, 3 for one; with few
// columns a bf16 A's own bytes, 64 per cycle (2048 tokens, 11008 × 4096, rank 64).
int64_t kblock_cycles(int ak, int terms, int mh, int bn) {
  return std::max<int64_t>(a_is_blocks(ak) ? (mh == 2 ? 1040 : 720) : (mh * 16384 + terms * bn * 128) / 64,
                           int64_t(terms) * bn * (mh == 2 ? 5 : 3));
}

// Tile and split of an M × N × K product.
GemmShape shape_of(int ak, int64_t M, int64_t N, int64_t K, bool bmn, int terms, bool may_split) {
  GemmShape s;
  // With at least a tile per SM, 256-row tiles whose width makes the last round of
  // CTAs as full as it can be: time goes as rounds × columns (a K-block of fewer than
  // 160 columns costs the widening, not the MMAs).  2048 tokens × 11008 rows: 208
  // columns (2.9 rounds) against 256 (2.3 rounds, the third mostly idle).
  int64_t ntn = (N + 255) / 256;
  const int64_t t2 = (M + 255) / 256, t1 = (M + 127) / 128, nk = (K + 63) / 64;
  s.splits = 1;
  if (t2 * ntn >= 148) {
    s.MH = 2;
    int64_t best = INT64_MAX, at = ntn;
    for (int64_t c = ntn; c <= 2 * ntn; ++c) {
      const int64_t bn = round_up((N + c - 1) / c, 16);
      if (!rings_fit(ak, bmn, terms, 2, int(bn), 2)) continue;  // (128 columns always do)
      const int64_t cost = (t2 * c + 147) / 148 * std::max<int64_t>(bn, 160) *
                           (rings_fit(ak, bmn, terms, 2, int(bn), 3) ? 4 : 5);
      if (cost < best) {
        best = cost;
        at = c;
      }
    }
    ntn = at;
  }
  s.BN = int(round_up((N + ntn - 1) / ntn, 16));
  if (t2 * ntn < 148) {
    // Fewer tiles than SMs: K is split where the caller has room for partial sums and where that saves
    // more than the launch that adds them up, about 6000 cycles, and their way through HBM
    // and back, at about 3500 bytes per cycle.
    auto cost = [&](int mh, int64_t* splits) {
      const int64_t tiles = (mh == 2 ? t2 : t1) * ntn;
      const int64_t per = kblock_cycles(ak, terms, mh, s.BN), whole = nk * per * ((tiles + 147) / 148);
      *splits = may_split ? std::max<int64_t>(1, std::min<int64_t>(148 / tiles, nk / 4)) : 1;
      const int64_t cut = (nk + *splits - 1) / *splits * per + 6000 + *splits * M * N * 8 / 3500;
      if (*splits == 1 || whole <= cut) *splits = 1;
      return *splits == 1 ? whole : cut;
    };
    int64_t s1 = 1, s2 = 1;
    const int64_t c1 = cost(1, &s1), c2 = cost(2, &s2);
    s.MH = c2 < c1 && rings_fit(ak, bmn, terms, 2, s.BN, 2) ? 2 : 1;
    s.splits = int(s.MH == 2 ? s2 : s1);
  }
  fit_rings(&s, ak, bmn, terms);
  return s;
}

int tile_smem(int ak, bool bmn, int terms, int mh, bool staged, const GemmArgs& g) {
  int bytes = g.stages * stage_bytes(bmn, terms, mh, g.BN) + g.codes * code_bytes(ak, mh);
  if (staged) bytes = std::max(bytes, mh * 128 * g.BN * 2);  // the epilogue's tile
  return bytes + 1024;
}
int64_t tile_count(int mh, const GemmArgs& g) {
  return int64_t((g.M + 128 * mh - 1) / (128 * mh)) * ((g.N + g.BN - 1) / g.BN) * g.splits;
}

template <int AK, bool BMN, int TERMS, int MH, int OUT>
hsl_status launch_gemm(const GemmMaps& maps, const GemmArgs& g, bool chained, cudaStream_t s) {
  void (*fn)(const GemmMaps, const GemmArgs) = k_mx_gemm<AK, BMN, TERMS, MH, OUT>;
  const int bytes = tile_smem(AK, BMN, TERMS, MH, OUT == OUT_T, g);
  if (cudaError_t e = allow_dyn_smem(reinterpret_cast<const void*>(fn), bytes))
    return cuda_fail(e, "block product smem attribute");
  note_launch();
  return cuda_fail(launch_chained(fn, chained, dim3(unsigned(tile_count(MH, g))), G_THREADS, size_t(bytes), s, maps, g),
                   "block product launch");
}
template <int AK, bool BMN, int TERMS, int OUT>
hsl_status launch_gemm(int mh, const GemmMaps& maps, const GemmArgs& g, bool chained, cudaStream_t s) {
  return mh == 2 ? launch_gemm<AK, BMN, TERMS, 2, OUT>(maps, g, chained, s)
                 : launch_gemm<AK, BMN, TERMS, 1, OUT>(maps, g, chained, s);
}

const auto kBF = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
const auto kSW = CU_TENSOR_MAP_SWIZZLE_128B;

// The tiled store of C [T][M] and, where add allows it, the tiled load of add.
bool out_maps(GemmMaps* maps, GemmArgs* g, int64_t T, int64_t M, int mh) {
  g->cstore = (M % 8 == 0 && reinterpret_cast<uintptr_t>(g->C) % 16 == 0) ? 1 : 0;
  g->addt = (g->cstore && g->add && reinterpret_cast<uintptr_t>(g->add) % 16 == 0) ? 1 : 0;
  return (!g->cstore || make_tmap_2d(&maps->c, kBF, 2, g->C, T, M, M, 128 * mh, g->BN, CU_TENSOR_MAP_SWIZZLE_NONE)) &&
         (!g->addt || make_tmap_2d(&maps->add, kBF, 2, g->add, T, M, M, 128 * mh, g->BN, CU_TENSOR_MAP_SWIZZLE_NONE));
}

// The tensor maps of a factor in blocks (stored rows × cols).
bool block_maps(GemmMaps* maps, int ak, int mh, const MxOperand& o, int64_t rows) {
  const auto U8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const int row_bytes = (a_is_mmajor(ak) ? 128 * mh : 64) / (a_is_int8(ak) ? 1 : 2);
  const int inner = std::min(row_bytes, 128);
  const auto sw = inner == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                  : inner == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                : CU_TENSOR_MAP_SWIZZLE_32B;
  return make_tmap_2d(&maps->q, U8, 1, o.p, rows, o.pitch, o.pitch, inner, a_is_mmajor(ak) ? 64 : 128 * mh, sw) &&
         (!a_is_mmajor(ak) || make_tmap_2d(&maps->qs, U8, 1, o.scales, rows, o.spitch, o.spitch, 16, 64,
                                           CU_TENSOR_MAP_SWIZZLE_NONE));
}

hsl_status map_failed() {
  set_message("tensor map encoding failed");
  return HSL_ERR_CUDA;
}

int64_t up16(int64_t b) { return (b + 255) / 256 * 256; }

hsl_status pad_rows(const void* src, int64_t rows, int64_t n, int64_t pitch, void* dst, cudaStream_t s) {
  note_launch();
  const int64_t pieces = pitch / 8;
  const unsigned threads = unsigned(std::min<int64_t>(256, round_up(pieces, 32)));
  const unsigned per = unsigned((pieces + threads - 1) / threads);
  const uint16_t* x = static_cast<const uint16_t*>(src);
  k_mx_pad_rows<<<unsigned(rows * per), threads, 0, s>>>(x, x + rows * n, per, int(n), int(pitch),
                                                         static_cast<uint16_t*>(dst));
  return cuda_fail(cudaGetLastError(), "row padding launch");
}

}  // namespace
}  // namespace hsl
