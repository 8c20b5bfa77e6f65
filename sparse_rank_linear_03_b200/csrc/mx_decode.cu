// Y = X Dᵀ (+ add) for a few tokens, D in e2m1 blocks: one pass over the codes.
//
// bf16 (k_mx_decode): bound by the bytes of D, 17 per 32 values.  At 6.5 TB/s that is
// 44 values per SM and cycle, so a value may cost 2.9 instructions, of which 1.45 on the
// integer pipe (64 lanes per cycle).  Byte permutes that build bf16 values take 2.8
// integer instructions per value (28672 × 8192, one token: 60 µs).  What this kernel
// does takes about half an integer instruction:
//
//   cvt turns two codes into two fp16 values, which mma.sync (m16n8k16, fp32 sums)
//   multiplies with the tokens, 16 rows of D × 8 columns.  Each block has its own
//   MMAs, and its scale multiplies their 4 sums per lane (fp32 FMA).
//
//   The tokens become fp16 without losing a bit: a token's values are sorted into
//   windows of 32 binades below its largest, and each window, scaled by its own
//   power of two, is a column of its own (8 significant bits over 32 binades end at
//   2^−23, fp16 reaches 2^−24).  Activations fit one window nearly always; there is room
//   for two columns per token up to 4 tokens (and not too long ones), and what does not fit
//   takes another pass over D.  From two tokens on a kernel of its own makes the columns (k_mx_tokens),
//   while the main kernel's first copies of D are already under way.  At the end each column is scaled back.  Infinities
//   and NaN go to the first window as they are.  Block scales enter as 2^(e − 110): a column's smallest product,
//   2^−25, then keeps its bits at every e.  At the other end sums of blocks with e of about 200 and more
//   (weights of 2^70) may overflow although the result, for small tokens, does not.  That always shows, as an
//   infinity or a NaN, and such outputs are summed again at the end, as they are, by the warp that issued the
//   copies (dc_again; if it is every output of 28672 × 8192, 3 ms at one token).  A look at each unit's scales,
//   with a second loop for such units, took 33 µs for ordinary weights, where this takes 29; the same repair as
//   a call from the sixteen warps 31.
//
//   One CTA per SM keeps the columns in shared memory and walks over tiles of 16 rows.
//   Codes and scales come in tiled copies, one of each per stage, a ring of stages ahead of
//   the arithmetic: at 1.5 to 2 µs of latency 65 to 90 KB per SM have to be in flight.
//   Sixteen warps divide a stage in units of 256 values of K.  Lane (g, t) takes word t
//   (8 codes) of each block of rows g and g + 8, and the same 8 values of column g:
//   the order of the terms of a dot product is free.  The warps' sums are added
//   up in warp order, several row tiles at a time.  Where the columns do not fit, K is taken in slices; the rows'
//   sums stay in shared memory from slice to slice and pass to pass.
//
//   28672 × 8192, calls one behind the other: 29 µs at one token (4.3 TB/s, launch and tail included), 33 at two,
//   41 at eight.
//
// f32 (k_mx_decode_f32): a lane per row, tokens broadcast from shared memory, fp32 FMA, K in ranges.
#include <cuda.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cstring>

#include "common.cuh"
#include "internal.h"
#include "mx.cuh"
#include "mx_ops.h"
#include "tc.cuh"

namespace hsl {
namespace {

constexpr int DC_WARPS = 16;
constexpr int DC_UNIT = 256;                 // values of K per warp and step
constexpr int DC_SMEM_MAX = 224 * 1024;

// Eight codes (one word) → four fp16 pairs.
__device__ __forceinline__ void widen_word(uint32_t w, uint32_t (&v)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
      : "r"(w));
}
// Four scale bytes (one word) → 2^(e − 110) in fp32 (infinite from e = 238 on): the conversion gives 2^(e − 127)
// as bf16 pairs (2^−127 a subnormal, 255 a NaN), which widen by shifts.
__device__ __forceinline__ void widen_scales(uint32_t w, float* s) {
  uint32_t p[2];
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.bf16x2.ue8m0x2 %0, a;\n\t"
      "cvt.rn.bf16x2.ue8m0x2 %1, b;\n\t}"
      : "=r"(p[0]), "=r"(p[1])
      : "r"(w));
  constexpr float k = 131072.0f;
  s[0] = bf_lo(p[0]) * k;
  s[1] = bf_hi(p[0]) * k;
  s[2] = bf_lo(p[1]) * k;
  s[3] = bf_hi(p[1]) * k;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 2^k, −126 <= k <= 127.
__device__ __forceinline__ float pow2(int k) { return __uint_as_float(uint32_t(127 + k) << 23); }

// One output's sum by a warp, straight from the token, whose values are finite: every product but those with 0
// takes its block's power of two in two factors, so that only what is past fp32 itself overflows.  (Inlined: a
// call costs the kernel 2 µs.)
__device__ __forceinline__ float dc_again(const uint8_t* codes, const uint8_t* scales, const __nv_bfloat16* x, int n,
                                       int nb) {
  float v = 0.f;
  for (int b = threadIdx.x & 31; b < nb; b += 32) {
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(codes) + b);
    const int e = __ldg(scales + b), s = e - 127;
    const float f0 = pow2(s >> 1), f1 = pow2((s + 1) >> 1);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    for (int j = 0; j < min(32, n - b * 32); ++j) {
      const uint32_t d = (w[j >> 3] >> ((j & 7) * 4)) & 15u;
      if (d & 7u) v = fmaf(__bfloat162float(x[b * 32 + j]) * f0, mx::e2m1_f32(d) * f1, v);
    }
    if (e == 255) v = __uint_as_float(0x7FC00000u);
  }
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

struct DcMaps {
  CUtensorMap c3;  // codes as [unit][row][128 bytes]: box {128, 16·tps, su}
  CUtensorMap c2;  // codes as [row][bytes]: box {128, 16·tps} (stages with the row's ragged end)
  CUtensorMap s;   // scales: box {128, 16·tps}
};
struct DcArgs {
  const int2* tokens;   // per token: largest exponent field (+ kNotFinite), windows
  const uint4* columns;  // [window][token][cpieces] pieces of eight fp16
  const uint8_t *codes, *scales;  // for dc_again
  int64_t pitch, spitch;
  const __nv_bfloat16* X;  // kSelf, dc_again
  const __nv_bfloat16* add;
  __nv_bfloat16* Y;
  int m, n, nb, T;
  int vec;     // kSelf: rows of X start on 16 bytes
  int wcols;   // columns per token, at most
  int cpieces;  // pieces per column in global memory
  int slice;   // units of K whose columns are in shared memory at a time
  int su;      // units per stage and row tile
  int tps;     // row tiles per stage
  int stages;
  int ysum, ring;  // offsets in shared memory: the kept sums, the stages
};

// A stage: su units of codes, each `rows` rows of 128 bytes, then 128 scale bytes per row
// (two units in 16 bytes), all in the 128-byte swizzle: 16-byte chunk c of row r lies at
// chunk c ^ (r & 7), so that the eight rows of a warp's access lie in different banks.
__host__ __device__ constexpr int dc_stage_bytes(int su, int rows) { return (su + 1) * rows * 128; }

// A column's 16-byte pieces (eight values each) in shared memory: 64 bytes between columns, so
// that the eight lanes of an access (two columns × four neighbouring pieces) meet
// eight different bank groups.
__host__ __device__ constexpr int dc_col_pitch(int slice) { return slice * (DC_UNIT / 8) + 4; }

// Eight values of a token, zeros past n.
__device__ __forceinline__ uint4 load_piece(const __nv_bfloat16* x, int col, int n, int vec) {
  uint4 v = make_uint4(0, 0, 0, 0);
  const __nv_bfloat16* p = x + col;
  if (vec && col + 8 <= n) {
    v = __ldg(reinterpret_cast<const uint4*>(p));
  } else {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (col + j < n)
        w[j >> 1] |= uint32_t(__ldg(reinterpret_cast<const uint16_t*>(p) + j)) << ((j & 1) * 16);
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return v;
}
// Largest and smallest exponent field of a piece's finite values that are not zero (-1 and 255 if
// there is none), two values at a time.  Whether there is an infinity or a NaN.
__device__ __forceinline__ bool exponents(const uint4& v, int& hi, int& lo) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t h = 0, l = 0xFFFFFFFFu;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t m = w[j] & 0x7FFF7FFFu;
    h = __vmaxu2(h, m);
    l = __vminu2(l, ((m | 0x80008000u) - 0x00010001u) ^ 0x80008000u);  // m − 1; a zero is the largest
  }
  const uint32_t top = max(h >> 16, h & 0xFFFFu), low = min(l >> 16, l & 0xFFFFu);
  hi = -1;
  lo = 255;
  if (top >= 0x7F80u) {  // an infinity or a NaN among them
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t bits = (w[j >> 1] >> ((j & 1) * 16)) & 0x7FFFu;
      if (bits != 0 && bits < 0x7F80u) {
        hi = max(hi, int(bits >> 7));
        lo = min(lo, int(bits >> 7));
      }
    }
  } else if (top != 0) {
    hi = int(top >> 7);
    lo = int((low + 1) >> 7);
  }
  return top >= 0x7F80u;
}
// The values of a piece that belong to window `win` of a token whose largest exponent field is
// `top`, scaled by 2^(142 − top + 32 win) to fp16; zeros elsewhere.
// (`all`: there is one window, with every value in it).
__device__ __forceinline__ uint4 window_piece(const uint4& v, int top, int win, bool all) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const int k = 142 - top + 32 * win;  // in two factors: 2^k alone may not be an fp32 value
  const float f0 = __uint_as_float(uint32_t(127 + k / 2) << 23);
  const float f1 = __uint_as_float(uint32_t(127 + k - k / 2) << 23);
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float x[2] = {bf_lo(w[j]) * f0 * f1, bf_hi(w[j]) * f0 * f1};
    if (!all) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int b = int((w[j] >> (h * 16 + 7)) & 0xFFu);
        const int at = b == 255 ? 0 : (top - b) >> 5;
        if (at != win) x[h] = 0.f;
      }
    }
    const __half2 p = __floats2half2_rn(x[0], x[1]);
    o[j] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// A token's largest exponent field and windows.
constexpr int kNotFinite = 0x100;  // beside the exponent field: there is an infinity or a NaN
__device__ __forceinline__ int2 windows_of(int hi, int lo, bool odd) {
  if (hi < 0) hi = lo = 127;  // nothing but zeros, infinities and NaN
  return make_int2(hi + (odd ? kNotFinite : 0), (hi - lo) / 32 + 1);
}

// A CTA per token: its exponents, then its windows as columns of fp16 (in global memory).
constexpr int DC_TOKEN_THREADS = 512;
constexpr int DC_TOKEN_KEEP = 4;  // pieces that a thread keeps in registers from the first pass
__global__ void __launch_bounds__(DC_TOKEN_THREADS)
    k_mx_tokens(const __nv_bfloat16* __restrict__ X, int n, int vec, int pieces, int2* __restrict__ tokens,
                uint4* __restrict__ columns) {
  pdl_trigger();  // the product's copies of D need not wait
  __shared__ int red[2][DC_TOKEN_THREADS / 32];
  const int tok = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const __nv_bfloat16* x = X + int64_t(tok) * n;
  uint4 kept[DC_TOKEN_KEEP];
  int hi = -1, lo = 255;
  bool odd = false;
#pragma unroll
  for (int k = 0; k < DC_TOKEN_KEEP; ++k) {
    const int c = threadIdx.x + k * DC_TOKEN_THREADS;
    kept[k] = c < pieces ? load_piece(x, c * 8, n, vec) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int k = 0; k < DC_TOKEN_KEEP; ++k) {
    int h, l;
    odd |= exponents(kept[k], h, l);
    hi = max(hi, h);
    lo = min(lo, l);
  }
  for (int c = threadIdx.x + DC_TOKEN_KEEP * DC_TOKEN_THREADS; c < pieces; c += DC_TOKEN_THREADS) {
    int h, l;
    odd |= exponents(load_piece(x, c * 8, n, vec), h, l);
    hi = max(hi, h);
    lo = min(lo, l);
  }
  hi = __reduce_max_sync(0xFFFFFFFFu, hi);
  lo = __reduce_min_sync(0xFFFFFFFFu, lo);
  if (lane == 0) {
    red[0][warp] = hi;
    red[1][warp] = lo;
  }
  odd = __syncthreads_or(odd);
#pragma unroll
  for (int w = 0; w < DC_TOKEN_THREADS / 32; ++w) {
    hi = max(hi, red[0][w]);
    lo = min(lo, red[1][w]);
  }
  const int2 of = windows_of(hi, lo, odd);
  hi = of.x & 0xFF;
  const int windows = of.y;
  if (threadIdx.x == 0) tokens[tok] = of;
  for (int w = 0; w < windows; ++w) {
    uint4* out = columns + (int64_t(w) * gridDim.x + tok) * pieces;
#pragma unroll
    for (int k = 0; k < DC_TOKEN_KEEP; ++k) {
      const int c = threadIdx.x + k * DC_TOKEN_THREADS;
      if (c < pieces) out[c] = window_piece(kept[k], hi, w, windows == 1);
    }
    for (int c = threadIdx.x + DC_TOKEN_KEEP * DC_TOKEN_THREADS; c < pieces; c += DC_TOKEN_THREADS)
      out[c] = window_piece(load_piece(x, c * 8, n, vec), hi, w, windows == 1);
  }
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ uint32_t g_mx_decode_err;

constexpr int DC_MAX_STAGES = 8;
constexpr int DC_THREADS = (DC_WARPS + 1) * 32;
// Room for the warps' sums: of two row tiles with eight columns, of more with fewer columns.
constexpr int DC_RED_PITCH = 20;  // a column's 16 rows, spread over the banks
constexpr int DC_RED = DC_WARPS * 16 * DC_RED_PITCH * 4;

__device__ __forceinline__ void dc_sync() { asm volatile("barrier.sync 1, 512;" ::: "memory"); }  // the 16 warps

// kSelf: one token, whose columns each CTA makes for itself.
template <bool kSelf>
__global__ void __launch_bounds__(DC_THREADS, 1)
    k_mx_decode(const __grid_constant__ DcMaps maps, const DcArgs a) {
  constexpr int kRows = 16;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  // (an offset, not a rounded integer: the compiler still knows that this is shared memory)
  unsigned char* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ uint64_t full[DC_MAX_STAGES], empty[DC_MAX_STAGES];
  __shared__ uint64_t xfull;
  __shared__ int abort_flag;
  __shared__ int2 token[8], range[DC_WARPS];
  __shared__ float unscale[2][8];  // per column: 2^k in two factors
  __shared__ int odd_token;        // kSelf: there is an infinity or a NaN
  __shared__ int again;            // some outputs are to be summed again: those marked 1 in ysum
  float* red = reinterpret_cast<float*>(smem);  // [slot][DC_WARPS][columns][DC_RED_PITCH]
  const int pieces = a.slice * (DC_UNIT / 8), cpitch = dc_col_pitch(a.slice);
  uint4* xs = reinterpret_cast<uint4*>(smem + DC_RED);
  unsigned char* ring = smem + a.ring;
  float* ysum = reinterpret_cast<float*>(smem + a.ysum);  // [row tile of this CTA][token][kRows]
  const int srows = a.tps * kRows;
  const int sbytes = dc_stage_bytes(a.su, srows);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int units = (a.nb + 7) / 8, tiles = (a.m + kRows - 1) / kRows;
  const int groups = (tiles + a.tps - 1) / a.tps;  // row tiles are taken tps at a time
  volatile int* abrt = &abort_flag;

  if (threadIdx.x == 0) {
    abort_flag = 0;
    odd_token = again = 0;
    for (int i = 0; i < a.stages; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&empty[i], DC_WARPS);
    }
    tc::mbar_init(&xfull, 1);
    tc::fence_mbar_init();
  }
  __syncthreads();

  if (warp == DC_WARPS) {
    const uint64_t policy = tc::make_policy_evict_first();
    const int whole = a.nb / 8;  // units that a row has in full
    int s = 0, issued = 0;
    uint32_t ph = 1;
    for (int u0 = 0; u0 < units; u0 += a.slice) {
      const int uend = min(u0 + a.slice, units);
      int passes = 1;
      bool told = false;
      for (int pass = 0; pass < passes; ++pass) {
        int step = 0;
        for (int grp = blockIdx.x; grp < groups; grp += gridDim.x) {
          const int row0 = grp * srows;
          for (int u = u0; u < uend; u += a.su, ++step) {
            // One token: a ring full goes out without knowing the passes.  From two on one stage: more of
            // them only hold up the kernel that makes the columns (8192 × 28672, 8 tokens: 57.8 µs, with a
            // ring full 59.1; 28672 × 8192 the same either way).
            if (!told && step == (kSelf ? a.stages : 1)) {
              told = true;
              __syncthreads();
            }
            if (lane == 0) {
              if (!tc::mbar_try(&empty[s], ph) && (*abrt || !tc::mbar_wait(&empty[s], ph, &g_mx_decode_err)))
                *abrt = 1;
              // after a wait that gave up nothing more is copied, but the barriers are still met
              if (!*abrt) {
                unsigned char* c = ring + s * sbytes;
                const bool ragged = u + a.su > whole && whole < units;
                const int nu = ragged ? min(a.su, units - u) : a.su;
                tc::mbar_expect_tx(&full[s], uint32_t((nu + 1) * srows * 128));
                if (!ragged) {
                  tc::tma_load_3d_hint(c, &maps.c3, 0, row0, u, &full[s], policy);
                } else {
                  for (int q = 0; q < nu; ++q)
                    tc::tma_load_2d_hint(c + q * srows * 128, &maps.c2, (u + q) * 128, row0, &full[s], policy);
                }
                tc::tma_load_2d_hint(c + a.su * srows * 128, &maps.s, u * 8, row0, &full[s], policy);
                ++issued;
              }
            }
            __syncwarp();
            if (++s == a.stages) {
              s = 0;
              ph ^= 1;
            }
          }
        }
        if (!told) {
          told = true;
          __syncthreads();
        }
        if (pass == 0)
          for (int t = 0; t < a.T; ++t) passes = max(passes, (token[t].y + a.wcols - 1) / a.wcols);
      }
    }
    if (lane == 0 && *abrt)
      for (int q = 0; q < a.stages && q < issued; ++q)  // copies in flight land first
        tc::mbar_wait(&full[q], uint32_t((issued - 1 - q) / a.stages) & 1, &g_mx_decode_err);
    // when the sums are done: those to be done again, if any
    __syncwarp();
    asm volatile("barrier.sync 2, 544;" ::: "memory");
    if (!again) return;
    for (int grp = blockIdx.x, local = 0; grp < groups; grp += gridDim.x, ++local)
      for (int e = 0; e < kRows * a.T * a.tps; ++e) {
        const int row = (grp * a.tps + (e >> 4) / a.T) * kRows + (e & 15), tok = (e >> 4) % a.T;
        if (row >= a.m || ysum[int64_t(local) * a.tps * a.T * kRows + e] != 1.f) continue;
        float v = dc_again(a.codes + row * a.pitch, a.scales + row * a.spitch, a.X + int64_t(tok) * a.n, a.n, a.nb);
        const int64_t at = int64_t(tok) * a.m + row;
        if (a.add) v += __bfloat162float(a.add[at]);
        __syncwarp();  // (add may be Y)
        if (lane == 0) a.Y[at] = __float2bfloat16_rn(v);
      }
    return;
  }

  const int g = lane >> 2, t = lane & 3;
  // this warp's row tile within a stage and its unit there
  const int sub = warp / a.su, my = warp - sub * a.su;
  int s = 0;
  uint32_t ph = 0, round = 0;  // round: passes over D so far
  for (int u0 = 0; u0 < units; u0 += a.slice) {
    const int uend = min(u0 + a.slice, units);
    if (u0 == 0) {
      if (kSelf) {
        int hi = -1, lo = 255;
        bool odd = false;
#pragma unroll 4
        for (int c = threadIdx.x; c < a.cpieces; c += DC_WARPS * 32) {
          int h, l;
          odd |= exponents(load_piece(a.X, c * 8, a.n, a.vec), h, l);
          hi = max(hi, h);
          lo = min(lo, l);
        }
        hi = __reduce_max_sync(0xFFFFFFFFu, hi);
        lo = __reduce_min_sync(0xFFFFFFFFu, lo);
        if (lane == 0) range[warp] = make_int2(hi, lo);
        if (odd) odd_token = 1;
        dc_sync();
        if (threadIdx.x == 0) {
          for (int w = 1; w < DC_WARPS; ++w) {
            hi = max(hi, range[w].x);
            lo = min(lo, range[w].y);
          }
          token[0] = windows_of(hi, lo, odd_token != 0);
        }
      } else {
        pdl_wait();  // the columns are written
        if (threadIdx.x < a.T) token[threadIdx.x] = __ldcg(a.tokens + threadIdx.x);
      }
    }
    __syncthreads();
    int windows = 1;
    for (int k = 0; k < a.T; ++k) windows = max(windows, token[k].y);
    const int per_tok = min(windows, a.wcols), cols = a.T * per_tok;
    const int passes = (windows + a.wcols - 1) / a.wcols;

    for (int pass = 0; pass < passes; ++pass, ++round) {
      tc::fence_async_smem();
      dc_sync();  // the last round's columns are read
      const int have = min(pieces, a.cpieces - u0 * (DC_UNIT / 8));  // the last slice may be shorter
      if (kSelf) {
        for (int c = 0; c < cols && pass * a.wcols + c < windows; ++c) {
#pragma unroll 4
          for (int e = threadIdx.x; e < have; e += DC_WARPS * 32)
            xs[c * cpitch + e] = window_piece(load_piece(a.X, (u0 * (DC_UNIT / 8) + e) * 8, a.n, a.vec), token[0].x & 0xFF,
                                              pass * a.wcols + c, windows == 1);
        }
      } else if (threadIdx.x == 0) {
        int count = 0;
        for (int c = 0; c < cols; ++c) count += pass * a.wcols + c % per_tok < token[c / per_tok].y;
        tc::mbar_expect_tx(&xfull, uint32_t(count * have * 16));
        for (int c = 0; c < cols; ++c) {
          const int tok = c / per_tok, win = pass * a.wcols + c % per_tok;
          if (win < token[tok].y)
            tc::bulk_load(xs + c * cpitch, a.columns + (int64_t(win) * a.T + tok) * a.cpieces + u0 * (DC_UNIT / 8),
                          uint32_t(have * 16), &xfull);
        }
      }
      if (threadIdx.x < cols) {
        const int tok = threadIdx.x / per_tok;
        const int k = (token[tok].x & 0xFF) - 127 - 32 * (pass * a.wcols + int(threadIdx.x) % per_tok);
        // (a column past the token's windows is all zeros: any factor will do)
        // (2^(e − 110) and the columns' 2^15 together are 2^32 more than 2^(e − 127))
        const int k0 = max(k - 32, -252) / 2, k1 = max(k - 32, -252) - k0;
        unscale[0][threadIdx.x] = pow2(k0);
        unscale[1][threadIdx.x] = pow2(k1);
      }
      for (int c = 0; c < cols; ++c)  // windows that a token does not have
        if (pass * a.wcols + c % per_tok >= token[c / per_tok].y)
          for (int e = threadIdx.x; e < pieces; e += DC_WARPS * 32) xs[c * cpitch + e] = make_uint4(0, 0, 0, 0);
      if (!kSelf && !tc::mbar_wait(&xfull, round & 1, &g_mx_decode_err)) *abrt = 1;
      dc_sync();
      const bool first = u0 == 0 && pass == 0, last = uend == units && pass == passes - 1;
      // The warps' sums of several row tiles are kept before they are added up together: a
      // meeting of the warps per tile costs more than the tile's copies.
      const int slots = DC_RED / (DC_WARPS * DC_RED_PITCH * 4 * cols);
      int slot = 0, local = 0;
      // Column g at this lane's words (the last column where there are fewer: those sums are not used)
      const uint4* xb = xs + min(g, cols - 1) * cpitch + t;
      for (int grp = blockIdx.x; grp < groups; grp += gridDim.x) {
        float acc[4] = {};
        for (int u = u0; u < uend; u += a.su) {
          const bool got = tc::mbar_try(&full[s], ph) ||
                           (!*abrt && tc::mbar_wait(&full[s], ph, &g_mx_decode_err));
          if (!got) *abrt = 1;
          const int unit = u + my;
          if (got && sub < a.tps && unit < uend) {
            // (rows start on 128 bytes: chunk b ^ g by an exclusive or)
            const uint32_t cbase = tc::smem_u32(ring) + s * sbytes + (my * srows + sub * kRows + g) * 128 +
                                   (g << 4) + t * 4;
            const unsigned char* ebase = ring + s * sbytes + (a.su * srows + sub * kRows + g) * 128 +
                                         (((my >> 1) ^ g) << 4) + (my & 1) * 8;
            uint2 e0 = *reinterpret_cast<const uint2*>(ebase);
            uint2 e1 = *reinterpret_cast<const uint2*>(ebase + 1024);
            if (unit * 8 + 8 > a.nb) {  // padding after the row's last block counts as 0
              const int k = a.nb - unit * 8;
              const uint32_t mx = k >= 4 ? ~0u : (1u << (8 * k)) - 1, my4 = k <= 4 ? 0u : (1u << (8 * (k - 4))) - 1;
              e0.x &= mx; e1.x &= mx; e0.y &= my4; e1.y &= my4;
            }
            uint32_t w0[8], w1[8];
#pragma unroll
            for (int b = 0; b < 8; ++b) {
              w0[b] = lds32(cbase ^ (b << 4));
              w1[b] = lds32((cbase ^ (b << 4)) + 1024);
            }
            float s0[8], s1[8];
            widen_scales(e0.x, s0);
            widen_scales(e0.y, s0 + 4);
            widen_scales(e1.x, s1);
            widen_scales(e1.y, s1 + 4);
            const int xu = (unit - u0) * 32;
#pragma unroll
            for (int b = 0; b < 8; ++b) {
              uint32_t v0[4], v1[4];
              widen_word(w0[b], v0);
              widen_word(w1[b], v1);
              const uint4 x = xb[xu + b * 4];
              float c[4] = {0.f, 0.f, 0.f, 0.f};
              mma16816(c, v0[0], v1[0], v0[1], v1[1], x.x, x.y);
              mma16816(c, v0[2], v1[2], v0[3], v1[3], x.z, x.w);
              acc[0] = fmaf(s0[b], c[0], acc[0]);
              acc[1] = fmaf(s0[b], c[1], acc[1]);
              acc[2] = fmaf(s1[b], c[2], acc[2]);
              acc[3] = fmaf(s1[b], c[3], acc[3]);
            }
          }
          tc::fence_async_smem();  // the loads are done before a copy may overwrite what they read
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&empty[s]);
          if (++s == a.stages) {
            s = 0;
            ph ^= 1;
          }
        }
        if (slot == 0 && local) dc_sync();  // the last sums are read
        float* out = red + (slot * DC_WARPS + warp) * cols * DC_RED_PITCH + g;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int col = 2 * t + q;
          if (col < cols) {
            out[col * DC_RED_PITCH] = acc[q];
            out[col * DC_RED_PITCH + 8] = acc[2 + q];
          }
        }
        ++slot;
        if (slot < slots && grp + int(gridDim.x) < groups) continue;
        dc_sync();
        // half of a warp per 16 rows, so that every warp has its share of few outputs; the warps go on
        // to the next row tile as they finish
        for (int e = warp * 16 + (lane & 15) + (lane >> 4) * (DC_WARPS * 16); e < kRows * a.T * a.tps * slot;
             e += DC_WARPS * 32) {
          const int i = e & 15, tile = (e >> 4) / a.T, tok = (e >> 4) - tile * a.T;
          const int q = a.tps == 1 ? tile : tile / a.tps, ts = tile - q * a.tps;
          const int row = ((grp - (slot - 1 - q) * int(gridDim.x)) * a.tps + ts) * kRows + i;
          if (row >= a.m) continue;
          const int64_t at = int64_t(tok) * a.m + row;
          const float plus = last && a.add ? __bfloat162float(a.add[at]) : 0.f;
          const float* p = red + ((q * DC_WARPS + ts * a.su) * cols + tok * per_tok) * DC_RED_PITCH + i;
          float v = 0.f;
          for (int c = per_tok - 1; c >= 0; --c) {
            float col = p[c * DC_RED_PITCH];
#pragma unroll 8
            for (int w = 1; w < a.su; ++w) col += p[(w * cols + c) * DC_RED_PITCH];
            v += col * unscale[0][tok * per_tok + c] * unscale[1][tok * per_tok + c];
          }
          float* keep = ysum + ((int64_t(local + q) * a.tps + ts) * a.T + tok) * kRows + i;
          if (!first) v += *keep;
          if (!last) {
            *keep = v;
            continue;
          }
          const bool odd = !(fabsf(v) < INFINITY) && token[tok].x < kNotFinite;
          *keep = odd ? 1.f : 0.f;
          if (odd) {
            again = 1;
            continue;
          }
          if (a.add) v += plus;
          a.Y[at] = __float2bfloat16_rn(v);
        }
        local += slot;
        slot = 0;
      }
    }
  }
  asm volatile("barrier.arrive 2, 544;" ::: "memory");  // the copying warp may look at the marks
}

// ---- f32 ------------------------------------------------------------------------
constexpr int DF_WARPS = 8;
constexpr int DF_TOK = 8;      // tokens of a pass
constexpr int DF_SLAB = 512;   // values of K staged at a time: 64 per warp

// A CTA takes 32 rows (a lane each) × up to 8 tokens; its eight warps divide each slab of K.
// A row's 16 bytes of codes are read by one lane, which uses a whole 32-byte sector with its two blocks.  What
// bounds it is widening and FMA issue once per 8 tokens, and below that latency: K goes in ranges to
// about five CTAs per SM, whose sums a second kernel adds in order (4096 × 4096, 8 tokens: 54 µs
// in one range, 27 in eight; one token 18.5 µs; slabs of 1024 values cost 2 to 10 µs more).
__global__ void __launch_bounds__(DF_WARPS * 32)
    k_mx_decode_f32(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t cpitch,
                    int64_t spitch, const float* __restrict__ X, const float* add, float* Y, int m, int n,
                    int nb, int T, int krange, float* __restrict__ part) {
  pdl_trigger();
  __shared__ __align__(16) float xs[DF_TOK][DF_SLAB];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = blockIdx.x * 32 + lane, row = min(i, m - 1);
  const int t0 = blockIdx.y * DF_TOK, nt = min(DF_TOK, T - t0);
  float acc[DF_TOK] = {};
  const int kend = min(n, int(blockIdx.z + 1) * krange);
  for (int k0 = blockIdx.z * krange; k0 < kend; k0 += DF_SLAB) {
    uint4 c[2];
    uint32_t s = 0;
    const int b0 = k0 / 32 + warp * 2;
    if (b0 < nb) s = __ldg(reinterpret_cast<const uint16_t*>(scales + int64_t(row) * spitch + b0));
#pragma unroll
    for (int q = 0; q < 2; ++q)
      c[q] = b0 + q < nb ? __ldg(reinterpret_cast<const uint4*>(codes + int64_t(row) * cpitch + int64_t(b0 + q) * 16))
                         : make_uint4(0, 0, 0, 0);
    __syncthreads();
    for (int e = threadIdx.x; e < nt * DF_SLAB; e += DF_WARPS * 32) {
      const int tok = e / DF_SLAB, k = e % DF_SLAB;
      xs[tok][k] = k0 + k < n ? X[int64_t(t0 + tok) * n + k0 + k] : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (b0 + q >= nb) break;
      const float scale = mx::scale_f32((s >> (8 * q)) & 0xFFu);
      const uint32_t w[4] = {c[q].x, c[q].y, c[q].z, c[q].w};
      float part[DF_TOK] = {};
#pragma unroll
      for (int z = 0; z < 8; ++z) {
        float d[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) d[p] = mx::e2m1_f32((w[z >> 1] >> ((z & 1) * 16 + p * 4)) & 15u) * scale;
#pragma unroll
        for (int tok = 0; tok < DF_TOK; ++tok) {
          if (tok >= nt) break;
          const float4 x = *reinterpret_cast<const float4*>(&xs[tok][warp * 64 + q * 32 + z * 4]);
          part[tok] = fmaf(d[0], x.x, part[tok]);
          part[tok] = fmaf(d[1], x.y, part[tok]);
          part[tok] = fmaf(d[2], x.z, part[tok]);
          part[tok] = fmaf(d[3], x.w, part[tok]);
        }
      }
#pragma unroll
      for (int tok = 0; tok < DF_TOK; ++tok) acc[tok] += part[tok];
    }
  }
  __syncthreads();
  float* red = &xs[0][0];  // [warp][token][row]
#pragma unroll
  for (int tok = 0; tok < DF_TOK; ++tok) red[(warp * DF_TOK + tok) * 32 + lane] = acc[tok];
  __syncthreads();
  // warp w adds up token w
  if (warp < nt && i < m) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < DF_WARPS; ++w) v += red[(w * DF_TOK + warp) * 32 + lane];
    const int64_t at = int64_t(t0 + warp) * m + i;
    if (part) {
      part[int64_t(blockIdx.z) * T * m + at] = v;
    } else {
      if (add) v += add[at];
      Y[at] = v;
    }
  }
}
static_assert(DF_WARPS * DF_TOK * 32 <= DF_TOK * DF_SLAB, "the sums fit where the tokens were");

// How a call is laid out in shared memory; stages = 0 where it does not fit.
struct DcPlan {
  int wcols, slice, su, tps, stages, ysum, ring, bytes, grid;
};
DcPlan decode_plan(int64_t T, int64_t m, int64_t n, int wcols) {
  DcPlan p = {};
  p.wcols = wcols;
  const int rows = 16;
  const int units = int((mx::blocks(n) + 7) / 8);
  const int64_t tiles = (m + rows - 1) / rows;
  // the widest slice (all of K at best) that leaves room for two stages at least; with
  // more than one, slices of whole stages of 16 units, or of an even number of units (a
  // copy of scales starts on 16 bytes)
  for (int count = 1; count <= units; ++count) {
    p.slice = (units + count - 1) / count;
    if (count > 1) p.slice = p.slice >= 16 ? p.slice / 16 * 16 : (p.slice + 1) / 2 * 2;
    p.su = std::min(p.slice, DC_WARPS);
    p.tps = DC_WARPS / p.su;
    const int64_t groups = (tiles + p.tps - 1) / p.tps;
    p.grid = int(std::min<int64_t>(groups, 148));
    const int64_t ysum = (groups + p.grid - 1) / p.grid * p.tps * T * rows * 4;
    const int64_t xs = T * p.wcols * dc_col_pitch(p.slice) * 16;
    const int stage = dc_stage_bytes(p.su, p.tps * rows);
    const int64_t left = DC_SMEM_MAX - round_up(DC_RED + xs, 1024) - ysum;
    if (left < 2 * stage) continue;
    p.stages = int(std::min<int64_t>(DC_MAX_STAGES, left / stage));
    p.ring = int(round_up(DC_RED + xs, 1024));
    p.ysum = p.ring + p.stages * stage;
    p.bytes = p.ysum + int(ysum) + 1024;
    return p;
  }
  p.stages = 0;
  return p;
}
// Two columns per token up to 4 tokens, unless their room costs stages or slices of K that one column
// would not.
DcPlan decode_plan(int64_t T, int64_t m, int64_t n) {
  const DcPlan one = decode_plan(T, m, n, 1);
  if (T > 4) return one;
  const DcPlan two = decode_plan(T, m, n, 2);
  return two.slice == one.slice && two.stages >= std::min(one.stages, 3) ? two : one;
}

}  // namespace

bool mx_decode_fits(int64_t T, int64_t m, int64_t n) {
  return T <= kMxDecodeMax && tmap_available() && decode_plan(T, m, n).stages >= 2;
}

// One token's columns cost a CTA less than a kernel that makes them for all, as the first stages of D are on
// their way meanwhile (28672 × 8192: 28.9 against 32.7 µs, 11008 × 4096: 12.3 against 14.4).  Of more tokens every
// CTA would make all columns.
bool decode_self(int64_t T) { return T == 1; }

// The workspace: per token its exponent and windows (256 bytes), then its columns: eight windows hold every
// bf16 value.
size_t mx_decode_workspace(int64_t T, int64_t n) {
  if (decode_self(T)) return 0;
  return size_t(256 + 8 * T * ((mx::blocks(n) + 7) / 8) * DC_UNIT * 2);
}

hsl_status mx_decode_run(const MxOperand& D, int64_t m, int64_t n, const void* X, const void* add, void* Y,
                         int64_t T, void* ws, cudaStream_t s) {
  const DcPlan p = decode_plan(T, m, n);
  DcArgs a;
  DcMaps maps;
  memset(&maps, 0, sizeof(maps));
  const int rows = 16 * p.tps;
  const auto U8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const auto SW = CU_TENSOR_MAP_SWIZZLE_128B;
  const int64_t whole = D.pitch / 128;
  if ((whole > 0 && !make_tmap_3d_bytes(&maps.c3, D.p, {128, m, whole}, D.pitch, 128, {128, rows, p.su}, SW)) ||
      !make_tmap_2d(&maps.c2, U8, 1, D.p, m, D.pitch, D.pitch, 128, rows, SW) ||
      !make_tmap_2d(&maps.s, U8, 1, D.scales, m, D.spitch, D.spitch, 128, rows, SW)) {
    set_message("tensor map encoding failed");
    return HSL_ERR_CUDA;
  }
  const bool self = decode_self(T);
  a.tokens = static_cast<const int2*>(ws);
  a.columns = self ? nullptr : reinterpret_cast<const uint4*>(static_cast<const char*>(ws) + 256);
  a.X = static_cast<const __nv_bfloat16*>(X);
  a.n = int(n);
  a.vec = n % 8 == 0 && reinterpret_cast<uintptr_t>(X) % 16 == 0 ? 1 : 0;
  a.cpieces = int((mx::blocks(n) + 7) / 8) * (DC_UNIT / 8);
  a.codes = static_cast<const uint8_t*>(D.p);
  a.scales = D.scales;
  a.pitch = D.pitch;
  a.spitch = D.spitch;
  a.add = static_cast<const __nv_bfloat16*>(add);
  a.Y = static_cast<__nv_bfloat16*>(Y);
  a.m = int(m);
  a.nb = int(mx::blocks(n));
  a.T = int(T);
  a.wcols = p.wcols;
  a.ring = p.ring;
  a.slice = p.slice;
  a.su = p.su;
  a.tps = p.tps;
  a.stages = p.stages;
  a.ysum = p.ysum;
  void (*fn)(const DcMaps, const DcArgs) = self ? k_mx_decode<true> : k_mx_decode<false>;
  if (cudaError_t e = allow_dyn_smem(reinterpret_cast<const void*>(fn), p.bytes))
    return cuda_fail(e, "4-bit decode smem attribute");
  note_launch(self ? 1 : 2);
  if (!self) {
    k_mx_tokens<<<unsigned(T), DC_TOKEN_THREADS, 0, s>>>(a.X, int(n), a.vec, a.cpieces, static_cast<int2*>(ws),
                                                         reinterpret_cast<uint4*>(static_cast<char*>(ws) + 256));
    if (hsl_status e = cuda_fail(cudaGetLastError(), "4-bit decode launch")) return e;
  }
  return cuda_fail(launch_chained(fn, !self, dim3(unsigned(p.grid)), DC_THREADS, size_t(p.bytes), s, maps, a),
                   "4-bit decode launch");
}

cudaError_t mx_decode_error_word(uint32_t** p) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_mx_decode_err);
}

// Ranges of K, each whole slabs: about five CTAs per SM.  Two slabs stay in one range, as the second launch and the
// scratch cost more than a slab (1024 × 1024, one token: 14.3 against 10.9 µs).
static int decode_f32_ranges(int64_t T, int64_t m, int64_t n, int64_t* krange) {
  const int64_t ctas = (m + 31) / 32 * ((T + DF_TOK - 1) / DF_TOK), slabs = (n + DF_SLAB - 1) / DF_SLAB;
  if (slabs <= 2) return *krange = slabs * DF_SLAB, 1;
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(slabs, (740 + ctas - 1) / ctas));
  const int64_t per = (slabs + want - 1) / want;
  *krange = per * DF_SLAB;
  return int((slabs + per - 1) / per);
}
size_t mx_decode_f32_workspace(int64_t T, int64_t m, int64_t n) {
  int64_t krange;
  const int ranges = decode_f32_ranges(T, m, n, &krange);
  return ranges > 1 ? size_t(ranges) * size_t(T * m) * 4 : 0;
}
hsl_status mx_decode_f32_run(const MxOperand& D, int64_t m, int64_t n, const void* X, const void* add,
                             void* Y, int64_t T, void* ws, cudaStream_t s) {
  int64_t krange;
  const int ranges = decode_f32_ranges(T, m, n, &krange);
  const dim3 grid(unsigned((m + 31) / 32), unsigned((T + DF_TOK - 1) / DF_TOK), unsigned(ranges));
  float* part = ranges > 1 ? static_cast<float*>(ws) : nullptr;
  note_launch();
  k_mx_decode_f32<<<grid, DF_WARPS * 32, 0, s>>>(static_cast<const uint8_t*>(D.p), D.scales, D.pitch, D.spitch,
                                                 static_cast<const float*>(X), static_cast<const float*>(add),
                                                 static_cast<float*>(Y), int(m), int(n), int(mx::blocks(n)),
                                                 int(T), int(krange), part);
  if (hsl_status e = cuda_fail(cudaGetLastError(), "4-bit f32 decode launch")) return e;
  return part ? mx_simt_sum_run(part, ranges, T * m, static_cast<const float*>(add), static_cast<float*>(Y), s) : HSL_OK;
}

}  // namespace hsl
