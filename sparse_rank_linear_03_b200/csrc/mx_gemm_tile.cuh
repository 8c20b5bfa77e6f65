// The body of a block-product CTA (mx_gemm.cuh): tile `block` of one product.  Included as text, inside a scope
// of a kernel that defines
//   AK, BMN, TERMS, MH, OUT   constants: kind of A, B N-major, terms of B, accumulators, result
//   maps, g, block            the product's GemmMaps and GemmArgs (kernel parameters), the tile
// because the same text as an inlined device function ran 8 % slower (2048 tokens × 11008 × 4096:
// 162 against 150 µs).  No include guard: a kernel of several products includes it once for each.
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  // (an offset, not a rounded integer: the compiler still knows that this is shared memory)
  unsigned char* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ uint64_t full[G_MAX_STAGES], empty[G_MAX_STAGES], accf[2], drained[2], quiet, addf;
  __shared__ uint64_t raw[G_MAX_STAGES], taken[G_MAX_STAGES];  // code tile landed, read
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ntn = (g.N + g.BN - 1) / g.BN;
  const int tile = block / g.splits, split = block % g.splits;
  const int i0 = (tile / ntn) * (128 * MH), j0 = (tile % ntn) * g.BN;
  const int kb0 = int(int64_t(g.nk) * split / g.splits);
  const int nk = int(int64_t(g.nk) * (split + 1) / g.splits) - kb0;
  constexpr int kA = MH * 128 * 128;  // bytes of the A tile
  const int bgroups = (g.BN + 63) / 64;
  const int kB = BMN ? bgroups * 8192 : g.BN * 128;
  using Code = CodeTile<AK, MH>;
  const int kStage = kA + TERMS * kB;
  unsigned char* cring = smem + g.stages * kStage;
  // The tensor unit cuts every sum off towards zero.  Over the hundreds of inexact terms of a gradient that
  // adds up to 2^−16 of the result (28672 × 8192, 4096 tokens), so there a chain of kChunk K-blocks goes to one of
  // two accumulators in turn, and the sixteen warps add the other to fp32 sums in registers, rounded to nearest.
  constexpr bool kFold = OUT == OUT_R;
  constexpr int kChunk = TERMS > 1 ? 2 : 4;
  constexpr int kSteps = kFold ? MH : 1;  // 32-column pieces of an accumulator per warp, at BN <= 128
  const int nchunks = (nk + kChunk - 1) / kChunk, aset = MH * g.BN;  // columns of a set of accumulators
  // (whole 32-column reads from the last accumulator stay inside)
  const uint32_t need = uint32_t((kFold ? 2 : 1) * aset - g.BN + (g.BN + 31) / 32 * 32);
  uint32_t cols = 32;
  while (cols < need) cols *= 2;

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < g.stages; ++s) {
      tc::mbar_init(&full[s], a_is_blocks(AK) ? 1 + 8 : 1);  // copies, and the eight widening warps
      tc::mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < g.codes; ++s) {
      tc::mbar_init(&raw[s], 1);
      tc::mbar_init(&taken[s], 8);
    }
    for (int p = 0; p < 2; ++p) {
      tc::mbar_init(&accf[p], 1);
      tc::mbar_init(&drained[p], 16);
    }
    tc::mbar_init(&quiet, 1);
    tc::mbar_init(&addf, 1);
    tc::fence_mbar_init();
    tc::prefetch_tmap(&maps.b[0]);
  }
  if (warp == 1) {
    tc::tmem_alloc(&tmem_slot, cols);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  // Every CTA of the grid holds its TMEM when the next kernel's may start: none of those can take it first.
  pdl_trigger();
  pdl_wait();
  const uint32_t tmem = tmem_slot;
  volatile int* abrt = &abort_flag;

  if (warp == 0) {
    if (lane == 0) {
      if (OUT == OUT_T && g.addt) tc::tma_prefetch_2d(&maps.add, i0, j0);  // into L2 for the epilogue
      int s = 0, issued = 0;
      uint32_t ph = 1;
      for (int kb = 0; kb < nk; ++kb) {
        if (!g_wait(&empty[s], ph, abrt)) break;
        unsigned char* a = smem + s * kStage;
        unsigned char* b = a + kA;
        const int k0 = (kb0 + kb) * G_BK;
        tc::mbar_expect_tx(&full[s], (a_is_blocks(AK) ? 0 : kA) + TERMS * kB);
        if (AK == A_BF16_K) {
#pragma unroll
          for (int h = 0; h < MH; ++h)
            tc::tma_load_2d(a + h * 16384, &maps.a, k0, i0 + h * 128, &full[s]);
        } else if (AK == A_BF16_M) {
#pragma unroll
          for (int h = 0; h < 2 * MH; ++h)
            tc::tma_load_2d(a + h * 8192, &maps.a, i0 + h * 64, k0, &full[s]);
        }
#pragma unroll
        for (int t = 0; t < TERMS; ++t) {
          if (BMN) {
            for (int q = 0; q < bgroups; ++q)
              tc::tma_load_2d(b + t * kB + q * 8192, &maps.b[t], j0 + q * 64, k0, &full[s]);
          } else {
            tc::tma_load_2d(b + t * kB, &maps.b[t], k0, j0, &full[s]);
          }
        }
        ++issued;
        if (++s == g.stages) {
          s = 0;
          ph ^= 1;
        }
      }
      // the copies in flight have landed before the CTA's shared memory is given up
      for (int q = 0; q < g.stages && q < issued; ++q) {
        const int last = (issued - 1 - q) / g.stages;  // uses of stage q before its last one
        if (*abrt) tc::mbar_wait(&full[q], uint32_t(last) & 1, &g_mx_gemm_err);
      }
    }
    __syncwarp();
  } else if (warp == 18) {
    if (lane == 0 && a_is_blocks(AK)) {
      int s = 0, issued = 0;
      uint32_t ph = 1;
      for (int kb = 0; kb < nk; ++kb) {
        if (!g_wait(&taken[s], ph, abrt)) break;
        unsigned char* q = cring + s * Code::kBytes;
        const int k0 = (kb0 + kb) * G_BK;
        const int qx = (a_is_mmajor(AK) ? i0 : k0) * Code::kElem / 2, qy = a_is_mmajor(AK) ? k0 : i0;
        tc::mbar_expect_tx(&raw[s], Code::kBytes);
#pragma unroll
        for (int x = 0; x < Code::kBoxes; ++x)
          tc::tma_load_2d(q + x * Code::kRows * Code::kInner, &maps.q, qx + x * Code::kInner, qy, &raw[s]);
        if (a_is_mmajor(AK)) tc::tma_load_2d(q + Code::kCodes, &maps.qs, (i0 / 32) & ~15, k0, &raw[s]);
        ++issued;
        if (++s == g.codes) {
          s = 0;
          ph ^= 1;
        }
      }
      for (int q = 0; q < g.codes && q < issued; ++q)
        if (*abrt) tc::mbar_wait(&raw[q], uint32_t((issued - 1 - q) / g.codes) & 1, &g_mx_gemm_err);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (OUT == OUT_T && g.add && !g.addt) {  // into L2 for the epilogue, line by line
      const int rows = min(g.BN, g.N - j0), len = min(128 * MH, g.M - i0);
      for (int e = lane; e < rows * 5; e += 32) {
        const int at = e % 5 * 64;
        const __nv_bfloat16* p = g.add + int64_t(j0 + e / 5) * g.M + i0;
        if (at < len + 63) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + min(at, len - 1)));
      }
    }
    if (tc::elect_one()) {
      const uint32_t idesc = tc::idesc_bf16(128, g.BN) | (a_is_mmajor(AK) ? 1u << 15 : 0u) |
                             (BMN ? 1u << 16 : 0u);
      int s = 0;
      uint32_t ph = 0;
      for (int kb = 0; kb < nk; ++kb) {
        const int chunk = kFold ? kb / kChunk : 0;
        const bool first = kFold ? kb % kChunk == 0 : kb == 0;
        if (kFold && first && !g_wait(&drained[chunk & 1], ((chunk >> 1) + 1) & 1, abrt)) break;
        if (!g_wait(&full[s], ph, abrt)) break;
        tc::tc_fence_after();
        unsigned char* a = smem + s * kStage;
        const uint32_t acc = tmem + uint32_t((chunk & 1) * aset);
#pragma unroll
        for (int t = 0; t < TERMS; ++t) {
          const uint64_t bd = BMN ? desc_mn_sw128(a + kA + t * kB) : tc::desc_sw128(a + kA + t * kB);
#pragma unroll
          for (int h = 0; h < MH; ++h) {
            const uint64_t ad =
                a_is_mmajor(AK) ? desc_mn_sw128(a + h * 16384) : tc::desc_sw128(a + h * 16384);
#pragma unroll
            for (int k = 0; k < G_BK / 16; ++k)
              tc::mma_bf16(acc + h * g.BN, tc::desc_advance(ad, k * (a_is_mmajor(AK) ? 2048 : 32)),
                           tc::desc_advance(bd, k * (BMN ? 2048 : 32)), idesc,
                           (!first || k > 0 || t > 0) ? 1u : 0u);
          }
        }
        tc::mma_commit(&empty[s]);
        if (kFold && (kb % kChunk == kChunk - 1 || kb == nk - 1)) tc::mma_commit(&accf[chunk & 1]);
        if (++s == g.stages) {
          s = 0;
          ph ^= 1;
        }
      }
      if (!kFold) tc::mma_commit(&accf[0]);
      if (kFold) {  // nothing may write to TMEM when it is given back, also where another warp has given up
        tc::mma_commit(&quiet);
        tc::mbar_wait(&quiet, 0, &g_mx_gemm_err);
      }
    }
    __syncwarp();
  } else {
    const int tid = (threadIdx.x - 64) & 255, group = (warp - 2) >> 3;
    // accumulators: warp w reaches TMEM lanes 32 (w mod 4) onwards; the four groups of four
    // warps divide the accumulators and their columns, in steps of 32 (the last step may reach past BN,
    // inside the allocation)
    int R, i, c_lo, c_hi;
    uint32_t tb;
    auto place = [&] {  // (called where it is first needed: these registers are dear to the widening)
      const int grp = (warp - 2) >> 2;
      const int half = MH == 2 ? grp & 1 : 0;
      R = half * 128 + (((warp & 3) << 5) | lane);
      i = i0 + R;
      tb = tmem + (uint32_t((warp & 3) * 32) << 16) + uint32_t(half * g.BN);
      const int steps = (g.BN + 31) / 32;
      constexpr int kShare = 4 / MH;  // groups of four warps per accumulator
      c_lo = steps * (grp / MH) / kShare;
      c_hi = steps * (grp / MH + 1) / kShare;
    };
    if (kFold) place();
    float sum[kSteps][32];
    if (kFold) {
#pragma unroll
      for (int q = 0; q < kSteps; ++q)
#pragma unroll
        for (int z = 0; z < 32; ++z) sum[q][z] = 0.f;
    }
    int folded = 0;
    bool live = true;
    // adds the chunks before `end` to the sums
    auto fold = [&](int end) {
      for (; live && folded < end; ++folded) {
        const int p = folded & 1;
        live = __all_sync(0xFFFFFFFFu, g_wait(&accf[p], (folded >> 1) & 1, abrt));
        if (!live) break;
        tc::tc_fence_after();
#pragma unroll
        for (int q = 0; q < 2 * kSteps; ++q) {
          const int c0 = c_lo * 32 + q * 16;
          if (c0 >= min(c_hi * 32, g.BN)) continue;
          float v[16];
          tc::tmem_ld16(tb + uint32_t(p * aset + c0), v);
#pragma unroll
          for (int z = 0; z < 16; ++z) sum[q >> 1][(q & 1) * 16 + z] += v[z];
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&drained[p]);
      }
      return live;
    };
    if (a_is_blocks(AK)) {
      constexpr bool kInt8 = a_is_int8(AK);
      // MH = 2: tile row tid, both blocks; MH = 1: two threads share a tile row
      const int trow = MH == 2 ? tid : (tid & 127);
      const int half0 = MH == 2 ? 0 : (tid >> 7);
      // The two groups of eight warps take the K-blocks in turn, so that one group's wait for
      // its codes and its hand-over overlap the other's arithmetic.
      // [M][K]: the row's scales, 16 blocks (8 K-blocks) at a time, one load ahead
      const bool row_ok = i0 + trow < g.arows;
      const uint4* srow = reinterpret_cast<const uint4*>(g.scales + int64_t(i0 + trow) * g.spitch);
      const int sgroups = int(g.spitch / 16);
      int sgrp = (kb0 + group) >> 3;
      uint4 sc = make_uint4(0, 0, 0, 0), sn = sc;
      if (!a_is_mmajor(AK) && row_ok) {
        if (sgrp < sgroups) sc = __ldg(srow + sgrp);
        if (sgrp + 1 < sgroups) sn = __ldg(srow + sgrp + 1);
      }
      int s = group, cs = group;
      uint32_t ph = 1, cph = 0;
      const uint32_t smem32 = tc::smem_u32(smem) + trow * 128 + ((trow & 7) << 4);
      for (int kb = group; kb < nk; kb += 2) {
        Block<kInt8> blk[MH];
        // (behind the widening of a chunk the MMAs of the one before are done, or soon will be)
        if (kFold && !fold(kb / kChunk - 1)) break;
        if (!g_wait(&raw[cs], cph, abrt)) break;
        const unsigned char* q = cring + cs * Code::kBytes;
#pragma unroll
        for (int b = 0; b < MH; ++b) {
          const int r = a_is_mmajor(AK) ? (trow & 63) : trow;
          const int n0 = (a_is_mmajor(AK) ? (trow >> 6) * 2 : 0) + half0 + b;  // block in the row
          if (kInt8) {
            blk[b].c[0] = *reinterpret_cast<const uint4*>(q + Code::at(r, 2 * n0));
            blk[b].c[kInt8 ? 1 : 0] = *reinterpret_cast<const uint4*>(q + Code::at(r, 2 * n0 + 1));
          } else {
            blk[b].c[0] = *reinterpret_cast<const uint4*>(q + Code::at(r, n0));
          }
          if (a_is_mmajor(AK)) blk[b].e = q[Code::kCodes + r * 16 + ((i0 / 32) & 15) + n0];
        }
        if (!a_is_mmajor(AK)) {
          const int kk = kb0 + kb;
          if ((kk >> 3) != sgrp) {  // steps of 2: the next group of 8 K-blocks
            sgrp = kk >> 3;
            sc = sn;
            if (row_ok && sgrp + 1 < sgroups) sn = __ldg(srow + sgrp + 1);
          }
          const uint32_t w = (kk & 4) ? ((kk & 2) ? sc.w : sc.z) : ((kk & 2) ? sc.y : sc.x);
          const uint32_t pair = (kk & 1) ? w >> 16 : w;
#pragma unroll
          for (int b = 0; b < MH; ++b)  // padding bytes after the last block count as 0
            blk[b].e = kk * 2 + half0 + b < g.nb ? (pair >> (8 * (half0 + b))) & 0xFFu : 0u;
        }
        const int read = cs;
        cs += 2;
        if (cs >= g.codes) {
          cs -= g.codes;
          cph ^= 1;
        }
        // (A parity tells one completion from the next only.  A warp that waits for the MMAs of
        // K-block kb − stages has seen those of kb − 2 − stages done, so it is never two
        // completions ahead; code tiles are an even number, so that a tile's place belongs to
        // one group, which has seen every earlier completion of its barrier.)
        if (!g_wait(&empty[s], ph, abrt)) break;
#pragma unroll
        for (int b = 0; b < MH; ++b) widen(blk[b], smem32 + s * kStage, half0 + b);
        // The fence also orders the reads of the codes before the copy that may overwrite them: an
        // arrival alone was seen to overtake loads still under way.
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          tc::mbar_arrive(&full[s]);
          tc::mbar_arrive(&taken[read]);
        }
        s += 2;
        if (s >= g.stages) {
          s -= g.stages;
          ph ^= 1;
        }
      }
    }
    __syncwarp();
    bool ok = (kFold ? fold(nchunks) : tc::mbar_wait(&accf[0], 0, &g_mx_gemm_err)) && !*abrt;
    __nv_bfloat16* stg = reinterpret_cast<__nv_bfloat16*>(smem);
    if (OUT == OUT_T && g.addt && ok) {
      // the tile of add into the idle ring, where each value is replaced by the result (loads of
      // single values from global memory took five times as long as the product)
      if (threadIdx.x == 64) {
        tc::mbar_expect_tx(&addf, uint32_t(128 * MH * g.BN * 2));
        tc::tma_load_2d(stg, &maps.add, i0, j0, &addf);
      }
      ok = tc::mbar_wait(&addf, 0, &g_mx_gemm_err);
    }
    if (ok) {
      tc::tc_fence_after();
      if (!kFold) place();
      const int mine = kFold ? kSteps : c_hi - c_lo;
#pragma unroll (kFold ? kSteps : 1)
      for (int q32 = 0; q32 < mine; ++q32) {
        const int c0 = (c_lo + q32) * 32;
        if (kFold && c_lo + q32 >= c_hi) break;
        float v[32];
        if (kFold) {
#pragma unroll
          for (int q = 0; q < 32; ++q) v[q] = sum[kFold ? q32 : 0][q];
        } else {
          tc::tmem_ld32(tb + c0, v);
        }
        const int jn = min(32, min(g.BN - c0, g.N - j0 - c0));  // columns of this step in the tile
        if (OUT == OUT_T || OUT == OUT_T_PART) {
          if (OUT == OUT_T_PART) {
            float* p = g.part + (int64_t(split) * g.N + j0 + c0) * g.M + i;
            if (i < g.M) {
#pragma unroll
              for (int q = 0; q < 32; ++q)
                if (q < jn) p[int64_t(q) * g.M] = v[q];
            }
          } else {
            if (g.addt) {
#pragma unroll
              for (int q = 0; q < 32; ++q)
                if (c0 + q < g.BN) v[q] += __bfloat162float(stg[(c0 + q) * (128 * MH) + R]);
            } else if (g.add && i < g.M && jn > 0) {
              const __nv_bfloat16* p = g.add + int64_t(j0 + c0) * g.M + i;
              __nv_bfloat16 av[32];  // all loads on their way before the first is used
#pragma unroll
              for (int q = 0; q < 32; ++q) av[q] = p[int64_t(min(q, jn - 1)) * g.M];
#pragma unroll
              for (int q = 0; q < 32; ++q) v[q] += __bfloat162float(av[q]);
            }
            if (g.cstore) {
#pragma unroll
              for (int q = 0; q < 32; ++q)
                if (c0 + q < g.BN) stg[(c0 + q) * (128 * MH) + R] = __float2bfloat16_rn(v[q]);
            } else if (i < g.M) {
              __nv_bfloat16* p = g.C + int64_t(j0 + c0) * g.M + i;
#pragma unroll
              for (int q = 0; q < 32; ++q)
                if (q < jn) p[int64_t(q) * g.M] = __float2bfloat16_rn(v[q]);
            }
          }
        } else if (i < g.M && jn > 0) {
          if (g.part) {
            float* p = g.part + (int64_t(split) * g.M + i) * g.N + j0 + c0;
            if (jn == 32 && g.N % 4 == 0) {
#pragma unroll
              for (int q = 0; q < 32; q += 4)
                *reinterpret_cast<float4*>(p + q) = make_float4(v[q], v[q + 1], v[q + 2], v[q + 3]);
            } else {
#pragma unroll
              for (int q = 0; q < 32; ++q)
                if (q < jn) p[q] = v[q];
            }
          } else {
            __nv_bfloat16* p = g.C + int64_t(i) * g.N + j0 + c0;
            if (jn == 32 && g.cstore) {  // rows of C start on 16 bytes
#pragma unroll
              for (int q = 0; q < 32; q += 8) {
                uint4 o;
                uint32_t* w = &o.x;
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                  const __nv_bfloat162 h = __floats2bfloat162_rn(v[q + 2 * z], v[q + 2 * z + 1]);
                  w[z] = *reinterpret_cast<const uint32_t*>(&h);
                }
                *reinterpret_cast<uint4*>(p + q) = o;
              }
            } else {
#pragma unroll
              for (int q = 0; q < 32; ++q)
                if (q < jn) p[q] = __float2bfloat16_rn(v[q]);
            }
          }
        }
      }
    } else {
      *abrt = 1;
    }
    if (OUT == OUT_T && g.cstore) {
      // the rounded tile [column][row] lies in the idle ring: one tiled store.  All sixteen
      // warps meet here, whether or not a wait gave up before.
      tc::fence_async_smem();
      asm volatile("barrier.sync 1, 512;" ::: "memory");
      if (threadIdx.x == 64 && ok && !*abrt) {
        tc::tma_store_2d(&maps.c, stg, i0, j0);
        tc::bulk_commit();
        tc::bulk_wait_read_all();
      }
    }
  }
  tc::tc_fence_before();
  tc::cta_sync();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, cols);
  }
