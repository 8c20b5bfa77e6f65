// The body of a block-product CTA (mx_gemm.cuh): tile `block` of one product.  Included as text, inside a scope
// of a kernel that defines
//   AK, BMN, TERMS, MH, OUT   constants: kind of A, B N-major, terms of B, accumulators, result
//   maps, g, block            the product's GemmMaps and GemmArgs (kernel parameters), the tile
// because the same text as an inlined device function ran 8 % slower (2048 tokens × 11008 × 4096:
// 162 against 150 µs).  No include guard: a kernel of several products includes it once for each.
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  // (an offset, not a rounded integer: the compiler still knows that this is shared memory)
  unsigned char* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ uint64_t full[G_MAX_STAGES], empty[G_MAX_STAGES], accf, addf;
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
  uint32_t cols = MH == 2 ? 64 : 32;  // whole 32-column reads past 2 × 16 columns stay inside
  while (cols < uint32_t(MH * g.BN)) cols *= 2;

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
    tc::mbar_init(&accf, 1);
    tc::mbar_init(&addf, 1);
    tc::fence_mbar_init();
    tc::prefetch_tmap(&maps.b0);
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
          const CUtensorMap* map = t ? &maps.b1 : &maps.b0;
          if (BMN) {
            for (int q = 0; q < bgroups; ++q)
              tc::tma_load_2d(b + t * kB + q * 8192, map, j0 + q * 64, k0, &full[s]);
          } else {
            tc::tma_load_2d(b + t * kB, map, k0, j0, &full[s]);
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
        if (!g_wait(&full[s], ph, abrt)) break;
        tc::tc_fence_after();
        unsigned char* a = smem + s * kStage;
#pragma unroll
        for (int t = 0; t < TERMS; ++t) {
          const uint64_t bd = BMN ? desc_mn_sw128(a + kA + t * kB) : tc::desc_sw128(a + kA + t * kB);
#pragma unroll
          for (int h = 0; h < MH; ++h) {
            const uint64_t ad =
                a_is_mmajor(AK) ? desc_mn_sw128(a + h * 16384) : tc::desc_sw128(a + h * 16384);
#pragma unroll
            for (int k = 0; k < G_BK / 16; ++k)
              tc::mma_bf16(tmem + h * g.BN, tc::desc_advance(ad, k * (a_is_mmajor(AK) ? 2048 : 32)),
                           tc::desc_advance(bd, k * (BMN ? 2048 : 32)), idesc,
                           (kb > 0 || k > 0 || t > 0) ? 1u : 0u);
          }
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
    const int tid = (threadIdx.x - 64) & 255, group = (warp - 2) >> 3;
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
    // epilogue: warp w reaches TMEM lanes 32 (w mod 4) onwards; the four groups of four
    // warps divide the accumulators and their columns
    __syncwarp();
    bool ok = tc::mbar_wait(&accf, 0, &g_mx_gemm_err) && !*abrt;
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
      const int grp = (warp - 2) >> 2;
      const int acc = MH == 2 ? grp & 1 : 0;
      const int L = ((warp & 3) << 5) | lane;
      const int R = acc * 128 + L;
      const int i = i0 + R;
      const uint32_t tb = tmem + (uint32_t((warp & 3) * 32) << 16) + uint32_t(acc * g.BN);
      // columns in steps of 32 (the last step may reach past BN, inside the allocation)
      const int steps = (g.BN + 31) / 32;
      constexpr int kShare = 4 / MH;  // groups of four warps per accumulator
      const int part = grp / MH;
      const int c_lo = steps * part / kShare, c_hi = steps * (part + 1) / kShare;
#pragma unroll 1
      for (int c = c_lo; c < c_hi; ++c) {
        const int c0 = c * 32;
        float v[32];
        tc::tmem_ld32(tb + c0, v);
        if (nk == 0) {
#pragma unroll
          for (int q = 0; q < 32; ++q) v[q] = 0.f;
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
