// fp8.cu -- grouped 8-bit product with a scale for each block of 128 on tcgen05 (kind::f8f6f4):
//
//   y[m, n] = sum_kb xs[m, kb] ws[n / 128, kb] ( sum_{k in block kb} xq[m, k] wq[n, k] )
//
// for the rows m each expert holds.  The inner sum of a block is exact products added in
// fp32 by the tensor cores into TMEM; the scales then enter once per block, in registers:
// acc += (xs ws) * block.  So the tensor cores never accumulate across blocks, and the outer
// sum is fp32 as well; y is rounded to bf16 once.
//
// A CTA pair (cta_group::2) computes 256 rows x TN = 256 columns; CTA r holds rows [128r, +128) of
// xq and columns [128r, +128) of wq, and all 256 columns of its rows in TMEM.  Two TMEM
// buffers of 256 columns take turns: while the MMAs fill one with block kb + 1, eight warps
// drain block kb from the other, each thread 128 columns of one row -- one row scale times
// one column scale per block and thread -- into 128 registers.  Warp 0 loads (TMA),
// warp 1 issues MMAs (the pair's first CTA) and owns TMEM, warps 4..11 drain.  A buffer is
// handed back as soon as its last column is in registers, by one arrival per warp (the second
// CTA's arrivals cross to the first).  Rows past the count are neither read as data nor
// written; every wait is bounded.
//
// With fewer tiles than pairs the depth of one tile bounds the product, and the drain of 256
// columns most of each block: then tiles of 128 or 64 columns, the narrowest that still fit on
// the pairs at once, a warp draining 64 or 32 (333 x 1456 x 2008: 12.4 -> 9.6 us; 130 rows of 3
// experts, 2752 x 360: 23.5 -> 13.3).  In a second wave they lose: xq is read for each column
// of tiles (8 x 256 rows, 1024 x 2048: 10.6 us in tiles of 256 columns, 13.1 in 128).
#include "common.cuh"
#include "internal.h"
#include "tc_tile.cuh"

namespace moe {

namespace {

constexpr int BK = 128;                 // depth of a stage = of a scale block (bytes)
constexpr int PM = 256;                 // rows of a tile; its columns TN: 256, 128 or 64
constexpr int kThreads = 384;           // loads, MMAs and two idle warps; eight draining warps
constexpr int kDrainWarps = 8;
// Registers: 384 threads launch with 168 each (64,512); 128 keep 40, 256 take 232 (the same).
constexpr int kRegsLoad = 40, kRegsDrain = 232;
constexpr uint32_t A_BYTES = 128 * BK, STAGE_BYTES = 2 * A_BYTES;     // A, and up to as much of B
constexpr int STAGES = 5;
constexpr double kBlockUs = 0.3;        // 256 x 64 x 128 on a pair, drained
constexpr uint32_t TILE_BYTES = 4096;   // 32 rows x 64 bf16 columns
constexpr uint32_t kPeerBitMask = 0xFEFFFFFFu;
constexpr uint32_t kBars = 256;
constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE_BYTES + 8 * TILE_BYTES + kBars + 16 + 4 * (3 * kMaxExperts + 1);
static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
static_assert(SMEM + 81 * 1024 > 228 * 1024, "a CTA must own its SM");

struct Fp8Pair {
  const int32_t* n;
  int E, C, K, N, KB, NB;
  int n_max;             // counts are read as min(max(n, 0), n_max)
  const float* xs;       // [E, C, KB]
  const float* ws;       // [E, NB, KB]
  __nv_bfloat16* y;
  int splits, rows;      // shares of a tile's depth (split.cu); most rows an expert holds
  float* part;           // splits > 1: [splits][E, rows, N] fp32 sums instead of y
  unsigned* err;
  uint64_t limit_ns;
};

template <bool SPLIT, int TN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    fp8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmD, const Fp8Pair a) {
  constexpr uint32_t TMEM_COLS = 2 * TN;
  constexpr int COLS = TN / 2;                         // columns of a CTA's part of B, and of a draining warp
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t base = (raw_base + 1023u) & ~1023u;   // same offset in both CTAs
  unsigned char* gbase = smem_raw + (base - raw_base);
  const uint32_t tiles0 = base + STAGES * STAGE_BYTES;
  const uint32_t bar0 = tiles0 + 8 * TILE_BYTES;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto tfull_bar = [&](int i) { return bar0 + 8u * (2 * STAGES + i); };
  auto tempty_bar = [&](int i) { return bar0 + 8u * (2 * STAGES + 2 + i); };
  const uint32_t done_bar = bar0 + 8u * (2 * STAGES + 4);
  unsigned char* misc = gbase + STAGES * STAGE_BYTES + 8 * TILE_BYTES + kBars;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 4);
  int* tile_pre = reinterpret_cast<int*>(misc + 16);   // [E + 1]
  int* mtiles = tile_pre + (kMaxExperts + 1);          // [E]
  int* nrows = mtiles + kMaxExperts;                   // [E]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int NT = (a.N + TN - 1) / TN;
  const int KB = a.KB, splits = SPLIT ? a.splits : 1;
  // item -> tile, and the item's blocks of depth
  auto tile_of = [&](int item) { return SPLIT ? item / splits : item; };
  auto depth_of = [&](int item, int& from, int& to) {
    const int s = SPLIT ? item % splits : 0;
    from = SPLIT ? KB * s / splits : 0;
    to = SPLIT ? KB * (s + 1) / splits : KB;
    return s;
  };

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(tfull_bar(i), 1);
      mbar_init(tempty_bar(i), 2 * kDrainWarps);   // draining warps of both CTAs
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32((const void*)tmem_slot), TMEM_COLS);
    tmem_relinquish_pair();
  }
  pdl_trigger();
  pdl_wait();
  if (warp == 2) {
    const int per = (a.E + 31) / 32;
    const int e0 = lane * per;
    int sum = 0;
    for (int e = e0; e < min(a.E, e0 + per); ++e) {
      nrows[e] = min(max(a.n[e], 0), a.n_max);
      mtiles[e] = (nrows[e] + PM - 1) / PM;
      sum += mtiles[e] * NT;
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    int run = inc - sum;
    for (int e = e0; e < min(a.E, e0 + per); ++e) {
      tile_pre[e] = run;
      run += mtiles[e] * NT;
    }
    if (lane == 31) tile_pre[a.E] = inc;
  }
  tc_fence_before();
  cluster_sync_all();          // barriers of both CTAs initialised, TMEM allocated
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp < 4) {
    reg_dec<kRegsLoad>();
  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    if (lane == 0) {
      TileIter it{tile_pre, mtiles, a.E, NT, 0};
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      int e, mt, nt;
      for (int tile = pair; ok && it.decode(tile_of(tile), e, mt, nt); tile += npairs) {
        const int rowA = e * a.C + mt * PM + (int)rank * 128;
        const int rowB = e * a.N + nt * TN + (int)rank * COLS;
        int from, to;
        depth_of(tile, from, to);
        for (int kb = from; kb < to; ++kb) {
          if (*abort_flag || !mbar_wait(empty_bar(s), ph ^ 1u, a.err, a.limit_ns)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          const uint32_t sa = base + s * STAGE_BYTES;
          const uint32_t fb = full_bar(s) & kPeerBitMask;
          if (leader) mbar_arrive_expect_tx(full_bar(s), 2 * (A_BYTES + COLS * BK));
          // depth past K (a last block cut short) reads as zeros
          tma_load_2d_pair(sa, &tmA, fb, kb * BK, rowA);
          tma_load_2d_pair(sa + A_BYTES, &tmB, fb, kb * BK, rowB);
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader only)
    if (lane == 0 && leader) {
      TileIter it{tile_pre, mtiles, a.E, NT, 0};
      // kind::f8f6f4, D fp32, A and B e4m3 (0) with contiguous depth, M = 256, N = TN
      const uint32_t idesc = (1u << 4) | ((uint32_t)(TN >> 3) << 17) | ((uint32_t)(PM >> 4) << 24);
      int s = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = true;
      int e, mt, nt;
      for (int tile = pair; ok && it.decode(tile_of(tile), e, mt, nt); tile += npairs) {
        int from, to;
        depth_of(tile, from, to);
        for (int kb = from; kb < to; ++kb) {
          if (*abort_flag || !mbar_wait(tempty_bar(acc), aph ^ 1u, a.err, a.limit_ns) ||
              !mbar_wait(full_bar(s), ph, a.err, a.limit_ns)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = base + s * STAGE_BYTES;
#pragma unroll
          for (int kk = 0; kk < BK / 32; ++kk)
            tc_mma_f8_pair(tmem_base + acc * TN, desc_sw128(sa + kk * 32u, 16u, 1024u),
                           desc_sw128(sa + A_BYTES + kk * 32u, 16u, 1024u), idesc, kk != 0);
          tc_commit_pair(tfull_bar(acc), 0x3);
          tc_commit_pair(empty_bar(s), 0x3);
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
          acc ^= 1;
          if (acc == 0) aph ^= 1u;
        }
      }
      if (!ok) {
        tc_commit_pair(done_bar, 0x1);
        mbar_wait(done_bar, 0, a.err, a.limit_ns);
      }
    }
    __syncwarp();
  }
  } else {
    // ------------------------------------------------------------ drain (warps 4..11, both CTAs)
    reg_inc<kRegsDrain>();
    const int q = warp & 3;                        // TMEM lane quarter of this warp
    const int half = (warp - 4) >> 2;              // its half of the tile's columns
    const uint32_t tile0 = tiles0 + (warp - 4) * TILE_BYTES;
    TileIter it{tile_pre, mtiles, a.E, NT, 0};
    int e, mt, nt, acc = 0;
    uint32_t aph = 0;
    bool ok = true;
    for (int tile = pair; ok && it.decode(tile_of(tile), e, mt, nt); tile += npairs) {
      const int local = mt * PM + (int)rank * 128 + q * 32;
      const int nvalid = min(32, nrows[e] - local);
      const int64_t row0 = (int64_t)e * a.C + local;
      const int col0 = nt * TN + half * COLS;
      const int nb = col0 >> 7;
      const bool live = lane < nvalid && nb < a.NB;
      const float* xs = a.xs + (row0 + (live ? lane : 0)) * KB;
      const float* ws = a.ws + ((int64_t)e * a.NB + (live ? nb : 0)) * KB;
      int from, to;
      depth_of(tile, from, to);
      uint64_t sum[COLS / 2];                    // two columns per register pair
#pragma unroll
      for (int j = 0; j < COLS / 2; ++j) sum[j] = 0ull;
      auto scale = [&](int kb, float& x, float& w) {
        x = live && kb < to ? __ldg(xs + kb) : 0.f;
        w = live && kb < to ? __ldg(ws + kb) : 0.f;
      };
      // adds block kb; its scales were loaded four blocks ago, those of block kb + 4 are now
      auto drain = [&](int kb, float& x, float& w) -> bool {
        if (!warp_wait(abort_flag, tfull_bar(acc), aph, a.err, a.limit_ns)) return false;
        tc_fence_after();
        const float f = x * w;
        const uint64_t sc = pack_f32x2(f, f);
        scale(kb + 4, x, w);
        const uint32_t tm = tmem_base + ((uint32_t)(q * 32) << 16) + acc * TN + half * COLS;
        // two groups of 32 columns in flight; the last two are on their way while the first two
        // are added, and the buffer is handed back before those are added
        uint32_t r0[32], r1[32];
        auto add = [&](int c, const uint32_t (&r)[32]) {
#pragma unroll
          for (int j = 0; j < 16; ++j)         // two columns per instruction
            sum[c * 16 + j] = fma_f32x2(sc, pack_u32x2(r[2 * j], r[2 * j + 1]), sum[c * 16 + j]);
        };
        tmem_ld_32x32b_x32(tm, r0);            // (rows past the last one: garbage times 0, not stored)
        if (COLS > 32) tmem_ld_32x32b_x32(tm + 32, r1);
        tmem_ld_wait();
        if constexpr (COLS == 128) {
          add(0, r0);
          tmem_ld_32x32b_x32(tm + 64, r0);
          add(1, r1);
          tmem_ld_32x32b_x32(tm + 96, r1);
          tmem_ld_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (leader) mbar_arrive(tempty_bar(acc));
          else mbar_arrive_peer(mapa_shared(tempty_bar(acc), 0));
        }
        add(COLS == 128 ? 2 : 0, r0);
        if constexpr (COLS > 32) add(COLS == 128 ? 3 : 1, r1);
        acc ^= 1;
        if (acc == 0) aph ^= 1u;
        return true;
      };
      float x[4], w[4];
#pragma unroll
      for (int d = 0; d < 4; ++d) scale(from + d, x[d], w[d]);
      for (int kb = from; ok && kb < to; kb += 4)
#pragma unroll
        for (int d = 0; d < 4; ++d)
          if (ok && kb + d < to) ok = drain(kb + d, x[d], w[d]);
      if (SPLIT) {
        if (ok && lane < nvalid) {
          float* p = a.part + (((int64_t)depth_of(tile, from, to) * a.E + e) * a.rows + local + lane) * a.N;
#pragma unroll
          for (int j = 0; j < COLS / 4; ++j)
            if (col0 + j * 4 < a.N)            // N is a multiple of 8
              __stcg(reinterpret_cast<ulonglong2*>(p + col0 + j * 4), make_ulonglong2(sum[2 * j], sum[2 * j + 1]));
        }
      } else if (ok && nvalid > 0) {
        const bool whole = nvalid == 32 && COLS >= 64;      // by TMA, 64 columns at a time
#pragma unroll
        for (int b = 0; b < (COLS + 63) / 64; ++b) {
          const int col = col0 + b * 64;
          if (col < a.N) {
            if (whole) {
              if (lane == 0) bulk_wait_read0();
              __syncwarp();
            }
#pragma unroll
            for (int j = 0; j < (COLS < 64 ? COLS : 64) / 8; ++j) {
              uint32_t pk[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint64_t v = sum[b * 32 + j * 4 + i];
                pk[i] = pack_bf16x2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
              }
              if (whole)
                st_shared_v4(tile0 + lane * 128 + ((j ^ (lane & 7)) << 4), pk[0], pk[1], pk[2], pk[3]);
              else if (lane < nvalid && col + j * 8 < a.N)       // N is a multiple of 8
                *reinterpret_cast<uint4*>(a.y + (row0 + lane) * a.N + col + j * 8) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            }
            if (whole) {
              fence_async_smem();
              __syncwarp();
              if (lane == 0) {
                tma_store_2d_hint(&tmD, tile0, col, (int)row0, l2_policy_evict_first());
                bulk_commit();
              }
            }
          }
        }
      }
    }
    if (lane == 0) bulk_wait0();
    __syncwarp();
  }

  tc_fence_before();
  let_copies_land(abort_flag);
  __syncwarp();
  cluster_sync_all();          // no CTA leaves while its pair may still use its smem or TMEM
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

template <int TN, bool SPLIT>
cudaError_t launch(const CUtensorMap& tmA, const CUtensorMap& tmD, const Fp8Pair& p, const Fp8Args& a) {
  CUtensorMap tmB;
  if (!encode_2d_bytes(&tmB, a.wq, a.K, (uint64_t)a.E * a.N, BK, TN / 2)) return cudaErrorInvalidValue;
  auto kern = fp8_pair_kernel<SPLIT, TN>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(a.num_sms & ~1), dim3(kThreads), SMEM, a.st, tmA, tmB, tmD, p);
}

int64_t tiles(const Fp8Args& a, int TN) { return (int64_t)a.E * ((a.rows + PM - 1) / PM) * ((a.N + TN - 1) / TN); }

}  // namespace

int fp8_shares(const Fp8Args& a) {
  return tiles(a, 64) > a.num_sms / 2 ? 1 : split_count(a.E, a.rows, a.N, 64, (a.K + 127) / 128, kBlockUs, a.num_sms);
}

cudaError_t fp8_pair(const Fp8Args& a) {
  CUtensorMap tmA, tmD;
  const uint64_t rows = (uint64_t)a.E * (uint64_t)a.C;
  if (!encode_2d_bytes(&tmA, a.xq, a.K, rows, BK, 128) || !encode_2d(&tmD, a.y, a.N, rows, 64, 32))
    return cudaErrorInvalidValue;
  Fp8Pair p{};
  p.n = a.n;
  p.E = a.E;
  p.C = (int)a.C;
  p.n_max = (int)a.rows;
  p.K = a.K;
  p.N = a.N;
  p.KB = (a.K + 127) / 128;
  p.NB = (a.N + 127) / 128;
  p.xs = a.xs;
  p.ws = a.ws;
  p.y = static_cast<__nv_bfloat16*>(a.y);
  p.rows = (int)a.rows;
  p.part = a.part;
  p.err = a.err;
  p.limit_ns = a.limit_ns;
  // the narrowest tiles that fit on the pairs at once; only those can be few enough for shares
  const int pairs = a.num_sms / 2;
  if (tiles(a, 128) > pairs) return launch<256, false>(tmA, tmD, p, a);
  if (tiles(a, 64) > pairs) return launch<128, false>(tmA, tmD, p, a);
  p.splits = fp8_shares(a);
  if (p.splits == 1) return launch<64, false>(tmA, tmD, p, a);
  const cudaError_t e = launch<64, true>(tmA, tmD, p, a);
  return e != cudaSuccess ? e : split_join(a.part, a.y, true, a.n, a.E, a.rows, a.C, a.N, p.splits, a.num_sms, a.st);
}

}  // namespace moe
