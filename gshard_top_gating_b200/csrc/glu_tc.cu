// glu_tc.cu -- gated experts on 5th-generation tensor cores (tcgen05), bf16 in, fp32 accumulate.
//
// For each expert e, with n = the rows it holds, W13 = [Wg | Wu] [M, 2H] and W2 [H, M]:
//
//   up     g = x Wg, u = x Wu, h = f(g) * u      one kernel: both products, f and the product
//   down   y = h W2
//   dh     dh = dy W2^T, dg = dh * u * f'(g), du = dh * f(g)    one kernel
//   dx     dx = [dg | du] W13^T
//   dW     dW13 = x^T [dg | du], dW2 = h^T dy                   reduction over the n rows
//
// Every product runs on CTA pairs (cta_group::2): a 256 x 256 tile of the accumulator, CTA r
// of the pair holding rows [128r, 128r + 128) of A and columns [128r, 128r + 128) of B, and,
// in its TMEM, its 128 rows of all 256 columns.  In `up` the pair's first CTA loads 128
// columns of Wg and the second the same 128 columns of Wu: g and u of one element then lie
// in one TMEM lane, 128 columns apart, and the epilogue forms h in registers.
//
// The caller's rows (x, y, dy, dx) are [E, C, width] with any C; rows at or past n are
// neither read as data nor written.  Whole 32-row groups leave by TMA; the last group of an
// expert is stored row by row.  The internal rows (h, [g|u], [dg|du]) are [E, Cp, width]
// with Cp a multiple of 256, and an expert's rows past n up to a multiple of 64 are stored as
// zeros in training, since the weight gradients reduce over whole blocks of 64 rows.
//
// Roles per CTA: warp 0 loads (TMA), warp 1 issues MMAs (the pair's first CTA) and owns TMEM,
// warps 2..5 drain the accumulator, double buffered, while the next tile's products run; but
// in `up`, `dh` and, for few rows, `dW`, warps 2..9, half of the columns each.  With four warps
// `dh` outlasted its products (545 against 346 us for 8 x 2048 rows, M = 2048, H = 8192), as did
// `up` for small M.  Every wait is bounded.
#include <type_traits>

#include "common.cuh"
#include "glu.cuh"
#include "internal.h"
#include "tc_tile.cuh"

namespace moe {

namespace {

constexpr int BK = 64;                 // depth of a stage
constexpr int PM = 256, PN = 256;      // pair tile
enum { kUp = 0, kUpSave = 1, kDown = 2, kDh = 3, kDx = 4, kDw = 5, kDwFew = 6 };
constexpr int epi_warps(int mode) { return mode == kDown || mode == kDx || mode == kDw ? 4 : 8; }
constexpr int threads(int mode) { return 64 + 32 * epi_warps(mode); }
constexpr uint32_t A_BYTES = 128 * BK * 2;            // 16 KB: 128 rows of A
constexpr uint32_t B_BYTES = 128 * BK * 2;            // 16 KB: 128 columns of B
constexpr uint32_t STAGE_BYTES = A_BYTES + B_BYTES;   // per CTA
constexpr uint32_t TMEM_COLS = 2 * PN;                // double-buffered accumulator
constexpr uint32_t TILE_BYTES = 4096;                 // a 32-row x 64-column bf16 store tile
constexpr uint32_t kPeerBitMask = 0xFEFFFFFFu;        // shared::cluster address -> the pair's first CTA

// Shared memory of an epilogue warp: tiles of 32 rows x 32 columns for h; for h, g and u; two
// buffers of them for g and u, which dg and du leave through; else one of 32 x 64.
constexpr uint32_t NARROW_BYTES = 2048;
constexpr uint32_t epi_bytes(int mode) {
  return mode == kUp ? NARROW_BYTES : mode == kUpSave ? 3 * NARROW_BYTES : mode == kDh ? 4 * NARROW_BYTES : TILE_BYTES;
}
constexpr int stages(int mode) { return mode == kUpSave ? 5 : mode == kDh ? 4 : 6; }
constexpr uint32_t kBars = 512;
constexpr size_t smem_bytes(int mode) {
  // alignment slack, stages, store tiles, barriers, misc, tile tables (kDw: the counts alone)
  return 1024 + (size_t)stages(mode) * STAGE_BYTES + epi_warps(mode) * epi_bytes(mode) + kBars + 16 +
         4 * (mode >= kDw ? kMaxExperts : 3 * kMaxExperts + 1);
}
// A CTA owns its SM (see the expert GEMMs of ffn_tc.cu): no other TMEM user fits beside it.
constexpr bool owns_sm(int mode) { return smem_bytes(mode) <= 227 * 1024 && smem_bytes(mode) + 81 * 1024 > 228 * 1024; }
static_assert(owns_sm(kUp) && owns_sm(kUpSave) && owns_sm(kDown) && owns_sm(kDh) && owns_sm(kDw) && owns_sm(kDwFew),
              "shared memory per CTA");

struct PairArgs {
  const int32_t* n;      // [E] rows per expert, clamped to [0, C]
  int E, C;
  int64_t Ca, Cd;        // rows per expert of A and of the output
  int K, N;              // depth and output columns (kUp: H)
  __nv_bfloat16* D;      // output, for the row-by-row stores (kDown, kDx)
  int splits, rows;      // kDown, kDx: shares of the depth (split.cu); most rows an expert holds
  float* part;           // splits > 1: [splits][E, rows, N] fp32 sums instead of D
  const uint4 *x, *dy;   // kDh, if tx: the rows whose last, partial blocks go to tx and tdy
  uint4 *tx, *tdy;
  unsigned* err;
  uint64_t limit_ns;
};

// One weight gradient, D[e] = A[e, :n]^T B[e, :n] ([P, Q] per expert).
struct DwProduct {
  CUtensorMap tmA, tmB, tmD, tmAt, tmBt;
  int64_t Ca, Cb;        // rows per expert of A and of B
  int P, Q;
  int tailA, tailB;      // the last, partial 64-row block comes from the tail maps
};
struct DwArgs {
  DwProduct d[2];
  int products;          // 1 or 2, the tiles of d[1] after those of d[0]
  const int32_t* n;
  int E, C;
  int store_zero;        // experts without rows get zeros (else keep what they hold)
  unsigned* err;
  uint64_t limit_ns;
};

template <typename A>
__device__ __forceinline__ int rows_of(const A& a, int e) { return min(max(a.n[e], 0), a.C); }

// idesc: kind::f16, D fp32, A and B bf16, M = 256, N = 256; a_mn / b_mn: operand's rows or
// columns contiguous instead of its depth.
__device__ __forceinline__ uint32_t idesc_pair(bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(PN >> 3) << 17) | ((uint32_t)(PM >> 4) << 24);
}

// 32 packed bf16 (16 words) of this lane's row into a 128-byte-swizzled store tile, columns
// [32 half, 32 half + 32).
__device__ __forceinline__ void put_half(uint32_t tile, int lane, int half, const uint32_t (&pk)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    st_shared_v4(tile + lane * 128 + (((half * 4 + j) ^ (lane & 7)) << 4), pk[4 * j], pk[4 * j + 1], pk[4 * j + 2],
                 pk[4 * j + 3]);
}
// Plain output of one warp: 32 rows x WIDTH columns from column col0 (N columns, a multiple
// of 64), nvalid of the rows kept (and row stores where that is fewer than 32).
template <int WIDTH>
__device__ __forceinline__ void store_plain(const CUtensorMap* tmD, uint32_t tmem, uint32_t tile, int64_t row0, int col0,
                                            int N, int nvalid, bool zero, __nv_bfloat16* D, int lane) {
#pragma unroll 1
  for (int b = 0; b < WIDTH / 64; ++b) {
    const int col = col0 + b * 64;
    if (col >= N) return;
    if (nvalid == 32) {
      if (lane == 0) bulk_wait_read0();
      __syncwarp();
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t r[32], pk[16];
      if (zero) {
#pragma unroll
        for (int j = 0; j < 16; ++j) pk[j] = 0u;
      } else {
        tmem_ld_32x32b_x32(tmem + b * 64 + half * 32, r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) pk[j] = pack_bf16x2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
      }
      if (nvalid == 32) {
        put_half(tile, lane, half, pk);
      } else if (lane < nvalid) {
        uint4* p = reinterpret_cast<uint4*>(D + (row0 + lane) * N + col + half * 32);
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] = make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
      }
    }
    if (nvalid == 32) {
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d_hint(tmD, tile, col, (int)row0, l2_policy_evict_first());
        bulk_commit();
      }
    }
  }
}

// The fp32 sums of one warp's rows (this lane's at p, N columns from column col0).
__device__ __forceinline__ void store_sums(uint32_t tmem, float* p, int col0, int N, bool live) {
#pragma unroll 1
  for (int b = 0; b < PN / 32 && col0 + b * 32 < N; ++b) {
    uint32_t r[32];
    tmem_ld_32x32b_x32(tmem + b * 32, r);
    tmem_ld_wait();
    if (live) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        __stcg(reinterpret_cast<uint4*>(p + col0 + b * 32) + j, make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]));
    }
  }
}

// 32 packed bf16 of this lane's row in a 32-column tile with 64-byte swizzle.
__device__ __forceinline__ void put_narrow(uint32_t tile, int lane, const uint32_t (&pk)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    st_shared_v4(tile + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4), pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
}
__device__ __forceinline__ void get_narrow(uint32_t tile, int lane, uint32_t (&pk)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 v = ld_shared_v4(tile + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4));
    pk[4 * j] = v.x;
    pk[4 * j + 1] = v.y;
    pk[4 * j + 2] = v.z;
    pk[4 * j + 3] = v.w;
  }
}

// g and u of one warp's 32 rows x 64 elements (accumulator columns tmem and tmem + 128) -> h
// (tmD), and with SAVE g and u as well (tmD2, [.., 2H]: g at column n, u at H + n); rows past
// nvalid become zeros with SAVE.
template <int FN, bool SAVE>
__device__ __forceinline__ void store_up(const CUtensorMap* tmD, const CUtensorMap* tmD2, uint32_t tmem, uint32_t tile,
                                         int row0, int col0, int H, int nvalid, int lane) {
  const bool live = !SAVE || lane < nvalid;
  if (col0 >= H) return;                         // H is a multiple of 64
#pragma unroll 1
  for (int half = 0; half < 2; ++half) {
    const int col = col0 + half * 32;
    uint32_t g[32], u[32], pk[16];
    tmem_ld_32x32b_x32(tmem + half * 32, g);
    tmem_ld_32x32b_x32(tmem + 128 + half * 32, u);
    if (lane == 0) bulk_wait_read0();
    __syncwarp();
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float h0 = glu_f<FN, true>(__uint_as_float(g[2 * j])) * __uint_as_float(u[2 * j]);
      const float h1 = glu_f<FN, true>(__uint_as_float(g[2 * j + 1])) * __uint_as_float(u[2 * j + 1]);
      pk[j] = live ? pack_bf16x2(h0, h1) : 0u;
    }
    put_narrow(tile, lane, pk);
    if (SAVE) {
      pack_gu(g, live, pk);
      put_narrow(tile + NARROW_BYTES, lane, pk);
      pack_gu(u, live, pk);
      put_narrow(tile + 2 * NARROW_BYTES, lane, pk);
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d_hint(tmD, tile, col, row0, l2_policy_evict_first());
      if (SAVE) {
        tma_store_2d_hint(tmD2, tile + NARROW_BYTES, col, row0, l2_policy_evict_first());
        tma_store_2d_hint(tmD2, tile + 2 * NARROW_BYTES, H + col, row0, l2_policy_evict_first());
      }
      bulk_commit();
    }
  }
}

// g and u of 32 columns from column col, by TMA into a pair of narrow tiles.
__device__ __forceinline__ void load_gu(const CUtensorMap* tmGU, uint32_t tile, uint32_t bar, int row0, int col, int H) {
  mbar_arrive_expect_tx(bar, 2 * NARROW_BYTES);
  tma_load_2d(tile, tmGU, bar, col, row0);
  tma_load_2d(tile + NARROW_BYTES, tmGU, bar, H + col, row0);
}

// The last, partial block of 64 rows of each expert of x and dy, zero-filled, to tx and tdy:
// what the weight gradients read instead of the caller's rows past the last one.  Warp `gw` of
// `warps` takes pieces of 128 x 16 bytes.
__device__ __forceinline__ void copy_tails(const PairArgs& a, const int* nrows, int gw, int warps, int lane) {
  const int row16 = a.K / 8;             // dh's depth is M, the rows' width: a multiple of 64
  const int per = BK * row16 / 128, total = 2 * a.E * per;
  for (int c = gw; c < total; c += warps) {
    const int b = c / per, e = b >> 1, at = (c - b * per) * 128 + lane;
    const int n = nrows[e], rem = n & (BK - 1);
    if (rem == 0) continue;
    const uint4* src = (b & 1 ? a.dy : a.x) + (e * a.Ca + n - rem) * row16;
    uint4* dst = (b & 1 ? a.tdy : a.tx) + (int64_t)e * BK * row16;
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = at + 32 * j < rem * row16 ? src[at + 32 * j] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int j = 0; j < 4; ++j) dst[at + 32 * j] = v[j];
  }
}

// MODE kUp, kUpSave, kDown, kDh, kDx.  tmD2: kUpSave the [g|u] output, kDh the [g|u] input.
template <int MODE, int FN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(threads(MODE), 1)
    glu_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmD, const __grid_constant__ CUtensorMap tmD2,
                    const PairArgs a) {
  constexpr int STAGES = stages(MODE);
  constexpr bool UP = MODE == kUp || MODE == kUpSave;
  constexpr bool BKM = MODE == kDh || MODE == kDx;     // B's depth is contiguous
  constexpr int COLS = UP ? 128 : PN;                  // output columns of a tile
  constexpr bool SPLIT = MODE == kDown || MODE == kDx; // a tile's depth may be cut into shares
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t base = (raw_base + 1023u) & ~1023u;   // same offset in both CTAs
  unsigned char* gbase = smem_raw + (base - raw_base);
  const uint32_t tiles0 = base + STAGES * STAGE_BYTES;
  const uint32_t bar0 = tiles0 + epi_warps(MODE) * epi_bytes(MODE);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto tfull_bar = [&](int i) { return bar0 + 8u * (2 * STAGES + i); };
  auto tempty_bar = [&](int i) { return bar0 + 8u * (2 * STAGES + 2 + i); };
  const uint32_t done_bar = bar0 + 8u * (2 * STAGES + 4);
  auto gu_bar = [&](int w, int i) { return bar0 + 8u * (2 * STAGES + 5 + 2 * w + i); };
  unsigned char* misc = gbase + STAGES * STAGE_BYTES + epi_warps(MODE) * epi_bytes(MODE) + kBars;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 4);
  int* tile_pre = reinterpret_cast<int*>(misc + 16);   // [E + 1]
  int* mtiles = tile_pre + (kMaxExperts + 1);          // [E]
  int* nrows = mtiles + kMaxExperts;                   // [E]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int NT = (a.N + COLS - 1) / COLS;
  const int KB = a.K / BK;
  const int splits = SPLIT ? a.splits : 1;
  // item -> tile, and the item's blocks of depth
  auto tile_of = [&](int item) { return SPLIT && splits > 1 ? item / splits : item; };
  auto depth_of = [&](int item, int& from, int& to) {
    const int s = SPLIT && splits > 1 ? item % splits : 0;
    from = s == 0 ? 0 : KB * s / splits;
    to = s + 1 == splits ? KB : KB * (s + 1) / splits;
    return s;
  };

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(tfull_bar(i), 1);
      mbar_init(tempty_bar(i), 2 * epi_warps(MODE));       // epilogue warps of both CTAs
    }
    mbar_init(done_bar, 1);
    if (MODE == kDh)
      for (int w = 0; w < 8; ++w)
        for (int i = 0; i < 2; ++i) mbar_init(gu_bar(w, i), 1);
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
  pdl_wait();                          // the producing kernel's rows and counts are complete
  if (warp == 2) {
    const int per = (a.E + 31) / 32;
    const int e0 = lane * per;
    int sum = 0;
    for (int e = e0; e < min(a.E, e0 + per); ++e) {
      nrows[e] = rows_of(a, e);
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

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    if (lane == 0) {
      TileIter it{tile_pre, mtiles, a.E, NT, 0};
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      int e, mt, nt;
      for (int tile = pair; ok && it.decode(tile_of(tile), e, mt, nt); tile += npairs) {
        const int rowA = (int)(e * a.Ca) + mt * PM + (int)rank * 128;
        // first column of this CTA's half of B: the same 128 elements of Wg or of Wu, or 128
        // of the tile's 256 columns
        const int colB = UP ? (int)rank * a.N + nt * COLS : nt * COLS + (int)rank * 128;
        int from, to;
        depth_of(tile, from, to);
        for (int kb = from; kb < to; ++kb) {
          if (*abort_flag || !mbar_wait(empty_bar(s), ph ^ 1u, a.err, a.limit_ns)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          const uint32_t sa = base + s * STAGE_BYTES;
          const uint32_t fb = full_bar(s) & kPeerBitMask;     // the leader's full barrier
          if (leader) mbar_arrive_expect_tx(full_bar(s), 2 * STAGE_BYTES);
          tma_load_2d_pair(sa, &tmA, fb, kb * BK, rowA);
          if (BKM) {
            tma_load_2d_pair(sa + A_BYTES, &tmB, fb, kb * BK, e * a.N + colB);
          } else {
#pragma unroll
            for (int j = 0; j < 2; ++j)
              tma_load_2d_pair(sa + A_BYTES + j * 8192u, &tmB, fb, colB + j * 64, e * a.K + kb * BK);
          }
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
      const uint32_t idesc = idesc_pair(false, !BKM);
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      int e, mt, nt, i = 0;
      for (int tile = pair; ok && it.decode(tile_of(tile), e, mt, nt); tile += npairs, ++i) {
        const int acc = i & 1;
        const uint32_t aph = (i >> 1) & 1;
        if (*abort_flag || !mbar_wait(tempty_bar(acc), aph ^ 1u, a.err, a.limit_ns)) {
          *abort_flag = 1;
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * PN;
        int from, to;
        depth_of(tile, from, to);
        for (int kb = from; kb < to; ++kb) {
          if (*abort_flag || !mbar_wait(full_bar(s), ph, a.err, a.limit_ns)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = base + s * STAGE_BYTES;
          const uint32_t sb = sa + A_BYTES;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk) {
            const uint64_t ad = desc_sw128(sa + kk * 32u, 16u, 1024u);
            const uint64_t bd = BKM ? desc_sw128(sb + kk * 32u, 16u, 1024u)
                                    : desc_sw128(sb + kk * 2048u, 8192u, 1024u);
            tc_mma_f16_pair(d_tmem, ad, bd, idesc, kb != from || kk != 0);
          }
          tc_commit_pair(empty_bar(s), 0x3);
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (ok) tc_commit_pair(tfull_bar(acc), 0x3);
      }
      if (!ok) {
        tc_commit_pair(done_bar, 0x1);
        mbar_wait(done_bar, 0, a.err, a.limit_ns);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue (from warp 2, both CTAs)
    const int q = warp & 3;
    const int part = (warp - 2) >> 2;            // kUp, kDh: which half of the tile's columns
    const uint32_t tile0 = tiles0 + (warp - 2) * epi_bytes(MODE);
    TileIter it{tile_pre, mtiles, a.E, NT, 0};
    int e, mt, nt, i = 0;
    uint32_t gph = 0;            // kDh: phase bits of the two (g, u) buffers
    if (MODE == kDh && a.tx)     // while the first tile's products run
      copy_tails(a, nrows, blockIdx.x * epi_warps(MODE) + warp - 2, gridDim.x * epi_warps(MODE), lane);
    for (int tile = pair; it.decode(tile_of(tile), e, mt, nt); tile += npairs, ++i) {
      const int acc = i & 1;
      const uint32_t aph = (i >> 1) & 1;
      const int local = mt * PM + (int)rank * 128 + q * 32;     // row within the expert
      const int64_t row0 = e * a.Cd + local;
      const int nvalid = min(32, nrows[e] - local);
      const int col0 = nt * COLS + part * (COLS / 2);
      if (MODE == kDh && nvalid > 0 && col0 < a.N && lane == 0) {
        bulk_wait_read0();       // the previous tile's stores have read their buffers
        load_gu(&tmD2, tile0, gu_bar(warp - 2, 0), (int)row0, col0, a.N);
        // the other columns into L2 while the products run
        for (int b = 1; b < 4 && col0 + b * 32 < a.N; ++b) {
          tma_prefetch_l2_2d(&tmD2, col0 + b * 32, (int)row0);
          tma_prefetch_l2_2d(&tmD2, a.N + col0 + b * 32, (int)row0);
        }
      }
      if (!warp_wait(abort_flag, tfull_bar(acc), aph, a.err, a.limit_ns)) {
        if (MODE == kDh && nvalid > 0 && col0 < a.N) mbar_wait(gu_bar(warp - 2, 0), gph & 1u, a.err, a.limit_ns);
        break;
      }
      tc_fence_after();
      const uint32_t tm = tmem_base + ((uint32_t)(q * 32) << 16) + acc * PN;
      if constexpr (UP) {
        if (MODE == kUpSave ? local < ((nrows[e] + BK - 1) & ~(BK - 1)) : nvalid > 0)
          store_up<FN, MODE == kUpSave>(&tmD, &tmD2, tm + part * 64, tile0, (int)row0, col0, a.N, nvalid, lane);
      } else if constexpr (MODE == kDh) {
        bool ok = true;
        const int nb = max(0, min(4, (a.N - col0) / 32));      // N is a multiple of 64
        if (nvalid > 0) {
#pragma unroll 1
          for (int b = 0; b < nb; ++b) {
            const uint32_t buf = tile0 + (b & 1) * 2 * NARROW_BYTES;
            if (b + 1 < nb && lane == 0) {
              // the other buffer's stores (columns b - 1) have left; bring in the next ones
              bulk_wait_read0();
              load_gu(&tmD2, tile0 + ((b + 1) & 1) * 2 * NARROW_BYTES, gu_bar(warp - 2, (b + 1) & 1), (int)row0,
                      col0 + (b + 1) * 32, a.N);
            }
            __syncwarp();
            uint32_t r[32], pg[16], pu[16];
            tmem_ld_32x32b_x32(tm + part * 128 + b * 32, r);
            ok = ok && mbar_wait(gu_bar(warp - 2, b & 1), (gph >> (b & 1)) & 1u, a.err, a.limit_ns);
            gph ^= 1u << (b & 1);
            get_narrow(buf, lane, pg);
            get_narrow(buf + NARROW_BYTES, lane, pu);
            tmem_ld_wait();
            const bool fg = gu_is_fine(pg[0]), fu = gu_is_fine(pu[0]), live = lane < nvalid;
            auto gradients = [&](auto all_fine) {
              constexpr bool FINE = decltype(all_fine)::value;
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float d0 = __uint_as_float(r[2 * j]), d1 = __uint_as_float(r[2 * j + 1]);
                float g0, g1, u0, u1, f0, df0, f1, df1;
                unpack_gu<FINE>(pg[j], fg, g0, g1);
                unpack_gu<FINE>(pu[j], fu, u0, u1);
                glu_f_df<FN, true>(g0, f0, df0);
                glu_f_df<FN, true>(g1, f1, df1);
                pg[j] = live ? pack_bf16x2(d0 * u0 * df0, d1 * u1 * df1) : 0u;
                pu[j] = live ? pack_bf16x2(d0 * f0, d1 * f1) : 0u;
              }
            };
            if (__all_sync(0xffffffffu, (fg && fu) || !live)) gradients(std::true_type{});
            else gradients(std::false_type{});
            put_narrow(buf, lane, pg);
            put_narrow(buf + NARROW_BYTES, lane, pu);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d_hint(&tmD, buf, col0 + b * 32, (int)row0, l2_policy_evict_first());
              tma_store_2d_hint(&tmD, buf + NARROW_BYTES, a.N + col0 + b * 32, (int)row0, l2_policy_evict_first());
              bulk_commit();
            }
          }
        } else if (nb > 0 && local < ((nrows[e] + BK - 1) & ~(BK - 1))) {
          // rows past the last one, up to a multiple of 64: zeros, so that the block that holds
          // it reduces over nothing else
          if (lane == 0) bulk_wait_read0();
          __syncwarp();
          const uint32_t z[16] = {};
          put_narrow(tile0, lane, z);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            for (int b = 0; b < nb; ++b) {
              tma_store_2d_hint(&tmD, tile0, col0 + b * 32, (int)row0, l2_policy_evict_first());
              tma_store_2d_hint(&tmD, tile0, a.N + col0 + b * 32, (int)row0, l2_policy_evict_first());
            }
            bulk_commit();
          }
        }
        if (!ok) *abort_flag = 1;
      } else {
        if (SPLIT && splits > 1) {
          int from, to;
          const int s = depth_of(tile, from, to);
          if (nvalid > 0)
            store_sums(tm, a.part + (((int64_t)s * a.E + e) * a.rows + local + lane) * a.N, col0, a.N, lane < nvalid);
        } else if (nvalid > 0) store_plain<PN>(&tmD, tm, tile0, row0, col0, a.N, nvalid, false, a.D, lane);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (leader) mbar_arrive(tempty_bar(acc));
        else mbar_arrive_peer(mapa_shared(tempty_bar(acc), 0));
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

// Weight gradients D[e] = A[e, :n]^T B[e, :n]: both operands with their rows as the depth.
// Rows n .. ceil64(n) - 1 of an operand hold zeros, or its last, partial block is read from a
// tail copy ([E, 64, width], zero-filled; tailA / tailB).  dW2 and dW13 go as one launch, so
// that the second's tiles fill the first's last wave and a step has a launch less (3 x 361 rows,
// M = 64, H = 1664: the step 60 -> 53 us, with the tails copied by `dh`).
template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(threads(MODE), 1)
    glu_dw_kernel(const __grid_constant__ DwArgs a) {
  constexpr int STAGES = stages(MODE);
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t base = (raw_base + 1023u) & ~1023u;
  unsigned char* gbase = smem_raw + (base - raw_base);
  const uint32_t tiles0 = base + STAGES * STAGE_BYTES;
  const uint32_t bar0 = tiles0 + epi_warps(MODE) * TILE_BYTES;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto tfull_bar = [&](int i) { return bar0 + 8u * (2 * STAGES + i); };
  auto tempty_bar = [&](int i) { return bar0 + 8u * (2 * STAGES + 2 + i); };
  const uint32_t done_bar = bar0 + 8u * (2 * STAGES + 4);
  unsigned char* misc = gbase + STAGES * STAGE_BYTES + epi_warps(MODE) * TILE_BYTES + kBars;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 4);
  int* nrows = reinterpret_cast<int*>(misc + 16);      // [E]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int QT0 = (a.d[0].Q + PN - 1) / PN, QT1 = (a.d[1].Q + PN - 1) / PN;
  const int per0 = (a.d[0].P + PM - 1) / PM * QT0, per1 = (a.d[1].P + PM - 1) / PM * QT1;
  const int first1 = a.E * per0, total = first1 + (a.products > 1 ? a.E * per1 : 0);
  // item -> product, expert and tile
  auto decode = [&](int item, int& e, int& pt, int& qt) -> const DwProduct& {
    const bool second = item >= first1;
    const int tile = second ? item - first1 : item, per = second ? per1 : per0, QT = second ? QT1 : QT0;
    e = tile / per;
    const int r = tile - e * per;
    pt = r / QT;
    qt = r - pt * QT;
    return a.d[second];
  };

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(tfull_bar(i), 1);
      mbar_init(tempty_bar(i), 2 * epi_warps(MODE));
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_desc(&a.d[0].tmA);
    tma_prefetch_desc(&a.d[0].tmB);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32((const void*)tmem_slot), TMEM_COLS);
    tmem_relinquish_pair();
  }
  pdl_trigger();
  pdl_wait();
  if (warp == 2)
    for (int e = lane; e < a.E; e += 32) nrows[e] = rows_of(a, e);
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = pair; ok && tile < total; tile += npairs) {
        int e, pt, qt;
        const DwProduct& d = decode(tile, e, pt, qt);
        const int KB = (nrows[e] + BK - 1) / BK;
        const bool part = (nrows[e] % BK) != 0;
        const int colA = pt * PM + (int)rank * 128, colB = qt * PN + (int)rank * 128;
        for (int kb = 0; kb < KB; ++kb) {
          if (*abort_flag || !mbar_wait(empty_bar(s), ph ^ 1u, a.err, a.limit_ns)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          const uint32_t sa = base + s * STAGE_BYTES;
          const uint32_t fb = full_bar(s) & kPeerBitMask;
          if (leader) mbar_arrive_expect_tx(full_bar(s), 2 * STAGE_BYTES);
          const bool last = part && kb == KB - 1;
          const bool ta = last && d.tailA, tb = last && d.tailB;
          const int rowA = ta ? e * BK : (int)(e * d.Ca) + kb * BK;
          const int rowB = tb ? e * BK : (int)(e * d.Cb) + kb * BK;
          // columns past P or Q (a last tile cut short) read as zeros
#pragma unroll
          for (int j = 0; j < 2; ++j) tma_load_2d_pair(sa + j * 8192u, ta ? &d.tmAt : &d.tmA, fb, colA + j * 64, rowA);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            tma_load_2d_pair(sa + A_BYTES + j * 8192u, tb ? &d.tmBt : &d.tmB, fb, colB + j * 64, rowB);
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      const uint32_t idesc = idesc_pair(true, true);
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      int i = 0;
      for (int tile = pair; ok && tile < total; tile += npairs) {
        const int KB = (nrows[tile >= first1 ? (tile - first1) / per1 : tile / per0] + BK - 1) / BK;
        if (KB == 0) continue;                  // zero tile: the epilogues store zeros
        const int acc = i & 1;
        const uint32_t aph = (i >> 1) & 1;
        ++i;
        if (*abort_flag || !mbar_wait(tempty_bar(acc), aph ^ 1u, a.err, a.limit_ns)) {
          *abort_flag = 1;
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * PN;
        for (int kb = 0; kb < KB; ++kb) {
          if (*abort_flag || !mbar_wait(full_bar(s), ph, a.err, a.limit_ns)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = base + s * STAGE_BYTES;
          const uint32_t sb = sa + A_BYTES;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk) {
            const uint64_t ad = desc_sw128(sa + kk * 2048u, 8192u, 1024u);
            const uint64_t bd = desc_sw128(sb + kk * 2048u, 8192u, 1024u);
            tc_mma_f16_pair(d_tmem, ad, bd, idesc, (kb | kk) != 0);
          }
          tc_commit_pair(empty_bar(s), 0x3);
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (ok) tc_commit_pair(tfull_bar(acc), 0x3);
      }
      if (!ok) {
        tc_commit_pair(done_bar, 0x1);
        mbar_wait(done_bar, 0, a.err, a.limit_ns);
      }
    }
    __syncwarp();
  } else {
    constexpr int WIDTH = PN * 4 / epi_warps(MODE);      // columns of a warp
    const int q = warp & 3, part = (warp - 2) >> 2;      // its 32 rows, and columns
    const uint32_t tile0 = tiles0 + (warp - 2) * TILE_BYTES;
    int i = 0;
    for (int tile = pair; tile < total; tile += npairs) {
      int e, pt, qt;
      const DwProduct& d = decode(tile, e, pt, qt);
      const bool zero = nrows[e] == 0;
      const int prow = pt * PM + (int)rank * 128 + q * 32;     // P is a multiple of 64: 32 rows or none
      int acc = 0;
      if (!zero) {
        acc = i & 1;
        const uint32_t aph = (i >> 1) & 1;
        ++i;
        if (!warp_wait(abort_flag, tfull_bar(acc), aph, a.err, a.limit_ns)) break;
        tc_fence_after();
      }
      if (prow < d.P && (!zero || a.store_zero))
        store_plain<WIDTH>(&d.tmD, tmem_base + ((uint32_t)(q * 32) << 16) + acc * PN + part * WIDTH, tile0,
                         (int64_t)e * d.P + prow, qt * PN + part * WIDTH, d.Q, 32, zero, nullptr, lane);
      if (!zero) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (leader) mbar_arrive(tempty_bar(acc));
          else mbar_arrive_peer(mapa_shared(tempty_bar(acc), 0));
        }
      }
    }
    if (lane == 0) bulk_wait0();
    __syncwarp();
  }

  tc_fence_before();
  let_copies_land(abort_flag);
  __syncwarp();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

template <int MODE, int FN>
cudaError_t launch_pair(const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap& tmD, const CUtensorMap& tmD2,
                        const PairArgs& p, const GluArgs& a) {
  auto kern = glu_pair_kernel<MODE, FN>;
  const size_t smem = smem_bytes(MODE);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(a.num_sms & ~1), dim3(threads(MODE)), smem, a.st, tmA, tmB, tmD, tmD2, p);
}

template <int MODE>
cudaError_t launch_fn(const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap& tmD, const CUtensorMap& tmD2,
                      const PairArgs& p, const GluArgs& a) {
  if (a.fn == kGluSilu) return launch_pair<MODE, kGluSilu>(tmA, tmB, tmD, tmD2, p, a);
  if (a.fn == kGluGelu) return launch_pair<MODE, kGluGelu>(tmA, tmB, tmD, tmD2, p, a);
  return launch_pair<MODE, kGluRelu>(tmA, tmB, tmD, tmD2, p, a);
}

PairArgs pair_args(const GluArgs& a) {
  PairArgs p{};
  p.n = a.n;
  p.E = a.E;
  p.C = (int)a.rows;      // no expert holds more
  p.err = a.err;
  p.limit_ns = a.limit_ns;
  return p;
}

// kDown, kDx: with too few tiles for the device, in shares of the depth.
constexpr double kBlockUs = 0.28;      // 256 x 256 x 64 on a pair
int shares_of(const GluArgs& a, int N, int K) {
  return split_count(a.E, a.rows, N, PN, K / BK, kBlockUs, a.num_sms);
}
template <int MODE>
cudaError_t launch_split(const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap& tmD, PairArgs p,
                         const GluArgs& a, void* out) {
  p.splits = shares_of(a, p.N, p.K);
  p.rows = (int)a.rows;
  p.part = a.part;
  const cudaError_t e = launch_pair<MODE, kGluSilu>(tmA, tmB, tmD, tmD, p, a);
  if (e != cudaSuccess || p.splits == 1) return e;
  return split_join(a.part, out, true, a.n, a.E, a.rows, a.C, p.N, p.splits, a.num_sms, a.st);
}

uint64_t rows(int E, int64_t per) { return (uint64_t)E * (uint64_t)per; }

bool dw_product(DwProduct* d, const GluArgs& a, const void* A, int64_t Ca, int P, const void* At, const void* B, int64_t Cb,
                int Q, const void* Bt, void* D) {
  d->Ca = Ca;
  d->Cb = Cb;
  d->P = P;
  d->Q = Q;
  d->tailA = At != nullptr;
  d->tailB = Bt != nullptr;
  return encode_2d(&d->tmA, A, P, rows(a.E, Ca), 64, BK) && encode_2d(&d->tmB, B, Q, rows(a.E, Cb), 64, BK) &&
         encode_2d(&d->tmD, D, Q, rows(a.E, P), 64, 32) &&
         encode_2d(&d->tmAt, At ? At : A, P, At ? rows(a.E, BK) : rows(a.E, Ca), 64, BK) &&
         encode_2d(&d->tmBt, Bt ? Bt : B, Q, Bt ? rows(a.E, BK) : rows(a.E, Cb), 64, BK);
}

bool dw2_product(DwProduct* d, const GluArgs& a) {
  return dw_product(d, a, a.h, a.Cp, a.H, nullptr, a.dy, a.C, a.M, a.tdy, a.dW2);
}

bool dw13_product(DwProduct* d, const GluArgs& a) {
  return dw_product(d, a, a.x, a.C, a.M, a.tx, a.dgu, a.Cp, 2 * a.H, nullptr, a.dW13);
}

cudaError_t launch_dw(const GluArgs& a, DwArgs& g, int products) {
  g.products = products;
  if (products == 1) g.d[1] = g.d[0];
  g.n = a.n;
  g.E = a.E;
  g.C = (int)a.rows;      // no expert holds more
  g.store_zero = !a.skip_empty;
  g.err = a.err;
  g.limit_ns = a.limit_ns;
  // Up to 8 blocks of 64 rows a tile's products end before four warps have drained the last one
  // (2.3 us): eight warps (25 x 18 rows, M = 768, H = 3776: 106 -> 89 us; 683 rows: equal).  Past
  // that eight cost the products more than they gain (step of 10 x 760 rows: 980 -> 1011 us).
  const bool few = a.rows <= 8 * BK;
  auto kern = few ? glu_dw_kernel<kDwFew> : glu_dw_kernel<kDw>;
  const size_t smem = few ? smem_bytes(kDwFew) : smem_bytes(kDw);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(a.num_sms & ~1), dim3(few ? threads(kDwFew) : threads(kDw)), smem, a.st, g);
}

}  // namespace

int glu_down_shares_bf16(const GluArgs& a) { return shares_of(a, a.M, a.H); }
int glu_dx_shares_bf16(const GluArgs& a) { return shares_of(a, a.M, 2 * a.H); }

cudaError_t glu_up_bf16(const GluArgs& a) {
  CUtensorMap tmA, tmB, tmD, tmD2;
  if (!encode_2d(&tmA, a.x, a.M, rows(a.E, a.C), BK, 128) ||
      !encode_2d(&tmB, a.W13, 2 * (uint64_t)a.H, rows(a.E, a.M), 64, BK) ||
      !encode_2d_narrow(&tmD, a.h, a.H, rows(a.E, a.Cp), 32) ||
      !encode_2d_narrow(&tmD2, a.gu ? a.gu : a.h, a.gu ? 2 * (uint64_t)a.H : a.H, rows(a.E, a.Cp), 32))
    return cudaErrorInvalidValue;
  PairArgs p = pair_args(a);
  p.Ca = a.C;
  p.Cd = a.Cp;
  p.K = a.M;
  p.N = a.H;
  return a.gu ? launch_fn<kUpSave>(tmA, tmB, tmD, tmD2, p, a) : launch_fn<kUp>(tmA, tmB, tmD, tmD2, p, a);
}

cudaError_t glu_down_bf16(const GluArgs& a) {
  CUtensorMap tmA, tmB, tmD;
  if (!encode_2d(&tmA, a.h, a.H, rows(a.E, a.Cp), BK, 128) ||
      !encode_2d(&tmB, a.W2, a.M, rows(a.E, a.H), 64, BK) || !encode_2d(&tmD, a.y, a.M, rows(a.E, a.C), 64, 32))
    return cudaErrorInvalidValue;
  PairArgs p = pair_args(a);
  p.Ca = a.Cp;
  p.Cd = a.C;
  p.K = a.H;
  p.N = a.M;
  p.D = static_cast<__nv_bfloat16*>(a.y);
  return launch_split<kDown>(tmA, tmB, tmD, p, a, a.y);
}

cudaError_t glu_dh_bf16(const GluArgs& a) {
  CUtensorMap tmA, tmB, tmD, tmG;
  if (!encode_2d(&tmA, a.dy, a.M, rows(a.E, a.C), BK, 128) ||
      !encode_2d(&tmB, a.W2, a.M, rows(a.E, a.H), BK, 128) ||
      !encode_2d_narrow(&tmD, a.dgu, 2 * (uint64_t)a.H, rows(a.E, a.Cp), 32) ||
      !encode_2d_narrow(&tmG, a.gu, 2 * (uint64_t)a.H, rows(a.E, a.Cp), 32))
    return cudaErrorInvalidValue;
  PairArgs p = pair_args(a);
  p.Ca = a.C;
  p.Cd = a.Cp;
  p.K = a.M;
  p.N = a.H;
  p.x = static_cast<const uint4*>(a.x);
  p.dy = static_cast<const uint4*>(a.dy);
  p.tx = static_cast<uint4*>(a.tx);
  p.tdy = static_cast<uint4*>(a.tdy);
  return launch_fn<kDh>(tmA, tmB, tmD, tmG, p, a);
}

cudaError_t glu_dx_bf16(const GluArgs& a) {
  CUtensorMap tmA, tmB, tmD;
  if (!encode_2d(&tmA, a.dgu, 2 * (uint64_t)a.H, rows(a.E, a.Cp), BK, 128) ||
      !encode_2d(&tmB, a.W13, 2 * (uint64_t)a.H, rows(a.E, a.M), BK, 128) ||
      !encode_2d(&tmD, a.dx, a.M, rows(a.E, a.C), 64, 32))
    return cudaErrorInvalidValue;
  PairArgs p = pair_args(a);
  p.Ca = a.Cp;
  p.Cd = a.C;
  p.K = 2 * a.H;
  p.N = a.M;
  p.D = static_cast<__nv_bfloat16*>(a.dx);
  return launch_split<kDx>(tmA, tmB, tmD, p, a, a.dx);
}

cudaError_t glu_dw_bf16(const GluArgs& a) {
  DwArgs g;
  if (!dw13_product(&g.d[0], a) || !dw2_product(&g.d[1], a)) return cudaErrorInvalidValue;
  return launch_dw(a, g, 2);
}

cudaError_t glu_dw2_bf16(const GluArgs& a) {
  DwArgs g;
  return dw2_product(&g.d[0], a) ? launch_dw(a, g, 1) : cudaErrorInvalidValue;
}

cudaError_t glu_dw13_bf16(const GluArgs& a) {
  DwArgs g;
  return dw13_product(&g.d[0], a) ? launch_dw(a, g, 1) : cudaErrorInvalidValue;
}

}  // namespace moe
