// few_rows.cu -- the grouped products of gated experts and of 8-bit weights when experts hold
// few rows, or when 256 x 256 tiles would leave most of the device idle: the weights are what
// has to be read, so they stream through every SM, and the rows ride along.
//
// The product is transposed: a tile is 128 columns of the result (features) times NT rows,
// with the weights as the MMA's 128-row operand and the rows as its NT-column operand, so the
// tensor cores' work follows the number of rows (16 at least) instead of 128-row tiles.
//
// Work is cut along the depth.  All tiles of all experts form one line of tiles x KB blocks
// (a block: 64 deep in bf16, 128 in e4m3), of which every CTA takes an equal, contiguous
// share, whatever the counts are: an expert without rows has no tiles, and two busy experts
// of 256 keep all SMs at work.  A CTA's share may end inside a tile.  It then writes its
// partial sum (fp32) to the workspace, and the last of the tile's CTAs to arrive adds all
// parts in the order of the depth, so that results do not depend on timing, and finishes the
// tile.  Nobody waits for another CTA.
//
// What bounds it: the bytes of the weights.  32 KB (16 KB) of weights per stage and up to
// 12 stages keep about 200 KB per SM in flight.  Warp 0 loads (TMA), warp 1 issues MMAs and
// owns TMEM, warps 2..5 take the accumulator out.  For 8-bit weights they do so after every
// block, since its scales differ: acc += (xs ws) * block, as in fp8.cu.  `down` starts its
// weight loads while `up` drains; only the loads of h wait for it.  Every wait is bounded.
#include "common.cuh"
#include "glu.cuh"
#include "internal.h"
#include "tc_tile.cuh"

namespace moe {

namespace {

constexpr int kThreads = 192;
constexpr uint32_t A_BYTES = 16384;         // 128 features x 128 bytes of depth
enum { kUp = 0, kDown = 1, kFp8 = 2 };
constexpr int kMinShare = 4;                // blocks per CTA, at least

template <int KIND, int NT>
struct Few {
  static constexpr int ACC = KIND == kUp ? 2 : 1;               // accumulators (g and u)
  static constexpr uint32_t STAGE = ACC * A_BYTES + NT * 128;
  static constexpr int FIT = (int)((220 * 1024) / STAGE);
  static constexpr int STAGES = FIT < 12 ? FIT : 12;
  static constexpr int BUFS = KIND == kFp8 ? 4 : 2;             // accumulator buffers in TMEM
  static constexpr int COLS = BUFS * ACC * NT;
  static constexpr uint32_t TMEM_COLS = COLS <= 32 ? 32 : COLS <= 64 ? 64 : COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
  static constexpr uint32_t kBars = 512;
  static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE + kBars + 16 + 4 * (3 * kMaxExperts + 1);
  static_assert(COLS <= 512, "TMEM columns");
  static_assert(8 * (2 * STAGES + 2 * BUFS + 1) <= (int)kBars, "barriers");
  static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
  static_assert(SMEM + 81 * 1024 > 228 * 1024, "a CTA must own its SM");
};

struct FewArgs {
  const int32_t* n;      // [E] rows per expert, clamped to [0, C]
  int E, C, N, KB, NTn;  // features, blocks of depth, tiles of 128 features
  int64_t Cb, Cd;        // rows per expert of the rows' operand and of the output
  int K;                 // rows of a bf16 weight matrix (its depth)
  __nv_bfloat16* D;      // output, N columns
  __nv_bfloat16* gu;     // kUp: [g|u], 2N columns, or null
  const float* xs;       // kFp8: [E, C, KB]
  const float* ws;       // kFp8: [E, NTn, KB]
  float* part;           // [2 * grid][ACC * NT][128] partial sums
  unsigned* count;       // [grid] parts of a tile that have arrived; zero between launches
  unsigned* err;
  uint64_t limit_ns;
};

// The line of blocks and this CTA's share of it.
struct Share {
  long long U;           // blocks in all
  int G;                 // CTAs that have a share
  __device__ long long first(int i) const { return U * i / G; }
  // the CTA whose share holds block u: the largest i with U i / G <= u
  __device__ int owner(long long u) const { return (int)(((u + 1) * G - 1) / U); }
};

// Tiles in the order (expert, features, rows), rows fastest: a weight tile is read by
// neighbours in the line.
struct Tile {
  int e, nt, rt;
};
__device__ __forceinline__ Tile tile_at(int t, const int* pre, const int* rtiles, int& e) {
  while (t >= pre[e + 1]) ++e;
  const int local = t - pre[e];
  return Tile{e, local / rtiles[e], local % rtiles[e]};
}

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The four epilogue warps meet.
__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// One finished element: feature f of row c of the tile (c may lie past the expert's rows only
// where zeros are wanted).
template <int KIND, int FN>
__device__ __forceinline__ void put(const FewArgs& a, int64_t row, int f, float v0, float v1, bool live) {
  if (KIND == kUp) {
    const float h = glu_f<FN, true>(v0) * v1;
    a.D[row * a.N + f] = __float2bfloat16_rn(live ? h : 0.f);
    if (a.gu) {
      a.gu[row * 2 * a.N + f] = __float2bfloat16_rn(live ? v0 : 0.f);
      a.gu[row * 2 * a.N + a.N + f] = __float2bfloat16_rn(live ? v1 : 0.f);
    }
  } else {
    a.D[row * a.N + f] = __float2bfloat16_rn(v0);
  }
}

template <int KIND, int NT, int FN>
__global__ void __launch_bounds__(kThreads, 1)
    few_rows_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const FewArgs a) {
  using F = Few<KIND, NT>;
  constexpr int ACC = F::ACC, STAGES = F::STAGES, BUFS = F::BUFS;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t base = (raw_base + 1023u) & ~1023u;
  unsigned char* gbase = smem_raw + (base - raw_base);
  const uint32_t bar0 = base + STAGES * F::STAGE;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * STAGES + b); };
  auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * STAGES + BUFS + b); };
  const uint32_t done_bar = bar0 + 8u * (2 * STAGES + 2 * BUFS);
  unsigned char* misc = gbase + STAGES * F::STAGE + F::kBars;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 4);
  volatile unsigned* arrived = reinterpret_cast<volatile unsigned*>(misc + 8);
  int* pre = reinterpret_cast<int*>(misc + 16);        // [E + 1] first tile of each expert
  int* rtiles = pre + (kMaxExperts + 1);               // [E] tiles of NT rows
  int* nrows = rtiles + kMaxExperts;                   // [E]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < BUFS; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), 4);
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32((const void*)tmem_slot), F::TMEM_COLS);
    tmem_relinquish();
  }
  // `up` and the 8-bit product follow whatever wrote the rows and counts.  `down` follows `up`
  // of the same call, which released it after its own wait: the counts are complete.
  if (KIND != kDown) {
    pdl_wait();
    pdl_trigger();
  }
  if (warp == 2) {
    const int per = (a.E + 31) / 32;
    const int e0 = lane * per;
    int sum = 0;
    for (int e = e0; e < min(a.E, e0 + per); ++e) {
      nrows[e] = min(max(a.n[e], 0), a.C);
      rtiles[e] = (nrows[e] + NT - 1) / NT;
      sum += rtiles[e] * a.NTn;
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    int run = inc - sum;
    for (int e = e0; e < min(a.E, e0 + per); ++e) {
      pre[e] = run;
      run += rtiles[e] * a.NTn;
    }
    if (lane == 31) pre[a.E] = inc;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int KB = a.KB;
  Share sh;
  sh.U = (long long)pre[a.E] * KB;
  sh.G = (int)min((long long)gridDim.x, (sh.U + kMinShare - 1) / kMinShare);
  const int me = blockIdx.x;
  const bool mine = me < sh.G;
  const long long u0 = mine ? sh.first(me) : 0, u1 = mine ? sh.first(me + 1) : 0;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int s = 0, e = 0;
      uint32_t ph = 0, issued = 0, issued_par = 0;
      bool ok = true;
      auto load_w = [&](int st, const Tile& t, int kb) {
        const uint32_t sa = base + st * F::STAGE;
        mbar_arrive_expect_tx(full_bar(st), F::STAGE);
        if (KIND == kFp8) {
          tma_load_2d(sa, &tmW, full_bar(st), kb * 128, t.e * a.N + t.nt * 128);
        } else {
          // features past N read the next columns or zeros; they are not stored
#pragma unroll
          for (int c = 0; c < ACC; ++c)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              tma_load_2d(sa + c * A_BYTES + j * 8192u, &tmW, full_bar(st), c * a.N + t.nt * 128 + j * 64, t.e * a.K + kb * 64);
        }
      };
      auto load_x = [&](int st, const Tile& t, int kb) {
        tma_load_2d(base + st * F::STAGE + ACC * A_BYTES, &tmX, full_bar(st), kb * (KIND == kFp8 ? 128 : 64),
                    (int)(t.e * a.Cb) + t.rt * NT);
      };
      long long u = u0;
      if (KIND == kDown) {
        // the first stages' weights before `up` has finished, then the rows it wrote
        const int lead = (int)min((long long)STAGES, u1 - u0);
        int e2 = 0;
        for (int i = 0; i < lead; ++i) load_w(i, tile_at((int)((u0 + i) / KB), pre, rtiles, e2), (int)((u0 + i) % KB));
        pdl_wait();
        for (int i = 0; i < lead; ++i) load_x(i, tile_at((int)((u0 + i) / KB), pre, rtiles, e), (int)((u0 + i) % KB));
        issued = (1u << lead) - 1u;
        u += lead;
        s = lead % STAGES;
        ph = lead == STAGES ? 1u : 0u;
      }
      while (ok && u < u1) {
        const Tile t = tile_at((int)(u / KB), pre, rtiles, e);
        int kb = (int)(u % KB);
        const int end = (int)min((long long)KB, kb + (u1 - u));
        u += end - kb;
        for (; kb < end; ++kb) {
          if (*abort_flag || !mbar_wait(empty_bar(s), ph ^ 1u, a.err, a.limit_ns)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          load_w(s, t, kb);
          load_x(s, t, kb);
          issued |= 1u << s;
          issued_par = (issued_par & ~(1u << s)) | (ph << s);
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (!ok) {   // let copies in flight land before the CTA exits
        for (int q = 0; q < STAGES; ++q)
          if ((issued >> q) & 1u) mbar_wait(full_bar(q), (issued_par >> q) & 1u, a.err, a.limit_ns);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      int s = 0, buf = 0, e = 0;
      uint32_t ph = 0, bph = 0;
      bool ok = true;
      for (long long u = u0; ok && u < u1;) {
        const Tile t = tile_at((int)(u / KB), pre, rtiles, e);
        const int kb0 = (int)(u % KB);
        const int len = (int)min((long long)(KB - kb0), u1 - u);
        u += len;
        // rows of this tile, rounded up to the MMA's step of 16 columns
        const int cols = (min(NT, nrows[t.e] - t.rt * NT) + 15) & ~15;
        // D fp32, M = 128, N = cols; bf16: A with its rows (features) contiguous, B its depth
        const uint32_t idesc = (1u << 4) | (KIND == kFp8 ? 0u : (1u << 7) | (1u << 10) | (1u << 15)) |
                               ((uint32_t)(cols >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
        for (int i = 0; i < len; ++i) {
          const bool fresh = KIND == kFp8 || i == 0;
          if (*abort_flag || (fresh && !mbar_wait(tempty_bar(buf), bph ^ 1u, a.err, a.limit_ns)) ||
              !mbar_wait(full_bar(s), ph, a.err, a.limit_ns)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = base + s * F::STAGE, sb = sa + ACC * A_BYTES;
          const uint32_t d = tmem_base + buf * (ACC * NT);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t bd = desc_sw128(sb + kk * 32u, 16u, 1024u);
            if (KIND == kFp8) {
              tc_mma_f8(d, desc_sw128(sa + kk * 32u, 16u, 1024u), bd, idesc, kk != 0);
            } else {
#pragma unroll
              for (int c = 0; c < ACC; ++c)
                tc_mma_f16(d + c * NT, desc_sw128(sa + c * A_BYTES + kk * 2048u, 8192u, 1024u), bd, idesc, (i | kk) != 0);
            }
          }
          tc_commit(empty_bar(s));
          if (KIND == kFp8 || i == len - 1) {
            tc_commit(tfull_bar(buf));
            if (++buf == BUFS) {
              buf = 0;
              bph ^= 1u;
            }
          }
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (!ok) {   // let issued MMAs finish before TMEM is released
        tc_commit(done_bar);
        mbar_wait(done_bar, 0, a.err, a.limit_ns);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue (warps 2..5)
    const int q = warp & 3;                    // TMEM lane quarter of this warp
    const int lane128 = q * 32 + lane;         // this thread's feature within a tile
    if (KIND == kDown) pdl_wait();             // the workspace is `up`'s until it has finished
    int buf = 0, e = 0;
    uint32_t bph = 0;
    bool ok = true;
    for (long long u = u0; ok && u < u1;) {
      const int ti = (int)(u / KB);
      const Tile t = tile_at(ti, pre, rtiles, e);
      const int kb0 = (int)(u % KB);
      const int len = (int)min((long long)(KB - kb0), u1 - u);
      u += len;
      const int row0 = t.rt * NT, left = nrows[t.e] - row0;
      const int nvalid = min(NT, left);
      const bool whole = len == KB;
      const int f = t.nt * 128 + lane128;
      const int64_t drow = t.e * a.Cd + row0;
      // training: the rows up to the next multiple of 64 are zeros (weight gradients reduce
      // over whole blocks of 64)
      const int nzero = KIND == kUp && a.gu && left <= NT ? (nrows[t.e] + 63) / 64 * 64 - row0 : 0;
      float* part = a.part + (size_t)(2 * me + (kb0 == 0)) * ACC * NT * 128 + lane128;
      const uint32_t tm0 = tmem_base + ((uint32_t)(q * 32) << 16);
      if constexpr (KIND == kFp8) {
        float sum[NT];
#pragma unroll
        for (int c = 0; c < NT; ++c) sum[c] = 0.f;
        const float* ws = a.ws + ((int64_t)t.e * a.NTn + t.nt) * KB;
        const float* xs = a.xs + (t.e * a.Cb + row0) * KB;
        constexpr int XR = (NT + 31) / 32;     // lane l holds the scales of rows l, l + 32, ...
        float x[2][XR], w[2];
        auto scales = [&](int i, float (&xv)[XR], float& wv) {
          const int kb = kb0 + i;
          wv = i < len ? __ldg(ws + kb) : 0.f;
#pragma unroll
          for (int r = 0; r < XR; ++r)
            xv[r] = i < len && r * 32 + lane < nvalid ? __ldg(xs + (int64_t)(r * 32 + lane) * KB + kb) : 0.f;
        };
        auto drain = [&](int i, float (&xv)[XR], float& wv) -> bool {
          if (*abort_flag || !mbar_wait(tfull_bar(buf), bph, a.err, a.limit_ns)) {
            *abort_flag = 1;
            return false;
          }
          tc_fence_after();
          float sc[XR];
#pragma unroll
          for (int r = 0; r < XR; ++r) sc[r] = xv[r] * wv;
          scales(i + 2, xv, wv);
          uint32_t v[NT / 16][16];
#pragma unroll
          for (int c = 0; c < NT / 16; ++c)
            if (c * 16 < nvalid) tmem_ld_32x32b_x16(tm0 + buf * NT + c * 16, v[c]);
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(tempty_bar(buf));
          if (++buf == BUFS) {
            buf = 0;
            bph ^= 1u;
          }
#pragma unroll
          for (int c = 0; c < NT / 16; ++c)
            if (c * 16 < nvalid) {
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const int col = c * 16 + j;
                sum[col] = fmaf(__shfl_sync(0xffffffffu, sc[col / 32], col % 32), __uint_as_float(v[c][j]), sum[col]);
              }
            }
          return true;
        };
        scales(0, x[0], w[0]);
        scales(1, x[1], w[1]);
        for (int i = 0; ok && i < len; i += 2) {
          ok = drain(i, x[0], w[0]);
          if (ok && i + 1 < len) ok = drain(i + 1, x[1], w[1]);
        }
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < NT; ++c)
          if (c < nvalid) {
            if (!whole) __stcg(part + c * 128, sum[c]);
            else if (f < a.N) put<KIND, FN>(a, drow + c, f, sum[c], 0.f, true);
          }
      } else {
        if (*abort_flag || !mbar_wait(tfull_bar(buf), bph, a.err, a.limit_ns)) {
          *abort_flag = 1;
          break;
        }
        tc_fence_after();
        const uint32_t tm = tm0 + buf * (ACC * NT);
#pragma unroll 1
        for (int c0 = 0; c0 < nvalid; c0 += 16) {
          uint32_t v[ACC][16];
#pragma unroll
          for (int c = 0; c < ACC; ++c) tmem_ld_32x32b_x16(tm + c * NT + c0, v[c]);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            if (c0 + j >= nvalid) break;
            if (!whole) {
#pragma unroll
              for (int c = 0; c < ACC; ++c) __stcg(part + (c * NT + c0 + j) * 128, __uint_as_float(v[c][j]));
            } else if (f < a.N) {
              put<KIND, FN>(a, drow + c0 + j, f, __uint_as_float(v[0][j]), __uint_as_float(v[ACC - 1][j]), true);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty_bar(buf));
        if (++buf == BUFS) {
          buf = 0;
          bph ^= 1u;
        }
      }
      bool finish = whole;
      if (!whole) {
        // a part of a tile: the last CTA to bring one adds them all, in the order of the depth
        const long long first = (long long)ti * KB;
        const int i0 = sh.owner(first), i1 = sh.owner(first + KB - 1);
        __threadfence();
        epi_sync();
        if (threadIdx.x == 64) *arrived = atomicAdd(a.count + i0, 1u);
        epi_sync();
        finish = *arrived == (unsigned)(i1 - i0);
        if (finish) {
          __threadfence();
          if (threadIdx.x == 64) a.count[i0] = 0u;
          if (f < a.N) {
#pragma unroll 1
            for (int c0 = 0; c0 < nvalid; c0 += 8) {
              float s[ACC][8] = {};
#pragma unroll 2
              for (int i = i0; i <= i1; ++i) {
                const float* p = a.part + (size_t)(2 * i + (i == i0)) * ACC * NT * 128 + lane128;
#pragma unroll
                for (int c = 0; c < ACC; ++c)
#pragma unroll
                  for (int j = 0; j < 8; ++j)
                    if (c0 + j < nvalid) s[c][j] += __ldcg(p + (c * NT + c0 + j) * 128);
              }
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (c0 + j < nvalid) put<KIND, FN>(a, drow + c0 + j, f, s[0][j], s[ACC - 1][j], true);
            }
          }
        }
      }
      if (KIND == kUp && finish && f < a.N)
        for (int c = nvalid; c < nzero; ++c) put<KIND, FN>(a, drow + c, f, 0.f, 0.f, false);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, F::TMEM_COLS);
  }
}

template <int KIND, int NT, int FN>
cudaError_t launch(const CUtensorMap& tmW, const CUtensorMap& tmX, const FewArgs& f, int num_sms, cudaStream_t st) {
  auto kern = few_rows_kernel<KIND, NT, FN>;
  const size_t smem = Few<KIND, NT>::SMEM;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(num_sms), dim3(kThreads), smem, st, tmW, tmX, f);
}

template <int KIND, int FN>
cudaError_t launch_nt(int nt, const CUtensorMap& tmW, const CUtensorMap& tmX, const FewArgs& f, int num_sms, cudaStream_t st) {
  switch (nt) {
    case 16: return launch<KIND, 16, FN>(tmW, tmX, f, num_sms, st);
    case 32: return launch<KIND, 32, FN>(tmW, tmX, f, num_sms, st);
    case 64: return launch<KIND, 64, FN>(tmW, tmX, f, num_sms, st);
  }
  if constexpr (KIND != kFp8) return launch<KIND, 128, FN>(tmW, tmX, f, num_sms, st);
  else return cudaErrorInvalidValue;
}

// Rows per tile: the smallest that holds C.
int row_tile(int64_t C, int most) {
  int nt = 16;
  while (nt < C && nt < most) nt *= 2;
  return nt;
}

constexpr int kMostBf16 = 128, kMostFp8 = 64;

}  // namespace

size_t few_rows_workspace(int64_t C_max, bool fp8, int num_sms, size_t* counts) {
  const int nt = row_tile(C_max, fp8 ? kMostFp8 : kMostBf16);
  *counts = (size_t)num_sms;
  return (size_t)2 * num_sms * (fp8 ? 1 : 2) * nt * 128;
}

cudaError_t glu_few_up(const GluArgs& a) {
  const int nt = row_tile(a.C, kMostBf16);
  CUtensorMap tmW, tmX;
  if (!encode_2d(&tmW, a.W13, 2 * (uint64_t)a.H, (uint64_t)a.E * a.M, 64, 64) ||
      !encode_2d(&tmX, a.x, a.M, (uint64_t)a.E * a.C, 64, nt))
    return cudaErrorInvalidValue;
  FewArgs f{};
  f.n = a.n;
  f.E = a.E;
  f.C = (int)a.C;
  f.N = a.H;
  f.K = a.M;
  f.KB = a.M / 64;
  f.NTn = (a.H + 127) / 128;
  f.Cb = a.C;
  f.Cd = a.Cp;
  f.D = static_cast<__nv_bfloat16*>(a.h);
  f.gu = static_cast<__nv_bfloat16*>(a.gu);
  f.part = a.part;
  f.count = a.count;
  f.err = a.err;
  f.limit_ns = a.limit_ns;
  if (a.fn == kGluSilu) return launch_nt<kUp, kGluSilu>(nt, tmW, tmX, f, a.num_sms, a.st);
  if (a.fn == kGluGelu) return launch_nt<kUp, kGluGelu>(nt, tmW, tmX, f, a.num_sms, a.st);
  return launch_nt<kUp, kGluRelu>(nt, tmW, tmX, f, a.num_sms, a.st);
}

cudaError_t glu_few_down(const GluArgs& a) {
  const int nt = row_tile(a.C, kMostBf16);
  CUtensorMap tmW, tmX;
  if (!encode_2d(&tmW, a.W2, a.M, (uint64_t)a.E * a.H, 64, 64) ||
      !encode_2d(&tmX, a.h, a.H, (uint64_t)a.E * a.Cp, 64, nt))
    return cudaErrorInvalidValue;
  FewArgs f{};
  f.n = a.n;
  f.E = a.E;
  f.C = (int)a.C;
  f.N = a.M;
  f.K = a.H;
  f.KB = a.H / 64;
  f.NTn = (a.M + 127) / 128;
  f.Cb = a.Cp;
  f.Cd = a.C;
  f.D = static_cast<__nv_bfloat16*>(a.y);
  f.part = a.part;
  f.count = a.count;
  f.err = a.err;
  f.limit_ns = a.limit_ns;
  return launch_nt<kDown, kGluSilu>(nt, tmW, tmX, f, a.num_sms, a.st);
}

cudaError_t fp8_few(const Fp8Args& a) {
  const int nt = row_tile(a.C, kMostFp8);
  CUtensorMap tmW, tmX;
  if (!encode_2d_bytes(&tmW, a.wq, a.K, (uint64_t)a.E * a.N, 128, 128) ||
      !encode_2d_bytes(&tmX, a.xq, a.K, (uint64_t)a.E * a.C, 128, nt))
    return cudaErrorInvalidValue;
  FewArgs f{};
  f.n = a.n;
  f.E = a.E;
  f.C = (int)a.C;
  f.N = a.N;
  f.KB = (a.K + 127) / 128;
  f.NTn = (a.N + 127) / 128;
  f.Cb = a.C;
  f.Cd = a.C;
  f.D = static_cast<__nv_bfloat16*>(a.y);
  f.xs = a.xs;
  f.ws = a.ws;
  f.part = a.part;
  f.count = a.count;
  f.err = a.err;
  f.limit_ns = a.limit_ns;
  return launch_nt<kFp8, kGluSilu>(nt, tmW, tmX, f, a.num_sms, a.st);
}

}  // namespace moe
