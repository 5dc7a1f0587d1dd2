// few_rows.cu -- the grouped products of gated experts and of 8-bit weights when experts hold
// few rows, or when 256 x 256 tiles would leave most of the device idle: the weights are what
// has to be read, so they stream through every SM, and the rows ride along.
//
// The product is transposed: a tile is 128 or 256 columns of the result (features; `up`: 128 of
// g and the same of u) times NT rows, with the weights as the MMA's 128-row operand and the rows
// as its NT-column operand, so the tensor cores' work follows the number of rows (16 at least)
// instead of 128-row tiles.
//
// Work is cut along the depth.  All tiles of all experts form one line of tiles x KB blocks
// (a block: 64 deep in bf16, 128 in e4m3): an expert without rows has no tiles, and two busy
// experts of 256 keep all SMs at work.  Most of the line is dealt out beforehand, an equal,
// contiguous share to every CTA; where shares are long (kLongShare blocks), its last fifth is
// cut into pieces that CTAs fetch as they finish, since SMs do not get the same share of the
// memory's bandwidth.  The cuts depend on the counts alone.  A CTA that holds part of a tile
// writes its sum (fp32) to the workspace, and the last of the tile's parts to arrive adds all
// of them in the order of the depth -- so results do not depend on timing -- and finishes the
// tile.  Nobody waits for another CTA.
//
// What bounds it: the bytes of the weights.  Stages of 32 KB of weights keep about 200 KB per
// SM in flight (16 KB stages lost 10-15% to the hand-over of a stage).  Warp 0 loads (TMA), warp 1
// issues MMAs and owns TMEM, warps 2..5 take the accumulator out, warps 6..9 join parts: the memory fence, the
// arrival and the other parts' loads take several us beside a saturated memory, which the
// accumulators of the next pieces must not wait for.  For 8-bit weights they do so after every
// block, since its scales differ: acc += (xs ws) * block, as in fp8.cu.  `down` starts its
// weight loads while `up` drains; only the loads of h wait for it.  Every wait is bounded.
#include <type_traits>

#include "common.cuh"
#include "glu.cuh"
#include "internal.h"
#include "tc_tile.cuh"

namespace moe {

namespace {

constexpr int kThreads = 320;               // loads, MMAs, four epilogue and four joining warps
constexpr uint32_t A_BYTES = 16384;         // 128 features x 128 bytes of depth
enum { kUp = 0, kDown = 1, kFp8 = 2 };
constexpr int kMinShare = 4;                // blocks per CTA, at least
constexpr int kLongShare = 32;              // blocks per CTA from which the last fifth is fetched
constexpr int kPieces = 4;                  // pieces per CTA in it, at most
constexpr uint32_t kPieceBytes = 256 * 1024;   // weights of a piece, at least (about 6 us of an SM's bandwidth)
constexpr int kRing = 4;                    // fetched pieces known ahead
constexpr int kJoin = 4;                    // parts on their way to the joining warps

template <int KIND, int NT>
struct Few {
  static constexpr int ACC = 2;                                 // accumulators: g and u, or two times 128 features
  static constexpr int FEATURES = KIND == kUp ? 128 : 128 * ACC;   // of a tile
  static constexpr uint32_t STAGE = ACC * A_BYTES + NT * 128;
  static constexpr int FIT = (int)((220 * 1024) / STAGE);
  static constexpr int STAGES = FIT < 12 ? FIT : 12;
  static constexpr int BUFS = KIND == kFp8 ? 4 : 2;             // accumulator buffers in TMEM
  static constexpr int COLS = BUFS * ACC * NT;
  static constexpr uint32_t TMEM_COLS = COLS <= 32 ? 32 : COLS <= 64 ? 64 : COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
  static constexpr uint32_t kBars = 512;
  static constexpr uint32_t kMisc = 256;
  static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE + kBars + kMisc + 4 * (3 * kMaxExperts + 1);
  static_assert(COLS <= 512, "TMEM columns");
  static_assert(8 * (2 * STAGES + 2 * BUFS + 1 + 2 * kRing + 2 * kJoin) <= (int)kBars, "barriers");
  static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
  static_assert(SMEM + 81 * 1024 > 228 * 1024, "a CTA must own its SM");
};

struct FewArgs {
  const int32_t* n;      // [E] rows per expert, clamped to [0, C]
  int E, C, N, KB, NB;   // features, blocks of depth, blocks of 128 features
  int64_t Cb, Cd;        // rows per expert of the rows' operand and of the output
  int K;                 // rows of a bf16 weight matrix (its depth)
  __nv_bfloat16* D;      // output, N columns
  uint16_t* gu;          // kUp: [g|u], 2N columns (glu.cuh), or null
  const float* xs;       // kFp8: [E, C, KB]
  const float* ws;       // kFp8: [E, NB, KB]
  float* part;           // [(2 + kPieces) * grid][ACC * NT][128] partial sums
  unsigned* count;       // arrivals: [grid] tiles of shares, [kPieces * grid] fetched tiles; then
                         // the next piece, and CTAs that found none.  Zero between launches
  unsigned* err;
  uint64_t limit_ns;
};

// How the line is cut, and where this CTA's share of it begins (one copy per CTA).
struct Cuts {
  int T, Ts;             // tiles in all, and those dealt out as shares
  int G;                 // CTAs that have a share
  int P;                 // pieces of each of the other tiles
  int t0, kb0, len;      // this CTA's share: tile, block, blocks
  int pad;
};

// floor(i * U / G) and the CTA whose share holds block u: the largest i with U i / G <= u
__device__ __forceinline__ long long share_first(long long U, int G, int i) {
  return U * i <= 0xFFFFFFFFll ? (long long)((uint32_t)(U * i) / (uint32_t)G) : U * i / G;
}
__device__ __forceinline__ int share_owner(long long U, int G, long long u) {
  const long long a = (u + 1) * G - 1;
  return (a | U) <= 0xFFFFFFFFll ? (int)((uint32_t)a / (uint32_t)U) : (int)(a / U);
}

// Tiles in the order (expert, features, rows), rows fastest: a weight tile is read by
// neighbours in the line.
struct Tile {
  int e, nt, rt;
};
__device__ __forceinline__ Tile tile_at(int t, const int* pre, const int* rtiles, int E) {
  int lo = 0, hi = E;        // pre[lo] <= t < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int local = t - pre[lo], r = rtiles[lo];
  const int nt = r == 1 ? local : local / r;
  return Tile{lo, nt, local - nt * r};
}

// The walk of one role over the CTA's work: its share, tile by tile, then fetched pieces,
// whose numbers the producer passes on through a ring.
struct Step {
  int t, kb, len;        // tile, first block, blocks
  int piece;             // fetched: its number, else -1
};

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

// Arrival of a part: orders the part's stores (which the joining warps' mbarrier has brought
// before it) ahead of it, and the loads of the other parts behind it.
__device__ __forceinline__ unsigned atom_add_acq_rel(unsigned* p, unsigned v) {
  unsigned old;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}

// Finished values of one row: feature f (and f + 128) of a tile.  `live` false: zeros.
template <int KIND, int ACC, int FN>
__device__ __forceinline__ void put(const FewArgs& a, int64_t row, int f, const float (&v)[ACC], bool live) {
  if (KIND == kUp) {
    if (f >= a.N) return;
    const float h = glu_f<FN, true>(v[0]) * v[1];
    a.D[row * a.N + f] = __float2bfloat16_rn(live ? h : 0.f);
    if (a.gu) {
      a.gu[row * 2 * a.N + f] = pack_gu_lane(v[0], live);
      a.gu[row * 2 * a.N + a.N + f] = pack_gu_lane(v[1], live);
    }
  } else {
#pragma unroll
    for (int j = 0; j < ACC; ++j)
      if (f + j * 128 < a.N) a.D[row * a.N + f + j * 128] = __float2bfloat16_rn(v[j]);
  }
}

// Training: the rows of h and [g|u] from an expert's last one to the next multiple of 64 are
// zeros, since the weight gradients reduce over whole blocks of 64.
template <int KIND, int ACC, int FN>
__device__ __forceinline__ void zero_rows(const FewArgs& a, int64_t drow, int f, int from, int to) {
  const float zero[ACC] = {};
  for (int k = from; k < to; ++k) put<KIND, ACC, FN>(a, drow + k, f, zero, false);
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
  auto pfull_bar = [&](int r) { return bar0 + 8u * (2 * STAGES + 2 * BUFS + 1 + r); };
  auto pempty_bar = [&](int r) { return bar0 + 8u * (2 * STAGES + 2 * BUFS + 1 + kRing + r); };
  auto jfull_bar = [&](int r) { return bar0 + 8u * (2 * STAGES + 2 * BUFS + 1 + 2 * kRing + r); };
  auto jempty_bar = [&](int r) { return bar0 + 8u * (2 * STAGES + 2 * BUFS + 1 + 2 * kRing + kJoin + r); };
  unsigned char* misc = gbase + STAGES * F::STAGE + F::kBars;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 4);
  volatile int* ring = reinterpret_cast<volatile int*>(misc + 16);
  Cuts* cuts = reinterpret_cast<Cuts*>(misc + 32);
  volatile int4* joins = reinterpret_cast<volatile int4*>(misc + 64);    // Steps of written parts
  int* pre = reinterpret_cast<int*>(misc + F::kMisc);  // [E + 1] first tile of each expert
  int* rtiles = pre + (kMaxExperts + 1);               // [E] tiles of NT rows
  int* nrows = rtiles + kMaxExperts;                   // [E]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int KB = a.KB, grid = (int)gridDim.x, me = (int)blockIdx.x;
  const int NTn = (a.N + F::FEATURES - 1) / F::FEATURES;
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
    for (int r = 0; r < kRing; ++r) {
      mbar_init(pfull_bar(r), 1);
      mbar_init(pempty_bar(r), 5);             // the MMA thread and four epilogue warps
    }
    for (int r = 0; r < kJoin; ++r) {
      mbar_init(jfull_bar(r), 128);
      mbar_init(jempty_bar(r), 4);
    }
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
      sum += rtiles[e] * NTn;
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
      run += rtiles[e] * NTn;
    }
    if (lane == 31) {
      pre[a.E] = inc;
      Cuts c{};
      c.T = c.Ts = inc;
      c.P = 1;
      if ((long long)inc * KB >= (long long)kLongShare * grid) {
        const int td = min(inc / 5, kPieces * grid);
        if (td > 0) {
          c.Ts = inc - td;
          c.P = max(1, min((int)(KB * (ACC * A_BYTES) / kPieceBytes), kPieces * grid / td));
        }
      }
      const long long U = (long long)c.Ts * KB;
      c.G = (int)min((long long)grid, (U + kMinShare - 1) / kMinShare);
      if (me < c.G) {
        const long long u0 = share_first(U, c.G, me), u1 = share_first(U, c.G, me + 1);
        c.t0 = u0 <= 0xFFFFFFFFll ? (int)((uint32_t)u0 / (uint32_t)KB) : (int)(u0 / KB);
        c.kb0 = (int)(u0 - (long long)c.t0 * KB);
        c.len = (int)(u1 - u0);
      }
      *cuts = c;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const Cuts c = *cuts;
  const int npieces = (c.T - c.Ts) * c.P;
  // training: the row of a tile up to which zeros follow its rows (its expert's last tile)
  auto zero_to = [&](int n, int row0, int nvalid) {
    return KIND == kUp && a.gu && row0 + nvalid == n ? (n + 63) / 64 * 64 - row0 : 0;
  };
  auto piece = [&](int id) {                           // a fetched piece
    const int i = id / c.P, p = id - i * c.P;
    const int kb = KB * p / c.P;
    return Step{c.Ts + i, kb, KB * (p + 1) / c.P - kb, id};
  };

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0, issued = 0, issued_par = 0;
      bool ok = true;
      auto load_w = [&](int st, const Tile& t, int kb) {
        const uint32_t sa = base + st * F::STAGE;
        mbar_arrive_expect_tx(full_bar(st), F::STAGE);
        // features past N read the next rows or columns, or zeros; they are not stored
        if (KIND == kFp8) {
          tma_load_2d(sa, &tmW, full_bar(st), kb * 128, t.e * a.N + t.nt * F::FEATURES);
        } else if (KIND == kDown) {
          tma_load_3d(sa, &tmW, full_bar(st), 0, t.e * a.K + kb * 64, t.nt * 4);
        } else {
          tma_load_3d(sa, &tmW, full_bar(st), 0, t.e * a.K + kb * 64, t.nt * 2);
          tma_load_3d(sa + A_BYTES, &tmW, full_bar(st), 0, t.e * a.K + kb * 64, a.N / 64 + t.nt * 2);
        }
      };
      auto load_x = [&](int st, const Tile& t, int kb) {
        tma_load_2d(base + st * F::STAGE + ACC * A_BYTES, &tmX, full_bar(st), kb * (KIND == kFp8 ? 128 : 64),
                    (int)(t.e * a.Cb) + t.rt * NT);
      };
      auto load = [&](const Step& st) {
        const Tile t = tile_at(st.t, pre, rtiles, a.E);
        for (int kb = st.kb; kb < st.kb + st.len; ++kb) {
          if (*abort_flag || !mbar_wait(empty_bar(s), ph ^ 1u, a.err, a.limit_ns)) {
            *abort_flag = 1;
            ok = false;
            return;
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
      };
      int t = c.t0, kb = c.kb0, left = c.len;
      if (KIND == kDown) {
        // the first stages' weights before `up` has finished, then the rows it wrote
        const int lead = min(STAGES, left);
        for (int pass = 0; pass < 2; ++pass) {
          t = c.t0;
          kb = c.kb0;
          Tile tile = lead ? tile_at(t, pre, rtiles, a.E) : Tile{0, 0, 0};
          for (int i = 0; i < lead; ++i) {
            if (pass == 0) load_w(i, tile, kb);
            else load_x(i, tile, kb);
            if (++kb == KB) {
              kb = 0;
              if (++t < c.T) tile = tile_at(t, pre, rtiles, a.E);
            }
          }
          if (pass == 0) pdl_wait();
        }
        issued = (1u << lead) - 1u;
        left -= lead;
        s = lead % STAGES;
        ph = lead == STAGES ? 1u : 0u;
      }
      while (ok && left > 0) {
        const Step st{t, kb, min(KB - kb, left), -1};
        load(st);
        left -= st.len;
        ++t;
        kb = 0;
      }
      if (npieces > 0) {
        unsigned* next = a.count + (1 + kPieces) * grid;
        int id = ok ? (int)atomicAdd(next, 1u) : npieces;
        for (int r = 0;; ++r) {
          const int slot = r % kRing;
          if (!ok || *abort_flag || !mbar_wait(pempty_bar(slot), ((r / kRing) & 1) ^ 1, a.err, a.limit_ns)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          ring[slot] = id;
          mbar_arrive(pfull_bar(slot));
          if (id >= npieces) break;
          const int then = (int)atomicAdd(next, 1u);
          load(piece(id));
          id = then;
        }
        if (ok && atomicAdd(next + 1, 1u) == (unsigned)grid - 1u) {   // every CTA has found none left
          next[0] = 0u;
          next[1] = 0u;
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
      int s = 0, buf = 0;
      uint32_t ph = 0, bph = 0;
      bool ok = true;
      auto mma = [&](const Step& st) {
        const Tile t = tile_at(st.t, pre, rtiles, a.E);
        // rows of this tile, rounded up to the MMA's step of 16 columns
        const int cols = (min(NT, nrows[t.e] - t.rt * NT) + 15) & ~15;
        // D fp32, M = 128, N = cols; bf16: A with its rows (features) contiguous, B its depth
        const uint32_t idesc = (1u << 4) | (KIND == kFp8 ? 0u : (1u << 7) | (1u << 10) | (1u << 15)) |
                               ((uint32_t)(cols >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
        for (int i = 0; i < st.len; ++i) {
          const bool fresh = KIND == kFp8 || i == 0;
          if (*abort_flag || (fresh && !mbar_wait(tempty_bar(buf), bph ^ 1u, a.err, a.limit_ns)) ||
              !mbar_wait(full_bar(s), ph, a.err, a.limit_ns)) {
            *abort_flag = 1;
            ok = false;
            return;
          }
          tc_fence_after();
          const uint32_t sa = base + s * F::STAGE, sb = sa + ACC * A_BYTES;
          const uint32_t d = tmem_base + buf * (ACC * NT);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t bd = desc_sw128(sb + kk * 32u, 16u, 1024u);
#pragma unroll
            for (int j = 0; j < ACC; ++j) {
              if (KIND == kFp8)
                tc_mma_f8(d + j * NT, desc_sw128(sa + j * A_BYTES + kk * 32u, 16u, 1024u), bd, idesc, kk != 0);
              else
                tc_mma_f16(d + j * NT, desc_sw128(sa + j * A_BYTES + kk * 2048u, 8192u, 1024u), bd, idesc, (i | kk) != 0);
            }
          }
          tc_commit(empty_bar(s));
          if (KIND == kFp8 || i == st.len - 1) {
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
      };
      int t = c.t0, kb = c.kb0, left = c.len;
      while (ok && left > 0) {
        const Step st{t, kb, min(KB - kb, left), -1};
        mma(st);
        left -= st.len;
        ++t;
        kb = 0;
      }
      if (npieces > 0)
        for (int r = 0; ok; ++r) {
          const int slot = r % kRing;
          if (*abort_flag || !mbar_wait(pfull_bar(slot), (r / kRing) & 1, a.err, a.limit_ns)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          const int id = ring[slot];
          mbar_arrive(pempty_bar(slot));
          if (id >= npieces) break;
          mma(piece(id));
        }
      if (!ok) {   // let issued MMAs finish before TMEM is released
        tc_commit(done_bar);
        mbar_wait(done_bar, 0, a.err, a.limit_ns);
      }
    }
    __syncwarp();
  } else if (warp < 6) {
    // ------------------------------------------------------------ epilogue (warps 2..5)
    const int q = warp & 3;                    // TMEM lane quarter of this warp
    const int lane128 = q * 32 + lane;         // this thread's feature within a tile
    if (KIND == kDown) pdl_wait();             // the workspace is `up`'s until it has finished
    int buf = 0, jn = 0;
    uint32_t bph = 0;
    bool ok = true;
    // passes a written part (or, with len 0, the end) on to the joining warps
    auto pass_on = [&](const Step& st) {
      const int slot = jn % kJoin;
      if (!warp_wait(abort_flag, jempty_bar(slot), ((jn / kJoin) & 1) ^ 1, a.err, a.limit_ns)) {
        ok = false;
        return;
      }
      if (threadIdx.x == 64) {
        joins[slot].x = st.t;
        joins[slot].y = st.kb;
        joins[slot].z = st.len;
        joins[slot].w = st.piece;
      }
      mbar_arrive(jfull_bar(slot));            // after this thread's stores
      ++jn;
    };
    auto take = [&](const Step& st) {
      const Tile t = tile_at(st.t, pre, rtiles, a.E);
      const int row0 = t.rt * NT, nvalid = min(NT, nrows[t.e] - row0);
      const bool whole = st.len == KB;
      const int f = t.nt * F::FEATURES + lane128;
      const int64_t drow = t.e * a.Cd + row0;
      const int slot = st.piece >= 0 ? 2 * grid + st.piece : 2 * me + (st.kb == 0);
      float* part = a.part + (size_t)slot * (ACC * NT * 128) + lane128;
      const uint32_t tm0 = tmem_base + ((uint32_t)(q * 32) << 16);
      if constexpr (KIND == kFp8) {
        float sum[ACC][NT];
#pragma unroll
        for (int j = 0; j < ACC; ++j)
#pragma unroll
          for (int k = 0; k < NT; ++k) sum[j][k] = 0.f;
        const float* ws = a.ws + ((int64_t)t.e * a.NB + t.nt * ACC) * KB;
        const bool second = t.nt * ACC + 1 < a.NB;      // the tile has a second block of 128
        const float* xs = a.xs + (t.e * a.Cb + row0) * KB;
        constexpr int AHEAD = 4;               // blocks whose scales are on their way
        float x[AHEAD], w[AHEAD][ACC];         // lane l holds the scale of row l
        auto scales = [&](int i, float& xv, float (&wv)[ACC]) {
          const int kb = st.kb + i;
          wv[0] = i < st.len ? __ldg(ws + kb) : 0.f;
          wv[1] = i < st.len && second ? __ldg(ws + KB + kb) : 0.f;
          xv = i < st.len && lane < nvalid ? __ldg(xs + (int64_t)lane * KB + kb) : 0.f;
        };
        auto drain = [&](int i, float& xv, float (&wv)[ACC]) {
          if (!warp_wait(abort_flag, tfull_bar(buf), bph, a.err, a.limit_ns)) {
            ok = false;
            return;
          }
          tc_fence_after();
          const float sx = xv, sw[ACC] = {wv[0], wv[1]};
          scales(i + AHEAD, xv, wv);
#pragma unroll
          for (int k = 0; k < NT; k += 16) {
            uint32_t v[ACC][16];
            if (k < nvalid) {
#pragma unroll
              for (int j = 0; j < ACC; ++j) tmem_ld_32x32b_x16(tm0 + buf * (ACC * NT) + j * NT + k, v[j]);
            }
            tmem_ld_wait();
            if (k + 16 == NT) {                // the last columns are here: hand the buffer back
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(tempty_bar(buf));
            }
            if (k < nvalid) {
#pragma unroll
              for (int i2 = 0; i2 < 16; ++i2) {
                const float s = __shfl_sync(0xffffffffu, sx, k + i2);
#pragma unroll
                for (int j = 0; j < ACC; ++j)
                  sum[j][k + i2] = fmaf(s * sw[j], __uint_as_float(v[j][i2]), sum[j][k + i2]);
              }
            }
          }
          if (++buf == BUFS) {
            buf = 0;
            bph ^= 1u;
          }
        };
#pragma unroll
        for (int d = 0; d < AHEAD; ++d) scales(d, x[d], w[d]);
        for (int i = 0; ok && i < st.len; i += AHEAD)
#pragma unroll
          for (int d = 0; d < AHEAD; ++d)
            if (ok && i + d < st.len) drain(i + d, x[d], w[d]);
        if (!ok) return;
#pragma unroll
        for (int k = 0; k < NT; ++k)
          if (k < nvalid) {
            float v[ACC];
#pragma unroll
            for (int j = 0; j < ACC; ++j) v[j] = sum[j][k];
            if (whole) {
              put<KIND, ACC, FN>(a, drow + k, f, v, true);
            } else {
#pragma unroll
              for (int j = 0; j < ACC; ++j) __stcg(part + (j * NT + k) * 128, v[j]);
            }
          }
      } else {
        if (!warp_wait(abort_flag, tfull_bar(buf), bph, a.err, a.limit_ns)) {
          ok = false;
          return;
        }
        tc_fence_after();
        const uint32_t tm = tm0 + buf * (ACC * NT);
#pragma unroll 1
        for (int c0 = 0; c0 < nvalid; c0 += 16) {
          uint32_t v[ACC][16];
#pragma unroll
          for (int j = 0; j < ACC; ++j) tmem_ld_32x32b_x16(tm + j * NT + c0, v[j]);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (c0 + i >= nvalid) break;
            float s[ACC];
#pragma unroll
            for (int j = 0; j < ACC; ++j) s[j] = __uint_as_float(v[j][i]);
            if (whole) {
              put<KIND, ACC, FN>(a, drow + c0 + i, f, s, true);
            } else {
#pragma unroll
              for (int j = 0; j < ACC; ++j) __stcg(part + (j * NT + c0 + i) * 128, s[j]);
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
      if (!whole) pass_on(st);
      else if (KIND == kUp) zero_rows<KIND, ACC, FN>(a, drow, f, nvalid, zero_to(nrows[t.e], row0, nvalid));
    };
    int t = c.t0, kb = c.kb0, left = c.len;
    while (ok && left > 0) {
      const Step st{t, kb, min(KB - kb, left), -1};
      take(st);
      left -= st.len;
      ++t;
      kb = 0;
    }
    if (npieces > 0)
      for (int r = 0; ok; ++r) {
        const int slot = r % kRing;
        if (!warp_wait(abort_flag, pfull_bar(slot), (r / kRing) & 1, a.err, a.limit_ns)) {
          ok = false;
          break;
        }
        const int id = ring[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(pempty_bar(slot));
        if (id >= npieces) break;
        take(piece(id));
      }
    if (ok) pass_on(Step{0, 0, 0, 0});
  } else {
    // ------------------------------------------------------------ joining parts (warps 6..9)
    const int lane128 = (warp - 6) * 32 + lane;
    if (KIND == kDown) pdl_wait();
    for (int jn = 0;; ++jn) {
      const int slot = jn % kJoin;
      // a part comes when its depth has been read: a whole share may lie before the first one
      bool got = false;
      for (int tries = 0; !got && tries < 8 && !*abort_flag; ++tries) got = mbar_poll(jfull_bar(slot), (jn / kJoin) & 1, a.limit_ns);
      // The four warps go on together or not at all: one that has seen its part wait there, beside
      // one that has seen the CTA give up and left, would wait for good.
      if (!all_meet<1, 128>(got)) {
        if (!got && !*abort_flag) atomicOr(a.err, DEVERR_TIMEOUT);
        *abort_flag = 1;
        break;
      }
      const Step st{joins[slot].x, joins[slot].y, joins[slot].z, joins[slot].w};
      __syncwarp();
      if (lane == 0) mbar_arrive(jempty_bar(slot));
      if (st.len == 0) break;
      // the last part of a tile to come adds them all, in the order of the depth
      int first, parts, counter;
      if (st.piece >= 0) {
        const int i = st.t - c.Ts;
        first = 2 * grid + i * c.P;
        parts = c.P;
        counter = grid + i;
      } else {
        const long long U = (long long)c.Ts * KB, u = (long long)st.t * KB;
        const int i0 = share_owner(U, c.G, u);
        parts = share_owner(U, c.G, u + KB - 1) - i0 + 1;
        first = 2 * i0 + 1;                  // the tile's first CTA, then slot 0 of the next ones
        counter = i0;
      }
      bool last = false;
      if (lane128 == 0) {
        last = atom_add_acq_rel(a.count + counter, 1u) == (unsigned)parts - 1u;
        if (last) a.count[counter] = 0u;
      }
      if (!any_meets<1, 128>(last)) continue;
      const Tile t = tile_at(st.t, pre, rtiles, a.E);
      const int row0 = t.rt * NT, nvalid = min(NT, nrows[t.e] - row0);
      const int f = t.nt * F::FEATURES + lane128;
      const int64_t drow = t.e * a.Cd + row0;
      const float* p0 = a.part + (size_t)first * (ACC * NT * 128) + lane128;
      // from one part's slot to the next: 1 for pieces; for shares 2 i0 + 1, 2 i0 + 2, 2 i0 + 4, ...
      auto at = [&](int i) {
        const int d = st.piece >= 0 ? i : i == 0 ? 0 : 2 * i - 1;
        return p0 + (size_t)d * (ACC * NT * 128);
      };
      // COLS columns at a time, PARTS of their parts in flight
      auto add = [&](auto cols, auto pcs) {
        constexpr int COLS = decltype(cols)::value, PARTS = decltype(pcs)::value;
#pragma unroll 1
        for (int c0 = 0; c0 < nvalid; c0 += COLS) {
          float s[ACC][COLS] = {};
#pragma unroll 1
          for (int i = 0; i < parts; i += PARTS) {
            float v[PARTS][ACC][COLS];
#pragma unroll
            for (int d = 0; d < PARTS; ++d) {
              const float* p = at(i + d);
#pragma unroll
              for (int j = 0; j < ACC; ++j)
#pragma unroll
                for (int k = 0; k < COLS; ++k)
                  v[d][j][k] = i + d < parts && c0 + k < nvalid ? __ldcg(p + (j * NT + c0 + k) * 128) : 0.f;
            }
#pragma unroll
            for (int d = 0; d < PARTS; ++d)
#pragma unroll
              for (int j = 0; j < ACC; ++j)
#pragma unroll
                for (int k = 0; k < COLS; ++k) s[j][k] += v[d][j][k];
          }
#pragma unroll
          for (int k = 0; k < COLS; ++k)
            if (c0 + k < nvalid) {
              float v[ACC];
#pragma unroll
              for (int j = 0; j < ACC; ++j) v[j] = s[j][k];
              put<KIND, ACC, FN>(a, drow + c0 + k, f, v, true);
            }
        }
      };
      if (nvalid <= 2) add(std::integral_constant<int, 2>{}, std::integral_constant<int, 16>{});
      else add(std::integral_constant<int, 8>{}, std::integral_constant<int, 4>{});
      if (KIND == kUp) zero_rows<KIND, ACC, FN>(a, drow, f, nvalid, zero_to(nrows[t.e], row0, nvalid));
    }
  }

  tc_fence_before();
  let_copies_land(abort_flag);
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

constexpr int kRowsBf16 = 16, kRowsFp8 = 32;     // most rows an expert may hold, and the widest tile

}  // namespace

size_t few_rows_workspace(bool fp8, int num_sms, size_t* counts) {
  *counts = (size_t)(1 + kPieces) * num_sms + 2;
  return (size_t)(2 + kPieces) * num_sms * 2 * (fp8 ? kRowsFp8 : kRowsBf16) * 128;
}

cudaError_t glu_few_up(const GluArgs& a) {
  CUtensorMap tmW, tmX;
  if (!encode_column_blocks(&tmW, a.W13, 2 * (uint64_t)a.H, (uint64_t)a.E * a.M, 2) ||
      !encode_2d(&tmX, a.x, a.M, (uint64_t)a.E * a.C, 64, kRowsBf16))
    return cudaErrorInvalidValue;
  FewArgs f{};
  f.n = a.n;
  f.E = a.E;
  f.C = (int)a.C;
  f.N = a.H;
  f.K = a.M;
  f.KB = a.M / 64;
  f.Cb = a.C;
  f.Cd = a.Cp;
  f.D = static_cast<__nv_bfloat16*>(a.h);
  f.gu = static_cast<uint16_t*>(a.gu);
  f.part = a.part;
  f.count = a.count;
  f.err = a.err;
  f.limit_ns = a.limit_ns;
  if (a.fn == kGluSilu) return launch<kUp, kRowsBf16, kGluSilu>(tmW, tmX, f, a.num_sms, a.st);
  if (a.fn == kGluGelu) return launch<kUp, kRowsBf16, kGluGelu>(tmW, tmX, f, a.num_sms, a.st);
  return launch<kUp, kRowsBf16, kGluRelu>(tmW, tmX, f, a.num_sms, a.st);
}

cudaError_t glu_few_down(const GluArgs& a) {
  CUtensorMap tmW, tmX;
  if (!encode_column_blocks(&tmW, a.W2, a.M, (uint64_t)a.E * a.H, 4) ||
      !encode_2d(&tmX, a.h, a.H, (uint64_t)a.E * a.Cp, 64, kRowsBf16))
    return cudaErrorInvalidValue;
  FewArgs f{};
  f.n = a.n;
  f.E = a.E;
  f.C = (int)a.C;
  f.N = a.M;
  f.K = a.H;
  f.KB = a.H / 64;
  f.Cb = a.Cp;
  f.Cd = a.C;
  f.D = static_cast<__nv_bfloat16*>(a.y);
  f.part = a.part;
  f.count = a.count;
  f.err = a.err;
  f.limit_ns = a.limit_ns;
  return launch<kDown, kRowsBf16, kGluSilu>(tmW, tmX, f, a.num_sms, a.st);
}

cudaError_t fp8_few(const Fp8Args& a) {
  const int nt = a.rows <= 16 ? 16 : 32;
  CUtensorMap tmW, tmX;
  if (!encode_2d_bytes(&tmW, a.wq, a.K, (uint64_t)a.E * a.N, 128, 256) ||
      !encode_2d_bytes(&tmX, a.xq, a.K, (uint64_t)a.E * a.C, 128, nt))
    return cudaErrorInvalidValue;
  FewArgs f{};
  f.n = a.n;
  f.E = a.E;
  f.C = (int)a.C;
  f.N = a.N;
  f.KB = (a.K + 127) / 128;
  f.NB = (a.N + 127) / 128;
  f.Cb = a.C;
  f.Cd = a.C;
  f.D = static_cast<__nv_bfloat16*>(a.y);
  f.xs = a.xs;
  f.ws = a.ws;
  f.part = a.part;
  f.count = a.count;
  f.err = a.err;
  f.limit_ns = a.limit_ns;
  return nt == 16 ? launch<kFp8, 16, kGluSilu>(tmW, tmX, f, a.num_sms, a.st) : launch<kFp8, 32, kGluSilu>(tmW, tmX, f, a.num_sms, a.st);
}

// When this file's kernels run.  Measured with all experts full, in us, this file's kernels :
// 256 x 256 tiles.  The joining of parts grows with the rows, so few rows win, and in bf16, where tiles come near the memory's
// rate too, with 9 to 16 rows only many weights.
//   gated experts, E x M x H, rows 1 / 8 / 16 / 32:
//     1 x 1024 x 4096    19 : 24    22 : 23    27 : 23    37 : 23
//     1 x 2048 x 8192    29 : 45    33 : 42    41 : 44    53 : 40
//     8 x 1024 x 4096    47 : 60    50 : 51    54 : 53    66 : 52
//     32 x 1024 x 4096  135 : 168  142 : 162  155 : 165  178 : 168
//   8-bit product, E x K x N, rows 1 / 16 / 32 / 64:
//     1 x 1456 x 2008    10 : 11    11 : 13    14 : 13    17 : 13
//     1 x 7168 x 4096    12 : 18    16 : 24    23 : 23    30 : 25
//     8 x 7168 x 4096    48 : 68    53 : 69    67 : 67    88 : 70
//     32 x 2048 x 7168   80 : 131   87 : 137  106 : 136  213 : 142
bool glu_few(const GluArgs& a) {
  return a.rows <= 8 || (a.rows <= kRowsBf16 && (int64_t)a.E * a.M * a.H >= (1 << 24));
}

// Both sides run both products of the gated experts alike, so that `down` finds `up` before it.
cudaError_t glu_up(const GluArgs& a, bool bf16) {
  if (!bf16) return glu_up_f32(a);
  return glu_few(a) ? glu_few_up(a) : glu_up_bf16(a);
}

cudaError_t glu_down(const GluArgs& a, bool bf16) {
  if (!bf16) return glu_down_f32(a);
  return glu_few(a) ? glu_few_down(a) : glu_down_bf16(a);
}

int glu_down_kernels(const GluArgs& a, bool bf16) {
  return (bf16 ? (glu_few(a) ? 1 : glu_down_shares_bf16(a)) : glu_down_shares_f32(a)) > 1 ? 2 : 1;
}

int glu_dx_kernels(const GluArgs& a, bool bf16) {
  return (bf16 ? glu_dx_shares_bf16(a) : glu_dx_shares_f32(a)) > 1 ? 2 : 1;
}

int fp8_matmul_kernels(const Fp8Args& a) { return a.rows > kRowsFp8 && fp8_shares(a) > 1 ? 2 : 1; }

cudaError_t fp8_matmul(const Fp8Args& a) { return a.rows <= kRowsFp8 ? fp8_few(a) : fp8_pair(a); }

}  // namespace moe
