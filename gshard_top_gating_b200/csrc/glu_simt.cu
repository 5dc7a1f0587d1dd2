// glu_simt.cu -- gated experts in fp32 on CUDA cores (FFMA): tensor cores would round the
// inputs to 11 bits.  The products of glu_tc.cu, one grouped kernel each:
//
//   C_e(i, j) = sum_k A_e(i, k) B_e(k, j)
//
// with the rows i (or, for the weight gradients, the depth k) limited to the n rows expert e
// holds; rows past them are neither read nor written.  A tile of T x T results per block
// of 256 threads; the depth comes in steps of TK through shared memory, four steps in flight
// (cp.async), each operand laid out as it lies in memory: along the depth, a thread reads four
// k of a row at once.  A thread's columns are SIDE apart, so that neighbours read and write
// neighbouring columns; in `up` the tile's first half holds columns of Wg and the second the
// same columns of Wu, so that g and u of an element meet in one thread.
#include "glu.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
enum { kSPlain = 0, kSUp = 1, kSDh = 2 };

struct SimtArgs {
  const float *A, *B;
  float* D;
  int64_t a_z, b_z, d_z;   // per expert
  int lda, ldb, ldd;
  int rows, cols, K;       // rows / K: 0 = the expert's count n
  int H;                   // kSUp, kSDh
  float* gu;               // kSUp: [g|u] out (or null); kSDh: in.  Rows of 2H, per expert gu_z
  int64_t gu_z;
  const int32_t* n;
  int C;
  int skip_empty;          // weight gradients of an expert without rows stay as they are
  int splits;              // shares of the depth: 1, or D is [splits][E, most rows, cols] (split.cu)
  int64_t s_z;             // splits > 1: from one share's sums to the next
};

__device__ __forceinline__ void cp_async16(float* dst, const float* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(live ? 16 : 0) : "memory");
}

constexpr int kSteps = 4;      // steps of the depth in flight

// Floats of one operand's step: rows of TK (its depth contiguous) or of T values, padded by 16
// bytes, which keeps both the copies' alignment and the reads free of bank conflicts.
template <int T, int TK>
constexpr int step_floats(bool along_k) { return along_k ? T * (TK + 4) : TK * (T + 4); }
template <int T, int TK, bool AT, bool BT>
constexpr size_t simt_smem() { return kSteps * (step_floats<T, TK>(!AT) + step_floats<T, TK>(BT)) * sizeof(float); }

// AT: A's rows are contiguous (A(i, k) at k * lda + i), else its depth (i * lda + k).
// BT: B's depth is contiguous (B(k, j) at j * ldb + k), else its columns (k * ldb + j).
template <int T, int TK, bool AT, bool BT, int EPI, int FN>
__global__ void __launch_bounds__(kThreads, 2) glu_simt_kernel(const SimtArgs g) {
  pdl_wait();
  pdl_trigger();
  // smaller tiles: four groups of 64 threads take a quarter of each step's depth each, so that
  // a thread still has 8 x 8 (4 x 4) results; with a quarter of them, shared-memory loads
  // bound the step
  constexpr int KS = T == 128 ? 1 : 4, SIDE = T == 128 ? 16 : 8;
  constexpr int R = T / SIDE, W = T / SIDE;   // rows and columns of a thread
  constexpr int FA = step_floats<T, TK>(!AT), FB = step_floats<T, TK>(BT);
  const int e = blockIdx.z / g.splits, share = blockIdx.z % g.splits;
  const int n = min(max(g.n[e], 0), g.C);
  const int rows = g.rows ? g.rows : n, K = g.K ? g.K : n;
  // `up`: the tile is T/2 columns of g beside the same T/2 columns of u
  constexpr int CW = EPI == kSUp ? T / 2 : T;
  const int i0 = blockIdx.y * T, j0 = blockIdx.x * CW;
  if (i0 >= rows || (g.skip_empty && n == 0)) return;
  const float* A = g.A + e * g.a_z;
  const float* B = g.B + e * g.b_z;
  extern __shared__ __align__(16) float simt_shared[];
  float* const As = simt_shared;
  float* const Bs = simt_shared + kSteps * FA;
  const int tid = threadIdx.x, ks = tid / (SIDE * SIDE);
  const int tx = tid % SIDE, ty = tid / SIDE % SIDE;

  // this thread's rows: contiguous where four of them are read at once, else SIDE apart, which
  // spreads a warp's rows over the banks
  auto row_of = [&](int r) { return AT ? ty * R + r : ty + SIDE * r; };

  auto load = [&](int step) {
    const int k0 = step * TK;
    float* as = As + step % kSteps * FA;
    float* bs = Bs + step % kSteps * FB;
    for (int idx = tid; idx < T * TK / 4; idx += kThreads) {
      if (AT) {            // four rows i of one k
        const int k = idx / (T / 4), i = idx % (T / 4) * 4;
        const bool in = k0 + k < K && i0 + i < rows;
        cp_async16(as + k * (T + 4) + i, in ? A + (int64_t)(k0 + k) * g.lda + i0 + i : A, in);
      } else {             // four k of one row i
        const int i = idx / (TK / 4), k = idx % (TK / 4) * 4;
        const bool in = i0 + i < rows && k0 + k < K;
        cp_async16(as + i * (TK + 4) + k, in ? A + (int64_t)(i0 + i) * g.lda + k0 + k : A, in);
      }
      if (BT) {
        const int j = idx / (TK / 4), k = idx % (TK / 4) * 4;
        const bool in = j0 + j < g.cols && k0 + k < K;
        cp_async16(bs + j * (TK + 4) + k, in ? B + (int64_t)(j0 + j) * g.ldb + k0 + k : B, in);
      } else {
        const int k = idx / (T / 4), j = idx % (T / 4) * 4;
        const int col = EPI == kSUp ? (j < CW ? j0 + j : g.H + j0 + j - CW) : j0 + j;
        const bool in = k0 + k < K && (EPI == kSUp ? j0 + (j < CW ? j : j - CW) < g.H : j0 + j < g.cols);
        cp_async16(bs + k * (T + 4) + j, in ? B + (int64_t)(k0 + k) * g.ldb + col : B, in);
      }
    }
  };

  const int all = (K + TK - 1) / TK;
  const int from = all * share / g.splits, steps = all * (share + 1) / g.splits;
#pragma unroll
  for (int s = 0; s < kSteps - 1; ++s) {
    if (from + s < steps) load(from + s);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  float acc[R][W] = {};
  for (int step = from; step < steps; ++step) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kSteps - 2) : "memory");
    __syncthreads();                 // this step is here for all, and all have read the one that `load` overwrites
    if (step + kSteps - 1 < steps) load(step + kSteps - 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
    const float* as = As + step % kSteps * FA;
    const float* bs = Bs + step % kSteps * FB;
#pragma unroll
    for (int kq = 0; kq < TK / KS; kq += 4) {
      const int k = ks * (TK / KS) + kq;
      float av[4][R], bv[4][W];
      if (AT) {
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
          for (int r = 0; r < R; r += 4)
            *reinterpret_cast<float4*>(&av[d][r]) = *reinterpret_cast<const float4*>(as + (k + d) * (T + 4) + ty * R + r);
      } else {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float4 v = *reinterpret_cast<const float4*>(as + row_of(r) * (TK + 4) + k);
          av[0][r] = v.x;
          av[1][r] = v.y;
          av[2][r] = v.z;
          av[3][r] = v.w;
        }
      }
      if (BT) {
#pragma unroll
        for (int c = 0; c < W; ++c) {
          const float4 v = *reinterpret_cast<const float4*>(bs + (tx + SIDE * c) * (TK + 4) + k);
          bv[0][c] = v.x;
          bv[1][c] = v.y;
          bv[2][c] = v.z;
          bv[3][c] = v.w;
        }
      } else {
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
          for (int c = 0; c < W; ++c) bv[d][c] = bs[(k + d) * (T + 4) + tx + SIDE * c];
      }
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int c = 0; c < W; ++c) acc[r][c] = fmaf(av[d][r], bv[d][c], acc[r][c]);
    }
  }

  if constexpr (KS > 1) {
    // the groups' sums meet in the operands' memory; group ks keeps rows ks, ks + 4, ...
    static_assert(KS * T * T <= kSteps * (FA + FB), "the sums fit into the operands' memory");
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    float* sums = simt_shared;
    const int t0 = tid % (SIDE * SIDE);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < W; ++c) sums[((r * W + c) * KS + ks) * SIDE * SIDE + t0] = acc[r][c];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (r % KS == ks) {
#pragma unroll
        for (int c = 0; c < W; ++c) {
          float s = 0.f;
#pragma unroll
          for (int k = 0; k < KS; ++k) s += sums[((r * W + c) * KS + k) * SIDE * SIDE + t0];
          acc[r][c] = s;
        }
      }
  }
  float* D = g.D + e * g.d_z + share * g.s_z;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = i0 + row_of(r);
    if (i >= rows || (KS > 1 && r % KS != ks)) continue;
    if (EPI == kSUp) {
#pragma unroll
      for (int c = 0; c < W / 2; ++c) {
        const int j = j0 + tx + SIDE * c;
        if (j >= g.H) continue;
        D[(int64_t)i * g.ldd + j] = glu_f<FN, false>(acc[r][c]) * acc[r][W / 2 + c];
        if (g.gu) {
          float* gu = g.gu + e * g.gu_z + (int64_t)i * 2 * g.H;
          gu[j] = acc[r][c];
          gu[g.H + j] = acc[r][W / 2 + c];
        }
      }
    } else {
#pragma unroll
      for (int c = 0; c < W; ++c) {
        const int j = j0 + tx + SIDE * c;
        if (j >= g.cols) continue;
        if (EPI == kSDh) {
          const float* gu = g.gu + e * g.gu_z + (int64_t)i * 2 * g.H;
          float f, df;
          glu_f_df<FN, false>(gu[j], f, df);
          D[(int64_t)i * g.ldd + j] = acc[r][c] * gu[g.H + j] * df;
          D[(int64_t)i * g.ldd + g.H + j] = acc[r][c] * f;
        } else {
          D[(int64_t)i * g.ldd + j] = acc[r][c];
        }
      }
    }
  }
}

template <int T, int TK, bool AT, bool BT, int EPI, int FN>
cudaError_t launch_tile(const SimtArgs& g, dim3 grid, cudaStream_t st) {
  auto kern = glu_simt_kernel<T, TK, AT, BT, EPI, FN>;
  constexpr size_t smem = simt_smem<T, TK, AT, BT>();
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kern, grid, dim3(kThreads), smem, st, g);
}

// Tiles of 128 x 128 when they fill the device twice over, else of 64 x 64 when those fill it,
// else of 32 x 32: small products are bound by the
// latency of their steps (a training step of 8 experts x 80 rows, M = 64, H = 256: 72 us with
// 64 x 64 tiles and one step in flight, 39 us).
int tile_of(int64_t rows, int cols, int E, int num_sms) {
  auto tiles = [&](int T) { return (rows + T - 1) / T * ((cols + T - 1) / T) * E; };
  return tiles(128) >= 2 * num_sms ? 128 : tiles(64) >= num_sms ? 64 : 32;
}

template <bool AT, bool BT, int EPI, int FN>
cudaError_t launch(const SimtArgs& g, int64_t rows, int cols, int E, int num_sms, cudaStream_t st) {
  const int T = tile_of(rows, cols, E, num_sms);
  const int cw = EPI == kSUp ? T / 2 : T;
  const dim3 grid((cols / (EPI == kSUp ? 2 : 1) + cw - 1) / cw, (unsigned)((rows + T - 1) / T), E * g.splits);
  if (T == 128) return launch_tile<128, 16, AT, BT, EPI, FN>(g, grid, st);
  if (T == 64) return launch_tile<64, 32, AT, BT, EPI, FN>(g, grid, st);
  return launch_tile<32, 32, AT, BT, EPI, FN>(g, grid, st);
}

// down and dx where 32 x 32 tiles leave SMs idle over a long depth: in shares of at least 256,
// joined by one more kernel (one row, M = 64, H = 2944, forward: 38 -> 15 us; 2 x 155 rows, M = 320, H = 4800: 186 -> 139 us).
constexpr int kShareK = 256;
int shares_of(const GluArgs& a, int cols, int K) {
  if (tile_of(a.rows, cols, a.E, a.num_sms) != 32) return 1;
  const int64_t tiles = (a.rows + 31) / 32 * ((cols + 31) / 32) * a.E, s = 2 * a.num_sms / tiles;
  const int most = K / kShareK;
  return s < 2 || most < 2 ? 1 : s < most ? (int)s : most;
}

template <bool BT>
cudaError_t launch_shares(SimtArgs g, const GluArgs& a, int K, float* out) {
  const int s = shares_of(a, g.cols, K);
  if (s == 1) return launch<false, BT, kSPlain, kGluSilu>(g, a.rows, g.cols, a.E, a.num_sms, a.st);
  g.splits = s;
  g.D = a.part;
  g.ldd = g.cols;
  g.d_z = a.rows * g.cols;
  g.s_z = a.E * g.d_z;
  const cudaError_t e = launch<false, BT, kSPlain, kGluSilu>(g, a.rows, g.cols, a.E, a.num_sms, a.st);
  if (e != cudaSuccess) return e;
  return split_join(a.part, out, false, a.n, a.E, a.rows, a.C, g.cols, s, a.num_sms, a.st);
}

template <bool AT, bool BT, int EPI>
cudaError_t launch_fn(int fn, const SimtArgs& g, int64_t rows, int cols, int E, int num_sms, cudaStream_t st) {
  if (fn == kGluSilu) return launch<AT, BT, EPI, kGluSilu>(g, rows, cols, E, num_sms, st);
  if (fn == kGluGelu) return launch<AT, BT, EPI, kGluGelu>(g, rows, cols, E, num_sms, st);
  return launch<AT, BT, EPI, kGluRelu>(g, rows, cols, E, num_sms, st);
}

SimtArgs simt_args(const GluArgs& a, const void* A, int64_t a_z, int lda, const void* B, int64_t b_z, int ldb, void* D,
                   int64_t d_z, int ldd, int rows, int cols, int K) {
  SimtArgs g{};
  g.A = static_cast<const float*>(A);
  g.B = static_cast<const float*>(B);
  g.D = static_cast<float*>(D);
  g.a_z = a_z;
  g.b_z = b_z;
  g.d_z = d_z;
  g.lda = lda;
  g.ldb = ldb;
  g.ldd = ldd;
  g.rows = rows;
  g.cols = cols;
  g.K = K;
  g.H = a.H;
  g.gu = static_cast<float*>(a.gu);
  g.gu_z = a.Cp * 2 * a.H;
  g.n = a.n;
  g.C = (int)a.rows;
  g.splits = 1;
  return g;
}

}  // namespace

// tiles x shares stays within two tiles of 32 x 32 per SM.
size_t glu_f32_workspace(int num_sms) { return (size_t)2 * num_sms * 32 * 32; }

int glu_down_shares_f32(const GluArgs& a) { return shares_of(a, a.M, a.H); }
int glu_dx_shares_f32(const GluArgs& a) { return shares_of(a, a.M, 2 * a.H); }

cudaError_t glu_up_f32(const GluArgs& a) {
  const int64_t w = (int64_t)a.M * 2 * a.H;
  const SimtArgs g = simt_args(a, a.x, a.C * a.M, a.M, a.W13, w, 2 * a.H, a.h, a.Cp * a.H, a.H, 0, 2 * a.H, a.M);
  return launch_fn<false, false, kSUp>(a.fn, g, a.rows, 2 * a.H, a.E, a.num_sms, a.st);
}

cudaError_t glu_down_f32(const GluArgs& a) {
  const int64_t w = (int64_t)a.H * a.M;
  const SimtArgs g = simt_args(a, a.h, a.Cp * a.H, a.H, a.W2, w, a.M, a.y, a.C * a.M, a.M, 0, a.M, a.H);
  return launch_shares<false>(g, a, a.H, static_cast<float*>(a.y));
}

cudaError_t glu_dh_f32(const GluArgs& a) {
  const int64_t w = (int64_t)a.H * a.M;
  const SimtArgs g = simt_args(a, a.dy, a.C * a.M, a.M, a.W2, w, a.M, a.dgu, a.Cp * 2 * a.H, 2 * a.H, 0, a.H, a.M);
  return launch_fn<false, true, kSDh>(a.fn, g, a.rows, a.H, a.E, a.num_sms, a.st);
}

cudaError_t glu_dx_f32(const GluArgs& a) {
  const int64_t w = (int64_t)a.M * 2 * a.H;
  const SimtArgs g =
      simt_args(a, a.dgu, a.Cp * 2 * a.H, 2 * a.H, a.W13, w, 2 * a.H, a.dx, a.C * a.M, a.M, 0, a.M, 2 * a.H);
  return launch_shares<true>(g, a, 2 * a.H, static_cast<float*>(a.dx));
}

cudaError_t glu_dw2_f32(const GluArgs& a) {
  SimtArgs g = simt_args(a, a.h, a.Cp * a.H, a.H, a.dy, a.C * a.M, a.M, a.dW2, (int64_t)a.H * a.M, a.M, a.H, a.M, 0);
  g.skip_empty = a.skip_empty;
  return launch<true, false, kSPlain, kGluSilu>(g, a.H, a.M, a.E, a.num_sms, a.st);
}

cudaError_t glu_dw13_f32(const GluArgs& a) {
  SimtArgs g = simt_args(a, a.x, a.C * a.M, a.M, a.dgu, a.Cp * 2 * a.H, 2 * a.H, a.dW13, (int64_t)a.M * 2 * a.H, 2 * a.H,
                         a.M, 2 * a.H, 0);
  g.skip_empty = a.skip_empty;
  return launch<true, false, kSPlain, kGluSilu>(g, a.M, 2 * a.H, a.E, a.num_sms, a.st);
}

}  // namespace moe
