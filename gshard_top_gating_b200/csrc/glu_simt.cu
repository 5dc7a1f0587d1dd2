// glu_simt.cu -- gated experts in fp32 on CUDA cores (FFMA): tensor cores would round the
// inputs to 11 bits.  The products of glu_tc.cu, one grouped kernel each:
//
//   C_e(i, j) = sum_k A_e(i, k) B_e(k, j)
//
// with the rows i (or, for the weight gradients, the depth k) limited to the n rows expert e
// holds; rows past them are neither read nor written.  A tile of T x T results per block
// of 256 threads, T/16 x T/16 each, depth in steps of TK through shared memory with the
// next step's operands in registers meanwhile.  A thread's columns lie in two groups, one in
// each half of the tile: in `up` the first half holds columns of Wg and the second the same
// columns of Wu, so that g and u of an element meet in one thread.
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
};

// AT: A's rows are contiguous (A(i, k) at k * lda + i), else its depth (i * lda + k).
// BT: B's depth is contiguous (B(k, j) at j * ldb + k), else its columns (k * ldb + j).
template <int T, int TK, bool AT, bool BT, int EPI, int FN>
__global__ void __launch_bounds__(kThreads) glu_simt_kernel(const SimtArgs g) {
  // small tiles: four groups of 64 threads take a quarter of each step's depth each, so that
  // every thread still has 4 x 4 results (with 2 x 2, shared-memory loads bound the step)
  constexpr int KS = T == 32 ? 4 : 1, SIDE = T == 32 ? 8 : 16;
  constexpr int R = T / SIDE, G = T / (2 * SIDE);       // rows and columns-per-half of a thread
  pdl_wait();
  pdl_trigger();
  const int e = blockIdx.z;
  const int n = min(max(g.n[e], 0), g.C);
  const int rows = g.rows ? g.rows : n, K = g.K ? g.K : n;
  // `up`: the tile is T/2 columns of g beside the same T/2 columns of u
  constexpr int CW = EPI == kSUp ? T / 2 : T;
  const int i0 = blockIdx.y * T, j0 = blockIdx.x * CW;
  if (i0 >= rows || (g.skip_empty && n == 0)) return;
  const float* A = g.A + e * g.a_z;
  const float* B = g.B + e * g.b_z;
  __shared__ __align__(16) float shared[2][TK][T + 4];
  auto& As = shared[0];
  auto& Bs = shared[1];
  const int tid = threadIdx.x, ks = tid / (SIDE * SIDE);
  const int tx = tid % SIDE, ty = tid / SIDE % SIDE;
  constexpr int L = T * TK / (4 * kThreads);   // float4 loads per thread and operand
  float4 ra[L], rb[L];

  auto load = [&](int k0) {
#pragma unroll
    for (int l = 0; l < L; ++l) {
      const int idx = tid + l * kThreads;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (AT) {            // four rows i of one k
        const int k = k0 + idx / (T / 4), i = i0 + idx % (T / 4) * 4;
        if (k < K && i < rows) v = *reinterpret_cast<const float4*>(A + (int64_t)k * g.lda + i);
      } else {             // four k of one row i
        const int i = i0 + idx / (TK / 4), k = k0 + idx % (TK / 4) * 4;
        if (i < rows && k < K) v = *reinterpret_cast<const float4*>(A + (int64_t)i * g.lda + k);
      }
      ra[l] = v;
      v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (BT) {
        const int j = j0 + idx / (TK / 4), k = k0 + idx % (TK / 4) * 4;
        if (j < g.cols && k < K) v = *reinterpret_cast<const float4*>(B + (int64_t)j * g.ldb + k);
      } else {
        const int k = k0 + idx / (T / 4);
        int j = idx % (T / 4) * 4;
        bool in;
        if (EPI == kSUp) {
          in = j0 + (j & (CW - 1)) < g.H;
          j = (j < CW ? j0 : g.H + j0 - CW) + j;
        } else {
          j += j0;
          in = j < g.cols;
        }
        if (k < K && in) v = *reinterpret_cast<const float4*>(B + (int64_t)k * g.ldb + j);
      }
      rb[l] = v;
    }
  };
  auto put = [&](float (&S)[TK][T + 4], const float4 (&r)[L], bool along_k) {
#pragma unroll
    for (int l = 0; l < L; ++l) {
      const int idx = tid + l * kThreads;
      if (along_k) {
        const int i = idx / (TK / 4), k = idx % (TK / 4) * 4;
        S[k][i] = r[l].x;
        S[k + 1][i] = r[l].y;
        S[k + 2][i] = r[l].z;
        S[k + 3][i] = r[l].w;
      } else {
        *reinterpret_cast<float4*>(&S[idx / (T / 4)][idx % (T / 4) * 4]) = r[l];
      }
    }
  };

  float acc[R][2 * G] = {};
  load(0);
  for (int k0 = 0; k0 < K; k0 += TK) {
    put(As, ra, !AT);
    put(Bs, rb, BT);
    __syncthreads();
    if (k0 + TK < K) load(k0 + TK);
#pragma unroll
    for (int kk = 0; kk < TK / KS; ++kk) {
      const int k = ks * (TK / KS) + kk;
      float av[R], bv[2 * G];
#pragma unroll
      for (int r = 0; r < R; ++r) av[r] = As[k][ty * R + r];
#pragma unroll
      for (int c = 0; c < G; ++c) {
        bv[c] = Bs[k][tx * G + c];
        bv[G + c] = Bs[k][T / 2 + tx * G + c];
      }
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < 2 * G; ++c) acc[r][c] = fmaf(av[r], bv[c], acc[r][c]);
    }
    __syncthreads();
  }

  if constexpr (KS > 1) {
    // the groups' sums meet in the operands' memory; group ks keeps row ks of each 4 x 4
    static_assert(KS == R && KS * T * T <= 2 * TK * (T + 4), "the sums fit into the operands' memory");
    float* sums = &shared[0][0][0];            // [group][thread][R][2 G]; the last step's reads are done
    const int t0 = tid % (SIDE * SIDE);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < 2 * G; ++c) sums[((r * 2 * G + c) * KS + ks) * SIDE * SIDE + t0] = acc[r][c];
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 2 * G; ++c) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k) s += sums[((ks * 2 * G + c) * KS + k) * SIDE * SIDE + t0];
#pragma unroll
      for (int r = 0; r < R; ++r) acc[r][c] = s;      // one of the rows below is used: r = ks
    }
  }
  float* D = g.D + e * g.d_z;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = i0 + ty * R + r;
    if (i >= rows || (KS > 1 && r != ks)) continue;
    if (EPI == kSUp) {
#pragma unroll
      for (int c = 0; c < G; ++c) {
        const int j = j0 + tx * G + c;
        if (j >= g.H) continue;
        D[(int64_t)i * g.ldd + j] = glu_f<FN, false>(acc[r][c]) * acc[r][G + c];
        if (g.gu) {
          float* gu = g.gu + e * g.gu_z + (int64_t)i * 2 * g.H;
          gu[j] = acc[r][c];
          gu[g.H + j] = acc[r][G + c];
        }
      }
    } else {
#pragma unroll
      for (int c = 0; c < 2 * G; ++c) {
        const int j = j0 + (c < G ? tx * G + c : T / 2 + tx * G + c - G);
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

// Tiles of 128 x 128 when they fill the device twice over, else of 64 x 64 when those fill it,
// else of 32 x 32 with four times the depth per step: small products are bound by the
// latency of their steps (a training step of 8 experts x 80 rows, M = 64, H = 256: 72 us with
// 64 x 64 tiles of depth 16 throughout, 55 us).
template <bool AT, bool BT, int EPI, int FN>
cudaError_t launch(const SimtArgs& g, int64_t rows, int cols, int E, int num_sms, cudaStream_t st) {
  auto tiles = [&](int T) { return (rows + T - 1) / T * ((cols + T - 1) / T) * E; };
  const int T = tiles(128) >= 2 * num_sms ? 128 : tiles(64) >= num_sms ? 64 : 32;
  const int cw = EPI == kSUp ? T / 2 : T;
  const dim3 grid((cols / (EPI == kSUp ? 2 : 1) + cw - 1) / cw, (unsigned)((rows + T - 1) / T), E);
  if (T == 128) return launch_pdl(glu_simt_kernel<128, 16, AT, BT, EPI, FN>, grid, dim3(kThreads), 0, st, g);
  if (T == 64) return launch_pdl(glu_simt_kernel<64, 16, AT, BT, EPI, FN>, grid, dim3(kThreads), 0, st, g);
  return launch_pdl(glu_simt_kernel<32, 64, AT, BT, EPI, FN>, grid, dim3(kThreads), 0, st, g);
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
  g.C = (int)a.C;
  return g;
}

}  // namespace

cudaError_t glu_up_f32(const GluArgs& a) {
  const int64_t w = (int64_t)a.M * 2 * a.H;
  const SimtArgs g = simt_args(a, a.x, a.C * a.M, a.M, a.W13, w, 2 * a.H, a.h, a.Cp * a.H, a.H, 0, 2 * a.H, a.M);
  return launch_fn<false, false, kSUp>(a.fn, g, a.C, 2 * a.H, a.E, a.num_sms, a.st);
}

cudaError_t glu_down_f32(const GluArgs& a) {
  const int64_t w = (int64_t)a.H * a.M;
  const SimtArgs g = simt_args(a, a.h, a.Cp * a.H, a.H, a.W2, w, a.M, a.y, a.C * a.M, a.M, 0, a.M, a.H);
  return launch<false, false, kSPlain, kGluSilu>(g, a.C, a.M, a.E, a.num_sms, a.st);
}

cudaError_t glu_dh_f32(const GluArgs& a) {
  const int64_t w = (int64_t)a.H * a.M;
  const SimtArgs g = simt_args(a, a.dy, a.C * a.M, a.M, a.W2, w, a.M, a.dgu, a.Cp * 2 * a.H, 2 * a.H, 0, a.H, a.M);
  return launch_fn<false, true, kSDh>(a.fn, g, a.C, a.H, a.E, a.num_sms, a.st);
}

cudaError_t glu_dx_f32(const GluArgs& a) {
  const int64_t w = (int64_t)a.M * 2 * a.H;
  const SimtArgs g =
      simt_args(a, a.dgu, a.Cp * 2 * a.H, 2 * a.H, a.W13, w, 2 * a.H, a.dx, a.C * a.M, a.M, 0, a.M, 2 * a.H);
  return launch<false, true, kSPlain, kGluSilu>(g, a.C, a.M, a.E, a.num_sms, a.st);
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
