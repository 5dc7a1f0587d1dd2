// split.cu -- products of 256-row tiles (fp32: of 32) that are too few for the device, cut
// along the depth: each of `splits` CTA pairs (blocks) takes a share of a tile's depth and
// stores its fp32 sums, and one more kernel adds them in order of the depth and rounds to the
// result's type.
//
// It costs that kernel, about 7 us, and the sums' way to memory and back, 0.13 us for every
// tile of them; it saves depth.  One expert of 256 rows, H = 4096 -> M = 1024, has 4 tiles for
// 74 pairs: the two products of the gated experts take 37 us in one piece, 28 us with the
// second in shares (2048 and 8192: 91 and 57 us).
#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

// 8 columns per thread, experts in grid.y.
template <typename T>
__global__ void __launch_bounds__(256) split_join_kernel(const float* __restrict__ part, T* __restrict__ y,
                                                         const int32_t* __restrict__ nexp, int rows, int64_t C, int N,
                                                         int splits) {
  pdl_wait();
  pdl_trigger();
  const int e = blockIdx.y, E = gridDim.y;
  const int n = min(max(nexp[e], 0), rows);
  const int per = N / 8;                      // N is a multiple of 8
  const int64_t step = (int64_t)E * rows * N;
  for (int i = blockIdx.x * 256 + threadIdx.x; i < n * per; i += gridDim.x * 256) {
    const int r = i / per, c = (i - r * per) * 8;
    const float4* p = reinterpret_cast<const float4*>(part + ((int64_t)e * rows + r) * N + c);
    float s[8] = {};
#pragma unroll 4
    for (int k = 0; k < splits; ++k) {
      const float4 a = __ldcg(p + k * step / 4), b = __ldcg(p + k * step / 4 + 1);
      s[0] += a.x;
      s[1] += a.y;
      s[2] += a.z;
      s[3] += a.w;
      s[4] += b.x;
      s[5] += b.y;
      s[6] += b.z;
      s[7] += b.w;
    }
    T* out = y + ((int64_t)e * C + r) * N + c;
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<uint4*>(out) =
          make_uint4(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]), pack_bf16x2(s[4], s[5]), pack_bf16x2(s[6], s[7]));
    } else {
      reinterpret_cast<float4*>(out)[0] = make_float4(s[0], s[1], s[2], s[3]);
      reinterpret_cast<float4*>(out)[1] = make_float4(s[4], s[5], s[6], s[7]);
    }
  }
}

constexpr int kMostSplits = 8;
constexpr double kJoinUs = 7.0, kTileUs = 0.13;     // measured: the kernel; a tile's sums, out and in

}  // namespace

int split_count(int E, int64_t rows, int N, int TN, int KB, double block_us, int num_sms) {
  const int64_t tiles = (int64_t)E * ((rows + 255) / 256) * ((N + TN - 1) / TN);
  const double sums = (double)E * rows * N / 65536.0;      // full tiles' worth
  int best = 1;
  double gain = 0.0;
  for (int s = 2; s <= kMostSplits && s * tiles <= num_sms / 2 && s <= KB; ++s) {
    const double g = KB * block_us * (1.0 - 1.0 / s) - kJoinUs - kTileUs * s * sums;
    if (g > gain) {
      gain = g;
      best = s;
    }
  }
  return best;
}

// tiles x splits stays within the pairs, so the sums take at most a tile per pair.
size_t split_workspace(int E, int N, int num_sms) {
  return (int64_t)E * ((N + 255) / 256) * 2 <= num_sms / 2 ? (size_t)(num_sms / 2) * 256 * 256 : 0;
}

namespace {

template <typename T>
cudaError_t launch_join(const float* part, T* y, const int32_t* n, int E, int64_t rows, int64_t C, int N, int splits,
                        int num_sms, cudaStream_t st) {
  const int64_t work = (rows * (N / 8) + 255) / 256, most = (num_sms * 8 + E - 1) / E;
  return launch_pdl(split_join_kernel<T>, dim3((unsigned)(work < most ? work : most), E), dim3(256), 0, st, part, y, n,
                    (int)rows, C, N, splits);
}

}  // namespace

cudaError_t split_join(const float* part, void* y, bool bf16, const int32_t* n, int E, int64_t rows, int64_t C, int N,
                       int splits, int num_sms, cudaStream_t st) {
  if (bf16) return launch_join(part, static_cast<__nv_bfloat16*>(y), n, E, rows, C, N, splits, num_sms, st);
  return launch_join(part, static_cast<float*>(y), n, E, rows, C, N, splits, num_sms, st);
}

}  // namespace moe
