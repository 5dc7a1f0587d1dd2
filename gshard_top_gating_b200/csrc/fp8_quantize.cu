// fp8_quantize.cu -- e4m3 values with one fp32 scale per block of 128: rows (1 x 128 blocks)
// and weights (128 x 128 blocks).
//
//   a = max(amax |x| over the block, 2^-100),  s = a / 448,  q = e4m3(x * (448 / a))
//
// rounded to nearest even; 448 is e4m3's largest value, and x * (448 / a) exceeds it by less
// than the half step that would round past it.  2^-100 keeps 448 / a finite: a block of
// zeros gets q = 0 and the scale 2^-100 / 448.  A block with a NaN becomes all NaN; one with
// an infinity gets s = inf, whose products are NaN or infinite as well.
#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr float kMax = 448.f;
constexpr float kTiny = 7.888609052210118e-31f;     // 2^-100

// max(|a|, |b|) that keeps a NaN
__device__ __forceinline__ float amax2(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

template <bool BF16>
__device__ __forceinline__ void load8(const void* x, int64_t i, float (&v)[8]) {
  if (BF16) {
    const uint4 r = ld_nc_v4(static_cast<const char*>(x) + i * 2);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = bf16lo(w[j]);
      v[2 * j + 1] = bf16hi(w[j]);
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 r = ld_nc_v4(static_cast<const char*>(x) + i * 4 + h * 16);
      v[4 * h] = __uint_as_float(r.x);
      v[4 * h + 1] = __uint_as_float(r.y);
      v[4 * h + 2] = __uint_as_float(r.z);
      v[4 * h + 3] = __uint_as_float(r.w);
    }
  }
}

// 16 lanes per block of 128 values, 8 values each.
template <bool BF16>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const void* __restrict__ x, uint2* __restrict__ q,
                                                            float* __restrict__ s, uint32_t nblocks, uint32_t KB, int K) {
  pdl_wait();
  const uint32_t lane = threadIdx.x & 15;
  for (uint32_t b = blockIdx.x * 16u + threadIdx.x / 16u; b < nblocks; b += gridDim.x * 16u) {
    const uint32_t row = b / KB, kb = b - row * KB;
    const int k = (int)(kb * 128u + lane * 8u);
    const int64_t i = (int64_t)row * K + k;
    float v[8] = {};
    if (k < K) load8<BF16>(x, i, v);
    float a = kTiny;
#pragma unroll
    for (int j = 0; j < 8; ++j) a = amax2(a, v[j]);
    const uint32_t mask = 0xFFFFu << (threadIdx.x & 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) a = amax2(a, __shfl_xor_sync(mask, a, o));
    const float r = __fdiv_rn(kMax, a);
    if (k < K)
      q[i / 8] = make_uint2(e4m3x4(v[0] * r, v[1] * r, v[2] * r, v[3] * r), e4m3x4(v[4] * r, v[5] * r, v[6] * r, v[7] * r));
    if (lane == 0) s[b] = __fdiv_rn(a, kMax);
  }
}

// One 128 x 128 tile of W[e] ([K, N]) per block of 256 threads, written transposed.
template <bool BF16>
__global__ void __launch_bounds__(256) quantize_weights_kernel(const void* __restrict__ W, uint8_t* __restrict__ q,
                                                               float* __restrict__ s, int K, int N) {
  __shared__ uint8_t tile[128][128 + 16];     // [n][k]
  __shared__ float part[8];
  const int e = blockIdx.z, k0 = blockIdx.y * 128, n0 = blockIdx.x * 128;
  const int tid = threadIdx.x;
  const int n = n0 + (tid & 15) * 8, kr = tid >> 4;      // 8 columns of rows kr, kr + 16, ...
  float v[8][8] = {};
  float a = kTiny;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int k = k0 + kr + 16 * r;
    if (k < K && n < N) load8<BF16>(W, ((int64_t)e * K + k) * N + n, v[r]);
#pragma unroll
    for (int j = 0; j < 8; ++j) a = amax2(a, v[r][j]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = amax2(a, __shfl_xor_sync(0xffffffffu, a, o));
  if ((tid & 31) == 0) part[tid >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) a = amax2(a, part[w]);
  const float m = __fdiv_rn(kMax, a);
#pragma unroll
  for (int r = 0; r < 8; ++r)
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const uint32_t p = e4m3x2(v[r][j] * m, v[r][j + 1] * m);
      tile[(tid & 15) * 8 + j][kr + 16 * r] = (uint8_t)p;
      tile[(tid & 15) * 8 + j + 1][kr + 16 * r] = (uint8_t)(p >> 8);
    }
  if (tid == 0) s[((int64_t)e * gridDim.x + blockIdx.x) * gridDim.y + blockIdx.y] = __fdiv_rn(a, kMax);
  __syncthreads();
  // K is a multiple of 16: whole 16-byte pieces of a row of q
  for (int p = tid; p < 128 * 8; p += 256) {
    const int row = p >> 3, c = (p & 7) * 16;
    if (n0 + row < N && k0 + c < K)
      *reinterpret_cast<uint4*>(q + ((int64_t)e * N + n0 + row) * K + k0 + c) = *reinterpret_cast<const uint4*>(&tile[row][c]);
  }
}

}  // namespace

cudaError_t fp8_quantize_rows(int64_t R, int K, bool bf16, const void* x, void* q, float* s, cudaStream_t st) {
  const uint32_t KB = (uint32_t)((K + 127) / 128), nblocks = (uint32_t)(R * KB);
  const uint32_t want = (nblocks + 15) / 16;
  const dim3 grid(want < 148 * 64 ? want : 148 * 64);
  if (bf16) return launch_pdl(quantize_rows_kernel<true>, grid, dim3(256), 0, st, x, static_cast<uint2*>(q), s, nblocks, KB, K);
  return launch_pdl(quantize_rows_kernel<false>, grid, dim3(256), 0, st, x, static_cast<uint2*>(q), s, nblocks, KB, K);
}

cudaError_t fp8_quantize_weights(int E, int K, int N, bool bf16, const void* W, void* q, float* s, cudaStream_t st) {
  const dim3 grid((N + 127) / 128, (K + 127) / 128, E);
  if (bf16) quantize_weights_kernel<true><<<grid, 256, 0, st>>>(W, static_cast<uint8_t*>(q), s, K, N);
  else quantize_weights_kernel<false><<<grid, 256, 0, st>>>(W, static_cast<uint8_t*>(q), s, K, N);
  return cudaGetLastError();
}

}  // namespace moe
