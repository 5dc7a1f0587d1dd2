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
#include "glu.cuh"
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

// Eight consecutive values as they are stored: 16 bytes of bf16, 32 of fp32.
template <bool BF16>
struct Raw8 {
  uint4 r[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* x, int64_t i) {
#pragma unroll
    for (int h = 0; h < (BF16 ? 1 : 2); ++h) r[h] = ld_nc_v4(static_cast<const char*>(x) + i * (BF16 ? 2 : 4) + h * 16);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int h = 0; h < (BF16 ? 1 : 2); ++h) r[h] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {r[0].x, r[0].y, r[0].z, r[0].w};
    const uint4 q = r[BF16 ? 0 : 1];
    const uint32_t z[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[BF16 ? 2 * j : j] = BF16 ? bf16lo(w[j]) : __uint_as_float(w[j]);
      v[BF16 ? 2 * j + 1 : 4 + j] = BF16 ? bf16hi(w[j]) : __uint_as_float(z[j]);
    }
  }
};

// 16 lanes per block of 128 values, 8 values each; BLOCKS blocks of one lane group are loaded
// before the first is used.  EVEN: K is a multiple of 128, so block b starts at value 128 b.
template <bool BF16, bool EVEN, int BLOCKS>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const void* __restrict__ x, uint2* __restrict__ q,
                                                            float* __restrict__ s, uint32_t nblocks, uint32_t KB, int K) {
  pdl_wait();
  const uint32_t lane = threadIdx.x & 15;
  const uint32_t mask = 0xFFFFu << (threadIdx.x & 16);
  // first value of this lane in block b, or -1 (past the row's end)
  auto at = [&](uint32_t b) -> int64_t {
    if (EVEN) return (int64_t)b * 128 + lane * 8u;
    const uint32_t row = b / KB, k = (b - row * KB) * 128u + lane * 8u;
    return k < (uint32_t)K ? (int64_t)row * K + k : -1;
  };
  const uint32_t group = blockIdx.x * 16u + threadIdx.x / 16u;
  const uint32_t b0 = group * BLOCKS;
  Raw8<BF16> raw[BLOCKS];
#pragma unroll
  for (int u = 0; u < BLOCKS; ++u) {
    raw[u].zero();
    if (b0 + u < nblocks) {
      const int64_t i = at(b0 + u);
      if (i >= 0) raw[u].load(x, i);
    }
  }
#pragma unroll
  for (int u = 0; u < BLOCKS; ++u) {
    if (b0 + u >= nblocks) break;                     // the same for all lanes of a group
    float v[8];
    raw[u].get(v);
    float a = kTiny;
#pragma unroll
    for (int j = 0; j < 8; ++j) a = amax2(a, v[j]);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) a = amax2(a, __shfl_xor_sync(mask, a, o));
    const float r = __fdiv_rn(kMax, a);
    const int64_t i = at(b0 + u);
    if (i >= 0)
      q[i / 8] = make_uint2(e4m3x4(v[0] * r, v[1] * r, v[2] * r, v[3] * r), e4m3x4(v[4] * r, v[5] * r, v[6] * r, v[7] * r));
    if (lane == 0) s[b0 + u] = __fdiv_rn(a, kMax);
  }
}

// The rows that experts hold: block (x, e) takes blocks of 128 of expert e's rows in turn.
// FN >= 0: the values are h = f(g) * u of [g | u], formed in 32 bits and quantised from there.
template <int FN>
__global__ void __launch_bounds__(256) quantize_held_kernel(const void* __restrict__ x, uint2* __restrict__ q,
                                                            float* __restrict__ s, const int32_t* __restrict__ nexp,
                                                            int64_t C, uint32_t KB, int K) {
  pdl_wait();
  const int e = blockIdx.y;
  const uint32_t lane = threadIdx.x & 15, mask = 0xFFFFu << (threadIdx.x & 16);
  const int64_t nblocks = min(max((int64_t)nexp[e], (int64_t)0), C) * KB;
  for (int64_t b = (int64_t)blockIdx.x * 16 + threadIdx.x / 16; b < nblocks; b += (int64_t)gridDim.x * 16) {
    const int64_t row = (int64_t)e * C + b / KB;
    const int k = (int)(b % KB) * 128 + (int)lane * 8;
    float v[8] = {};
    if (k < K) {
      Raw8<true> raw;
      if (FN < 0) {
        raw.load(x, row * K + k);
        raw.get(v);
      } else {
        float u[8];
        raw.load(x, row * 2 * K + k);
        raw.get(v);
        raw.load(x, row * 2 * K + K + k);
        raw.get(u);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = glu_f<FN < 0 ? 0 : FN, true>(v[j]) * u[j];
      }
    }
    float a = kTiny;
#pragma unroll
    for (int j = 0; j < 8; ++j) a = amax2(a, v[j]);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) a = amax2(a, __shfl_xor_sync(mask, a, o));
    const float r = __fdiv_rn(kMax, a);
    if (k < K)
      q[(row * K + k) / 8] =
          make_uint2(e4m3x4(v[0] * r, v[1] * r, v[2] * r, v[3] * r), e4m3x4(v[4] * r, v[5] * r, v[6] * r, v[7] * r));
    if (lane == 0) s[row * KB + (int)(b % KB)] = __fdiv_rn(a, kMax);
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
    if (k < K && n < N) {
      Raw8<BF16> raw;
      raw.load(W, ((int64_t)e * K + k) * N + n);
      raw.get(v[r]);
    }
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

template <bool BF16, bool EVEN>
cudaError_t launch_rows(uint32_t nblocks, uint32_t KB, int K, const void* x, void* q, float* s, cudaStream_t st) {
  // many blocks: several in flight per lane group (65536 x 7168 bf16: 267 us with one, 244 with
  // two, 229 with four, 224 with eight; copying the same bytes 218); few: one each, on more SMs
  constexpr int MANY = BF16 ? 8 : 4;
  int dev = 0, sms = 148;
  if (nblocks >= 128u * MANY) {          // (few rows: not worth the question)
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  }
  const bool many = nblocks >= (uint32_t)sms * 128u * MANY;
  const uint32_t per = 16u * (many ? MANY : 1);
  const dim3 grid((nblocks + per - 1) / per);
  auto kern = many ? quantize_rows_kernel<BF16, EVEN, MANY> : quantize_rows_kernel<BF16, EVEN, 1>;
  return launch_pdl(kern, grid, dim3(256), 0, st, x, static_cast<uint2*>(q), s, nblocks, KB, K);
}

}  // namespace

cudaError_t fp8_quantize_rows(int64_t R, int K, bool bf16, const void* x, void* q, float* s, cudaStream_t st) {
  const uint32_t KB = (uint32_t)((K + 127) / 128), nblocks = (uint32_t)(R * KB);
  if (K % 128 == 0)
    return bf16 ? launch_rows<true, true>(nblocks, KB, K, x, q, s, st) : launch_rows<false, true>(nblocks, KB, K, x, q, s, st);
  return bf16 ? launch_rows<true, false>(nblocks, KB, K, x, q, s, st) : launch_rows<false, false>(nblocks, KB, K, x, q, s, st);
}

namespace {

template <int FN>
cudaError_t launch_held(int E, int64_t C, int K, const int32_t* n, const void* x, void* q, float* s, int num_sms,
                        cudaStream_t st) {
  const uint32_t KB = (uint32_t)((K + 127) / 128);
  // about eight blocks of threads per SM over all experts, and no more than an expert can use
  int64_t per = (C * KB + 15) / 16, want = (num_sms * 8 + E - 1) / E;
  if (want > per) want = per;
  return launch_pdl(quantize_held_kernel<FN>, dim3((unsigned)want, E), dim3(256), 0, st, x, static_cast<uint2*>(q), s, n, C,
                    KB, K);
}

}  // namespace

cudaError_t fp8_quantize_held(int E, int64_t C, int K, const int32_t* n, const void* x, void* q, float* s, int num_sms,
                              cudaStream_t st) {
  return launch_held<-1>(E, C, K, n, x, q, s, num_sms, st);
}

cudaError_t fp8_quantize_glu(int E, int64_t C, int K, int fn, const int32_t* n, const void* gu, void* q, float* s,
                             int num_sms, cudaStream_t st) {
  if (fn == kGluSilu) return launch_held<kGluSilu>(E, C, K, n, gu, q, s, num_sms, st);
  if (fn == kGluGelu) return launch_held<kGluGelu>(E, C, K, n, gu, q, s, num_sms, st);
  return launch_held<kGluRelu>(E, C, K, n, gu, q, s, num_sms, st);
}

cudaError_t fp8_quantize_weights(int E, int K, int N, bool bf16, const void* W, void* q, float* s, cudaStream_t st) {
  const dim3 grid((N + 127) / 128, (K + 127) / 128, E);
  if (bf16) quantize_weights_kernel<true><<<grid, 256, 0, st>>>(W, static_cast<uint8_t*>(q), s, K, N);
  else quantize_weights_kernel<false><<<grid, 256, 0, st>>>(W, static_cast<uint8_t*>(q), s, K, N);
  return cudaGetLastError();
}

}  // namespace moe
