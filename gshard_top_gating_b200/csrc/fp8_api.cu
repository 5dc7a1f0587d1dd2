// fp8_api.cu -- the C ABI of 8-bit products (moe_fp8_* of include/moe.h).
#include <new>

#include "api_util.h"
#include "internal.h"

using namespace moe;

struct moe_fp8 {
  int32_t E;
  int64_t C_max, K, N;
  const void* wq;
  const float* ws;
  int device, num_sms;
  void* ws_dev;          // the handle's allocation
  float* part;           // few_rows.cu: partial sums, arrival counts
  unsigned* count;
  size_t ncount;
  unsigned* err;
};

extern "C" {

moe_status moe_fp8_quantize_rows(int64_t R, int64_t K, moe_dtype src, const void* x, void* q, float* s, void* stream) {
  if (R < 0 || K < 16 || (K % 16) || (src != MOE_F32 && src != MOE_BF16)) return MOE_ERR_INVALID_ARG;
  if (R > 0 && (!x || !q || !s || !is_aligned(x, 16) || !is_aligned(q, 16) || !is_aligned(s, 4)))
    return MOE_ERR_INVALID_ARG;
  if (K > (1 << 20) || R > INT32_MAX || R * ((K + 127) / 128) > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  if (R == 0) return MOE_OK;
  return status_of(fp8_quantize_rows(R, (int)K, src == MOE_BF16, x, q, s, static_cast<cudaStream_t>(stream)));
}

moe_status moe_fp8_quantize_weights(int32_t E, int64_t K, int64_t N, moe_dtype src, const void* W, void* q, float* s,
                                    void* stream) {
  if (E < 1 || K < 16 || (K % 16) || N < 8 || (N % 8) || (src != MOE_F32 && src != MOE_BF16)) return MOE_ERR_INVALID_ARG;
  if (!W || !q || !s || !is_aligned(W, 16) || !is_aligned(q, 16) || !is_aligned(s, 4)) return MOE_ERR_INVALID_ARG;
  if (E > kMaxExperts || K > (1 << 20) || N > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  return status_of(fp8_quantize_weights(E, (int)K, (int)N, src == MOE_BF16, W, q, s, static_cast<cudaStream_t>(stream)));
}

moe_status moe_fp8_create(moe_fp8_handle* out, int32_t E, int64_t C_max, int64_t K, int64_t N, const void* wq,
                          const float* ws) {
  if (!out) return MOE_ERR_INVALID_ARG;
  *out = nullptr;
  if (E < 1 || C_max < 1 || K < 16 || (K % 16) || N < 8 || (N % 8)) return MOE_ERR_INVALID_ARG;
  if (!wq || !ws || !is_aligned(wq, 16) || !is_aligned(ws, 4)) return MOE_ERR_INVALID_ARG;
  if (E > kMaxExperts || K > (1 << 20) || N > (1 << 20) || C_max > (1 << 21)) return MOE_ERR_UNSUPPORTED;
  if (E * C_max > INT32_MAX - 512 || E * N > INT32_MAX - 512) return MOE_ERR_UNSUPPORTED;   // 32-bit TMA row coordinates
  moe_fp8* h = new (std::nothrow) moe_fp8();
  if (!h) return MOE_ERR_OOM;
  h->E = E;
  h->C_max = C_max;
  h->K = K;
  h->N = N;
  h->wq = wq;
  h->ws = ws;
  cudaError_t ce = cudaGetDevice(&h->device);
  if (ce == cudaSuccess) ce = cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device);
  BufferCarver c{nullptr};
  for (int pass = 0; ce == cudaSuccess && pass < 2; ++pass) {
    c.off = 0;
    const size_t few = few_rows_workspace(true, h->num_sms, &h->ncount);
    const size_t split = split_workspace(E, (int)N, h->num_sms);
    h->part = c.take<float>(few > split ? few : split);
    h->err = c.take<unsigned>(1 + h->ncount);     // the error word, then the counts
    h->count = h->err + 1;
    if (pass == 0) {
      ce = cudaMalloc(&h->ws_dev, c.off + 256);
      c.base = static_cast<char*>(h->ws_dev);
    }
  }
  if (ce == cudaSuccess) ce = cudaMemset(h->err, 0, (1 + h->ncount) * sizeof(unsigned));
  if (ce != cudaSuccess) {
    cudaGetLastError();
    if (h->ws_dev) cudaFree(h->ws_dev);
    delete h;
    return status_of(ce);
  }
  *out = h;
  return MOE_OK;
}

moe_status moe_fp8_destroy(moe_fp8_handle h) {
  if (!h) return MOE_OK;
  cudaError_t ce = cudaDeviceSynchronize();
  const cudaError_t fe = cudaFree(h->ws_dev);
  delete h;
  return status_of(ce != cudaSuccess ? ce : fe);
}

moe_status moe_fp8_check(moe_fp8_handle h, void* stream) {
  if (!h || !on_device(h->device)) return MOE_ERR_INVALID_ARG;
  return take_device_error(h->err, static_cast<cudaStream_t>(stream), 1 + h->ncount);
}

moe_status moe_fp8_matmul(moe_fp8_handle h, int64_t C, const void* xq, const float* xs, const int32_t* nrows, void* y,
                          void* stream) {
  if (!h || C < 0 || C > h->C_max || !on_device(h->device)) return MOE_ERR_INVALID_ARG;
  if (C > 0 && (!xq || !xs || !nrows || !y || !is_aligned(xq, 16) || !is_aligned(xs, 4) || !is_aligned(nrows, 4) ||
                !is_aligned(y, 16)))
    return MOE_ERR_INVALID_ARG;
  if (C == 0) return MOE_OK;
  Fp8Args a{};
  a.E = h->E;
  a.K = (int)h->K;
  a.N = (int)h->N;
  a.C = a.rows = C;
  a.n = nrows;
  a.xq = xq;
  a.xs = xs;
  a.wq = h->wq;
  a.ws = h->ws;
  a.y = y;
  a.part = h->part;
  a.count = h->count;
  a.err = h->err;
  a.limit_ns = 2000000000ull;   // 2 s per wait: far above any legitimate one
  a.num_sms = h->num_sms;
  a.st = static_cast<cudaStream_t>(stream);
  return status_of(fp8_matmul(a));
}

}  // extern "C"
