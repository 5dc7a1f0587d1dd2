// glu_api.cu -- the C ABI of gated experts (moe_glu_* of include/moe.h): handle, workspace,
// launch sequence.  Forward: up, down.  Backward: dh (which copies the tails of x and dy too),
// dW2 and dW13, dx.
#include <new>

#include "api_util.h"
#include "internal.h"

using namespace moe;

struct moe_glu {
  int32_t E;
  int64_t C_max, Cp, M, H;
  moe_dtype act;
  int fn, device, num_sms;
  const void* W13;
  const void* W2;
  void* ws;
  void* h;               // [E, Cp, H] act
  float* part;           // few_rows.cu: partial sums, arrival counts
  unsigned* count;
  size_t ncount;
  unsigned* err;
  void* bws;             // the backward's allocation (moe_glu_enable_backward)
  void* gu;              // [E, Cp, 2H] act
  void* dgu;             // [E, Cp, 2H] act
  void* tx;              // [E, 64, M] act (bf16)
  void* tdy;
  int64_t saved_C;       // C of the last forward that kept g and u, or -1
  // A forward was captured into a CUDA graph without keeping g and u: a replay of that graph,
  // which the host cannot see, leaves those of another forward behind.
  bool graph_without_gu;
};

namespace {

constexpr uint64_t kWaitLimitNs = 2000000000ull;   // 2 s per wait: far above any legitimate one

GluArgs args_of(moe_glu_handle h, int64_t C, const void* x, const int32_t* n, cudaStream_t st) {
  GluArgs a{};
  a.E = h->E;
  a.M = (int)h->M;
  a.H = (int)h->H;
  a.fn = h->fn;
  a.C = a.rows = C;
  a.Cp = h->Cp;
  a.n = n;
  a.x = x;
  a.W13 = h->W13;
  a.W2 = h->W2;
  a.h = h->h;
  a.gu = h->gu;
  a.dgu = h->dgu;
  a.tx = h->tx;
  a.tdy = h->tdy;
  a.part = h->part;
  a.count = h->count;
  a.err = h->err;
  a.limit_ns = kWaitLimitNs;
  a.num_sms = h->num_sms;
  a.st = st;
  return a;
}

}  // namespace

#define GLU_TRY(call)                            \
  do {                                           \
    cudaError_t _e = (call);                     \
    if (_e != cudaSuccess) return status_of(_e); \
  } while (0)

extern "C" {

moe_status moe_glu_create(moe_glu_handle* out, int32_t E, int64_t C_max, int64_t M, int64_t H, moe_dtype act,
                          moe_glu_fn fn, const void* W13, const void* W2) {
  if (!out) return MOE_ERR_INVALID_ARG;
  *out = nullptr;
  if (E < 1 || C_max < 1 || M < 64 || H < 64 || (M % 64) || (H % 64)) return MOE_ERR_INVALID_ARG;
  if (act != MOE_F32 && act != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (fn != MOE_GLU_SILU && fn != MOE_GLU_GELU && fn != MOE_GLU_RELU) return MOE_ERR_INVALID_ARG;
  if (!W13 || !W2 || !is_aligned(W13, 16) || !is_aligned(W2, 16)) return MOE_ERR_INVALID_ARG;
  if (E > kMaxExperts || C_max > (1 << 21) || M > (1 << 16) || H > (1 << 16)) return MOE_ERR_UNSUPPORTED;
  const int64_t Cp = (C_max + 255) / 256 * 256;
  if (E * Cp > INT32_MAX) return MOE_ERR_UNSUPPORTED;     // 32-bit TMA row coordinates
  moe_glu* h = new (std::nothrow) moe_glu();
  if (!h) return MOE_ERR_OOM;
  h->E = E;
  h->C_max = C_max;
  h->Cp = Cp;
  h->M = M;
  h->H = H;
  h->act = act;
  h->fn = fn;
  h->W13 = W13;
  h->W2 = W2;
  h->saved_C = -1;
  cudaError_t ce = cudaGetDevice(&h->device);
  if (ce == cudaSuccess) ce = cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device);
  BufferCarver c{nullptr};
  for (int pass = 0; ce == cudaSuccess && pass < 2; ++pass) {
    c.off = 0;
    h->h = c.take<char>((size_t)E * Cp * H * act_bytes_of(act));
    if (act == MOE_BF16) {
      const size_t few = few_rows_workspace(false, h->num_sms, &h->ncount);
      const size_t split = split_workspace(E, (int)M, h->num_sms);
      h->part = c.take<float>(few > split ? few : split);
    } else {
      h->part = c.take<float>(glu_f32_workspace(h->num_sms));
    }
    h->err = c.take<unsigned>(1 + h->ncount);     // the error word, then the counts
    h->count = h->err + 1;
    if (pass == 0) {
      ce = cudaMalloc(&h->ws, c.off + 256);
      c.base = static_cast<char*>(h->ws);
    }
  }
  if (ce == cudaSuccess) ce = cudaMemset(h->err, 0, (1 + h->ncount) * sizeof(unsigned));
  if (ce != cudaSuccess) {
    cudaGetLastError();
    if (h->ws) cudaFree(h->ws);
    delete h;
    return status_of(ce);
  }
  *out = h;
  return MOE_OK;
}

moe_status moe_glu_destroy(moe_glu_handle h) {
  if (!h) return MOE_OK;
  cudaError_t ce = cudaDeviceSynchronize();
  const cudaError_t f1 = cudaFree(h->ws);
  const cudaError_t f2 = h->bws ? cudaFree(h->bws) : cudaSuccess;
  delete h;
  if (ce == cudaSuccess) ce = f1 != cudaSuccess ? f1 : f2;
  return status_of(ce);
}

moe_status moe_glu_check(moe_glu_handle h, void* stream) {
  if (!h || !on_device(h->device)) return MOE_ERR_INVALID_ARG;
  return take_device_error(h->err, static_cast<cudaStream_t>(stream), 1 + h->ncount);
}

moe_status moe_glu_enable_backward(moe_glu_handle h) {
  if (!h || !on_device(h->device)) return MOE_ERR_INVALID_ARG;
  if (h->bws) return MOE_OK;
  const size_t as = act_bytes_of(h->act), rows = (size_t)h->E * h->Cp;
  BufferCarver c{nullptr};
  void *gu = nullptr, *dgu = nullptr, *tx = nullptr, *tdy = nullptr, *bws = nullptr;
  for (int pass = 0; pass < 2; ++pass) {
    c.off = 0;
    gu = c.take<char>(rows * 2 * h->H * as);
    dgu = c.take<char>(rows * 2 * h->H * as);
    if (h->act == MOE_BF16) {
      tx = c.take<char>((size_t)h->E * 64 * h->M * as);
      tdy = c.take<char>((size_t)h->E * 64 * h->M * as);
    }
    if (pass == 0) {
      const cudaError_t ce = cudaMalloc(&bws, c.off + 256);
      if (ce != cudaSuccess) {
        cudaGetLastError();
        return status_of(ce);
      }
      c.base = static_cast<char*>(bws);
    }
  }
  h->bws = bws;
  h->gu = gu;
  h->dgu = dgu;
  h->tx = tx;
  h->tdy = tdy;
  return MOE_OK;
}

moe_status moe_glu_forward(moe_glu_handle h, int64_t C, const void* x, const int32_t* nrows, void* y, void* stream) {
  if (!h || C < 0 || C > h->C_max || !on_device(h->device)) return MOE_ERR_INVALID_ARG;
  if (C > 0 && (!x || !y || !nrows || !is_aligned(x, 16) || !is_aligned(y, 16) || !is_aligned(nrows, 4)))
    return MOE_ERR_INVALID_ARG;
  h->saved_C = -1;
  if (!h->bws && is_capturing(static_cast<cudaStream_t>(stream))) h->graph_without_gu = true;
  if (C > 0) {
    GluArgs a = args_of(h, C, x, nrows, static_cast<cudaStream_t>(stream));
    a.y = y;
    GLU_TRY(glu_up(a, h->act == MOE_BF16));
    GLU_TRY(glu_down(a, h->act == MOE_BF16));
  }
  if (h->bws) h->saved_C = C;
  return MOE_OK;
}

moe_status moe_glu_backward(moe_glu_handle h, int64_t C, const void* x, const int32_t* nrows, const void* dy, void* dx,
                            void* dW13, void* dW2, uint32_t flags, void* stream) {
  if (!h || C < 0 || C > h->C_max || !on_device(h->device) || (flags & ~(uint32_t)MOE_BWD_SKIP_EMPTY_EXPERTS))
    return MOE_ERR_INVALID_ARG;
  if (!h->bws || h->saved_C != C || h->graph_without_gu) return MOE_ERR_STATE;
  if (!dW13 || !dW2 || !is_aligned(dW13, 16) || !is_aligned(dW2, 16)) return MOE_ERR_INVALID_ARG;
  if (C > 0 && (!x || !dy || !dx || !nrows || !is_aligned(x, 16) || !is_aligned(dy, 16) || !is_aligned(dx, 16) ||
                !is_aligned(nrows, 4)))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (C == 0) {          // no rows: every expert is empty
    if (flags & MOE_BWD_SKIP_EMPTY_EXPERTS) return MOE_OK;
    const size_t w = (size_t)h->E * h->M * h->H * act_bytes_of(h->act);
    GLU_TRY(cudaMemsetAsync(dW13, 0, 2 * w, st));
    GLU_TRY(cudaMemsetAsync(dW2, 0, w, st));
    return MOE_OK;
  }
  GluArgs a = args_of(h, C, x, nrows, st);
  a.dy = dy;
  a.dx = dx;
  a.dW13 = dW13;
  a.dW2 = dW2;
  a.skip_empty = (flags & MOE_BWD_SKIP_EMPTY_EXPERTS) != 0;
  if (h->act == MOE_BF16) {
    GLU_TRY(glu_dh_bf16(a));
    GLU_TRY(glu_dw_bf16(a));
    GLU_TRY(glu_dx_bf16(a));
  } else {
    GLU_TRY(glu_dw2_f32(a));
    GLU_TRY(glu_dh_f32(a));
    GLU_TRY(glu_dw13_f32(a));
    GLU_TRY(glu_dx_f32(a));
  }
  return MOE_OK;
}

}  // extern "C"
