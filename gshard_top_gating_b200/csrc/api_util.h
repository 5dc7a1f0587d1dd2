// api_util.h -- host helpers of the C entry points: pointer checks, status of a CUDA error,
// carving one allocation into buffers.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe.h"
#include "common.cuh"

namespace moe {

inline size_t act_bytes_of(moe_dtype a) { return a == MOE_BF16 ? 2 : 4; }

inline bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline moe_status status_of(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  if (e == cudaErrorMemoryAllocation) return MOE_ERR_OOM;
  return MOE_ERR_CUDA;
}

// Takes 256-byte aligned buffers off one allocation; with base == nullptr only measures.
struct BufferCarver {
  char* base;
  size_t off = 0;
  template <typename T>
  T* take(size_t n) {
    off = (off + 255) & ~(size_t)255;
    T* p = base ? reinterpret_cast<T*>(base + off) : nullptr;
    off += n * sizeof(T);
    return p;
  }
};

inline bool on_device(int device) {
  int cur = -1;
  return cudaGetDevice(&cur) == cudaSuccess && cur == device;
}

// Whether `st` is being captured into a graph; an error (a capture elsewhere in global mode)
// counts as capturing.
inline bool is_capturing(cudaStream_t st) {
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  return cudaStreamIsCapturing(st, &cs) != cudaSuccess || cs != cudaStreamCaptureStatusNone;
}

// Synchronises `st`, reads a device error word and, if it is set, clears it and the words
// behind it (`words` in all).
inline moe_status take_device_error(unsigned* err, cudaStream_t st, size_t words = 1) {
  unsigned e = 0;
  cudaError_t ce = cudaMemcpyAsync(&e, err, sizeof(unsigned), cudaMemcpyDeviceToHost, st);
  if (ce == cudaSuccess) ce = cudaStreamSynchronize(st);
  if (ce != cudaSuccess) return status_of(ce);
  if (!e) return MOE_OK;
  ce = cudaMemsetAsync(err, 0, words * sizeof(unsigned), st);
  if (ce == cudaSuccess) ce = cudaStreamSynchronize(st);
  if (ce != cudaSuccess) return status_of(ce);
  return (e & DEVERR_TIMEOUT) ? MOE_ERR_TIMEOUT : MOE_ERR_CUDA;
}

}  // namespace moe
