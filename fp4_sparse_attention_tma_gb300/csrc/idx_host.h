// Argument checks and device queries shared by the C-ABI layers (host.cu,
// attn_host.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "idx_internal.h"
#include "idxtopk.h"

namespace idxk {

constexpr int kMaxDevices = 64;

struct DeviceState {
  bool init = false;
  int sm_count = 0;
  int cc_major = 0, cc_minor = 0;
  cudaMemPool_t pool = nullptr;
};

// The library's state of device `dev` (created on first use: its scratch pool and
// the tensor-map encoder).
int device_state(int dev, DeviceState** out);

// SM count and compute capability of `dev`, and the tensor-map encoder; unlike
// device_state this creates no memory pool.
int device_info_no_pool(int dev, int* sm, int* major, int* minor);

// ---------------------------------------------------------- validation ----

inline bool mul_ok(int64_t a, int64_t b, int64_t* out) {
  if (a < 0 || b < 0) return false;
  if (a != 0 && b > INT64_MAX / a) return false;
  *out = a * b;
  return true;
}

// Validates one descriptor: dtype, rank, non-negative shape, C-contiguous
// strides, 16-byte aligned base (unless empty or need_align is false: host
// tensors that are only copied).  Returns IDX_OK or an error.
inline int check_tensor(const idx_tensor_t* t, int dtype, int ndim, bool need_align = true) {
  if (!t) return IDX_ERR_INVALID_ARGUMENT;
  if (t->dtype != dtype || t->ndim != ndim) return IDX_ERR_INVALID_ARGUMENT;
  int64_t numel = 1;
  for (int i = 0; i < ndim; ++i) {
    if (t->shape[i] < 0) return IDX_ERR_INVALID_ARGUMENT;
    if (!mul_ok(numel, t->shape[i], &numel)) return IDX_ERR_OVERFLOW;
  }
  int64_t expect = 1;
  for (int i = ndim - 1; i >= 0; --i) {
    if (t->shape[i] > 1 && t->stride[i] != expect) return IDX_ERR_INVALID_ARGUMENT;
    if (!mul_ok(expect, t->shape[i] > 0 ? t->shape[i] : 1, &expect)) return IDX_ERR_OVERFLOW;
  }
  int64_t bytes;
  if (!mul_ok(numel, dtype == IDX_U8 ? 1 : 4, &bytes)) return IDX_ERR_OVERFLOW;
  if (numel > 0) {
    if (!t->data) return IDX_ERR_INVALID_ARGUMENT;
    if (need_align && ((uintptr_t)t->data & 15u) != 0) return IDX_ERR_INVALID_ARGUMENT;
  }
  return IDX_OK;
}

inline int64_t numel_of(const idx_tensor_t* t) {
  int64_t n = 1;
  for (int i = 0; i < t->ndim; ++i) n *= t->shape[i];
  return n;
}

// Device that owns `ptr` (device or managed memory), or -1.
inline int device_of(const void* ptr) {
  cudaPointerAttributes a;
  if (cudaPointerGetAttributes(&a, ptr) != cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  if (a.type != cudaMemoryTypeDevice && a.type != cudaMemoryTypeManaged) return -1;
  return a.device;
}

class DeviceGuard {
 public:
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev_) != cudaSuccess) {
      cudaGetLastError();
      prev_ = -1;
    }
    if (prev_ != dev) ok_ = cudaSetDevice(dev) == cudaSuccess;
  }
  ~DeviceGuard() {
    if (prev_ >= 0) cudaSetDevice(prev_);
  }
  bool ok() const { return ok_; }

 private:
  int prev_ = -1;
  bool ok_ = true;
};

// Every non-empty tensor must be device memory of one device; returns it.
inline int common_device(const idx_tensor_t* const* ts, int n, int* dev) {
  int d = -1;
  for (int i = 0; i < n; ++i) {
    const idx_tensor_t* t = ts[i];
    if (!t || numel_of(t) == 0) continue;
    const int td = device_of(t->data);
    if (td < 0) return IDX_ERR_INVALID_ARGUMENT;
    if (d >= 0 && td != d) return IDX_ERR_INVALID_ARGUMENT;
    d = td;
  }
  if (d < 0 && cudaGetDevice(&d) != cudaSuccess) {
    cudaGetLastError();
    return IDX_ERR_CUDA;
  }
  *dev = d;
  return IDX_OK;
}

inline int check_stream(cudaStream_t stream, int dev) {
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(stream, &cs) != cudaSuccess) {
    cudaGetLastError();
    return IDX_ERR_CUDA;
  }
  if (cs != cudaStreamCaptureStatusNone) return IDX_ERR_UNSUPPORTED;
  if (stream != nullptr) {
    int sd = -1;
    if (cudaStreamGetDevice(stream, &sd) != cudaSuccess) {
      cudaGetLastError();
      return IDX_ERR_INVALID_ARGUMENT;
    }
    if (sd != dev) return IDX_ERR_INVALID_ARGUMENT;
  }
  return IDX_OK;
}

}  // namespace idxk
