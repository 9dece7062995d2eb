// Argument checks, layouts and workspaces shared by the C-ABI layers of the operators on a
// layer's cache (attn_host.cu, cache_host.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "idx_host.h"

namespace idxk {

// Validates a tensor with free strides: type, rank, 16-byte aligned base, last dimension
// contiguous, other strides non-negative multiples of `unit` elements (16-bit tensors: 8)
// whose offsets stay within 63 bits.
inline int check_strided(const idx_tensor_t* t, int dtype, int ndim, int64_t unit = 8) {
  if (!t || t->dtype != dtype || t->ndim != ndim) return IDX_ERR_INVALID_ARGUMENT;
  int64_t reach = 0, numel = 1;
  for (int i = 0; i < ndim; ++i) {
    if (t->shape[i] < 0) return IDX_ERR_INVALID_ARGUMENT;
    if (!mul_ok(numel, t->shape[i], &numel)) return IDX_ERR_OVERFLOW;
  }
  if (numel == 0) return IDX_OK;
  for (int i = 0; i < ndim; ++i) {
    if (t->shape[i] <= 1) continue;
    if (i == ndim - 1 ? t->stride[i] != 1 : t->stride[i] < 0 || t->stride[i] % unit != 0)
      return IDX_ERR_INVALID_ARGUMENT;
    int64_t x;
    if (!mul_ok(t->shape[i] - 1, t->stride[i], &x) || x > (INT64_MAX / 4) - reach) return IDX_ERR_OVERFLOW;
    reach += x;
  }
  if (!t->data || ((uintptr_t)t->data & 15u) != 0) return IDX_ERR_INVALID_ARGUMENT;
  return IDX_OK;
}

// Whether no two elements of `t` share an address (its dimensions nest).
inline bool no_overlap(const idx_tensor_t* t) {
  bool used[4] = {false, false, false, false};
  int64_t span = 1;
  for (int k = 0; k < t->ndim; ++k) {
    int best = -1;
    for (int i = 0; i < t->ndim; ++i)
      if (!used[i] && (best < 0 || t->stride[i] < t->stride[best])) best = i;
    used[best] = true;
    if (t->shape[best] <= 1) continue;
    if (t->stride[best] < span) return false;
    span += t->stride[best] * (t->shape[best] - 1);
  }
  return true;
}

inline int elem_bytes(const idx_tensor_t* t) {
  return t->dtype == IDX_U8 ? 1 : t->dtype == IDX_BF16 || t->dtype == IDX_F16 ? 2 : 4;
}

// The bytes that `t` spans.
inline int64_t span_of(const idx_tensor_t* t) {
  int64_t reach = 1;
  for (int i = 0; i < t->ndim; ++i)
    if (t->shape[i] > 1) reach += (t->shape[i] - 1) * t->stride[i];
  return reach * elem_bytes(t);
}
constexpr int64_t kFar = ((int64_t)1 << 32) * 16 - 16;

// The addresses that `t` spans.
inline void range_of(const idx_tensor_t* t, uintptr_t* a, uintptr_t* b) {
  *a = (uintptr_t)t->data;
  *b = *a + (uintptr_t)span_of(t);
}

inline bool apart(const idx_tensor_t* x, const idx_tensor_t* y) {
  if (!x || !y || numel_of(x) == 0 || numel_of(y) == 0) return true;
  uintptr_t a, b, c, d;
  range_of(x, &a, &b);
  range_of(y, &c, &d);
  return b <= c || d <= a;
}

// Each of the outputs apart from every input and from the other outputs.
template <int NO, int NI>
bool all_apart(const idx_tensor_t* const (&outs)[NO], const idx_tensor_t* const (&ins)[NI]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < NI; ++j)
      if (!apart(outs[i], ins[j])) return false;
    for (int j = 0; j < i; ++j)
      if (!apart(outs[i], outs[j])) return false;
  }
  return true;
}

inline bool same_layout(const idx_tensor_t* x, const idx_tensor_t* y) {
  if (x->data != y->data || x->ndim != y->ndim) return false;
  for (int i = 0; i < x->ndim; ++i)
    if (x->shape[i] != y->shape[i] || (x->shape[i] > 1 && x->stride[i] != y->stride[i])) return false;
  return true;
}

inline bool same_strides(const idx_tensor_t* x, const idx_tensor_t* y) {
  for (int i = 0; i < x->ndim; ++i)
    if (x->shape[i] != y->shape[i] || (x->shape[i] > 1 && x->stride[i] != y->stride[i])) return false;
  return true;
}

// Elements from the address of x to that of y.
inline int64_t distance(const idx_tensor_t* x, const idx_tensor_t* y) {
  return ((int64_t)(uintptr_t)y->data - (int64_t)(uintptr_t)x->data) / elem_bytes(x);
}

// Whether two elements of a cache whose dimensions nest (no_overlap) lie `delta` apart, other than two of
// one position (`one_position`: those do not count).  Dimension by dimension, the largest stride first: of
// the steps along it only one or two leave a rest that the others can reach.
inline bool elements_apart(const idx_tensor_t* t, int64_t delta, bool one_position, uint32_t used = 0, bool moved = false) {
  int best = -1;
  int64_t inner = 0;
  for (int i = 0; i < 4; ++i)
    if (!(used >> i & 1) && t->shape[i] > 1 && (best < 0 || t->stride[i] > t->stride[best])) best = i;
  if (best < 0) return delta == 0 && (moved || !one_position);
  used |= 1u << best;
  for (int i = 0; i < 4; ++i)
    if (!(used >> i & 1) && t->shape[i] > 1) inner += (t->shape[i] - 1) * t->stride[i];
  const int64_t s = t->stride[best], n = t->shape[best] - 1;
  for (int64_t d = delta / s - 2; d <= delta / s + 2; ++d) {
    const int64_t rest = delta - d * s;
    if (d < -n || d > n || rest > inner || rest < -inner) continue;
    if (elements_apart(t, rest, one_position, used, moved || (best < 2 && d != 0))) return true;
  }
  return false;
}

// Whether two tensors of elements of one size whose first dimensions step alike keep apart between any
// two steps (pages that hold keys and values, rows of a fused projection).
inline bool interleaved(const idx_tensor_t* x, const idx_tensor_t* y) {
  const int64_t each = x->stride[0];
  if (x->shape[0] <= 1 || y->shape[0] <= 1 || y->stride[0] != each || each <= 0) return false;
  int64_t x_end = 1, y_end = 1;
  for (int i = 1; i < x->ndim; ++i)
    if (x->shape[i] > 1) x_end += (x->shape[i] - 1) * x->stride[i];
  for (int i = 1; i < y->ndim; ++i)
    if (y->shape[i] > 1) y_end += (y->shape[i] - 1) * y->stride[i];
  int64_t at = distance(x, y) % each;
  if (at < 0) at += each;
  return at >= x_end && at + y_end <= each;
}

// Whether two paged tensors (each without overlap in itself, of elements of one size) share no element,
// or (`alike`) only elements of the same position.
inline bool pages_apart(const idx_tensor_t* k_dst, const idx_tensor_t* v_dst, bool alike = false) {
  if (apart(k_dst, v_dst)) return true;
  if (same_strides(k_dst, v_dst)) return !elements_apart(k_dst, distance(k_dst, v_dst), alike);
  return interleaved(k_dst, v_dst);   // laid out differently: in every page apart
}

// Whether keys and values moved into k_dst and v_dst (each without overlap in itself) keep out of each
// other's way: the two share no element, or only elements that the caches' keys and values of a position
// share alike (a latent cache that both are views of: the same bytes are moved twice).
inline bool places_agree(const idx_tensor_t* k, const idx_tensor_t* v, const idx_tensor_t* k_dst, const idx_tensor_t* v_dst) {
  bool alike = same_strides(k, v) && distance(k, v) == distance(k_dst, v_dst);
  for (int i = 1; i < 4; ++i) alike &= k->shape[i] <= 1 || k->stride[i] == k_dst->stride[i];
  return pages_apart(k_dst, v_dst, alike);
}

// The stride of dimension i (0 where it has one element: nothing steps along it).
inline int64_t step(const idx_tensor_t* t, int i) { return t->shape[i] > 1 ? t->stride[i] : 0; }

struct Machine {
  int dev = -1, sm = 0;
  bool capturing = false;
};

// The device of the call's tensors and its stream's state; `status` and `workspace` are
// checked to be of the same device when they are given.
inline int find_machine(const idx_tensor_t* const* ts, int n, const void* status, const void* workspace, cudaStream_t stream,
                 Machine* m) {
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(stream, &cs) != cudaSuccess) {
    cudaGetLastError();
    return IDX_ERR_CUDA;
  }
  m->capturing = cs != cudaStreamCaptureStatusNone;
  if (m->capturing) {
    // pointer and stream-device queries fail while a stream is captured
    if (cudaGetDevice(&m->dev) != cudaSuccess) {
      cudaGetLastError();
      return IDX_ERR_CUDA;
    }
  } else {
    int st = common_device(ts, n, &m->dev);
    if (st) return st;
    if (status && device_of(status) != m->dev) return IDX_ERR_INVALID_ARGUMENT;
    if (workspace && device_of(workspace) != m->dev) return IDX_ERR_INVALID_ARGUMENT;
    if (stream != nullptr) {
      int sd = -1;
      if (cudaStreamGetDevice(stream, &sd) != cudaSuccess) {
        cudaGetLastError();
        return IDX_ERR_INVALID_ARGUMENT;
      }
      if (sd != m->dev) return IDX_ERR_INVALID_ARGUMENT;
    }
  }
  return IDX_OK;
}

// SM count, and whether the device is one that the kernels are built for: asked once a
// device (neither changes).
inline int check_arch(Machine* m) {
  static std::atomic<int> known[kMaxDevices];   // SM count + 1, or -1 for another architecture
  if (m->dev < 0 || m->dev >= kMaxDevices) return IDX_ERR_INVALID_ARGUMENT;
  int k = known[m->dev].load(std::memory_order_acquire);
  if (k == 0) {
    int sm = 0, major = 0, minor = 0;
    const int st = device_info_no_pool(m->dev, &sm, &major, &minor);
    if (st) return st;
    k = major == 10 && minor == 3 ? sm + 1 : -1;
    known[m->dev].store(k, std::memory_order_release);
  }
  m->sm = k - 1;
  return k > 0 ? IDX_OK : IDX_ERR_UNSUPPORTED;
}

// Where a call's workspace and status word come from.
struct Space {
  bool async;
  void* workspace;
  uint64_t bytes;
  uint32_t* status;
};

// Runs `enqueue(base, status)` with `bytes` of workspace.  Stream-ordered: the caller's,
// checked.  Synchronous: from the pool, and the call's result is the status that the
// device wrote, after `stream` has reached the end of the work.
template <typename F>
int with_space(const Space& s, size_t bytes, const Machine& m, cudaStream_t stream, F enqueue) {
  if (s.async) {
    if (bytes > 0 && (!s.workspace || ((uintptr_t)s.workspace & 255u) != 0 || s.bytes < bytes)) return IDX_ERR_INVALID_ARGUMENT;
    if (enqueue((char*)s.workspace, s.status) != cudaSuccess) {
      cudaGetLastError();
      return IDX_ERR_CUDA;
    }
    return IDX_OK;
  }
  DeviceState* ds = nullptr;
  int st = device_state(m.dev, &ds);
  if (st) return st;
  char* base = nullptr;
  if (cudaMallocFromPoolAsync((void**)&base, bytes + 256, ds->pool, stream) != cudaSuccess) {
    cudaGetLastError();
    return IDX_ERR_CUDA;
  }
  uint32_t* word = (uint32_t*)(base + bytes);
  bool ok = enqueue(base, word) == cudaSuccess;
  uint32_t status = 0;
  // pageable destination: returns once the copy (and all earlier work on the stream) is done
  ok &= cudaMemcpyAsync(&status, word, sizeof(status), cudaMemcpyDeviceToHost, stream) == cudaSuccess;
  ok &= cudaFreeAsync(base, stream) == cudaSuccess;
  if (!ok || cudaGetLastError() != cudaSuccess) {
    cudaStreamSynchronize(stream);
    cudaGetLastError();
    return IDX_ERR_CUDA;
  }
  return (int)status;
}

inline int check_space(const Space& s) {
  if (!s.async) return IDX_OK;
  return s.status && ((uintptr_t)s.status & 3u) == 0 ? IDX_OK : IDX_ERR_INVALID_ARGUMENT;
}

const Space kSync = {false, nullptr, 0, nullptr};

}  // namespace idxk
