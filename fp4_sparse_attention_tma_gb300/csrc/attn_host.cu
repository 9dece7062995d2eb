// C ABI of the attention and eviction operators (declared in include/idxtopk.h): their
// argument checks, workspaces and kernel sequences.  Every operator has a stream-ordered
// form (caller workspace, device status word, nothing synchronised or allocated) and a
// synchronous one, which takes its workspace from the library's pool and reads the status
// back.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>

#include "attn.h"
#include "idx_host.h"
#include "idxtopk.h"

using namespace idxk;

namespace {

// Positions of a request, at most: the kernels step past a range's end by less than the rest
// of an int32.
constexpr int64_t kMostPositions = INT32_MAX - 65536;

// Validates a 16-bit tensor with free strides: type, rank, 16-byte aligned base, last
// dimension contiguous, other strides non-negative multiples of 8 elements whose offsets
// stay within 63 bits.
int check_strided(const idx_tensor_t* t, int dtype, int ndim) {
  if (!t || t->dtype != dtype || t->ndim != ndim) return IDX_ERR_INVALID_ARGUMENT;
  int64_t reach = 0, numel = 1;
  for (int i = 0; i < ndim; ++i) {
    if (t->shape[i] < 0) return IDX_ERR_INVALID_ARGUMENT;
    if (!mul_ok(numel, t->shape[i], &numel)) return IDX_ERR_OVERFLOW;
  }
  if (numel == 0) return IDX_OK;
  for (int i = 0; i < ndim; ++i) {
    if (t->shape[i] <= 1) continue;
    if (i == ndim - 1 ? t->stride[i] != 1 : t->stride[i] < 0 || t->stride[i] % 8 != 0)
      return IDX_ERR_INVALID_ARGUMENT;
    int64_t x;
    if (!mul_ok(t->shape[i] - 1, t->stride[i], &x) || x > (INT64_MAX / 4) - reach) return IDX_ERR_OVERFLOW;
    reach += x;
  }
  if (!t->data || ((uintptr_t)t->data & 15u) != 0) return IDX_ERR_INVALID_ARGUMENT;
  return IDX_OK;
}

// Whether no two elements of `t` share an address (its dimensions nest).
bool no_overlap(const idx_tensor_t* t) {
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

int elem_bytes(const idx_tensor_t* t) {
  return t->dtype == IDX_U8 ? 1 : t->dtype == IDX_BF16 || t->dtype == IDX_F16 ? 2 : 4;
}

// The bytes that `t` spans.
int64_t span_of(const idx_tensor_t* t) {
  int64_t reach = 1;
  for (int i = 0; i < t->ndim; ++i)
    if (t->shape[i] > 1) reach += (t->shape[i] - 1) * t->stride[i];
  return reach * elem_bytes(t);
}
constexpr int64_t kFar = ((int64_t)1 << 32) * 16 - 16;

// The addresses that `t` spans.
void range_of(const idx_tensor_t* t, uintptr_t* a, uintptr_t* b) {
  *a = (uintptr_t)t->data;
  *b = *a + (uintptr_t)span_of(t);
}

bool apart(const idx_tensor_t* x, const idx_tensor_t* y) {
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

bool same_layout(const idx_tensor_t* x, const idx_tensor_t* y) {
  if (x->data != y->data || x->ndim != y->ndim) return false;
  for (int i = 0; i < x->ndim; ++i)
    if (x->shape[i] != y->shape[i] || (x->shape[i] > 1 && x->stride[i] != y->stride[i])) return false;
  return true;
}

bool same_strides(const idx_tensor_t* x, const idx_tensor_t* y) {
  for (int i = 0; i < x->ndim; ++i)
    if (x->shape[i] != y->shape[i] || (x->shape[i] > 1 && x->stride[i] != y->stride[i])) return false;
  return true;
}

// Elements from the address of x to that of y.
int64_t distance(const idx_tensor_t* x, const idx_tensor_t* y) {
  return ((int64_t)(uintptr_t)y->data - (int64_t)(uintptr_t)x->data) / elem_bytes(x);
}

// Whether two elements of a cache whose dimensions nest (no_overlap) lie `delta` apart, other than two of
// one position (`one_position`: those do not count).  Dimension by dimension, the largest stride first: of
// the steps along it only one or two leave a rest that the others can reach.
bool elements_apart(const idx_tensor_t* t, int64_t delta, bool one_position, uint32_t used = 0, bool moved = false) {
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

// Whether keys and values moved into k_dst and v_dst (each without overlap in itself) keep out of each
// other's way: the two share no element, or only elements that the caches' keys and values of a position
// share alike (a latent cache that both are views of: the same bytes are moved twice).
bool places_agree(const idx_tensor_t* k, const idx_tensor_t* v, const idx_tensor_t* k_dst, const idx_tensor_t* v_dst) {
  if (apart(k_dst, v_dst)) return true;
  if (same_strides(k_dst, v_dst)) {
    bool alike = same_strides(k, v) && distance(k, v) == distance(k_dst, v_dst);
    for (int i = 1; i < 4; ++i) alike &= k->shape[i] <= 1 || k->stride[i] == k_dst->stride[i];
    return !elements_apart(k_dst, distance(k_dst, v_dst), alike);
  }
  // laid out differently: in every page apart
  const int64_t page = k_dst->stride[0];
  if (k_dst->shape[0] <= 1 || v_dst->stride[0] != page || page <= 0) return false;
  int64_t k_end = 1, v_end = 1;
  for (int i = 1; i < 4; ++i) {
    if (k_dst->shape[i] <= 1) continue;
    k_end += (k_dst->shape[i] - 1) * k_dst->stride[i];
    v_end += (v_dst->shape[i] - 1) * v_dst->stride[i];
  }
  int64_t at = distance(k_dst, v_dst) % page;
  if (at < 0) at += page;
  return at >= k_end && at + v_end <= page;
}

// The stride of dimension i (0 where it has one element: nothing steps along it).
int64_t step(const idx_tensor_t* t, int i) { return t->shape[i] > 1 ? t->stride[i] : 0; }

struct Machine {
  int dev = -1, sm = 0;
  bool capturing = false;
};

// The device of the call's tensors and its stream's state; `status` and `workspace` are
// checked to be of the same device when they are given.
int find_machine(const idx_tensor_t* const* ts, int n, const void* status, const void* workspace, cudaStream_t stream,
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
int check_arch(Machine* m) {
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
    if (!s.workspace || ((uintptr_t)s.workspace & 255u) != 0 || s.bytes < bytes) return IDX_ERR_INVALID_ARGUMENT;
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

int check_space(const Space& s) {
  if (!s.async) return IDX_OK;
  return s.status && ((uintptr_t)s.status & 3u) == 0 ? IDX_OK : IDX_ERR_INVALID_ARGUMENT;
}

// --------------------------------------------------------------- attention ----

struct AttnPlan {
  int32_t group, chunks, chunk_heads, group_rows, row_cols, tile, workers;
  bool tensor_core;
};

// Which of the two kernels, at head dimension 128 (attn_tc.cuh knows no other; and its offsets
// end where a cache spans 64 GB, `far`).  attn_tc.cuh loads with fewer instructions and holds 64
// query heads a row, but two rows of a request at the most, and a unit's end costs it 3 us;
// attn.cuh holds 16 or 32 pairs of query head and row.  Measured (us; attn_tc.cuh, attn.cuh):
//   one or two rows a request, long: 64 heads on 8, 32 requests of 4096..65536, 1 row 648, 672,
//     2 rows 652, 677; 32 heads on 8 184, 192; 8 on 8 184, 192; 64 on 1, 2 rows 105, 402
//   up to 2000 positions: 64 on 8 76, 76; up to 1000: 32 on 8 110, 105; 64 on 1 36, 69
//   windows of 100 under a table of 4000, 32 on 8: 256 requests 74, 37, 76 requests 33, 21, 38 requests
//     25, 20; of 2000: 256 requests 324, 333 (hence: many units, which may be short, are attn.cuh's)
//   more rows than two: 64 on 8, 3 rows 1271, 1008 (as many walks as for 4 rows and half as many again: groups
//     begin at fixed row numbers), 4 rows 757 (attn.cuh); 8 on 1, 4 rows 165, 145; but 16 on 1, 4 rows
//     166, 237 (with 11 heads or more attn.cuh's tile holds two rows as well)
//   slots: 2048 rows of 1024, 32 on 4 480, 516; 64 rows of 1024, 32 on 8 46, 49; 2048 of 512,
//     16 on 1 87, 80, 24 on 1 88, 137; 4096 of 128, 16 on 1 96, 56
// `positions`: what a row sees at most, as far as the host knows (the page table's width).
bool tensor_core_for(int64_t group, int64_t rows, int64_t per_req, int64_t kv_heads, int64_t dim, int64_t positions,
                     bool slots, bool far, int sm) {
  if (dim != 128 || far) return false;
  if (group > 16) return true;
  if (slots) return positions >= 1024;
  if (group > 10 && group * per_req > 16) return true;
  return per_req <= 2 && positions >= 2048 && (rows + per_req - 1) / per_req * kv_heads <= 2 * sm;
}

// How the query heads of a key-value head are laid on the kernel's tiles.  The page table's rows stand for
// the number of requests, which the host does not know: under a table of more rows than the call has, rows
// are taken for single ones (one call between events: 32 requests x 2 rows x 64 heads on one 178 us, 120
// under a table of 32; x 4 rows x 64 heads on 8 1313, 756).  attn_tc.cuh: 64 columns
// a row, two rows of a request together where requests have several (32 requests x 2 rows x 64
// heads on one: 105 us, 166 one by one).  attn.cuh: a tile holds 16 (query head, row) pairs; where
// a group, or its rows that share the cache, need more, 32 (two tiles that share every key and
// value read; 32 requests x 4 rows x 64 heads on 8: 757 us, 1295 with 16), up to head dimension
// 128 (beyond it two tiles' sums do not fit a thread's registers).
AttnPlan plan_of(int64_t rows, int64_t num_req, int64_t q_heads, int64_t kv_heads, int64_t dim, int64_t positions,
                 bool slots, bool far, int sm) {
  AttnPlan a{};
  a.group = (int32_t)(q_heads / kv_heads);
  const int64_t per_req = rows > num_req && num_req > 0 ? (rows + num_req - 1) / num_req : 1;
  a.tensor_core = tensor_core_for(a.group, rows, per_req, kv_heads, dim, positions, slots, far, sm);
  const int32_t most = a.tensor_core ? 64 : dim <= 128 && (int64_t)a.group * per_req > 16 ? 32 : 16;
  a.chunks = (a.group + most - 1) / most;
  a.chunk_heads = (a.group + a.chunks - 1) / a.chunks;
  if (a.tensor_core) {
    a.group_rows = a.chunks == 1 && per_req > 1 ? 2 : 1;
    a.row_cols = most;
    a.tile = a.group_rows * most;
    a.workers = sm;
  } else {
    a.group_rows = a.chunks > 1 ? 1 : most / a.group;
    a.row_cols = a.chunk_heads;
    a.tile = most;
    a.workers = sm * attn_warps((int32_t)dim, most);
  }
  return a;
}

int check_heads(const idx_tensor_t* q, const idx_tensor_t* k, const idx_tensor_t* v, const idx_tensor_t* out) {
  if (!q || (q->dtype != IDX_BF16 && q->dtype != IDX_F16)) return IDX_ERR_INVALID_ARGUMENT;
  int st;
  if ((st = check_strided(q, q->dtype, 3)) || (st = check_strided(k, q->dtype, 4)) ||
      (st = check_strided(v, q->dtype, 4)) || (st = check_strided(out, q->dtype, 3)))
    return st;
  const int64_t D = q->shape[2], Hq = q->shape[1], Hk = k->shape[2];
  for (int i = 0; i < 4; ++i)
    if (k->shape[i] != v->shape[i]) return IDX_ERR_INVALID_ARGUMENT;
  for (int i = 0; i < 3; ++i)
    if (q->shape[i] != out->shape[i]) return IDX_ERR_INVALID_ARGUMENT;
  if (k->shape[3] != D || Hk < 1 || Hq < 1 || Hq % Hk != 0) return IDX_ERR_INVALID_ARGUMENT;
  if ((D != 64 && D != 128 && D != 256) || k->shape[1] != kPage) return IDX_ERR_UNSUPPORTED;
  if (!no_overlap(out)) return IDX_ERR_INVALID_ARGUMENT;
  if (q->shape[0] > INT32_MAX || Hq > 65536 || k->shape[0] * (int64_t)kPage > INT32_MAX) return IDX_ERR_OVERFLOW;
  return IDX_OK;
}

struct AttnCall {
  const idx_tensor_t *q, *k, *v, *page_table, *row_req, *row_start, *row_end, *slots;
  float scale;
  const idx_tensor_t *out, *lse, *weight_in, *weight_out;
};

AttnLayout layout_of(const AttnPlan& a, int sm, int64_t rows, int64_t q_heads, int64_t dim, int64_t max_pages,
                     bool weights) {
  return attn_layout(a.workers, sm, a.tile, dim, weights ? rows * q_heads : 0, weights ? max_pages * kPage : 0);
}

int run_attn(const AttnCall& c, const Space& space, cudaStream_t stream) {
  int st;
  if ((st = check_space(space))) return st;
  if ((st = check_heads(c.q, c.k, c.v, c.out))) return st;
  const int64_t R = c.q->shape[0], Hq = c.q->shape[1], D = c.q->shape[2], NP = c.k->shape[0], Hk = c.k->shape[2];
  const float scale_log2 = c.scale * 1.4426950408889634f;   // what the kernels work with
  if (!(c.scale > 0.f) || !std::isfinite(scale_log2)) return IDX_ERR_INVALID_ARGUMENT;
  if (c.lse && ((st = check_tensor(c.lse, IDX_F32, 2)))) return st;
  if (c.lse && (c.lse->shape[0] != R || c.lse->shape[1] != Hq)) return IDX_ERR_INVALID_ARGUMENT;
  int64_t NR = 1, MP = 0;
  if (c.slots) {
    if ((st = check_tensor(c.slots, IDX_I32, 2))) return st;
    if (c.slots->shape[0] != R || c.slots->shape[1] < 1) return IDX_ERR_INVALID_ARGUMENT;
    if (c.slots->shape[1] > kMostPositions) return IDX_ERR_OVERFLOW;
  } else {
    if ((st = check_tensor(c.page_table, IDX_I32, 2)) || (st = check_tensor(c.row_req, IDX_I32, 1)) ||
        (st = check_tensor(c.row_start, IDX_I32, 1)) || (st = check_tensor(c.row_end, IDX_I32, 1)))
      return st;
    NR = c.page_table->shape[0], MP = c.page_table->shape[1];
    if (c.row_req->shape[0] != R || c.row_start->shape[0] != R || c.row_end->shape[0] != R)
      return IDX_ERR_INVALID_ARGUMENT;
    if (MP * (int64_t)kPage > kMostPositions || NR > INT32_MAX) return IDX_ERR_OVERFLOW;
    if (R > 0 && (NR < 1 || MP < 1)) return IDX_ERR_INVALID_ARGUMENT;
  }
  if (c.weight_in && !c.weight_out) return IDX_ERR_INVALID_ARGUMENT;
  for (const idx_tensor_t* w : {c.weight_in, c.weight_out}) {
    if (!w) continue;
    if ((st = check_tensor(w, IDX_F32, 2))) return st;
    if (w->shape[0] != NR || w->shape[1] != MP * kPage) return IDX_ERR_INVALID_ARGUMENT;
  }
  if (R > 0 && NP < 1) return IDX_ERR_INVALID_ARGUMENT;
  const bool in_place = c.weight_in && c.weight_in->data == c.weight_out->data;
  const idx_tensor_t* outs[] = {c.out, c.lse, c.weight_out};
  const idx_tensor_t* ins[] = {c.q,       c.k,     c.v,    c.page_table, c.row_req, c.row_start,
                               c.row_end, c.slots, in_place ? nullptr : c.weight_in};
  if (!all_apart(outs, ins)) return IDX_ERR_INVALID_ARGUMENT;
  const idx_tensor_t* all[] = {c.q,       c.k,     c.v,   c.page_table, c.row_req, c.row_start,
                               c.row_end, c.slots, c.out, c.lse,        c.weight_in, c.weight_out};
  Machine m;
  if ((st = find_machine(all, 12, space.status, space.workspace, stream, &m))) return st;
  if (m.capturing && !space.async) return IDX_ERR_UNSUPPORTED;
  DeviceGuard guard(m.dev);
  if (!guard.ok()) return IDX_ERR_CUDA;
  if ((st = check_arch(&m))) return st;
  const bool weights = c.weight_out != nullptr && numel_of(c.weight_out) > 0;
  const bool far = span_of(c.k) >= kFar || span_of(c.v) >= kFar;
  const AttnPlan a = c.slots ? plan_of(R, R, Hq, Hk, D, c.slots->shape[1], true, far, m.sm)
                             : plan_of(R, NR, Hq, Hk, D, MP * kPage, false, far, m.sm);
  int64_t logit_rows, logit_bytes;
  if (weights && (!mul_ok(R * Hq, MP * kPage, &logit_rows) || !mul_ok(logit_rows, 4, &logit_bytes) ||
                  logit_bytes > (INT64_MAX >> 2)))
    return IDX_ERR_OVERFLOW;
  const AttnLayout L = layout_of(a, m.sm, R, Hq, D, MP, weights);
  AttnParams p{};
  p.q = c.q->data, p.k = c.k->data, p.v = c.v->data, p.out = c.out->data;
  p.lse = c.lse ? (float*)c.lse->data : nullptr;
  p.q_row = step(c.q, 0), p.q_head = step(c.q, 1);
  p.out_row = step(c.out, 0), p.out_head = step(c.out, 1);
  p.k_page = step(c.k, 0), p.k_slot = step(c.k, 1), p.k_head = step(c.k, 2);
  p.v_page = step(c.v, 0), p.v_slot = step(c.v, 1), p.v_head = step(c.v, 2);
  if (c.slots) {
    p.slots = (const int32_t*)c.slots->data;
    p.n_slots = (int32_t)c.slots->shape[1];
  } else {
    p.page_table = (const int32_t*)c.page_table->data;
    p.row_req = (const int32_t*)c.row_req->data;
    p.row_start = (const int32_t*)c.row_start->data;
    p.row_end = (const int32_t*)c.row_end->data;
  }
  p.rows = (int32_t)R, p.num_req = (int32_t)NR, p.max_pages = (int32_t)MP, p.num_pages = (int32_t)NP;
  p.q_heads = (int32_t)Hq, p.kv_heads = (int32_t)Hk;
  p.group = a.group, p.chunks = a.chunks, p.chunk_heads = a.chunk_heads, p.group_rows = a.group_rows;
  p.row_cols = a.row_cols, p.tensor_core = a.tensor_core;
  p.far = far;
  p.workers = R > 0 ? a.workers : 0;
  p.n_cta = R > 0 ? m.sm : 0;
  p.scale_log2 = scale_log2;
  p.tile = a.tile, p.dim = (int32_t)D;
  const bool bf16 = c.q->dtype == IDX_BF16;
  return with_space(space, L.total, m, stream, [&](char* base, uint32_t* status) -> cudaError_t {
    p.cta_status = (uint32_t*)(base + L.cta_status);
    p.active = (int32_t*)(base + L.active);
    p.open_parts = (int32_t*)(base + L.open_parts);
    p.open_info = (int4*)(base + L.open_info);
    p.part_ml = (float2*)(base + L.part_ml);
    p.part_o = (float*)(base + L.part_o);
    if (weights) {
      p.row_stat = (float2*)(base + L.row_stat);
      p.logits = (float*)(base + L.logits);
      p.weight_in = c.weight_in ? (const float*)c.weight_in->data : nullptr;
      p.weight_out = (float*)c.weight_out->data;
    }
    p.status_out = status;
    cudaError_t e = cudaSuccess;
    if (R > 0 && (e = launch_attn(p, bf16, m.sm, stream)) != cudaSuccess) return e;
    if ((e = launch_attn_join(p, bf16, m.sm, stream)) != cudaSuccess) return e;
    return weights ? launch_attn_weights(p, stream) : cudaSuccess;
  });
}

int attn_bytes(int64_t rows, int64_t q_heads, int64_t kv_heads, int64_t dim, int64_t num_req, int64_t max_pages,
               bool slots, bool weights, int32_t device, uint64_t* bytes) {
  if (!bytes || rows < 0 || kv_heads < 1 || q_heads < 1 || q_heads % kv_heads != 0 || max_pages < 0)
    return IDX_ERR_INVALID_ARGUMENT;
  if (dim != 64 && dim != 128 && dim != 256) return IDX_ERR_UNSUPPORTED;
  int sm = 0, major = 0, minor = 0;
  int st = device_info_no_pool(device, &sm, &major, &minor);
  if (st) return st;
  int64_t n;
  if (weights && (!mul_ok(rows * q_heads, max_pages * kPage, &n) || n > (INT64_MAX >> 4))) return IDX_ERR_OVERFLOW;
  // whichever kernel the caches' extent and the rows' length choose
  *bytes = 0;
  for (bool far : {false, true})
    for (int64_t positions : {(int64_t)1, kMostPositions}) {
      const AttnPlan a = plan_of(rows, num_req, q_heads, kv_heads, dim, positions, slots, far, sm);
      const uint64_t n = layout_of(a, sm, rows, q_heads, dim, max_pages, weights).total;
      if (n > *bytes) *bytes = n;
    }
  return IDX_OK;
}

// ---------------------------------------------------------------- eviction ----

struct EvictCall {
  const idx_tensor_t *k, *v, *page_table, *seq_len, *weight;
  int32_t budget, first, last;
  const idx_tensor_t *k_dst, *v_dst, *dst_table, *keep, *new_len, *new_table, *new_weight;
};

// Workspace: a status word per cluster, then the bitmaps (if they are not in shared memory).
size_t evict_space(int64_t num_req, int64_t dst_pages, size_t* mark) {
  *mark = align_up((size_t)(num_req + 1) * 4, 256);
  const size_t bitmap = evict_mark_shared(dst_pages) ? 0 : (size_t)((dst_pages + 31) / 32) * 4;
  return *mark + align_up(bitmap * 8, 256);   // a cluster has at most 8 CTAs
}

int run_evict(const EvictCall& c, const Space& space, cudaStream_t stream) {
  int st;
  if ((st = check_space(space))) return st;
  if (!c.k || (c.k->dtype != IDX_BF16 && c.k->dtype != IDX_F16)) return IDX_ERR_INVALID_ARGUMENT;
  for (const idx_tensor_t* t : {c.k, c.v, c.k_dst, c.v_dst})
    if ((st = check_strided(t, c.k->dtype, 4))) return st;
  if ((st = check_tensor(c.page_table, IDX_I32, 2)) || (st = check_tensor(c.seq_len, IDX_I32, 1)) ||
      (st = check_tensor(c.weight, IDX_F32, 2)) || (st = check_tensor(c.dst_table, IDX_I32, 2)) ||
      (st = check_tensor(c.keep, IDX_I32, 2)) || (st = check_tensor(c.new_len, IDX_I32, 1)) ||
      (st = check_tensor(c.new_table, IDX_I32, 2)) || (st = check_tensor(c.new_weight, IDX_F32, 2)))
    return st;
  const int64_t NP = c.k->shape[0], Hk = c.k->shape[2], D = c.k->shape[3], DN = c.k_dst->shape[0];
  const int64_t NR = c.page_table->shape[0], MP = c.page_table->shape[1], DP = c.dst_table->shape[1];
  for (int i = 0; i < 4; ++i) {
    if (c.k->shape[i] != c.v->shape[i] || c.k_dst->shape[i] != c.v_dst->shape[i]) return IDX_ERR_INVALID_ARGUMENT;
    if (i > 0 && c.k_dst->shape[i] != c.k->shape[i]) return IDX_ERR_INVALID_ARGUMENT;
  }
  if (Hk < 1) return IDX_ERR_INVALID_ARGUMENT;
  if ((D != 64 && D != 128 && D != 256) || c.k->shape[1] != kPage) return IDX_ERR_UNSUPPORTED;
  if (NP * kPage > INT32_MAX || DN * kPage > INT32_MAX || MP * kPage > kMostPositions || Hk > 65536 || NR >= INT32_MAX / 8)
    return IDX_ERR_OVERFLOW;
  if (c.budget < 1 || c.first < 0 || c.last < 0 || (int64_t)c.first + c.last > c.budget)
    return IDX_ERR_INVALID_ARGUMENT;
  const int64_t widest = c.budget < MP * kPage ? c.budget : MP * kPage;
  if (c.seq_len->shape[0] != NR || c.weight->shape[0] != NR || c.weight->shape[1] != MP * kPage ||
      c.dst_table->shape[0] != NR || DP > MP || DP * kPage < widest || c.keep->shape[0] != NR ||
      c.keep->shape[1] != c.budget || c.new_len->shape[0] != NR || c.new_table->shape[0] != NR ||
      c.new_table->shape[1] != MP || c.new_weight->shape[0] != NR || c.new_weight->shape[1] != MP * kPage)
    return IDX_ERR_INVALID_ARGUMENT;
  if (NR > 0 && (MP < 1 || NP < 1 || DN < 1)) return IDX_ERR_INVALID_ARGUMENT;
  const int64_t used = (c.budget + kPage - 1) / kPage;
  if (NR * used > INT32_MAX / 32) return IDX_ERR_OVERFLOW;   // CTAs of the copy
  // the fresh pages are pages of the same tensors, or of others that lie apart from them
  const bool same = NR > 0 && same_layout(c.k, c.k_dst) && same_layout(c.v, c.v_dst);
  if (!no_overlap(c.k_dst) || !no_overlap(c.v_dst)) return IDX_ERR_INVALID_ARGUMENT;
  if (NR > 0 && !places_agree(c.k, c.v, c.k_dst, c.v_dst)) return IDX_ERR_INVALID_ARGUMENT;
  for (const idx_tensor_t* d : {c.k_dst, c.v_dst})
    for (const idx_tensor_t* s : {c.k, c.v})
      if (!same && !apart(d, s)) return IDX_ERR_INVALID_ARGUMENT;
  const idx_tensor_t* outs[] = {c.keep, c.new_len, c.new_table, c.new_weight};
  const idx_tensor_t* ins[] = {c.k, c.v, c.page_table, c.seq_len, c.weight, c.k_dst, c.v_dst, c.dst_table};
  if (!all_apart(outs, ins)) return IDX_ERR_INVALID_ARGUMENT;
  const idx_tensor_t* moved[] = {c.page_table, c.seq_len, c.weight, c.dst_table};
  for (const idx_tensor_t* t : moved)
    if (!apart(t, c.k_dst) || !apart(t, c.v_dst)) return IDX_ERR_INVALID_ARGUMENT;
  const idx_tensor_t* all[] = {c.k,     c.v,         c.page_table, c.seq_len, c.weight,    c.k_dst,
                               c.v_dst, c.dst_table, c.keep,       c.new_len, c.new_table, c.new_weight};
  Machine m;
  if ((st = find_machine(all, 12, space.status, space.workspace, stream, &m))) return st;
  if (m.capturing && !space.async) return IDX_ERR_UNSUPPORTED;
  DeviceGuard guard(m.dev);
  if (!guard.ok()) return IDX_ERR_CUDA;
  if ((st = check_arch(&m))) return st;
  EvictParams p{};
  p.k = c.k->data, p.v = c.v->data, p.k_dst = c.k_dst->data, p.v_dst = c.v_dst->data;
  p.k_page = step(c.k, 0) * 2, p.k_slot = step(c.k, 1) * 2, p.k_head = step(c.k, 2) * 2;
  p.v_page = step(c.v, 0) * 2, p.v_slot = step(c.v, 1) * 2, p.v_head = step(c.v, 2) * 2;
  p.kd_page = step(c.k_dst, 0) * 2, p.kd_slot = step(c.k_dst, 1) * 2, p.kd_head = step(c.k_dst, 2) * 2;
  p.vd_page = step(c.v_dst, 0) * 2, p.vd_slot = step(c.v_dst, 1) * 2, p.vd_head = step(c.v_dst, 2) * 2;
  p.page_table = (const int32_t*)c.page_table->data;
  p.seq_len = (const int32_t*)c.seq_len->data;
  p.dst_table = (const int32_t*)c.dst_table->data;
  p.weight = (const float*)c.weight->data;
  p.keep = (int32_t*)c.keep->data;
  p.new_len = (int32_t*)c.new_len->data;
  p.new_table = (int32_t*)c.new_table->data;
  p.new_weight = (float*)c.new_weight->data;
  p.num_req = (int32_t)NR, p.max_pages = (int32_t)MP, p.num_pages = (int32_t)NP, p.dst_pages = (int32_t)DN;
  p.dst_width = (int32_t)DP;
  p.budget = c.budget, p.keep_first = c.first, p.keep_last = c.last;
  p.kv_heads = (int32_t)Hk, p.head_bytes = (int32_t)D * 2;
  p.same_pool = same ? 1 : 0;
  size_t mark;
  const size_t bytes = evict_space(NR, DN, &mark);
  return with_space(space, bytes, m, stream, [&](char* base, uint32_t* status) -> cudaError_t {
    if (NR == 0) return cudaMemsetAsync(status, 0, sizeof(uint32_t), stream);
    p.part_status = (uint32_t*)base;
    p.dst_mark = (uint32_t*)(base + mark);
    p.status_out = status;
    return launch_evict(p, m.sm, stream);
  });
}

const Space kSync = {false, nullptr, 0, nullptr};

}  // namespace

extern "C" {

int idx_attn_paged(const idx_tensor_t* q, const idx_tensor_t* k_cache, const idx_tensor_t* v_cache,
                   const idx_tensor_t* page_table, const idx_tensor_t* row_req, const idx_tensor_t* row_start,
                   const idx_tensor_t* row_end, float scale, const idx_tensor_t* out, const idx_tensor_t* out_lse,
                   const idx_tensor_t* weight_in, const idx_tensor_t* weight_out, idx_stream_t stream) {
  return run_attn({q, k_cache, v_cache, page_table, row_req, row_start, row_end, nullptr, scale, out, out_lse,
                   weight_in, weight_out},
                  kSync, (cudaStream_t)stream);
}

int idx_attn_paged_async(const idx_tensor_t* q, const idx_tensor_t* k_cache, const idx_tensor_t* v_cache,
                         const idx_tensor_t* page_table, const idx_tensor_t* row_req, const idx_tensor_t* row_start,
                         const idx_tensor_t* row_end, float scale, const idx_tensor_t* out,
                         const idx_tensor_t* out_lse, const idx_tensor_t* weight_in, const idx_tensor_t* weight_out,
                         void* workspace, uint64_t workspace_bytes, uint32_t* status, idx_stream_t stream) {
  return run_attn({q, k_cache, v_cache, page_table, row_req, row_start, row_end, nullptr, scale, out, out_lse,
                   weight_in, weight_out},
                  {true, workspace, workspace_bytes, status}, (cudaStream_t)stream);
}

int idx_attn_paged_scratch_bytes(int32_t rows, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t num_req,
                                 int32_t max_pages, int32_t with_weights, int32_t device, uint64_t* bytes) {
  return attn_bytes(rows, q_heads, kv_heads, head_dim, num_req, max_pages, false, with_weights != 0, device, bytes);
}

int idx_attn_selected(const idx_tensor_t* q, const idx_tensor_t* k_cache, const idx_tensor_t* v_cache,
                      const idx_tensor_t* slots, float scale, const idx_tensor_t* out, const idx_tensor_t* out_lse,
                      idx_stream_t stream) {
  if (!slots) return IDX_ERR_INVALID_ARGUMENT;
  return run_attn({q, k_cache, v_cache, nullptr, nullptr, nullptr, nullptr, slots, scale, out, out_lse, nullptr,
                   nullptr},
                  kSync, (cudaStream_t)stream);
}

int idx_attn_selected_async(const idx_tensor_t* q, const idx_tensor_t* k_cache, const idx_tensor_t* v_cache,
                            const idx_tensor_t* slots, float scale, const idx_tensor_t* out,
                            const idx_tensor_t* out_lse, void* workspace, uint64_t workspace_bytes, uint32_t* status,
                            idx_stream_t stream) {
  if (!slots) return IDX_ERR_INVALID_ARGUMENT;
  return run_attn({q, k_cache, v_cache, nullptr, nullptr, nullptr, nullptr, slots, scale, out, out_lse, nullptr,
                   nullptr},
                  {true, workspace, workspace_bytes, status}, (cudaStream_t)stream);
}

int idx_attn_selected_scratch_bytes(int32_t rows, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                    int32_t selected, int32_t device, uint64_t* bytes) {
  if (selected < 1) return IDX_ERR_INVALID_ARGUMENT;
  return attn_bytes(rows, q_heads, kv_heads, head_dim, rows, 0, true, false, device, bytes);
}

int idx_cache_evict(const idx_tensor_t* k_cache, const idx_tensor_t* v_cache, const idx_tensor_t* page_table,
                    const idx_tensor_t* seq_len, const idx_tensor_t* weight, int32_t budget, int32_t keep_first,
                    int32_t keep_last, const idx_tensor_t* k_dst, const idx_tensor_t* v_dst,
                    const idx_tensor_t* dst_page_table, const idx_tensor_t* out_keep_idx, const idx_tensor_t* out_len,
                    const idx_tensor_t* out_page_table, const idx_tensor_t* out_weight, idx_stream_t stream) {
  return run_evict({k_cache, v_cache, page_table, seq_len, weight, budget, keep_first, keep_last, k_dst, v_dst,
                    dst_page_table, out_keep_idx, out_len, out_page_table, out_weight},
                   kSync, (cudaStream_t)stream);
}

int idx_cache_evict_async(const idx_tensor_t* k_cache, const idx_tensor_t* v_cache, const idx_tensor_t* page_table,
                          const idx_tensor_t* seq_len, const idx_tensor_t* weight, int32_t budget, int32_t keep_first,
                          int32_t keep_last, const idx_tensor_t* k_dst, const idx_tensor_t* v_dst,
                          const idx_tensor_t* dst_page_table, const idx_tensor_t* out_keep_idx,
                          const idx_tensor_t* out_len, const idx_tensor_t* out_page_table,
                          const idx_tensor_t* out_weight, void* workspace, uint64_t workspace_bytes, uint32_t* status,
                          idx_stream_t stream) {
  return run_evict({k_cache, v_cache, page_table, seq_len, weight, budget, keep_first, keep_last, k_dst, v_dst,
                    dst_page_table, out_keep_idx, out_len, out_page_table, out_weight},
                   {true, workspace, workspace_bytes, status}, (cudaStream_t)stream);
}

int idx_cache_evict_scratch_bytes(int32_t num_req, int32_t max_pages, int32_t dst_pages, int32_t budget,
                                  int32_t device, uint64_t* bytes) {
  if (!bytes || num_req < 0 || max_pages < 0 || dst_pages < 0 || budget < 1 || device < 0)
    return IDX_ERR_INVALID_ARGUMENT;
  size_t mark;
  *bytes = evict_space(num_req, dst_pages, &mark);
  return IDX_OK;
}

}  // extern "C"
