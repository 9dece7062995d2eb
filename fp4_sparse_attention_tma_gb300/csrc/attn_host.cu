// C ABI of the attention and eviction operators (declared in include/idxtopk.h): their
// argument checks, workspaces and kernel sequences.  Every operator has a stream-ordered
// form (caller workspace, device status word, nothing synchronised or allocated) and a
// synchronous one, which takes its workspace from the library's pool and reads the status
// back.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>

#include "attn.h"
#include "idxtopk.h"
#include "op_host.h"

using namespace idxk;

namespace {

// Positions of a request, at most: the kernels step past a range's end by less than the rest
// of an int32.
constexpr int64_t kMostPositions = INT32_MAX - 65536;

// --------------------------------------------------------------- attention ----

struct AttnPlan {
  int32_t group, chunks, chunk_heads, group_rows, row_cols, tile, workers, team;
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

// The same for a 4-bit cache (attn_fp4.cuh; its form on tensor memory is attn_tc.cuh's).  There decoding the
// codes costs more than the products: attn_tc.cuh does it once for 64 pairs of query head and row, attn_fp4.cuh
// for 16 or 32, by more warps.  Measured (us between events; attn_tc.cuh, attn_fp4.cuh), fp16, heads on one:
//   32 requests of 4096..65536: 1 row, 8 heads 74, 75, 16 75, 82, 17 76, 118, 32 76, 127, 64 81, 212, 128 133, 357;
//     2 rows, 8 heads 105, 82, 12 106, 126, 16 109, 127, 17 108, 200, 32 112, 211, 64 120, 358, 128 239, 661
//     (2 rows, 64 heads on 4 351, 347); 4 rows, 12 heads 185, 206, 16 188, 211
//   2 rows of 700..1000 positions: 8 heads 29, 25, 12 29, 33, 16 30, 37, 24 29, 46, 64 33, 40
//   2 rows of 100..200: 12 heads 25, 23, 24 25, 24, 64 27, 28; windows of 100, 256 requests: 16 51, 40, 24 52, 43,
//     64 58, 56, 128 70, 73 (how long a window is, the host does not know)
//   chosen slots, 512 rows of 1024: 16 heads 61, 46, 20 58, 85, 64 67, 146; 8192 of 128: 16 277, 87, 24 235, 196,
//     32 230, 211, 64 267, 378; 64 of 16384: 16 72, 70, 20 72, 133
bool tensor_core_for_fp4(int64_t group, int64_t per_req, int64_t dim, bool slots, bool far) {
  if (dim != 128 || far) return false;
  return group > 16 || (!slots && group > 10 && group * per_req > 16);
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
                 bool slots, bool far, bool fp4, int sm) {
  AttnPlan a{};
  a.group = (int32_t)(q_heads / kv_heads);
  const int64_t per_req = rows > num_req && num_req > 0 ? (rows + num_req - 1) / num_req : 1;
  a.tensor_core = fp4 ? tensor_core_for_fp4(a.group, per_req, dim, slots, far)
                       : tensor_core_for(a.group, rows, per_req, kv_heads, dim, positions, slots, far, sm);
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
    a.workers = sm * (fp4 ? attn_fp4_warps((int32_t)dim, most, slots) : attn_warps((int32_t)dim, most));
  }
  a.team = fp4 && !a.tensor_core ? attn_fp4_team(kv_heads, a.workers / sm) : 1;
  return a;
}

// `fp4`: k and v are codes, [NP, 64, Hk, D / 2].
int check_heads(const idx_tensor_t* q, const idx_tensor_t* k, const idx_tensor_t* v, const idx_tensor_t* out, bool fp4) {
  if (!q || (q->dtype != IDX_BF16 && q->dtype != IDX_F16)) return IDX_ERR_INVALID_ARGUMENT;
  int st;
  const int cached = fp4 ? IDX_U8 : q->dtype;
  if ((st = check_strided(q, q->dtype, 3)) || (st = check_strided(k, cached, 4, fp4 ? 16 : 8)) ||
      (st = check_strided(v, cached, 4, fp4 ? 16 : 8)) || (st = check_strided(out, q->dtype, 3)))
    return st;
  const int64_t D = q->shape[2], Hq = q->shape[1], Hk = k->shape[2];
  for (int i = 0; i < 4; ++i)
    if (k->shape[i] != v->shape[i]) return IDX_ERR_INVALID_ARGUMENT;
  for (int i = 0; i < 3; ++i)
    if (q->shape[i] != out->shape[i]) return IDX_ERR_INVALID_ARGUMENT;
  if (k->shape[3] != (fp4 ? D / 2 : D) || Hk < 1 || Hq < 1 || Hq % Hk != 0) return IDX_ERR_INVALID_ARGUMENT;
  if ((D != 64 && D != 128 && D != 256) || k->shape[1] != kPage) return IDX_ERR_UNSUPPORTED;
  if (!no_overlap(out)) return IDX_ERR_INVALID_ARGUMENT;
  if (q->shape[0] > INT32_MAX || Hq > 65536 || k->shape[0] * (int64_t)kPage > INT32_MAX) return IDX_ERR_OVERFLOW;
  return IDX_OK;
}

struct AttnCall {
  const idx_tensor_t *q, *k, *v, *page_table, *row_req, *row_start, *row_end, *slots;
  float scale;
  const idx_tensor_t *out, *lse, *weight_in, *weight_out;
  const idx_tensor_t *k_scale, *v_scale;   // a cache in 4 bits
  bool fp4;
};

// The scales of a 4-bit cache's codes.
int check_scales(const idx_tensor_t* codes, const idx_tensor_t* scale, int64_t D) {
  const int st = check_strided(scale, IDX_U8, 4, D / 32);
  if (st) return st;
  for (int i = 0; i < 3; ++i)
    if (scale->shape[i] != codes->shape[i]) return IDX_ERR_INVALID_ARGUMENT;
  return scale->shape[3] == D / 32 ? IDX_OK : IDX_ERR_INVALID_ARGUMENT;
}

AttnLayout layout_of(const AttnPlan& a, int sm, int64_t rows, int64_t q_heads, int64_t dim, int64_t max_pages,
                     bool weights) {
  return attn_layout(a.workers, sm, a.tile, dim, weights ? rows * q_heads : 0, weights ? max_pages * kPage : 0);
}

int run_attn(const AttnCall& c, const Space& space, cudaStream_t stream) {
  int st;
  if ((st = check_space(space))) return st;
  if ((st = check_heads(c.q, c.k, c.v, c.out, c.fp4))) return st;
  if (c.fp4 && ((st = check_scales(c.k, c.k_scale, c.q->shape[2])) || (st = check_scales(c.v, c.v_scale, c.q->shape[2]))))
    return st;
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
  const idx_tensor_t* ins[] = {c.q,       c.k,     c.v,       c.page_table, c.row_req, c.row_start,
                               c.row_end, c.slots, c.k_scale, c.v_scale,    in_place ? nullptr : c.weight_in};
  if (!all_apart(outs, ins)) return IDX_ERR_INVALID_ARGUMENT;
  const idx_tensor_t* all[] = {c.q,   c.k,   c.v,         c.page_table, c.row_req, c.row_start, c.row_end, c.slots,
                               c.out, c.lse, c.weight_in, c.weight_out, c.k_scale, c.v_scale};
  Machine m;
  if ((st = find_machine(all, 14, space.status, space.workspace, stream, &m))) return st;
  if (m.capturing && !space.async) return IDX_ERR_UNSUPPORTED;
  DeviceGuard guard(m.dev);
  if (!guard.ok()) return IDX_ERR_CUDA;
  if ((st = check_arch(&m))) return st;
  const bool weights = c.weight_out != nullptr && numel_of(c.weight_out) > 0;
  const bool far = span_of(c.k) >= kFar || span_of(c.v) >= kFar ||
                   (c.fp4 && (span_of(c.k_scale) > UINT32_MAX || span_of(c.v_scale) > UINT32_MAX));
  const AttnPlan a = c.slots ? plan_of(R, R, Hq, Hk, D, c.slots->shape[1], true, far, c.fp4, m.sm)
                             : plan_of(R, NR, Hq, Hk, D, MP * kPage, false, far, c.fp4, m.sm);
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
  if (c.fp4) {
    p.k_scale = (const uint8_t*)c.k_scale->data, p.v_scale = (const uint8_t*)c.v_scale->data;
    p.ks_page = step(c.k_scale, 0), p.ks_slot = step(c.k_scale, 1), p.ks_head = step(c.k_scale, 2);
    p.vs_page = step(c.v_scale, 0), p.vs_slot = step(c.v_scale, 1), p.vs_head = step(c.v_scale, 2);
  }
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
  // (attn_fp4.cuh: offsets in 32 bits)
  p.far = c.fp4 && !a.tensor_core ? far || span_of(c.k) > UINT32_MAX || span_of(c.v) > UINT32_MAX : far;
  p.workers = R > 0 ? a.workers : 0;
  p.team = a.team, p.ranges = p.workers / a.team, p.kv_units = (int32_t)Hk / a.team;
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
               bool slots, bool weights, bool fp4, int32_t device, uint64_t* bytes) {
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
      const AttnPlan a = plan_of(rows, num_req, q_heads, kv_heads, dim, positions, slots, far, fp4, sm);
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
  return attn_bytes(rows, q_heads, kv_heads, head_dim, num_req, max_pages, false, with_weights != 0, false, device, bytes);
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
  return attn_bytes(rows, q_heads, kv_heads, head_dim, rows, 0, true, false, false, device, bytes);
}

int idx_attn_paged_fp4(const idx_tensor_t* q, const idx_tensor_t* k_codes, const idx_tensor_t* k_scale,
                       const idx_tensor_t* v_codes, const idx_tensor_t* v_scale, const idx_tensor_t* page_table,
                       const idx_tensor_t* row_req, const idx_tensor_t* row_start, const idx_tensor_t* row_end, float scale,
                       const idx_tensor_t* out, const idx_tensor_t* out_lse, idx_stream_t stream) {
  return run_attn({q, k_codes, v_codes, page_table, row_req, row_start, row_end, nullptr, scale, out, out_lse, nullptr,
                   nullptr, k_scale, v_scale, true},
                  kSync, (cudaStream_t)stream);
}

int idx_attn_paged_fp4_async(const idx_tensor_t* q, const idx_tensor_t* k_codes, const idx_tensor_t* k_scale,
                             const idx_tensor_t* v_codes, const idx_tensor_t* v_scale, const idx_tensor_t* page_table,
                             const idx_tensor_t* row_req, const idx_tensor_t* row_start, const idx_tensor_t* row_end,
                             float scale, const idx_tensor_t* out, const idx_tensor_t* out_lse, void* workspace,
                             uint64_t workspace_bytes, uint32_t* status, idx_stream_t stream) {
  return run_attn({q, k_codes, v_codes, page_table, row_req, row_start, row_end, nullptr, scale, out, out_lse, nullptr,
                   nullptr, k_scale, v_scale, true},
                  {true, workspace, workspace_bytes, status}, (cudaStream_t)stream);
}

int idx_attn_paged_fp4_scratch_bytes(int32_t rows, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t num_req,
                                     int32_t max_pages, int32_t device, uint64_t* bytes) {
  return attn_bytes(rows, q_heads, kv_heads, head_dim, num_req, max_pages, false, false, true, device, bytes);
}

int idx_attn_selected_fp4(const idx_tensor_t* q, const idx_tensor_t* k_codes, const idx_tensor_t* k_scale,
                          const idx_tensor_t* v_codes, const idx_tensor_t* v_scale, const idx_tensor_t* slots, float scale,
                          const idx_tensor_t* out, const idx_tensor_t* out_lse, idx_stream_t stream) {
  if (!slots) return IDX_ERR_INVALID_ARGUMENT;
  return run_attn({q, k_codes, v_codes, nullptr, nullptr, nullptr, nullptr, slots, scale, out, out_lse, nullptr, nullptr,
                   k_scale, v_scale, true},
                  kSync, (cudaStream_t)stream);
}

int idx_attn_selected_fp4_async(const idx_tensor_t* q, const idx_tensor_t* k_codes, const idx_tensor_t* k_scale,
                                const idx_tensor_t* v_codes, const idx_tensor_t* v_scale, const idx_tensor_t* slots,
                                float scale, const idx_tensor_t* out, const idx_tensor_t* out_lse, void* workspace,
                                uint64_t workspace_bytes, uint32_t* status, idx_stream_t stream) {
  if (!slots) return IDX_ERR_INVALID_ARGUMENT;
  return run_attn({q, k_codes, v_codes, nullptr, nullptr, nullptr, nullptr, slots, scale, out, out_lse, nullptr, nullptr,
                   k_scale, v_scale, true},
                  {true, workspace, workspace_bytes, status}, (cudaStream_t)stream);
}

int idx_attn_selected_fp4_scratch_bytes(int32_t rows, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                        int32_t selected, int32_t device, uint64_t* bytes) {
  if (selected < 1) return IDX_ERR_INVALID_ARGUMENT;
  return attn_bytes(rows, q_heads, kv_heads, head_dim, rows, 0, true, false, true, device, bytes);
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
