// C ABI of the operators that write a paged cache and read a 4-bit one back (declared in
// include/idxtopk.h): argument checks and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>

#include "append.h"
#include "idxtopk.h"
#include "op_host.h"

using namespace idxk;

namespace {

struct AppendCall {
  const idx_tensor_t *q, *k, *v, *page_table, *row_req, *row_pos, *q_weight, *k_weight;
  float eps;
  const idx_tensor_t* rope;
  int32_t rope_first, rope_pairs;
  const idx_tensor_t *out_q, *out_q_scale, *k_cache, *k_scale, *v_cache, *v_scale;
  bool fp4;
};

bool same_shape(const idx_tensor_t* a, const idx_tensor_t* b) {
  if (a->ndim != b->ndim) return false;
  for (int i = 0; i < a->ndim; ++i)
    if (a->shape[i] != b->shape[i]) return false;
  return true;
}

HeadsIn heads_in(const idx_tensor_t* t) {
  HeadsIn h{};
  if (t) h.data = t->data, h.row = step(t, 0), h.head = step(t, 1);
  return h;
}

// A paged destination of Hk heads of dimension D: [NP, 64, Hk, D] 16-bit, or codes [.., D / 2] and
// scales [.., D / 32].
int check_pages(const idx_tensor_t* t, const idx_tensor_t* scale, bool fp4, int dtype, int64_t Hk, int64_t D) {
  int st;
  if (!fp4) {
    if ((st = check_strided(t, dtype, 4))) return st;
  } else {
    if ((st = check_strided(t, IDX_U8, 4, 16)) || (st = check_strided(scale, IDX_U8, 4, D / 32))) return st;
    for (int i = 0; i < 3; ++i)
      if (t->shape[i] != scale->shape[i]) return IDX_ERR_INVALID_ARGUMENT;
    if (scale->shape[3] != D / 32 || !no_overlap(scale)) return IDX_ERR_INVALID_ARGUMENT;
  }
  if (t->shape[2] != Hk || t->shape[3] != (fp4 ? D / 2 : D) || !no_overlap(t)) return IDX_ERR_INVALID_ARGUMENT;
  if (t->shape[1] != kPage) return IDX_ERR_UNSUPPORTED;
  if (t->shape[0] * (int64_t)kPage > INT32_MAX) return IDX_ERR_OVERFLOW;
  return IDX_OK;
}

PagedOut paged_out(const idx_tensor_t* t, const idx_tensor_t* scale) {
  PagedOut o{};
  if (!t) return o;
  o.data = t->data, o.page = step(t, 0), o.slot = step(t, 1), o.head = step(t, 2);
  if (scale)
    o.scale = (uint8_t*)scale->data, o.s_page = step(scale, 0), o.s_slot = step(scale, 1), o.s_head = step(scale, 2);
  return o;
}

int run_append(const AppendCall& c, const Space& space, cudaStream_t stream) {
  int st;
  if ((st = check_space(space))) return st;
  if (!c.k || (c.k->dtype != IDX_BF16 && c.k->dtype != IDX_F16)) return IDX_ERR_INVALID_ARGUMENT;
  const int dtype = c.k->dtype;
  if ((st = check_strided(c.k, dtype, 3))) return st;
  const int64_t R = c.k->shape[0], Hk = c.k->shape[1], D = c.k->shape[2];
  if (D != 64 && D != 128 && D != 256) return IDX_ERR_UNSUPPORTED;
  if (Hk < 1) return IDX_ERR_INVALID_ARGUMENT;
  if ((c.v == nullptr) != (c.v_cache == nullptr) || (c.q == nullptr) != (c.out_q == nullptr)) return IDX_ERR_INVALID_ARGUMENT;
  if (c.v && ((st = check_strided(c.v, dtype, 3)))) return st;
  if (c.v && !same_shape(c.k, c.v)) return IDX_ERR_INVALID_ARGUMENT;
  if (c.fp4 && c.v && !c.v_scale) return IDX_ERR_INVALID_ARGUMENT;
  if (!c.v && c.v_scale) return IDX_ERR_INVALID_ARGUMENT;
  if ((st = check_pages(c.k_cache, c.k_scale, c.fp4, dtype, Hk, D))) return st;
  if (c.v && ((st = check_pages(c.v_cache, c.v_scale, c.fp4, dtype, Hk, D)))) return st;
  if (c.v && c.v_cache->shape[0] != c.k_cache->shape[0]) return IDX_ERR_INVALID_ARGUMENT;
  const int64_t NP = c.k_cache->shape[0];
  int64_t Hq = 0;
  const bool q4 = c.out_q && c.out_q->dtype == IDX_U8;
  if (c.q) {
    if ((st = check_strided(c.q, dtype, 3))) return st;
    Hq = c.q->shape[1];
    if (c.q->shape[0] != R || c.q->shape[2] != D || Hq < 1) return IDX_ERR_INVALID_ARGUMENT;
    if (q4) {
      if (!c.fp4 || !c.out_q_scale) return IDX_ERR_INVALID_ARGUMENT;
      if ((st = check_strided(c.out_q, IDX_U8, 3, 16)) || (st = check_strided(c.out_q_scale, IDX_U8, 3, D / 32))) return st;
      if (c.out_q_scale->shape[0] != R || c.out_q_scale->shape[1] != Hq || c.out_q_scale->shape[2] != D / 32 ||
          !no_overlap(c.out_q_scale))
        return IDX_ERR_INVALID_ARGUMENT;
    } else if ((st = check_strided(c.out_q, dtype, 3))) {
      return st;
    }
    if (c.out_q->shape[0] != R || c.out_q->shape[1] != Hq || c.out_q->shape[2] != (q4 ? D / 2 : D) || !no_overlap(c.out_q))
      return IDX_ERR_INVALID_ARGUMENT;
  }
  if (c.out_q_scale && !q4) return IDX_ERR_INVALID_ARGUMENT;
  if ((st = check_tensor(c.page_table, IDX_I32, 2)) || (st = check_tensor(c.row_req, IDX_I32, 1)) ||
      (st = check_tensor(c.row_pos, IDX_I32, 1)))
    return st;
  const int64_t NR = c.page_table->shape[0], MP = c.page_table->shape[1];
  if (c.row_req->shape[0] != R || c.row_pos->shape[0] != R) return IDX_ERR_INVALID_ARGUMENT;
  if (R > 0 && (NP < 1 || NR < 1 || MP < 1)) return IDX_ERR_INVALID_ARGUMENT;
  if (NR > INT32_MAX || MP * (int64_t)kPage > INT32_MAX || R > INT32_MAX || Hq > 65536 || Hk > 65536 ||
      R * (Hq + 2 * Hk) > INT32_MAX)
    return IDX_ERR_OVERFLOW;
  if (c.q_weight && !c.q) return IDX_ERR_INVALID_ARGUMENT;
  int weight_type = 0;
  for (const idx_tensor_t* w : {c.q_weight, c.k_weight}) {
    if (!w) continue;
    if (w->dtype != IDX_F32 && w->dtype != dtype) return IDX_ERR_INVALID_ARGUMENT;
    if (weight_type && weight_type != w->dtype) return IDX_ERR_INVALID_ARGUMENT;
    weight_type = w->dtype;
    if ((st = check_strided(w, weight_type, 1)) || w->shape[0] != D) return st ? st : IDX_ERR_INVALID_ARGUMENT;
  }
  if (!(c.eps >= 0.f) || !std::isfinite(c.eps)) return IDX_ERR_INVALID_ARGUMENT;
  int64_t rot = 0, P = 0;
  if (c.rope) {
    if ((st = check_tensor(c.rope, IDX_F32, 3))) return st;
    P = c.rope->shape[0], rot = 2 * c.rope->shape[2];
    if (c.rope->shape[1] != 2 || P < 1 || P > INT32_MAX || rot < 16 || rot > D) return IDX_ERR_INVALID_ARGUMENT;
    if (rot % 16 != 0 || c.rope_first % 8 != 0) return IDX_ERR_UNSUPPORTED;
    if (c.rope_first < 0 || c.rope_first + rot > D || (c.rope_pairs != 0 && c.rope_pairs != 1)) return IDX_ERR_INVALID_ARGUMENT;
  }
  // the places to write share no element; in place: the queries
  const bool in_place = c.q && !q4 && c.q->data == c.out_q->data && same_strides(c.q, c.out_q);
  const idx_tensor_t* places[] = {c.k_cache, c.v_cache, c.k_scale, c.v_scale};
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < i; ++j)
      if (places[i] && places[j] && numel_of(places[i]) > 0 && !pages_apart(places[i], places[j])) return IDX_ERR_INVALID_ARGUMENT;
  const idx_tensor_t* q_outs[] = {c.out_q, c.out_q_scale};
  const idx_tensor_t* q_apart[] = {in_place ? nullptr : c.q, c.page_table, c.row_req, c.row_pos, c.q_weight, c.k_weight,
                                   c.rope, c.k_cache, c.v_cache, c.k_scale, c.v_scale};
  if (!all_apart(q_outs, q_apart)) return IDX_ERR_INVALID_ARGUMENT;
  // (queries in place in a projection that they share with keys and values)
  for (const idx_tensor_t* o : q_outs)
    for (const idx_tensor_t* x : {c.k, c.v})
      if (!apart(o, x) && (q4 || !interleaved(o, x))) return IDX_ERR_INVALID_ARGUMENT;
  const idx_tensor_t* ins[] = {c.q, c.k, c.v, c.page_table, c.row_req, c.row_pos, c.q_weight, c.k_weight, c.rope};
  for (const idx_tensor_t* t : places)
    for (const idx_tensor_t* x : ins)
      if (!apart(t, x)) return IDX_ERR_INVALID_ARGUMENT;
  const idx_tensor_t* all[] = {c.q,        c.k,    c.v,     c.page_table,  c.row_req, c.row_pos, c.q_weight,
                               c.k_weight, c.rope, c.out_q, c.out_q_scale, c.k_cache, c.k_scale, c.v_cache, c.v_scale};
  Machine m;
  if ((st = find_machine(all, 15, space.status, space.workspace, stream, &m))) return st;
  if (m.capturing && !space.async) return IDX_ERR_UNSUPPORTED;
  DeviceGuard guard(m.dev);
  if (!guard.ok()) return IDX_ERR_CUDA;
  if ((st = check_arch(&m))) return st;
  AppendParams p{};
  p.q = heads_in(c.q), p.k = heads_in(c.k), p.v = heads_in(c.v);
  p.q_weight = c.q_weight ? c.q_weight->data : nullptr;
  p.k_weight = c.k_weight ? c.k_weight->data : nullptr;
  p.weight_f32 = weight_type == IDX_F32;
  p.eps = c.eps;
  if (c.rope) {
    p.rope = (const float*)c.rope->data;
    p.rope_rows = (int32_t)P, p.rot = (int32_t)rot, p.first = c.rope_first, p.pairs = c.rope_pairs;
  }
  p.page_table = (const int32_t*)c.page_table->data;
  p.row_req = (const int32_t*)c.row_req->data;
  p.row_pos = (const int32_t*)c.row_pos->data;
  p.rows = (int32_t)R, p.num_req = (int32_t)NR, p.max_pages = (int32_t)MP, p.num_pages = (int32_t)NP;
  p.q_heads = (int32_t)Hq, p.kv_heads = (int32_t)Hk;
  if (c.out_q) {
    p.out_q = c.out_q->data, p.oq_row = step(c.out_q, 0), p.oq_head = step(c.out_q, 1);
    if (q4) {
      p.out_q_scale = (uint8_t*)c.out_q_scale->data;
      p.oqs_row = step(c.out_q_scale, 0), p.oqs_head = step(c.out_q_scale, 1);
    }
  }
  p.q_in_place = in_place;
  p.k_dst = paged_out(c.k_cache, c.k_scale), p.v_dst = paged_out(c.v_cache, c.v_scale);
  return with_space(space, 0, m, stream, [&](char*, uint32_t* status) -> cudaError_t {
    p.status_out = status;
    if (R == 0) return cudaMemsetAsync(status, 0, sizeof(uint32_t), stream);
    return launch_append(p, dtype == IDX_BF16, (int)D, c.fp4, m.sm, stream);
  });
}

struct GatherCall {
  const idx_tensor_t *k, *k_scale, *v, *v_scale, *slots, *out_k, *out_v;
};

int run_gather(const GatherCall& c, const Space& space, cudaStream_t stream) {
  int st;
  if ((st = check_space(space))) return st;
  if (!c.k || c.k->dtype != IDX_U8 || c.k->ndim != 4 || !c.out_k) return IDX_ERR_INVALID_ARGUMENT;
  if (c.out_k->dtype != IDX_BF16 && c.out_k->dtype != IDX_F16) return IDX_ERR_INVALID_ARGUMENT;
  const int dtype = c.out_k->dtype;
  const int64_t NP = c.k->shape[0], Hk = c.k->shape[2], D = 2 * c.k->shape[3];
  if (D != 64 && D != 128 && D != 256) return IDX_ERR_UNSUPPORTED;
  if (Hk < 1 || Hk > 65536) return IDX_ERR_INVALID_ARGUMENT;
  if ((c.v == nullptr) != (c.out_v == nullptr) || (c.v == nullptr) != (c.v_scale == nullptr)) return IDX_ERR_INVALID_ARGUMENT;
  if ((st = check_tensor(c.slots, IDX_I32, 1))) return st;
  const int64_t N = c.slots->shape[0];
  for (int i = 0; i < 2; ++i) {
    const idx_tensor_t *t = i ? c.v : c.k, *s = i ? c.v_scale : c.k_scale, *o = i ? c.out_v : c.out_k;
    if (!t) continue;
    if ((st = check_pages(t, s, true, dtype, Hk, D)) || (st = check_strided(o, dtype, 3))) return st;
    if (t->shape[0] != NP || o->shape[0] != N || o->shape[1] != Hk || o->shape[2] != D || !no_overlap(o))
      return IDX_ERR_INVALID_ARGUMENT;
  }
  if (N > 0 && NP < 1) return IDX_ERR_INVALID_ARGUMENT;
  if (N > INT32_MAX / 2 || N * Hk > INT32_MAX / 2) return IDX_ERR_OVERFLOW;
  const idx_tensor_t* outs[] = {c.out_k, c.out_v};
  const idx_tensor_t* ins[] = {c.k, c.k_scale, c.v, c.v_scale, c.slots};
  if (!all_apart(outs, ins)) return IDX_ERR_INVALID_ARGUMENT;
  const idx_tensor_t* all[] = {c.k, c.k_scale, c.v, c.v_scale, c.slots, c.out_k, c.out_v};
  Machine m;
  if ((st = find_machine(all, 7, space.status, space.workspace, stream, &m))) return st;
  if (m.capturing && !space.async) return IDX_ERR_UNSUPPORTED;
  DeviceGuard guard(m.dev);
  if (!guard.ok()) return IDX_ERR_CUDA;
  if ((st = check_arch(&m))) return st;
  GatherParams p{};
  bool narrow = false;
  for (int i = 0; i < 2; ++i) {
    const idx_tensor_t *t = i ? c.v : c.k, *s = i ? c.v_scale : c.k_scale, *o = i ? c.out_v : c.out_k;
    if (!t) continue;
    GatherParams::From& f = p.t[i];
    f.codes = (const uint8_t*)t->data, f.page = step(t, 0), f.slot = step(t, 1), f.head = step(t, 2);
    f.scale = (const uint8_t*)s->data, f.s_page = step(s, 0), f.s_slot = step(s, 1), f.s_head = step(s, 2);
    f.out = o->data, f.row = step(o, 0), f.out_head = step(o, 1);
    p.far |= span_of(t) >= kFar || span_of(s) > UINT32_MAX;
    narrow |= ((uintptr_t)o->data | (uintptr_t)(f.row * 2) | (uintptr_t)(f.out_head * 2)) % 32 != 0;
  }
  p.wide = !narrow;
  p.slots = (const int32_t*)c.slots->data;
  p.n = (int32_t)N, p.num_pages = (int32_t)NP, p.kv_heads = (int32_t)Hk;
  return with_space(space, 0, m, stream, [&](char*, uint32_t* status) -> cudaError_t {
    p.status_out = status;
    if (N == 0) return cudaMemsetAsync(status, 0, sizeof(uint32_t), stream);
    return launch_gather(p, dtype == IDX_BF16, (int)D, m.sm, stream);
  });
}

// Nothing of the caller's but the status word.
Space with_status(uint32_t* status) { return {true, nullptr, 0, status}; }

}  // namespace

extern "C" {

int idx_cache_append(const idx_tensor_t* q, const idx_tensor_t* k, const idx_tensor_t* v, const idx_tensor_t* page_table,
                     const idx_tensor_t* row_req, const idx_tensor_t* row_pos, const idx_tensor_t* q_weight,
                     const idx_tensor_t* k_weight, float eps, const idx_tensor_t* rope, int32_t rope_first,
                     int32_t rope_pairs, const idx_tensor_t* out_q, const idx_tensor_t* k_cache,
                     const idx_tensor_t* v_cache, idx_stream_t stream) {
  return run_append({q, k, v, page_table, row_req, row_pos, q_weight, k_weight, eps, rope, rope_first, rope_pairs, out_q,
                     nullptr, k_cache, nullptr, v_cache, nullptr, false},
                    kSync, (cudaStream_t)stream);
}

int idx_cache_append_async(const idx_tensor_t* q, const idx_tensor_t* k, const idx_tensor_t* v,
                           const idx_tensor_t* page_table, const idx_tensor_t* row_req, const idx_tensor_t* row_pos,
                           const idx_tensor_t* q_weight, const idx_tensor_t* k_weight, float eps, const idx_tensor_t* rope,
                           int32_t rope_first, int32_t rope_pairs, const idx_tensor_t* out_q, const idx_tensor_t* k_cache,
                           const idx_tensor_t* v_cache, uint32_t* status, idx_stream_t stream) {
  return run_append({q, k, v, page_table, row_req, row_pos, q_weight, k_weight, eps, rope, rope_first, rope_pairs, out_q,
                     nullptr, k_cache, nullptr, v_cache, nullptr, false},
                    with_status(status), (cudaStream_t)stream);
}

int idx_cache_append_fp4(const idx_tensor_t* q, const idx_tensor_t* k, const idx_tensor_t* v,
                         const idx_tensor_t* page_table, const idx_tensor_t* row_req, const idx_tensor_t* row_pos,
                         const idx_tensor_t* q_weight, const idx_tensor_t* k_weight, float eps, const idx_tensor_t* rope,
                         int32_t rope_first, int32_t rope_pairs, const idx_tensor_t* out_q, const idx_tensor_t* out_q_scale,
                         const idx_tensor_t* k_codes, const idx_tensor_t* k_scale, const idx_tensor_t* v_codes,
                         const idx_tensor_t* v_scale, idx_stream_t stream) {
  return run_append({q, k, v, page_table, row_req, row_pos, q_weight, k_weight, eps, rope, rope_first, rope_pairs, out_q,
                     out_q_scale, k_codes, k_scale, v_codes, v_scale, true},
                    kSync, (cudaStream_t)stream);
}

int idx_cache_append_fp4_async(const idx_tensor_t* q, const idx_tensor_t* k, const idx_tensor_t* v,
                               const idx_tensor_t* page_table, const idx_tensor_t* row_req, const idx_tensor_t* row_pos,
                               const idx_tensor_t* q_weight, const idx_tensor_t* k_weight, float eps,
                               const idx_tensor_t* rope, int32_t rope_first, int32_t rope_pairs, const idx_tensor_t* out_q,
                               const idx_tensor_t* out_q_scale, const idx_tensor_t* k_codes, const idx_tensor_t* k_scale,
                               const idx_tensor_t* v_codes, const idx_tensor_t* v_scale, uint32_t* status,
                               idx_stream_t stream) {
  return run_append({q, k, v, page_table, row_req, row_pos, q_weight, k_weight, eps, rope, rope_first, rope_pairs, out_q,
                     out_q_scale, k_codes, k_scale, v_codes, v_scale, true},
                    with_status(status), (cudaStream_t)stream);
}

int idx_cache_gather_fp4(const idx_tensor_t* k_codes, const idx_tensor_t* k_scale, const idx_tensor_t* v_codes,
                         const idx_tensor_t* v_scale, const idx_tensor_t* slots, const idx_tensor_t* out_k,
                         const idx_tensor_t* out_v, idx_stream_t stream) {
  return run_gather({k_codes, k_scale, v_codes, v_scale, slots, out_k, out_v}, kSync, (cudaStream_t)stream);
}

int idx_cache_gather_fp4_async(const idx_tensor_t* k_codes, const idx_tensor_t* k_scale, const idx_tensor_t* v_codes,
                               const idx_tensor_t* v_scale, const idx_tensor_t* slots, const idx_tensor_t* out_k,
                               const idx_tensor_t* out_v, uint32_t* status, idx_stream_t stream) {
  return run_gather({k_codes, k_scale, v_codes, v_scale, slots, out_k, out_v}, with_status(status), (cudaStream_t)stream);
}

}  // extern "C"
