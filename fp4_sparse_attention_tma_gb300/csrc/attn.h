// Shared definitions of the attention operators (attention of new tokens over a
// paged key-value cache, and over lists of physical slots): parameters, the
// division of the work, the workspace layout and the launchers.
//
// The work of a call is a list of units.  A unit is one key-value head (or, where
// more query heads share it than one matrix tile holds, one chunk of them) of one
// row group: consecutive rows of one request that share a tile and, in attn.cuh, whose
// windows meet, so that their cached positions are read once.  A unit is cut into subtiles of kSub
// positions; the units' subtiles, one after another, are dealt to the workers (one
// warp each; in attn_tc.cuh one CTA each, with tiles of 128 positions) in equal
// contiguous ranges, each unit counted as kUnitCost subtiles more than it has (its
// beginning and end take a worker's time too; they precede its own).  A unit that lies inside one worker's range
// is finished there; one that is cut leaves partial sums (the maximum, the sum of
// the exponentials and the weighted values, all fp32), which attn_join_kernel
// combines.  A worker's range cuts at most two units, so the workspace is bounded by
// the machine, not by rows or context.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "idx_internal.h"

namespace idxk {

constexpr int kSub = 16;           // cached positions per subtile
// 48 ragged requests x 3 rows x 16 heads, one of them of one position: 61 us with 0, 51 with 1 or 2, 49 with 3;
// 32 requests x 2 rows x 64 heads on one (tiles of 128 positions): 113, 111, 110, 110.
constexpr int kUnitCost = 2;

struct AttnParams {
  const void *q, *k, *v;
  void* out;
  float* lse;                       // [rows, q_heads] or null
  int64_t q_row, q_head;            // strides in elements
  int64_t k_page, k_slot, k_head;
  int64_t v_page, v_slot, v_head;
  int64_t out_row, out_head;
  // a cache in 4 bits: k and v are its codes (strides in bytes), with these scales; else null
  const uint8_t *k_scale, *v_scale;
  int64_t ks_page, ks_slot, ks_head;
  int64_t vs_page, vs_slot, vs_head;
  const int32_t *page_table, *row_req, *row_start, *row_end;
  const int32_t* slots;             // [rows, n_slots]: attention over slot lists, else null
  int32_t n_slots;
  int32_t rows, num_req, max_pages, num_pages;
  int32_t q_heads, kv_heads;
  int32_t group;                    // query heads per key-value head
  int32_t chunks, chunk_heads;      // a key-value head's query heads in chunks of at most a tile
  int32_t group_rows;               // rows per group, at most (1 where there are several chunks)
  int32_t row_cols;                 // tile rows between the rows of a group (chunk_heads of them in use)
  int32_t tensor_core;              // 1: the kernel of attn_tc.cuh
  int32_t far;                      // 1: a cache spans 64 GB or more (attn_fp4.cuh: 4 GB)
  int32_t workers;                  // warps of the grid
  int32_t team;                     // (attn_fp4.cuh) warps that walk over the same range, a key-value head each; else 1
  int32_t ranges;                   // workers / team
  int32_t kv_units;                 // kv_heads / team
  float scale_log2;                 // softmax scale x log2(e)
  // workspace
  uint32_t* cta_status;             // [CTAs] first error that the CTA saw
  int32_t n_cta;
  int32_t* active;                  // workers that have a range (the first so many)
  int32_t* open_parts;              // [active] parts of the unit that the range's end cuts first, or 0
  int4* open_info;                  // [workers] {first row of its group, rows, unit index in the group, 0}
  float2* part_ml;                  // [workers][2][tile] maximum (of the products, not scaled) and sum (shifted)
  float* part_o;                    // [workers][2][tile][dim]
  int32_t tile;                     // tile rows of a unit: 16 or 32; tensor_core: 64 or 128
  int32_t dim;
  // accumulated weights
  float* logits;                    // [rows * q_heads][max_pages * 64] or null
  float2* row_stat;                 // [rows * q_heads] maximum (not scaled) and 1 / sum, or null
  const float* weight_in;           // [num_req][max_pages * 64] or null
  float* weight_out;
  uint32_t* status_out;
};

// Byte offsets of a call's workspace.
struct AttnLayout {
  size_t cta_status, active, open_parts, open_info, part_ml, part_o, row_stat, logits, total;
};

inline AttnLayout attn_layout(int64_t workers, int64_t n_cta, int64_t tile, int64_t dim, int64_t stat_rows,
                              int64_t logit_width) {
  AttnLayout L{};
  size_t off = 0;
  L.cta_status = off; off = align_up(off + (size_t)n_cta * 4, 256);
  L.active = off;     off = align_up(off + 4, 256);
  L.open_parts = off; off = align_up(off + (size_t)workers * 4, 256);
  L.open_info = off;  off = align_up(off + (size_t)workers * 16, 256);
  L.part_ml = off;    off = align_up(off + (size_t)workers * 2 * tile * 8, 256);
  L.part_o = off;     off = align_up(off + (size_t)workers * 2 * tile * dim * 4, 256);
  L.row_stat = off;   off = align_up(off + (size_t)stat_rows * 8, 256);
  L.logits = off;     off = align_up(off + (size_t)stat_rows * (size_t)logit_width * 4, 256);
  L.total = off;
  return L;
}

// Warps of a CTA of the kernel of attn.cuh (with its ring stages, what fits the shared
// memory of an SM).
inline int attn_warps(int32_t dim, int32_t tile) { return dim == 256 ? 4 : dim == 128 ? 8 : tile == 32 ? 12 : 16; }

// The same of the kernel of attn_fp4.cuh.  Measured (us between events), head dimension 128, tiles of 16: 12 and 8 warps, 32
// requests x 2 rows x 64 heads on 8 314, 328; over slots, whose addresses take more registers than 12 warps leave, 64 rows
// x 1024 x 32 heads on 8 52, 48, 512 rows 239, 220.  64: 12 and 16 warps 195, 205; over slots 512 rows 138, 134; 64 rows
// 35, 37.  256: 6 and 4 warps 947, 985; over slots 679, 672.
inline int attn_fp4_warps(int32_t dim, int32_t tile, bool slots) {
  return dim == 256 ? 6 : tile == 32 || (slots && dim == 128) ? 8 : 12;
}

// Warps of a team there: key-value heads whose scales (4 bytes a position at head dimension 128) may share a sector of
// memory are read at the same time, by warps of one CTA.  32 requests x 2 rows x 64 heads on 8, slot by slot: each
// head by itself reads twice the cache's bytes.
inline int attn_fp4_team(int64_t kv_heads, int warps) {
  for (int t : {4, 3, 2})
    if (kv_heads % t == 0 && warps % t == 0) return t;
  return 1;
}

#ifdef __CUDACC__
// What exponents are counted from, where a row's maximum is `top`: the maximum, or 0 where it is
// infinite.  Below -infinity every weight is 0.  Above it a score of +infinity weighs +infinity, so
// that the sum is infinite (NaN only with a score of NaN), log sum exp is +infinity and the outputs,
// infinity over infinity, are NaN.
__device__ __forceinline__ float reference(float top) { return fabsf(top) == INFINITY ? 0.f : top; }

// The exponent of a product of a row, counted from the row's reference `ref` (finite; c the scale in
// units of log2).  The difference is formed before it is scaled: it is 0 where the two are equal, and
// not above 0 where the product is not above the reference.  (Formed after it, in one fused
// operation, it would keep the rounding of the scaled reference, which beyond 2^31 can be more than
// fp32's exponents hold: the largest weight would be infinite or 0.)
__device__ __forceinline__ float exponent(float product, float ref, float c) {
  return __fmul_rn(__fsub_rn(product, ref), c);
}

// Weights are rounded to the inputs' type for the product with the values.  bf16 has fp32's range; fp16
// loses bits below 2^-14 and ends at 2^-25, where a long tail under one heavy position would be lost
// while its sum is not.  So fp16 weights, their sums and the weighted values are 2^kShift times what they
// stand for: bits are lost below 2^-24 of a row's largest weight, nothing above 2^-35 vanishes, and n
// positions together are off by n 2^-35 max |v| at the most.
template <bool BF16>
constexpr float kShift = BF16 ? 0.f : 10.f;
template <bool BF16>
constexpr float kShiftUp = BF16 ? 1.f : 1024.f;   // 2^kShift

// The row's log sum exp from its maximum and its (shifted) sum.
template <bool BF16>
__device__ __forceinline__ float log_sum_exp(float top, float sum, float c) {
  return (__fmul_rn(top, c) + log2f(sum * (1.f / kShiftUp<BF16>))) * 0.6931471805599453f;
}
#endif

// The attention kernel; bf16: the inputs' type (else fp16).
cudaError_t launch_attn(const AttnParams& p, bool bf16, int sm_count, cudaStream_t stream);
// Combines the units that were cut, publishes the status, fails closed.
cudaError_t launch_attn_join(const AttnParams& p, bool bf16, int sm_count, cudaStream_t stream);
// weight_out = weight_in + the weights that every position received.
cudaError_t launch_attn_weights(const AttnParams& p, cudaStream_t stream);

// ------------------------------------------------------------- eviction ----

struct EvictParams {
  const void *k, *v;
  void *k_dst, *v_dst;
  // strides in bytes
  int64_t k_page, k_slot, k_head, v_page, v_slot, v_head;
  int64_t kd_page, kd_slot, kd_head, vd_page, vd_slot, vd_head;
  const int32_t *page_table, *seq_len, *dst_table;
  const float* weight;
  int32_t *keep, *new_len, *new_table;
  float* new_weight;
  int32_t num_req, max_pages, num_pages, dst_pages, dst_width;
  int32_t budget, keep_first, keep_last;
  int32_t kv_heads, head_bytes;
  int32_t same_pool;                // the destination pages are pages of the source tensors
  int32_t slice_cap;                // keys of a CTA's slice that fit its shared memory
  int32_t mark_shared;              // the bitmap of the fresh pages fits shared memory
  int32_t copy_rows;                // rows of a page that a CTA of the copy moves
  uint32_t* part_status;            // workspace: [num_req + 1] first error of each cluster
  uint32_t* dst_mark;               // workspace: [CTAs of a cluster] bitmaps, where shared memory is too small
  uint32_t* status_out;
};

// CTAs of a cluster, and whether the fresh pages' bitmap lies in shared memory.
int evict_cluster(int64_t num_req, int64_t max_pages, int sm_count);
bool evict_mark_shared(int64_t dst_pages);
cudaError_t launch_evict(EvictParams p, int sm_count, cudaStream_t stream);

}  // namespace idxk
