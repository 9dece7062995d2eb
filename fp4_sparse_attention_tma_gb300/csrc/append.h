// Writing a paged cache, and reading a 4-bit one back: parameters and launchers.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "idx_internal.h"

namespace idxk {

// A row's heads in a call's input, or its place in a paged destination (strides in elements).
struct HeadsIn {
  const void* data;                 // or null
  int64_t row, head;
};
struct PagedOut {
  void* data;                       // 16-bit elements, or bytes of codes
  uint8_t* scale;                   // 4-bit form: the scales, else null
  int64_t page, slot, head;
  int64_t s_page, s_slot, s_head;
};

struct AppendParams {
  HeadsIn q, k, v;
  const void *q_weight, *k_weight;  // [D] in the inputs' type or fp32, or null
  int32_t weight_f32;
  float eps;
  const float* rope;                // [rope_rows][2][rot / 2] cosines, sines; or null
  int32_t rope_rows, rot, first, pairs;
  const int32_t *page_table, *row_req, *row_pos;
  int32_t rows, num_req, max_pages, num_pages, q_heads, kv_heads;
  void* out_q;                      // [R, Hq, D], or codes [R, Hq, D / 2] with scales [R, Hq, D / 32]
  uint8_t* out_q_scale;
  int64_t oq_row, oq_head, oqs_row, oqs_head;
  int32_t q_in_place;
  PagedOut k_dst, v_dst;
  int32_t table_bytes;              // of what finds slots named twice, in shared memory before the rings of the warps
  int32_t table_bits;               // log2 of its words: slots' numbers, or (bitmap) a bit for each slot
  int32_t bitmap;
  uint32_t* status_out;
};

cudaError_t launch_append(const AppendParams& p, bool bf16, int dim, bool fp4, int sm_count, cudaStream_t stream);

struct GatherParams {
  struct From {
    const uint8_t *codes, *scale;   // or null
    int64_t page, slot, head, s_page, s_slot, s_head;
    void* out;
    int64_t row, out_head;
  } t[2];
  const int32_t* slots;
  int32_t n, num_pages, kv_heads;
  int32_t far;                      // codes that span 64 GB or scales that span 4
  int32_t wide;                     // outputs' heads begin at 32-byte boundaries
  uint32_t* status_out;
};

cudaError_t launch_gather(const GatherParams& p, bool bf16, int dim, int sm_count, cudaStream_t stream);

}  // namespace idxk
