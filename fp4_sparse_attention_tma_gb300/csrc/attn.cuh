// The attention kernel: one pass over the cached positions of every row with the
// running maximum and sum of the softmax,
//
//   s_hj = c * q_h . k_j,  m_h = max_j s_hj,  l_h = sum_j 2^(s_hj - m_h),
//   out_h = (1 / l_h) sum_j 2^(s_hj - m_h) v_j,   c = scale * log2(e),
//
// products in 16 bits with fp32 accumulation, everything else in fp32; the weights
// 2^(s - m) are rounded to the inputs' type for the second product (their sum is
// not), which the matrix instruction asks for: an error of u sum p |v| at most beside the
// output's own u |out| (u half a unit in the last place; fp16's range: kShift in attn.h).
//
// What bounds it is the cache's traffic: a key and a value are read for 4 flops per
// query head of their group and element, far below the tensor cores' ratio to HBM for
// the 16 or 32 (query head, row) pairs of a tile.  Hence warps that never wait for one
// another: every warp owns a ring of asynchronous 16-byte copies (kSub positions of
// keys and values a stage) and a range of subtiles (attn.h), and one warp-level matrix
// instruction chain consumes a stage while the others are in flight.  The copies take
// any page, slot and head stride and any list of slots, and fill with zero what no row
// sees, so that what lies there cannot reach a sum.  As many warps as the shared memory
// has rings for (3 stages of 16 positions).  48 requests x 3 rows x 16 heads of dimension
// 64 over up to 1002 positions: 160 MB in 50 us, of which 5 us pass before the first copy
// and 8 in the join; 32 requests x 3 rows x 64 heads on 8: 4.45 GB in 1008 us (groups of four rows begin at
// every fourth row of the call, so the 32 requests are walked over 48 times).
#pragma once

#include "attn_common.cuh"

namespace idxk {
namespace attn {

template <bool BF16, int D, int TILE, int WARPS, int STAGES, bool SLOTS>
__global__ void __launch_bounds__(WARPS * 32, 1) attn_kernel(const __grid_constant__ AttnParams p) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr int MT = TILE / 16;          // matrix tiles of 16 query heads x rows
  constexpr int KS = D / 16;             // steps of the first product
  constexpr int NT = D / 8;              // tiles of 8 of the output's columns
  constexpr int CH = D / 8;              // 16-byte pieces of a cached head
  constexpr uint32_t kHalf = kSub * D * 2;  // bytes of a stage's keys (and of its values)

  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ uint32_t err;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t worker = warp * gridDim.x + blockIdx.x;
  allow_launch_after();
  if (threadIdx.x == 0) err = kOk;
  __syncthreads();

  Split sp;
  Cursor<SLOTS> at;
  Rows rows{};
  int64_t end;   // of the worker's range, counted from the unit's first subtile
  const bool work = find_range<Cursor<SLOTS>, SLOTS, WARPS>(p, rows, sp, at, end, worker, ring, &err);
  if (worker < sp.active && lane == 0) p.open_parts[worker] = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.active = sp.active;
  uint32_t warp_err = kOk;
  if (work) {
    const uint32_t my_ring = smem_addr(ring) + (uint32_t)warp * (STAGES * 2 * kHalf);

    // ---- fetching side: runs STAGES - 1 subtiles ahead, over the ends of segments ----
    constexpr int ROWS = 32 / CH > 0 ? 32 / CH : 1;   // positions that one copy of the warp covers
    constexpr int COPIES = kSub / ROWS;
    const int piece = lane % CH, row_in = ROWS > 1 ? lane / CH : 0;
    uint32_t to[8 / ROWS > 0 ? 8 / ROWS : 1];         // where the lane's pieces go: the swizzle repeats every 8 rows
    constexpr int TO = sizeof(to) / sizeof(to[0]);
#pragma unroll
    for (int i = 0; i < TO; ++i) {
      const int r = i * ROWS + row_in;
      to[i] = (uint32_t)(r * (D * 2) + ((piece ^ (r & 7)) << 4));
    }
    Cursor<SLOTS> f = at;
    int64_t f_end = end;                              // as `end`; 0 when everything has been fetched
    const T *f_k, *f_v;                               // the head's keys and values, at this lane's piece
    const int32_t* f_list;                            // the request's pages, or the row's slots
    int32_t entry;                                    // page of the next subtile, or slot of its position lane % 16
    uint64_t shown = 0;                               // (slots) which positions of the fetched subtiles are one, 16 bits each
    auto look_up = [&]() {
      if constexpr (SLOTS) {
        const int32_t j = f.s * kSub + (lane & 15);
        entry = j < p.n_slots ? f_list[j] : -1;
      } else {
        entry = f_list[(f.base + f.s) / (kPage / kSub)];
      }
    };
    auto begin_fetch = [&]() {
      f_k = (const T*)p.k + f.kv * p.k_head + piece * 8;
      f_v = (const T*)p.v + f.kv * p.v_head + piece * 8;
      f_list = SLOTS ? p.slots + (int64_t)f.row0 * p.n_slots : p.page_table + (int64_t)f.req * p.max_pages;
      look_up();
    };
    begin_fetch();
    auto fetch = [&](int stage) {
      if (f_end > 0) {
        const uint32_t dk = my_ring + (uint32_t)stage * (2 * kHalf), dv = dk + kHalf;
        auto place = [&](int i) { return to[i % TO] + (uint32_t)(i / TO) * (8 * D * 2); };
        if constexpr (SLOTS) {
          const bool on = entry >= 0 && entry < p.num_pages * kPage;
          if (!on && entry != -1) warp_err = kErrInvalidPage;
          const uint32_t mask = __ballot_sync(~0u, on) & 0xFFFFu;
          shown |= (uint64_t)mask << ((STAGES - 1) * 16);
          const int32_t page = on ? entry / kPage : 0, off = on ? entry % kPage : 0;
          if (!p.far) {
            // offsets in units of 16 bytes
            const uint32_t ok = on ? (uint32_t)page * (uint32_t)(p.k_page / 8) + (uint32_t)off * (uint32_t)(p.k_slot / 8) : 0u;
            const uint32_t ov = on ? (uint32_t)page * (uint32_t)(p.v_page / 8) + (uint32_t)off * (uint32_t)(p.v_slot / 8) : 0u;
#pragma unroll
            for (int i = 0; i < COPIES; ++i) {
              const int r = i * ROWS + row_in;
              const uint32_t bytes = mask >> r & 1u ? 16u : 0u;
              copy16(dk + place(i), f_k + (uint64_t)__shfl_sync(~0u, ok, r) * 8, bytes);
              copy16(dv + place(i), f_v + (uint64_t)__shfl_sync(~0u, ov, r) * 8, bytes);
            }
          } else {
            const unsigned long long ok = page * p.k_page + off * p.k_slot, ov = page * p.v_page + off * p.v_slot;
#pragma unroll
            for (int i = 0; i < COPIES; ++i) {
              const int r = i * ROWS + row_in;
              const uint32_t bytes = mask >> r & 1u ? 16u : 0u;
              copy16(dk + place(i), f_k + __shfl_sync(~0u, ok, r), bytes);
              copy16(dv + place(i), f_v + __shfl_sync(~0u, ov, r), bytes);
            }
          }
        } else {
          const bool there = entry >= 0 && entry < p.num_pages;
          if (!there) warp_err = kErrInvalidPage;
          const int32_t pos0 = (f.base + f.s) * kSub, off = pos0 % kPage + row_in;
          const int64_t page = there ? entry : 0;
          const T* k = f_k + page * p.k_page + off * p.k_slot;
          const T* v = f_v + page * p.v_page + off * p.v_slot;
          const int64_t ks = ROWS * p.k_slot, vs = ROWS * p.v_slot;
          if (there && pos0 >= f.lo && pos0 + kSub <= f.hi) {
#pragma unroll
            for (int i = 0; i < COPIES; ++i, k += ks, v += vs) {
              copy16(dk + place(i), k, 16u);
              copy16(dv + place(i), v, 16u);
            }
          } else {
#pragma unroll
            for (int i = 0; i < COPIES; ++i, k += ks, v += vs) {
              const int32_t pos = pos0 + i * ROWS + row_in;
              const bool on = there && pos >= f.lo && pos < f.hi;
              copy16(dk + place(i), on ? k : (const T*)p.k, on ? 16u : 0u);
              copy16(dv + place(i), on ? v : (const T*)p.v, on ? 16u : 0u);
            }
          }
        }
        if (++f.s < min((int64_t)f.nsub, f_end)) {
          look_up();
        } else {
          f_end = max((int64_t)0, f_end - f.nsub - kUnitCost);
          if (f_end > 0) {
            f.next_unit(p, rows);
            begin_fetch();
          }
        }
      }
      copy_commit();
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) {
      fetch(i);
      shown >>= 16;
    }

    // ---- computing side ----
    int stage = 0;
    const float c = p.scale_log2;
    while (end > 0) {
      const int32_t v0 = at.s, v1 = (int32_t)min((int64_t)at.nsub, end);
      const bool cut_front = v0 > 0;      // the segment starts inside its unit
      const int32_t h0 = at.kv * p.group + at.chunk * p.chunk_heads;
      const int32_t heads = min(p.chunk_heads, p.group - at.chunk * p.chunk_heads);
      uint32_t qf[MT][KS][4];
      float o[MT][NT][4];
      float mx[MT][2], sum[MT][2];
      int32_t w_lo[MT][2], w_hi[MT][2];   // windows of the thread's tile rows
      uint32_t live = 0;                  // bit 2t + e: the thread's tile row is a row that sees something
      bool seen = false;                  // (slots) some slot of the segment was one
      int32_t full_lo = 0, full_hi = INT32_MAX;   // positions that every row of the group sees
      // tile row m: row m / chunk_heads of the group, head h0 + m % chunk_heads
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int m = t * 16 + e * 8 + lane / 4;
          const int j = m / p.chunk_heads, h = m - j * p.chunk_heads;
          bool on = j < at.nrows && h < heads;
          int32_t a = at.lo, b = at.hi;
          if constexpr (!SLOTS) {
            if (on) {
              a = rows.start[at.row0 + j], b = rows.end[at.row0 + j];
              if (b <= a) on = false, a = at.lo, b = at.hi;
            }
          }
          if (on) live |= 1u << (2 * t + e);
          w_lo[t][e] = a, w_hi[t][e] = b;
          full_lo = max(full_lo, a), full_hi = min(full_hi, b);
          mx[t][e] = kNegInf, sum[t][e] = 0.f;
          const uint32_t* src =
              (const uint32_t*)((const T*)p.q + (int64_t)(at.row0 + j) * p.q_row + (int64_t)(h0 + h) * p.q_head);
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            qf[t][k][e] = on ? src[k * 8 + (lane & 3)] : 0u;
            qf[t][k][2 + e] = on ? src[k * 8 + 4 + (lane & 3)] : 0u;
          }
        }
      full_lo = __reduce_max_sync(~0u, full_lo);
      full_hi = __reduce_min_sync(~0u, full_hi);
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) o[t][n][x] = 0.f;

      for (int32_t sub = v0; sub < v1; ++sub) {
      // the next stage goes where the last one computed was
      copy_wait<STAGES - 2>();
      __syncwarp();
      const uint32_t on = (uint32_t)shown & 0xFFFFu;
      fetch(stage == 0 ? STAGES - 1 : stage - 1);
      shown >>= 16;
      const uint32_t sk = my_ring + (uint32_t)stage * (2 * kHalf), sv = sk + kHalf;
      stage = stage == STAGES - 1 ? 0 : stage + 1;

      // scores of the subtile: two tiles of 8 positions
      float s[MT][2][4];
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) s[t][n][x] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; k += 2)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          uint32_t b[4];
          const int r = n * 8 + (lane & 7);
          ldsm4(sk + (uint32_t)(r * (D * 2) + (((k * 2 + lane / 8) ^ (r & 7)) << 4)), b);
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            mma16816<BF16>(s[t][n], qf[t][k], b[0], b[1]);
            mma16816<BF16>(s[t][n], qf[t][k + 1], b[2], b[3]);
          }
        }

      const int32_t pos0 = (at.base + sub) * kSub;
      bool edge;
      if constexpr (SLOTS) {
        edge = on != 0xFFFFu;
        seen |= on != 0;
        if (edge) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x)
              if (!(on >> (n * 8 + (lane & 3) * 2 + x) & 1)) {
#pragma unroll
                for (int t = 0; t < MT; ++t) s[t][n][x] = s[t][n][2 + x] = kNegInf;
              }
        }
      } else {
        edge = pos0 < full_lo || pos0 + kSub > full_hi;
        if (edge) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int32_t pos = pos0 + n * 8 + (lane & 3) * 2 + x;
#pragma unroll
              for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (pos < w_lo[t][e] || pos >= w_hi[t][e]) s[t][n][2 * e + x] = kNegInf;
            }
        }
        if (p.logits) {
          const int64_t width = (int64_t)p.max_pages * kPage;
#pragma unroll
          for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int m = t * 16 + e * 8 + lane / 4;
              const int j = m / p.chunk_heads, h = m - j * p.chunk_heads;
              if (live >> (2 * t + e) & 1) {
                float* dst = p.logits + ((int64_t)(at.row0 + j) * p.q_heads + h0 + h) * width + pos0 + (lane & 3) * 2;
#pragma unroll
                for (int n = 0; n < 2; ++n) *(float2*)(dst + n * 8) = make_float2(s[t][n][2 * e], s[t][n][2 * e + 1]);
              }
            }
        }
      }

      // running maximum; the sums are scaled where it moved
      float ref[MT][2];
      bool moved = false;
      float alpha[MT][2];
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float m = fmaxf(fmaxf(s[t][0][2 * e], s[t][0][2 * e + 1]), fmaxf(s[t][1][2 * e], s[t][1][2 * e + 1]));
          m = fmaxf(m, __shfl_xor_sync(~0u, m, 1));
          m = fmaxf(m, __shfl_xor_sync(~0u, m, 2));
          m = fmaxf(m, mx[t][e]);
          ref[t][e] = reference(m);
          alpha[t][e] = m == mx[t][e] ? 1.f : ex2(exponent(mx[t][e], ref[t][e], c));
          moved |= m != mx[t][e];
          mx[t][e] = m;
        }
      if (__any_sync(~0u, moved)) {
#pragma unroll
        for (int t = 0; t < MT; ++t) {
#pragma unroll
          for (int e = 0; e < 2; ++e) sum[t][e] *= alpha[t][e];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            o[t][n][0] *= alpha[t][0];
            o[t][n][1] *= alpha[t][0];
            o[t][n][2] *= alpha[t][1];
            o[t][n][3] *= alpha[t][1];
          }
        }
      }
      uint32_t pf[MT][4];
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float a = ex2(fmaf(__fsub_rn(s[t][n][2 * e], ref[t][e]), c, kShift<BF16>));
            const float b = ex2(fmaf(__fsub_rn(s[t][n][2 * e + 1], ref[t][e]), c, kShift<BF16>));
            sum[t][e] += a + b;
            pf[t][n * 2 + e] = pack2<BF16>(a, b);
          }

      const uint32_t va = sv + (uint32_t)((lane & 15) * (D * 2));
      const uint32_t vx = (uint32_t)(lane & 7);
      if (SLOTS || !edge || at.nrows == 1) {
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
          uint32_t b[4];
          ldsm4t(va + (((uint32_t)(n + lane / 16) ^ vx) << 4), b);
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            mma16816<BF16>(o[t][n], pf[t], b[0], b[1]);
            mma16816<BF16>(o[t][n + 1], pf[t], b[2], b[3]);
          }
        }
      } else {
        // some rows of the group see a position and others do not: row by row, with the values that the
        // row does not see set to zero (0 x infinity or NaN would not be)
        for (int j = 0; j < at.nrows; ++j) {
          const int32_t a0 = rows.start[at.row0 + j], b0 = rows.end[at.row0 + j];
          if (b0 <= a0) continue;
          uint32_t keep[2];   // of the thread's pairs of positions
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int32_t pos = pos0 + x * 8 + (lane & 3) * 2;
            keep[x] = (pos >= a0 && pos < b0 ? 0xFFFFu : 0u) | (pos + 1 >= a0 && pos + 1 < b0 ? 0xFFFF0000u : 0u);
          }
#pragma unroll
          for (int n = 0; n < NT; n += 2) {
            uint32_t b[4];
            ldsm4t(va + (((uint32_t)(n + lane / 16) ^ vx) << 4), b);
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                float d[4] = {0.f, 0.f, 0.f, 0.f};
                mma16816<BF16>(d, pf[t], b[2 * y] & keep[0], b[2 * y + 1] & keep[1]);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if ((t * 16 + e * 8 + lane / 4) / p.chunk_heads == j) {
                    o[t][n + y][2 * e] += d[2 * e];
                    o[t][n + y][2 * e + 1] += d[2 * e + 1];
                  }
              }
          }
        }
      }

      }

      // the segment ends: finish the unit, or leave its part
      {
        const bool unit_end = v1 == at.nsub, whole = unit_end && !cut_front;
        const int which = cut_front ? 0 : 1;
        if (!unit_end && !cut_front && lane == 0) {
          p.open_parts[worker] = sp.holder(sp.first(worker + 1) - end + at.nsub - 1) - worker + 1;
          p.open_info[worker] = make_int4(at.row0, at.nrows, at.kv * p.chunks + at.chunk, 0);
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float l = sum[t][e];
            l += __shfl_xor_sync(~0u, l, 1);
            l += __shfl_xor_sync(~0u, l, 2);
            const int m = t * 16 + e * 8 + lane / 4;
            const int j = m / p.chunk_heads, h = m - j * p.chunk_heads;
            const bool on = live >> (2 * t + e) & 1;
            if (!whole) {
              const int64_t at_part = ((int64_t)worker * 2 + which) * TILE + m;
              if (on) {
                // a sum of -1: the part saw no position at all
                if ((lane & 3) == 0) p.part_ml[at_part] = make_float2(mx[t][e], SLOTS && !seen ? -1.f : l);
                float2* dst = (float2*)(p.part_o + at_part * D) + (lane & 3);
#pragma unroll
                for (int n = 0; n < NT; ++n) dst[n * 4] = make_float2(o[t][n][2 * e], o[t][n][2 * e + 1]);
              }
            } else if (on) {
              const int64_t row = at.row0 + j;
              const int32_t qh = h0 + h;
              const float inv = SLOTS && !seen ? 0.f : 1.f / l;
              T* dst = (T*)p.out + row * p.out_row + (int64_t)qh * p.out_head + (lane & 3) * 2;
#pragma unroll
              for (int n = 0; n < NT; ++n)
                *(uint32_t*)(dst + n * 8) = pack2<BF16>(o[t][n][2 * e] * inv, o[t][n][2 * e + 1] * inv);
              if ((lane & 3) == 0) {
                if (p.lse) p.lse[row * p.q_heads + qh] = log_sum_exp<BF16>(mx[t][e], l, c);
                if (p.row_stat)
                  p.row_stat[row * p.q_heads + qh] =
                      make_float2(mx[t][e] == kNegInf ? 0.f : mx[t][e], inv * kShiftUp<BF16>);
              }
            }
          }
      }
      end -= at.nsub + kUnitCost;
      if (end > 0) at.next_unit(p, rows);
    }
    copy_wait<0>();
  }
  // rows that see nothing
  if constexpr (!SLOTS) {
    for (int64_t i = (int64_t)blockIdx.x * (WARPS * 32) + threadIdx.x; i < p.rows * (int64_t)p.q_heads;
         i += (int64_t)gridDim.x * (WARPS * 32)) {
      const int32_t r = (int32_t)(i / p.q_heads), h = (int32_t)(i - (int64_t)r * p.q_heads);
      if (p.row_end[r] > p.row_start[r]) continue;
      uint4* o = (uint4*)((T*)p.out + r * p.out_row + h * p.out_head);
      for (int j = 0; j < CH; ++j) o[j] = make_uint4(0, 0, 0, 0);
      if (p.lse) p.lse[i] = kNegInf;
      if (p.row_stat) p.row_stat[i] = make_float2(0.f, 0.f);
    }
  }
  warp_err = __reduce_max_sync(~0u, warp_err);
  if (lane == 0 && warp_err != kOk) atomicMax(&err, warp_err);
  __syncthreads();
  if (threadIdx.x == 0) p.cta_status[blockIdx.x] = err;
}

template <bool BF16, int D, int TILE, int WARPS, int STAGES, bool SLOTS>
cudaError_t launch_one(const AttnParams& p, int sm_count, cudaStream_t stream) {
  auto* kernel = attn_kernel<BF16, D, TILE, WARPS, STAGES, SLOTS>;
  constexpr int smem = WARPS * STAGES * 2 * kSub * D * 2;
  static std::atomic<bool> done[64];
  cudaError_t e = set_smem_once(kernel, smem, done);
  if (e != cudaSuccess) return e;
  kernel<<<sm_count, WARPS * 32, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace attn
}  // namespace idxk
