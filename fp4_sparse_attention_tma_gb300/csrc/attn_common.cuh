// Device code that the attention kernels share: the asynchronous copies, the division of
// the work, and the walk over the units.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "attn.h"
#include "idx_launch.h"

namespace idxk {
namespace attn {

constexpr float kNegInf = -INFINITY;

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// 16-byte asynchronous copy; bytes = 0 writes zeros and reads nothing.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (BF16) {
    __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
    return *(uint32_t*)&t;
  } else {
    __half2 t = __floats2half2_rn(lo, hi);
    return *(uint32_t*)&t;
  }
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Divides the units' subtiles among the workers.
struct Split {
  int64_t total = 0;    // subtiles of all units, and what they are counted more
  int32_t active = 0;   // workers with a range
  __device__ void divide(const AttnParams& p, int64_t subtiles) {
    total = subtiles;
    active = (int32_t)(total < p.workers ? total : p.workers);
  }
  __device__ int64_t first(int64_t w) const { return total * w / active; }
  // the worker whose range holds subtile x
  __device__ int32_t holder(int64_t x) const { return (int32_t)(((x + 1) * active - 1) / total); }
};

// The rows' metadata: the caller's arrays, or a copy in shared memory (of up to so many rows;
// every role and warp walks over them, and its waits for them would add up).
constexpr int kRowCopies = 512;
struct Rows {
  const int32_t *req, *start, *end;
};

// Row groups: a row starts one where the request changes, and every group_rows rows of the call (counted
// from its first row, so a request's rows may fall into two groups).
__device__ __forceinline__ bool starts_group(const AttnParams& p, const Rows& rows, int32_t r) {
  return r < p.rows && (r % p.group_rows == 0 || rows.req[r - 1] != rows.req[r]);
}

// Whether a row's window [a, b) does not meet the window [a0, b0) of the row before it.  Groups whose rows
// are walked over together (Cursor) end there: their windows then have no gap between them, so that every
// position that is read is under some row's window, and no page is asked for that none needs.
__device__ __forceinline__ bool apart(int32_t a0, int32_t b0, int32_t a, int32_t b) {
  return b > a && (b0 <= a0 || max(a, a0) > min(b, b0));
}

// What a unit of the group that starts at row r counts; 0 where none does, or it sees nothing.  (A call of
// its own: within the kernel it costs the loops there registers, 51.5 us for 50.8 at 48 requests x 3 rows x
// 16 heads of dimension 64.)
inline __device__ __noinline__ int32_t joint_count(Rows rows, int32_t n_rows, int32_t group_rows, int32_t r) {
  if (r >= n_rows) return 0;
  const int32_t req = rows.req[r], stop = min(n_rows, (r / group_rows + 1) * group_rows);
  int32_t a0 = rows.start[r], b0 = rows.end[r];
  if (r % group_rows != 0 && rows.req[r - 1] == req && !apart(rows.start[r - 1], rows.end[r - 1], a0, b0)) return 0;
  int32_t a = b0 > a0 ? a0 : INT32_MAX, b = b0 > a0 ? b0 : 0;
  for (int32_t i = r + 1; i < stop && rows.req[i] == req; ++i) {
    const int32_t a1 = rows.start[i], b1 = rows.end[i];
    if (apart(a0, b0, a1, b1)) break;
    if (b1 > a1) a = min(a, a1), b = max(b, b1);
    a0 = a1, b0 = b1;
  }
  return b > a ? (b + kSub - 1) / kSub - a / kSub + kUnitCost : 0;
}

// A place in the list of units: subtile `s` of one unit of the group at row0.
template <bool SLOTS>
struct Cursor {
  int32_t row0, nrows, req;   // the group
  int32_t lo, hi;             // positions of its rows' windows, together
  int32_t base, nsub;         // first subtile (absolute) and their number
  int32_t kv, chunk, s;       // the unit: key-value head and chunk of its query heads

  // The group that starts at `row`.  Called by the whole warp.
  __device__ void load(const AttnParams& p, const Rows& rows, int32_t row) {
    row0 = row;
    if constexpr (SLOTS) {
      nrows = 1;
      req = 0;
      lo = 0;
      hi = p.n_slots;
      base = 0;
    } else {
      const int lane = threadIdx.x & 31;
      const int32_t r = row + lane;
      const int32_t stop = min(p.rows, (row / p.group_rows + 1) * p.group_rows);
      const bool in = r < stop;
      const int32_t rr = in ? rows.req[r] : -1;
      int32_t a = in ? rows.start[r] : 0, b = in ? rows.end[r] : 0;
      const int32_t a0 = __shfl_up_sync(~0u, a, 1), b0 = __shfl_up_sync(~0u, b, 1);
      req = __shfl_sync(~0u, rr, 0);
      const uint32_t other = ~__ballot_sync(~0u, in && rr == req && (lane == 0 || !apart(a0, b0, a, b)));
      nrows = other ? __ffs(other) - 1 : 32;
      if (lane >= nrows || b <= a) a = INT32_MAX, b = 0;
      lo = __reduce_min_sync(~0u, a);
      hi = __reduce_max_sync(~0u, b);
      if (lo > hi) lo = hi;
      base = lo / kSub;
    }
    nsub = hi > lo ? (hi + kSub - 1) / kSub - base : 0;
  }
  __device__ static int32_t count(const AttnParams& p, const Rows& rows, int32_t r) {
    return joint_count(rows, p.rows, p.group_rows, r);
  }
  // The same for a row of a call over slots.
  __device__ static int32_t row_count(const AttnParams& p) { return (p.n_slots + kSub - 1) / kSub + kUnitCost; }
  // Place t of the group's units, one after another; returns how far it is behind the unit's first subtile.
  __device__ int32_t place(const AttnParams& p, int64_t t) {
    const int32_t n = nsub + kUnitCost, u = (int32_t)(t / n), off = (int32_t)(t - (int64_t)u * n) - kUnitCost;
    s = max(0, off);
    kv = u / p.chunks;
    chunk = u % p.chunks;
    return off;
  }
  // The next unit, at its first subtile; the caller has not passed the end of the list.
  __device__ void next_unit(const AttnParams& p, const Rows& rows) {
    s = 0;
    if (++chunk < p.chunks) return;
    chunk = 0;
    if (++kv < p.kv_heads) return;
    kv = 0;
    do {
      load(p, rows, row0 + nrows);
    } while (nsub == 0);
  }
};

// Checks the rows' metadata (all of it, by every CTA, so that all agree), counts the
// subtiles, and leaves the place where the worker's range starts in `cur` (`worker` may
// differ from warp to warp), and where it ends, counted from the unit's first subtile, in
// `end`.  Called by the whole CTA.  False: an error (recorded in *err) or nothing to do for
// this warp.  `room`: 8 bytes of shared memory a thread.
template <class Cur, bool SLOTS, int WARPS>
__device__ bool find_range(const AttnParams& p, Rows& rows, Split& sp, Cur& cur, int64_t& end, int32_t worker, void* room,
                           uint32_t* err) {
  const int32_t units = p.kv_heads * p.chunks;
  if constexpr (SLOTS) {
    const int32_t n = Cur::row_count(p);
    sp.divide(p, (int64_t)p.rows * units * n);
    if (worker >= sp.active) return false;
    const int64_t t = sp.first(worker);
    const int64_t per_row = (int64_t)units * n;
    const int32_t row = (int32_t)(t / per_row);
    cur.load(p, rows, row);
    end = sp.first(worker + 1) - t + cur.place(p, t - row * per_row);
    return end > cur.s;
  } else {
    constexpr int N = WARPS * 32;
    __shared__ int64_t warp_sum[WARPS];
    int64_t* pre = (int64_t*)room;      // [N] subtiles before each row of the pass, in the pass
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    __shared__ int32_t copy[3][kRowCopies];
    const bool copied = p.rows <= kRowCopies;
    int64_t sum = 0;
    bool bad = false;
    const bool one_pass = p.rows <= N;
    for (int32_t r = tid; r < p.rows; r += N) {
      const int32_t q = p.row_req[r], a = p.row_start[r], b = p.row_end[r];
      bad |= q < 0 || q >= p.num_req || a < 0 || b < a || (int64_t)b > (int64_t)p.max_pages * kPage;
      if (copied) copy[0][r] = q, copy[1][r] = a, copy[2][r] = b;
    }
    rows = copied ? Rows{copy[0], copy[1], copy[2]} : Rows{p.row_req, p.row_start, p.row_end};
    if (__syncthreads_or(bad)) {
      if (tid == 0) *err = kErrInvalidMetadata;
      return false;
    }
    int32_t mine = 0;
    for (int32_t r = tid; r < p.rows; r += N) sum += mine = Cur::count(p, rows, r);
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if (lane == 0) warp_sum[warp] = sum;
    __syncthreads();
    sum = 0;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) sum += warp_sum[i];
    sp.divide(p, sum * units);
    const bool some = worker < sp.active;
    const int64_t t = some ? sp.first(worker) : 0;
    bool found = false;
    int64_t before = 0;   // subtiles (of one unit each) before the pass
    for (int32_t r0 = 0; r0 < p.rows; r0 += N) {
      if (!one_pass) mine = Cur::count(p, rows, r0 + tid);
      int64_t inc = mine;
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(~0u, inc, o);
        if (lane >= o) inc += x;
      }
      __syncthreads();
      if (lane == 31) warp_sum[warp] = inc;
      __syncthreads();
      int64_t base = 0, all = 0;
#pragma unroll
      for (int i = 0; i < WARPS; ++i) {
        if (i < warp) base += warp_sum[i];
        all += warp_sum[i];
      }
      pre[tid] = base + inc - mine;
      __syncthreads();
      if (some && !found && t < (before + all) * units) {
        // the last row of the pass whose subtiles start at or before t: the first row of the group that
        // holds it (rows without a count of their own come before it, or start after t)
        const int32_t n = min(N, p.rows - r0);
        int32_t at = 0;
        for (int32_t i = lane; i < n; i += 32)
          if ((before + pre[i]) * units <= t) at = i;   // pre is non-decreasing
        at = __reduce_max_sync(~0u, at);
        cur.load(p, rows, r0 + at);
        end = sp.first(worker + 1) - t + cur.place(p, t - (before + pre[at]) * units);
        found = true;
      }
      before += all;
    }
    __syncthreads();   // `room` is free again
    return found && end > cur.s;
  }
}

}  // namespace attn
}  // namespace idxk
