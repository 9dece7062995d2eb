// The attention kernel for head dimension 128 on the fifth-generation tensor cores: up to 64 query
// heads of a key-value head at once (a chunk), for one or two rows of a request.
//
// With more than 16 heads the products, not the copies, bound warps that load every key and value
// once per 16 heads (attn.cuh); with fewer, over long contexts, what counts is how few instructions
// the copies take.  A CTA takes tiles of 128 positions for a matrix of 128 rows:
//
//   S [128 x 128 positions] = Q K^T      (queries and keys in shared memory, K-major)
//   O [128 x 128] += P V                 (weights in tensor memory, values as they lie in the cache)
//
// A matrix row is a tensor memory lane and a thread of each softmax warpgroup: its sum and its
// weights need no other thread, the weights are written over the scores they come from, and next to
// nothing of a visit passes through shared memory.  O is scaled only when a row's maximum exceeds
// the reference of its weights by kRaise (in units of log2); a weight, at most 2^kRaise then (fp16:
// 2^(kRaise + kShift), within its range), is rounded to the inputs' type for the second product (its
// sum is not), which the matrix instruction asks for: u sum p |v| at most beside the output's u |out|.
//
// What bounds it: HBM where the cache is long (32 requests x 2 rows x 64 heads on 8, 4096..65536
// positions: 4.45 GB in 652 us, 6.8 TB/s; one row of 262143 positions: 163 us, 6.6 TB/s).  The same
// batch with one key-value head: 0.56 GB in 105 us, of which 5 us pass before the first copies, 4 us
// in a segment's end and 8 us in the join.  Where rows pick 1024 slots of a cache that L2 holds, the
// copies (64 KB a visit), the products and the softmax each take 0.7 to 0.8 us a visit and overlap to
// 1.0, and a unit of 8 visits ends in 2.5 us (8192 rows: 555 us, 495 TFLOP/s; without the copies 15 %
// less, without the products 13 %).
//
// Two rows of one request: matrix rows 0..63 and 64..127 are theirs; both use the tiles that both
// see in full.  What only one row sees is visited for it alone, in an order and with a second
// accumulator such that it never meets the other's sums (0 x infinity is not 0): first the first
// row's own tiles, then (the second row's lanes set back to 0) the common ones, then the second
// row's own into the second accumulator.
//
// One row: its heads stand in both halves of the matrix.  The lower half weighs and sums the first 64
// positions of every tile, the upper half the others, each with its own reference and accumulator;
// they are joined at the segment's end.
//
// Roles: two warpgroups of softmax (the same rows, half of the positions each; a row's maximum is
// the only thing that its two threads exchange), one that copies keys (and the queries), one that copies values
// (16-byte asynchronous copies into the 128-byte swizzle, any stride, page or slot), one warp that
// issues the scores' products and one the outputs'.  Every wait is bounded.
#pragma once

#include "attn_common.cuh"
#include "idx_device.cuh"

namespace idxk {
namespace attn {
namespace tc {

constexpr int kPos = 128;                 // positions of a tile
constexpr int kCols = 64;                 // matrix rows of one row of the call (query heads of a chunk)
constexpr int kHead = 128;                // head dimension
constexpr uint32_t kHalfTile = kPos * 128;      // 64 of the dimension's elements of 128 rows
constexpr uint32_t kTileBytes = 2 * kHalfTile;  // a tile of keys, of values or of queries
constexpr int kWarps = 20;
constexpr int kThreads = kWarps * 32;
constexpr int kLoaders = 128;             // threads that copy keys (and as many values)
template <bool BF16>
constexpr float kRaise = BF16 ? 8.f : 5.f;   // weights are at most 2^(kRaise + kShift)
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOut = 256;            // first column of the accumulators, after two tiles of scores
constexpr int kRingK = 3, kRingV = 2;     // tiles of keys and of values in shared memory
constexpr uint32_t kKeys = 0, kValues = kKeys + kRingK * kTileBytes, kQueries = kValues + kRingV * kTileBytes,
                   kStage = kQueries + kTileBytes;   // offsets; then room to pass sums between the halves
constexpr int kStageRow = 17;             // floats
constexpr int kSmemBytes = (int)kStage + 4 * kCols * kStageRow * 4 + 1024;   // the base is aligned to 1024 by hand

// D += A B^T with both operands in shared memory, or A in tensor memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 8 columns of tensor memory, this warp's 32 lanes, loaded (and waited for) or stored.
__device__ __forceinline__ void tmem_load8(uint32_t a, float (&r)[8]) {
  uint32_t u[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
      : "r"(a)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = __uint_as_float(u[i]);
}
__device__ __forceinline__ void tmem_store8(uint32_t a, const float (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(a),
               "r"(__float_as_uint(r[0])), "r"(__float_as_uint(r[1])), "r"(__float_as_uint(r[2])),
               "r"(__float_as_uint(r[3])), "r"(__float_as_uint(r[4])), "r"(__float_as_uint(r[5])),
               "r"(__float_as_uint(r[6])), "r"(__float_as_uint(r[7]))
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(a),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// Shared-memory matrix descriptor with the 128-byte swizzle.  K-major: 8-row groups `stride`
// apart.  MN-major: groups of 8 along K `stride` apart, groups of 64 along M or N `lead` apart.
__device__ __forceinline__ uint64_t desc128(uint32_t addr, uint32_t lead, uint32_t stride) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(stride >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// Instruction descriptor, kind::f16 with fp32 accumulation, A K-major; `mn`: B MN-major.
template <bool BF16>
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t M, uint32_t N, bool mn) {
  return (1u << 4) | ((BF16 ? 1u : 0u) << 7) | ((BF16 ? 1u : 0u) << 10) | ((mn ? 1u : 0u) << 16) | ((N >> 3) << 17) |
         ((M >> 4) << 24);
}

// The walk over the units; a unit's steps are visits of (tile, rows).
template <int NB, bool SLOTS>
struct Walk {
  int32_t row0, nrows, req;
  int32_t a[NB], b[NB];          // windows of the group's rows (0, 0: none)
  int32_t c0, c1;                // tiles that both rows see in full
  int32_t nsub;                  // visits of a unit
  int32_t kv, chunk, s;

  __device__ static int32_t lo(int32_t a) { return a / kPos; }
  __device__ static int32_t hi(int32_t b) { return (b + kPos - 1) / kPos; }
  // Visits of a unit whose rows see these windows; c0 and c1 as above.
  __device__ static int32_t visits(const int32_t (&a)[NB], const int32_t (&b)[NB], int32_t& c0, int32_t& c1) {
    int32_t n = 0;
    c0 = 0, c1 = 0;
#pragma unroll
    for (int j = 0; j < NB; ++j) n += b[j] > a[j] ? hi(b[j]) - lo(a[j]) : 0;
    if constexpr (NB == 2) {
      if (b[0] > a[0] && b[1] > a[1]) {
        c0 = max(hi(a[0]), hi(a[1]));
        c1 = min(lo(b[0]), lo(b[1]));
        if (c1 <= c0) c0 = c1 = 0;
        n -= c1 - c0;
      }
    }
    return n;
  }
  __device__ static int32_t count(const AttnParams& p, const Rows& rows, int32_t r) {
    if (!starts_group(p, rows, r)) return 0;
    int32_t a[NB], b[NB], c0, c1;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int32_t i = r + j;
      const bool in = i < p.rows && (j == 0 || (i % p.group_rows != 0 && rows.req[i] == rows.req[r]));
      a[j] = in ? rows.start[i] : 0;
      b[j] = in ? rows.end[i] : 0;
    }
    const int32_t n = visits(a, b, c0, c1);
    return n ? n + kUnitCost : 0;
  }
  __device__ static int32_t row_count(const AttnParams& p) { return hi(p.n_slots) + kUnitCost; }

  __device__ void load(const AttnParams& p, const Rows& rows, int32_t row) {
    row0 = row;
    req = 0;
    nrows = 1;
    if constexpr (SLOTS) {
      a[0] = 0;
      b[0] = p.n_slots;
    } else {
      req = rows.req[row];
      if constexpr (NB == 2)
        if (row + 1 < p.rows && (row + 1) % p.group_rows != 0 && rows.req[row + 1] == req) nrows = 2;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        a[j] = j < nrows ? rows.start[row + j] : 0;
        b[j] = j < nrows ? rows.end[row + j] : 0;
        if (b[j] <= a[j]) a[j] = b[j] = 0;
      }
    }
    nsub = visits(a, b, c0, c1);
  }
  // Place t of the group's units, one after another; returns how far it is behind the unit's first visit.
  __device__ int32_t place(const AttnParams& p, int64_t t) {
    const int32_t n = nsub + kUnitCost, u = (int32_t)(t / n), off = (int32_t)(t - (int64_t)u * n) - kUnitCost;
    s = max(0, off);
    kv = u / p.chunks;
    chunk = u % p.chunks;
    return off;
  }
  // The next unit, at its first visit; the caller has not passed the end of the list.
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
  // Visit v of the unit: its tile and its rows (bit j).
  __device__ void visit(int32_t v, int32_t& tile, uint32_t& rows) const {
    if constexpr (NB == 1) {
      tile = lo(a[0]) + v;
      rows = 1;
    } else {
      // what only the first row sees in full, what both see, what only the second does
      const bool both = c1 > c0;
      rows = 1;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int32_t front = both ? c0 - lo(a[j]) : hi(b[j]) - lo(a[j]), back = both ? hi(b[j]) - c1 : 0;
        if (v < front + back) {
          tile = v < front ? lo(a[j]) + v : c1 + v - front;
          rows = 1u << j;
          return;
        }
        v -= front + back;
        if (j == 0) {
          if (v < c1 - c0) {
            tile = c0 + v;
            rows = 3;
            return;
          }
          v -= c1 - c0;
        }
      }
      tile = 0;   // (not reached)
    }
  }
};

// Two fp32 operations in one instruction, and a maximum of three.  exponent2: `exponent` of two products
// (minus the reference is given), and the shift.
__device__ __forceinline__ void exponent2(float& x, float& y, float minus_ref, float c, float shift) {
  asm("{\n\t.reg .b64 v, m, s, h;\n\t"
      "mov.b64 v, {%0, %1};\n\tmov.b64 s, {%2, %2};\n\tmov.b64 m, {%3, %3};\n\tmov.b64 h, {%4, %4};\n\t"
      "add.rn.f32x2 v, v, s;\n\tfma.rn.f32x2 v, v, m, h;\n\tmov.b64 {%0, %1}, v;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(minus_ref), "f"(c), "f"(shift));
}
__device__ __forceinline__ void add2(float& x, float& y, float a, float b) {
  asm("{\n\t.reg .b64 v, s;\n\t"
      "mov.b64 v, {%0, %1};\n\tmov.b64 s, {%2, %3};\n\t"
      "add.rn.f32x2 v, v, s;\n\tmov.b64 {%0, %1}, v;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 8 floats to a 32-byte boundary: half as many store instructions, of 32 rows each, as of 16 bytes.
__device__ __forceinline__ void store32(float* a, const float (&z)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(a), "f"(z[0]), "f"(z[1]), "f"(z[2]),
               "f"(z[3]), "f"(z[4]), "f"(z[5]), "f"(z[6]), "f"(z[7])
               : "memory");
}

// One lane of the warp, the same each time: what it commits is what it issued.
__device__ __forceinline__ bool elect_one() {
  uint32_t on;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(on));
  return on != 0;
}

// Arrives on `bar` (one of its expected arrivals) when this thread's copies so far have landed.
__device__ __forceinline__ void arrive_when_copied(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void copy_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// A bounded wait: false when it gave up (after kWaitLimitNs, or because another role did).
__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort, uint32_t* err) {
  uint64_t t0 = 0;
  if (*abort) return false;
  for (uint32_t i = 0;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 63u) {
      if (*abort) return false;
      const uint64_t now = global_timer_ns();
      if (t0 == 0) {
        t0 = now;
      } else if (now - t0 > kWaitLimitNs) {
        *abort = 1;
        atomicMax(err, (uint32_t)kErrTimeout);
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* abort, uint32_t* err) {
  if (mbar_try_wait(bar, parity)) return true;
  return wait_slow(bar, parity, abort, err);
}

template <bool BF16, int NB, bool SLOTS>
__global__ void __launch_bounds__(kThreads, 1) attn_tc_kernel(const __grid_constant__ AttnParams p) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr bool SPLIT = NB == 1;           // one row: either half of the matrix takes half of a tile's positions
  constexpr int kSoft = 256;                // softmax threads

  extern __shared__ __align__(16) unsigned char raw[];
  __shared__ uint32_t err, tmem_base;
  __shared__ int abort_flag;
  __shared__ __align__(8) uint64_t bars[2 * kRingK + 2 * kRingV + 1 + 3 * 2 + 1];
  __shared__ float2 half_ml[2][kCols];      // (one row) reference and sum of either half, -1 where nothing was seen
  __shared__ float row_max[2][2][128];      // by visit and warpgroup
  __shared__ float row_sum[2][128];         // by warpgroup, -1 where nothing was seen
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t smem = (smem_addr(raw) + 1023u) & ~1023u;
  const uint32_t bar0 = smem_addr(bars);
  auto full_k = [&](uint32_t i) { return bar0 + 8 * i; };
  auto empty_k = [&](uint32_t i) { return bar0 + 8 * (kRingK + i); };
  auto full_v = [&](uint32_t i) { return bar0 + 8 * (2 * kRingK + i); };
  auto empty_v = [&](uint32_t i) { return bar0 + 8 * (2 * kRingK + kRingV + i); };
  constexpr uint32_t kRest = 2 * kRingK + 2 * kRingV;
  const uint32_t empty_q = bar0 + 8 * kRest, drain = bar0 + 8 * (kRest + 7);
  // by tile of scores (visits take them in turn):
  auto full_s = [&](uint32_t b) { return bar0 + 8 * (kRest + 1 + b); };    // scores are there
  auto full_p = [&](uint32_t b) { return bar0 + 8 * (kRest + 3 + b); };    // weights are there
  auto done_pv = [&](uint32_t b) { return bar0 + 8 * (kRest + 5 + b); };   // and summed: the tile is free

  allow_launch_after();
  if (threadIdx.x == 0) {
    err = kOk;
    abort_flag = 0;
    for (int i = 0; i < kRingK; ++i) mbar_init(full_k(i), kLoaders), mbar_init(empty_k(i), 1);
    for (int i = 0; i < kRingV; ++i) mbar_init(full_v(i), kLoaders), mbar_init(empty_v(i), 1);
    mbar_init(empty_q, 1);
    for (int b = 0; b < 2; ++b) mbar_init(full_s(b), 1), mbar_init(full_p(b), kSoft), mbar_init(done_pv(b), 1);
    mbar_init(drain, 2);
    fence_mbar_init();
  }
  if (warp == 16) {
    tmem_alloc(smem_addr(&tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  volatile int* abort = &abort_flag;

  // A role walks over its segments (the part of a unit in the CTA's range) and a segment's visits.
  // What only a segment's ends need lies in shared memory, a copy a warp: in registers it would push
  // the visits' own values out to local memory, for which no L1 is left.
  struct Place {
    Walk<NB, SLOTS> at;
    int64_t end;   // of the CTA's range, counted from the unit's first visit
  };
  __shared__ Place places[kWarps];
  __shared__ Split split;
  __shared__ Rows meta;
  Walk<NB, SLOTS>& at = places[warp].at;
  bool work;
  {
    Split sp;
    Walk<NB, SLOTS> first;
    Rows rows{};
    int64_t end;
    work = find_range<Walk<NB, SLOTS>, SLOTS, kWarps>(p, rows, sp, first, end, blockIdx.x, raw, &err);
    if (threadIdx.x == 0) {
      if ((int32_t)blockIdx.x < sp.active) p.open_parts[blockIdx.x] = 0;
      if (blockIdx.x == 0) *p.active = sp.active;
      split = sp;
      meta = rows;
    }
    if (work && lane == 0) {
      places[warp].at = first;
      places[warp].end = end;
    }
  }
  __syncthreads();
  // The segment's last visit (and one more); then, on to the next segment: false at the range's end.
  auto segment_end = [&]() { return (int32_t)min((int64_t)at.nsub, places[warp].end); };
  auto next_segment = [&]() {
    __syncwarp();
    if (lane == 0) {
      places[warp].end -= at.nsub + kUnitCost;
      if (places[warp].end > 0) at.next_unit(p, meta);
    }
    __syncwarp();
    return places[warp].end > 0;
  };
  // Whether the range goes on after the segment, and with the next row (else another unit of this one).
  auto goes_on = [&]() { return places[warp].end > at.nsub + kUnitCost; };
  auto next_is_row = [&]() { return at.chunk + 1 == p.chunks && at.kv + 1 == p.kv_heads; };
  if (work) {
    // registers: 640 threads are launched with 96 each; two warpgroups of 120 and three of 80 are as many
    if (warp < 8) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 120;");
      // ------------------------------------------------------------ softmax ----
      const int x = threadIdx.x & 127;                 // matrix row, tensor memory lane
      const int g = warp >> 2;                         // warpgroup
      const uint32_t pair = 2 + (warp & 3);            // barrier of the two warps that have the same rows
      const uint32_t part_of = (uint32_t)(warp & 3) >> 1;   // half of the matrix: the row of the group, or the positions' half
      constexpr uint32_t kAll = 1;                     // barrier of all softmax threads
      constexpr int CH = SPLIT ? 1 : 2;                // 32 positions each: what a thread weighs of a tile
      const int c0 = SPLIT ? (int)part_of * 2 + g : 2 * g;
      const uint32_t lanes = (uint32_t)(warp & 3) << 21;    // this warp's 32 lanes
      const uint32_t out_a = tmem + lanes + kOut + (SPLIT ? part_of * kHead : 0), out_b = tmem + lanes + kOut + kHead;
      uint32_t n = 0;                // visits so far
      bool ok = true;
      bool more = true;
      // (slots) the slots of the next visit's positions, asked for a visit ahead
      int32_t slot[CH];
      const int32_t* list = nullptr;
      auto ask = [&](int32_t v) {
#pragma unroll
        for (int k = 0; k < CH; ++k) {
          const int32_t pos = v * kPos + (c0 + k) * 32 + lane;
          slot[k] = pos < p.n_slots ? list[pos] : -1;
        }
      };
      if constexpr (SLOTS) {
        list = p.slots + (int64_t)at.row0 * p.n_slots;
        ask(at.s);
      }
      while (more) {
        const int32_t v1 = segment_end();
        float ref = kNegInf, sum[4] = {0.f, 0.f, 0.f, 0.f};
        bool had_a = false, had_b = false;   // the accumulators hold something of this matrix row
        bool foreign = false;                // the first accumulator holds the other row's tiles alone in this row's lanes
        bool seen = false;
        for (int32_t v = at.s; v < v1; ++v, ++n) {
          const uint32_t b = n & 1;
          int32_t tile;
          uint32_t rows;
          at.visit(v, tile, rows);
          const bool mine = SPLIT || (rows >> part_of & 1);
          // which of the positions this row sees
          uint32_t on[CH];
#pragma unroll
          for (int k = 0; k < CH; ++k) on[k] = ~0u;
          if constexpr (SLOTS) {
#pragma unroll
            for (int k = 0; k < CH; ++k) on[k] = __ballot_sync(~0u, slot[k] >= 0 && slot[k] < p.num_pages * kPage);
            if (v + 1 < v1) ask(v + 1);
          } else if (rows != 3) {
            const int32_t a = at.a[SPLIT ? 0 : part_of], z = at.b[SPLIT ? 0 : part_of];
            if (tile * kPos < a || tile * kPos + kPos > z) {
#pragma unroll
              for (int k = 0; k < CH; ++k) {
                const int32_t pos = tile * kPos + (c0 + k) * 32 + lane;
                on[k] = __ballot_sync(~0u, pos >= a && pos < z);
              }
            }
          }
          ok &= wait(full_s(b), n >> 1 & 1, abort, &err);
          tc_fence_after();
          const uint32_t s = tmem + lanes + b * kPos + c0 * 32, w_at = tmem + lanes + b * kPos + c0 * 16;
          if (mine) {
            uint32_t r[CH][32];
            // chunk k's maximum (its scores put down first, where the weights are to be added up)
            float top = kNegInf, top2 = kNegInf;
            auto look = [&](int k, uint32_t (&r)[32]) {
              if constexpr (!SLOTS) {
                if (p.logits) {
                  const int64_t width = (int64_t)p.max_pages * kPage;
                  const int32_t pos = tile * kPos + (c0 + k) * 32, h = at.chunk * p.chunk_heads + (x & (kCols - 1));
                  if ((x & (kCols - 1)) < p.chunk_heads && h < p.group && pos < width) {
                    float4* dst = (float4*)(p.logits +
                                            ((int64_t)(at.row0 + (SPLIT ? 0 : part_of)) * p.q_heads + at.kv * p.group + h) *
                                                width + pos);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                      dst[i] = make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]),
                                           __uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3]));
                  }
                }
              }
              if (on[k] != ~0u) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (!(on[k] >> i & 1)) r[i] = __float_as_uint(kNegInf);
              }
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                top = max3(top, __uint_as_float(r[i]), __uint_as_float(r[i + 1]));
                top2 = max3(top2, __uint_as_float(r[i + 2]), __uint_as_float(r[i + 3]));
              }
              seen |= on[k] != 0;
            };
#pragma unroll
            for (int k = 0; k < CH; ++k) tmem_ld32(s + k * 32, r[k]);
#pragma unroll
            for (int k = 0; k < CH; ++k) tmem_wait_ld32(r[k]);
#pragma unroll
            for (int k = 0; k < CH; ++k) look(k, r[k]);
            // of the whole row: the other warpgroup's thread has seen the other positions
            top = fmaxf(top, top2);
            row_max[b][g][x] = top;
            bar_sync(pair, 64);
            top = fmaxf(top, row_max[b][g ^ 1][x]);
            // does its weights' reference have to follow?
            if (__any_sync(~0u, exponent(top, ref, p.scale_log2) > kRaise<BF16>)) {   // (false where both are -infinity)
              const float raised = fmaxf(ref, top), f = raised == ref ? 1.f : ex2(exponent(ref, raised, p.scale_log2));
              ref = raised;
#pragma unroll
              for (int i = 0; i < 4; ++i) sum[i] *= f;
              if (had_a || had_b) {
                ok &= wait(done_pv(b ^ 1), (n - 1) >> 1 & 1, abort, &err);   // the last visit that added to them
                tc_fence_after();
                // a half of the columns each
#pragma unroll 1
                for (int y = 0; y < kHead; y += 8) {
                  if (y < 64 ? !had_a : !had_b) continue;
                  const uint32_t o = (y < 64 ? out_a : out_b - 64) + g * 64 + y;
                  float z[8];
                  tmem_load8(o, z);
#pragma unroll
                  for (int i = 0; i < 8; ++i) z[i] *= f;
                  tmem_store8(o, z);
                }
                tmem_wait_st();
              }
            }
            // the weights, over the scores
            const float base = -reference(ref);
            auto weigh = [&](int k, const uint32_t (&r)[32]) {
              uint32_t w[16];
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                float d0 = __uint_as_float(r[i]), d1 = __uint_as_float(r[i + 1]);
                exponent2(d0, d1, base, p.scale_log2, kShift<BF16>);
                const float e0 = ex2(d0), e1 = ex2(d1);
                add2(sum[i & 2], sum[(i & 2) + 1], e0, e1);
                w[i / 2] = pack2<BF16>(e0, e1);
              }
              tmem_st16(w_at + k * 16, w);
            };
#pragma unroll
            for (int k = 0; k < CH; ++k) weigh(k, r[k]);
            if (!SPLIT && rows == 2) {
              had_b = true;
            } else {
              had_a = true;
            }
          }
          if (!SPLIT) {
            // the first row's own tiles end: what they left in the second row's lanes means nothing
            if (!mine && rows == 1) foreign = true;
            if (foreign && rows == 3) {
              foreign = false;
              if (n > 0) ok &= wait(done_pv(b ^ 1), (n - 1) >> 1 & 1, abort, &err);
              tc_fence_after();
              const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
              for (int y = 0; y < 64; y += 8) tmem_store8(out_a + g * 64 + y, zero);
            }
          }
          tmem_wait_st();
          tc_fence_before();
          // (after a wait that gave up the visits go on, without further waiting, to the vote below)
          mbar_arrive(full_p(b));
        }

        if constexpr (SLOTS) {
          // the next unit's first: of this row, or of the next
          if (goes_on()) {
            if (next_is_row()) list += p.n_slots;
            ask(0);
          }
        }

        // the segment ends: finish the unit, or leave its part
        const bool cut_front = at.s > 0, unit_end = v1 == at.nsub, whole = unit_end && !cut_front;
        const int which = cut_front ? 0 : 1;
        if (!unit_end && !cut_front && threadIdx.x == 0) {
          p.open_parts[blockIdx.x] =
              split.holder(split.first(blockIdx.x + 1) - places[warp].end + at.nsub - 1) - (int32_t)blockIdx.x + 1;
          p.open_info[blockIdx.x] = make_int4(at.row0, at.nrows, at.kv * p.chunks + at.chunk, 0);
        }
        // the last visit of each tile of scores that this segment (or one before it) had
        if (n > 0) ok &= wait(done_pv((n - 1) & 1), (n - 1) >> 1 & 1, abort, &err);
        if (n > 1) ok &= wait(done_pv(n & 1), (n - 2) >> 1 & 1, abort, &err);
        tc_fence_after();
        float l = (sum[0] + sum[1]) + (sum[2] + sum[3]);
        // of the whole row
        row_sum[g][x] = (had_a || had_b) && (!SLOTS || seen) ? l : -1.f;
        bar_sync(pair, 64);
        const float l0 = row_sum[0][x], l1 = row_sum[1][x];
        const bool has = l0 != -1.f || l1 != -1.f;
        l = (l0 != -1.f ? l0 : 0.f) + (l1 != -1.f ? l1 : 0.f);
        if (SPLIT && g == 0) half_ml[part_of][x & (kCols - 1)] = make_float2(ref, has ? l : -1.f);
        // every softmax thread votes on the waits, so that all leave together
        if (bar_red_or(kAll, kSoft, !ok)) break;

        const int32_t row_in = SPLIT ? 0 : (int32_t)part_of, col = x & (kCols - 1);
        const int32_t head = at.chunk * p.chunk_heads + col;
        const bool live = col < p.chunk_heads && head < p.group && at.b[row_in] > at.a[row_in];
        const int64_t row = at.row0 + row_in;
        const int32_t qh = at.kv * p.group + head;
        const int64_t part = ((int64_t)blockIdx.x * 2 + which) * (NB * kCols) + row_in * kCols + col;
        float top = ref, f = 1.f;
        bool any = has;
        if constexpr (SPLIT) {
          const float2 o = half_ml[part_of ^ 1][col];
          const bool other = o.y != -1.f;
          top = fmaxf(has ? ref : kNegInf, other ? o.x : kNegInf);
          const float base = reference(top);
          f = has ? ex2(exponent(ref, base, p.scale_log2)) : 0.f;
          l = (has ? l * f : 0.f) + (other ? o.y * ex2(exponent(o.x, base, p.scale_log2)) : 0.f);
          any = has || other;
        }
        const float inv = any ? 1.f / l : 0.f;
        if (live && g == 0 && (!SPLIT || part_of == 0)) {
          if (!whole) {
            p.part_ml[part] = make_float2(top, any ? l : -1.f);
          } else {
            const int64_t i = row * p.q_heads + qh;
            if (p.lse) p.lse[i] = log_sum_exp<BF16>(top, l, p.scale_log2);
            if (p.row_stat) p.row_stat[i] = make_float2(top == kNegInf ? 0.f : top, inv * kShiftUp<BF16>);
          }
        }
        if (whole) f *= inv;
        T* out = (T*)p.out + row * p.out_row + (int64_t)qh * p.out_head;
        float* po = p.part_o + part * kHead;
        auto emit = [&](int c, const float (&z)[8]) {   // 8 columns of the thread's row
          if (!live) return;
          if (whole) {
            uint4 u;
            u.x = pack2<BF16>(z[0], z[1]), u.y = pack2<BF16>(z[2], z[3]);
            u.z = pack2<BF16>(z[4], z[5]), u.w = pack2<BF16>(z[6], z[7]);
            *(uint4*)(out + c) = u;
          } else if (any) {
            store32(po + c, z);
          }
        };
        if constexpr (SPLIT) {
          // each half finishes 64 columns, 32 a thread; the other half's share of them comes through shared
          // memory, 16 at a time
          float* stage = (float*)(raw + (smem - smem_addr(raw)) + kStage);
          float* give = stage + ((part_of * 2 + g) * kCols + col) * kStageRow;
          const float* take = stage + (((part_of ^ 1) * 2 + g) * kCols + col) * kStageRow;
#pragma unroll 1
          for (int at_col = 0; at_col < 32; at_col += 16) {
#pragma unroll 1
            for (int c = 0; c < 16; c += 8) {
              float r[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
              if (has) tmem_load8(out_a + (part_of ^ 1) * 64 + g * 32 + at_col + c, r);
#pragma unroll
              for (int i = 0; i < 8; ++i) give[c + i] = has ? r[i] * f : 0.f;
            }
            bar_sync(kAll, kSoft);
#pragma unroll 1
            for (int c = 0; c < 16; c += 8) {
              float r[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
              if (has) tmem_load8(out_a + part_of * 64 + g * 32 + at_col + c, r);
#pragma unroll
              for (int i = 0; i < 8; ++i) r[i] = (has ? r[i] * f : 0.f) + take[c + i];
              emit((int)part_of * 64 + g * 32 + at_col + c, r);
            }
            bar_sync(kAll, kSoft);
          }
        } else {
#pragma unroll 1
          for (int c = g * 64; c < g * 64 + 64; c += 8) {
            float r[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, s[8];
            if (had_a) tmem_load8(out_a + c, r);
            if (had_b) {
              tmem_load8(out_b + c, s);
#pragma unroll
              for (int i = 0; i < 8; ++i) r[i] += s[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) r[i] *= f;
            emit(c, r);
          }
        }
        tc_fence_before();
        more = next_segment();
      }
    } else if (warp < 16) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
      // ------------------------------------------------------------- copies ----
      const bool values = warp >= 12;
      const int quarter = warp & 3, t = threadIdx.x & (kLoaders - 1);
      const uint32_t depth = values ? kRingV : kRingK;
      const uint32_t ring = smem + (values ? kValues : kKeys);
      const T* cache = (const T*)(values ? p.v : p.k);
      const int64_t s_page = values ? p.v_page : p.k_page, s_slot = values ? p.v_slot : p.k_slot,
                    s_head = values ? p.v_head : p.k_head;
      // Offsets are in units of 16 bytes (the caches span less than 64 GB).
      const uint32_t page16 = (uint32_t)(s_page / 8), slot16 = (uint32_t)(s_slot / 8);
      const int x = lane & 15, r0 = lane / 16;   // this lane's piece of a head, and its rows r0 + 2 i of the warp's 32
      uint32_t n = 0, seg = 0;                   // tiles, segments
      bool ok = true;
      uint32_t bad = kOk;
      // the slot of this thread's position, or the page of the warp's 32, of the next visit: asked for a
      // visit ahead (and a row's slots brought to L2 a row ahead)
      int32_t entry;
      auto ask = [&](const int32_t* list, int32_t tile) {
        if constexpr (SLOTS) {
          const int32_t pos = tile * kPos + quarter * 32 + lane;
          entry = pos < p.n_slots ? list[pos] : -1;
        } else {
          const int32_t i = tile * 2 + quarter / 2;
          entry = i < p.max_pages ? list[i] : -1;
        }
      };
      if constexpr (SLOTS) ask(p.slots + (int64_t)at.row0 * p.n_slots, at.s);
      bool more = true;
      while (more) {
        const int32_t v0 = at.s, v1 = segment_end();
        int32_t tile;
        uint32_t rows;
        const int32_t* list;
        if constexpr (SLOTS) {
          list = p.slots + (int64_t)at.row0 * p.n_slots;
          if (warp == 12 && at.row0 + 1 < p.rows)
            for (int32_t i = lane * 32; i < p.n_slots; i += 32 * 32)
              asm volatile("prefetch.global.L2 [%0];" ::"l"(list + p.n_slots + i));
        } else {
          list = p.page_table + (int64_t)at.req * p.max_pages;
          at.visit(v0, tile, rows);
          ask(list, tile);
        }
        if (!values) {
          // the queries, with the segment's first tile of keys (one row's stand in both halves)
          ok = __all_sync(~0u, wait(empty_q, (seg & 1) ^ 1, abort, &err));
          if (!ok) break;
          const int32_t h0 = at.kv * p.group + at.chunk * p.chunk_heads;
          const int32_t heads = min(p.chunk_heads, p.group - at.chunk * p.chunk_heads);
#pragma unroll 4
          for (int i = t; i < 128 * 16; i += kLoaders) {
            const int r = i / 16, y = i % 16, j = SPLIT ? 0 : r / kCols, h = r % kCols;
            const bool in = at.b[j] > at.a[j] && h < heads;
            const T* q = (const T*)p.q + (in ? (int64_t)(at.row0 + j) * p.q_row + (int64_t)(h0 + h) * p.q_head : 0);
            copy16(smem + kQueries + (y / 8) * kHalfTile + r * 128 + (((y & 7) ^ (r & 7)) << 4), q + y * 8, in ? 16u : 0u);
          }
          ++seg;
        }
        const char* base = (const char*)(cache + at.kv * s_head + x * 8);
        for (int32_t v = v0; v < v1; ++v) {
          at.visit(v, tile, rows);
          uint32_t from;   // where this lane's position lies, or ~0
          if constexpr (SLOTS) {
            const bool on = entry >= 0 && entry < p.num_pages * kPage;
            if (!on && entry != -1) bad = kErrInvalidPage;
            from = on ? (uint32_t)(entry / kPage) * page16 + (uint32_t)(entry % kPage) * slot16 : ~0u;
            if (v + 1 < v1) {
              ask(list, v + 1);
            } else if (goes_on()) {
              // the next unit's first: of this row, or of the next
              ask(list + (next_is_row() ? p.n_slots : 0), 0);
            }
          } else {
            int32_t lo = 0, hi = INT32_MAX;   // seen by every row of the visit
#pragma unroll
            for (int j = 0; j < NB; ++j)
              if (rows >> j & 1) lo = max(lo, at.a[j]), hi = min(hi, at.b[j]);
            const int32_t first = tile * kPos + quarter * 32;
            const bool any = first < hi && first + 32 > lo, there = entry >= 0 && entry < p.num_pages;
            if (any && !there) bad = kErrInvalidPage;
            const bool on = there && first + lane >= lo && first + lane < hi;
            from = on ? (uint32_t)entry * page16 + (uint32_t)((quarter & 1) * 32 + lane) * slot16 : ~0u;
            if (v + 1 < v1) {
              int32_t next_tile;
              uint32_t next_rows;
              at.visit(v + 1, next_tile, next_rows);
              ask(list, next_tile);
            }
          }
          const bool all = __all_sync(~0u, from != ~0u);
          const uint32_t slot = n % depth;
          ok = __all_sync(~0u, wait(values ? empty_v(slot) : empty_k(slot), (n / depth & 1) ^ 1, abort, &err));
          if (!ok) break;
          const uint32_t dst = ring + slot * kTileBytes + (x / 8) * kHalfTile + (uint32_t)quarter * (32 * 128);
          uint32_t to[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) to[i] = dst + (2 * i + r0) * 128 + (((x & 7) ^ (2 * i + r0)) << 4);
          if (all) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              copy16(to[i & 3] + (i >> 2) * 1024, base + (uint64_t)__shfl_sync(~0u, from, 2 * i + r0) * 16, 16u);
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint32_t o = __shfl_sync(~0u, from, 2 * i + r0);
              const bool in = o != ~0u;
              copy16(to[i & 3] + (i >> 2) * 1024, base + (uint64_t)(in ? o : 0u) * 16, in ? 16u : 0u);
            }
          }
          arrive_when_copied(values ? full_v(slot) : full_k(slot));
          ++n;
        }
        if (!ok) break;
        more = next_segment();
      }
      copy_wait_all();
      bad = __reduce_max_sync(~0u, bad);
      if (lane == 0 && bad != kOk) atomicMax(&err, bad);
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
      if (warp == 16) {
      // ----------------------------------------------------- scores' products ----
      constexpr uint32_t kQK = idesc_f16<BF16>(128, kPos, false);
      const uint64_t q = desc128(smem + kQueries, 16, 1024);
      uint32_t n = 0;
      bool ok = true, more = true;
      while (more) {
        const int32_t v1 = segment_end();
        for (int32_t v = at.s; v < v1; ++v, ++n) {
          const uint32_t slot = n % kRingK, b = n & 1;
          ok = __all_sync(~0u, wait(full_k(slot), n / kRingK & 1, abort, &err));
          ok = ok && __all_sync(~0u, wait(done_pv(b), (n >> 1 & 1) ^ 1, abort, &err));
          if (!ok) break;
          fence_proxy_async_smem();   // the copies' writes before the products' reads
          tc_fence_after();
          if (elect_one()) {
            const uint64_t k = desc128(smem + kKeys + slot * kTileBytes, 16, 1024);
#pragma unroll
            for (int i = 0; i < kHead / 16; ++i)   // 16 elements: 32 bytes of a row
              mma_ss(tmem + b * kPos, q + (i / 4) * (kHalfTile >> 4) + (i % 4) * 2, k + (i / 4) * (kHalfTile >> 4) + (i % 4) * 2,
                     kQK, i > 0);
            tc_commit(full_s(b));
            tc_commit(empty_k(slot));
          }
          __syncwarp();
        }
        if (!ok) break;
        if (elect_one()) tc_commit(empty_q);
        __syncwarp();
        more = next_segment();
      }
      } else if (warp == 17) {
      // ---------------------------------------------------- outputs' products ----
      constexpr uint32_t kPV = idesc_f16<BF16>(128, kHead, true);
      uint32_t n = 0;
      bool ok = true, more = true;
      while (more) {
        const int32_t v1 = segment_end();
        bool fresh[2] = {true, true};   // the accumulator is to be begun anew
        for (int32_t v = at.s; v < v1; ++v, ++n) {
          int32_t tile;
          uint32_t rows;
          at.visit(v, tile, rows);
          const uint32_t slot = n % kRingV, b = n & 1;
          const uint32_t to = !SPLIT && rows == 2 ? 1u : 0u;
          ok = __all_sync(~0u, wait(full_v(slot), n / kRingV & 1, abort, &err));
          ok = ok && __all_sync(~0u, wait(full_p(b), n >> 1 & 1, abort, &err));
          if (!ok) break;
          fence_proxy_async_smem();   // the copies' writes before the products' reads
          tc_fence_after();
          const bool anew = to ? fresh[1] : fresh[0];
          // 16 positions a product: 8 columns of weights, 2048 bytes of values
          if (elect_one()) {
            const uint64_t val = desc128(smem + kValues + slot * kTileBytes, kHalfTile, 1024);
#pragma unroll
            for (int i = 0; i < kPos / 16; ++i) {
              const uint32_t out = tmem + kOut + (SPLIT ? i / 4 : to) * kHead;
              mma_ts(out, tmem + b * kPos + i * 8, val + i * (2048 >> 4), kPV, !anew || (SPLIT ? i % 4 : i) > 0);
            }
            tc_commit(done_pv(b));
            tc_commit(empty_v(slot));
          }
          __syncwarp();
          if (to) fresh[1] = false; else fresh[0] = false;
        }
        if (!ok) break;
        more = next_segment();
      }
      }
    }
  }

  // rows that see nothing
  if constexpr (!SLOTS) {
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < p.rows * (int64_t)p.q_heads;
         i += (int64_t)gridDim.x * kThreads) {
      const int32_t r = (int32_t)(i / p.q_heads), h = (int32_t)(i - (int64_t)r * p.q_heads);
      if (p.row_end[r] > p.row_start[r]) continue;
      uint4* o = (uint4*)((T*)p.out + r * p.out_row + h * p.out_head);
      for (int k = 0; k < kHead / 8; ++k) o[k] = make_uint4(0, 0, 0, 0);
      if (p.lse) p.lse[i] = kNegInf;
      if (p.row_stat) p.row_stat[i] = make_float2(0.f, 0.f);
    }
  }
  // the products in flight end before the tensor memory is given back
  if (warp == 16 || warp == 17) {
    __syncwarp();
    if (elect_one()) tc_commit(drain);
    __syncwarp();
    for (uint32_t i = 0; i < 1u << 20; ++i)
      if (mbar_try_wait(drain, 0)) break;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0) p.cta_status[blockIdx.x] = err;
  if (warp == 16) tmem_dealloc(tmem, kTmemCols);
}

template <bool BF16, int NB, bool SLOTS>
cudaError_t launch(const AttnParams& p, int sm_count, cudaStream_t stream) {
  auto* kernel = attn_tc_kernel<BF16, NB, SLOTS>;
  static std::atomic<bool> done[64];
  cudaError_t e = set_smem_once(kernel, kSmemBytes, done);
  if (e != cudaSuccess) return e;
  kernel<<<sm_count, kThreads, kSmemBytes, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace tc
}  // namespace attn
}  // namespace idxk
