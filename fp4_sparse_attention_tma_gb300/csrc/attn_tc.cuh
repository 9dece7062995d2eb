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
#include "attn_fp4.cuh"
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
// The shared memory: tiles of keys and of values, the queries, room to pass sums between the halves, and (4 bits) each
// copying warp's codes and scales on their way.
template <bool FP4>
struct Memory {
  static constexpr int kRingK = FP4 ? 2 : 3, kRingV = 2;
  static constexpr uint32_t kKeys = 0, kValues = kKeys + kRingK * kTileBytes, kQueries = kValues + kRingV * kTileBytes,
                            kStage = kQueries + kTileBytes;
  static constexpr int kStageCols = 16, kStageRow = kStageCols + 1;   // floats
  static constexpr uint32_t kRaw = kStage + 4 * kCols * kStageRow * 4;
  static constexpr uint32_t kRawDepth = 2, kRawStage = 2048 + 128;   // codes and scales of 32 positions
  static constexpr int kBytes = (int)(kRaw + (FP4 ? 8 * kRawDepth * kRawStage : 0)) + 1024;   // the base is aligned to 1024 by hand
};

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
// 16 columns; one or two such loads waited for.
__device__ __forceinline__ void tmem_ld16(uint32_t a, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(a));
}
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&r)[16], uint32_t (&s)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(s[0]),
                 "+r"(s[1]), "+r"(s[2]), "+r"(s[3]), "+r"(s[4]), "+r"(s[5]), "+r"(s[6]), "+r"(s[7]), "+r"(s[8]),
                 "+r"(s[9]), "+r"(s[10]), "+r"(s[11]), "+r"(s[12]), "+r"(s[13]), "+r"(s[14]), "+r"(s[15])
               :
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
    if (++kv < p.kv_units) return;
    kv = 0;
    do {
      load(p, rows, row0 + nrows);
    } while (nsub == 0);
  }
  // Visit v of the unit: its tile and its rows (bit j); with it `run` - 1 more visits have the tiles that follow, and the
  // same rows.
  __device__ void visit(int32_t v, int32_t& tile, uint32_t& rows) const {
    int32_t run;
    visit(v, tile, rows, run);
  }
  __device__ void visit(int32_t v, int32_t& tile, uint32_t& rows, int32_t& run) const {
    run = INT32_MAX;
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
          run = v < front ? front - v : front + back - v;
          return;
        }
        v -= front + back;
        if (j == 0) {
          if (v < c1 - c0) {
            tile = c0 + v;
            rows = 3;
            run = c1 - c0 - v;
            return;
          }
          v -= c1 - c0;
        }
      }
      tile = 0;   // (not reached)
    }
  }
};

// A unit's visits one after another.
template <int NB, bool SLOTS>
struct Steps {
  int32_t tile, run;
  uint32_t rows;
  __device__ void start(const Walk<NB, SLOTS>& at, int32_t v) { at.visit(v, tile, rows, run); }
  __device__ void next(const Walk<NB, SLOTS>& at, int32_t v) {   // from visit v - 1 to v
    if (NB == 1 || --run > 0)
      ++tile;
    else
      at.visit(v, tile, rows, run);
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

template <bool BF16, int NB, bool SLOTS, bool FP4>
__global__ void __launch_bounds__(kThreads, 1) attn_tc_kernel(const __grid_constant__ AttnParams p) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr bool MB = BF16 && !FP4;         // the matrices' type: bf16, or fp16
  using M = Memory<FP4>;
  constexpr int kRingK = M::kRingK, kRingV = M::kRingV;
  constexpr uint32_t kKeys = M::kKeys, kValues = M::kValues, kQueries = M::kQueries;
  constexpr bool SPLIT = NB == 1;           // one row: either half of the matrix takes half of a tile's positions
  constexpr int kSoft = 256;                // softmax threads

  extern __shared__ __align__(16) unsigned char raw[];
  __shared__ uint32_t err, tmem_base;
  __shared__ int abort_flag;
  __shared__ __align__(8) uint64_t bars[2 * kRingK + 2 * kRingV + 1 + 3 * 2 + 2];
  __shared__ float2 half_ml[2][kCols];      // (one row) reference and sum of either half, -1 where nothing was seen
  __shared__ float row_max[2][2][128];      // by visit and warpgroup
  __shared__ float row_sum[2][128];         // by warpgroup, -1 where nothing was seen
  // (4 bits) what the queries were divided by, by segment, and the references of keys and values by visit and quarter
  // of the tile: the copies run no more than so far ahead of the softmax
  constexpr int kAhead = FP4 ? 8 : 1;
  __shared__ float q_unit[FP4 ? 4 : 1][128];
  __shared__ __align__(16) int32_t refs[kAhead][2][4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t smem = (smem_addr(raw) + 1023u) & ~1023u;
  const uint32_t bar0 = smem_addr(bars);
  auto full_k = [&](uint32_t i) { return bar0 + 8 * i; };
  auto empty_k = [&](uint32_t i) { return bar0 + 8 * (kRingK + i); };
  auto full_v = [&](uint32_t i) { return bar0 + 8 * (2 * kRingK + i); };
  auto empty_v = [&](uint32_t i) { return bar0 + 8 * (2 * kRingK + kRingV + i); };
  constexpr uint32_t kRest = 2 * kRingK + 2 * kRingV;
  const uint32_t empty_q = bar0 + 8 * kRest, drain = bar0 + 8 * (kRest + 7), full_q = bar0 + 8 * (kRest + 8);
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
    mbar_init(full_q, 64);
    for (int b = 0; b < 2; ++b) mbar_init(full_s(b), FP4 ? 2 : 1), mbar_init(full_p(b), kSoft), mbar_init(done_pv(b), 1);
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
  __shared__ Place asking[FP4 ? 8 : 1];   // (4 bits) of the copying warps: what they copy, ahead
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
      uint32_t n = 0, seg = 0;       // visits, segments so far
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
        int32_t o_ref = (int32_t)fp4::kLowest;   // (4 bits) the weighted values' reference
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
              if constexpr (!SLOTS && !FP4) {
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
            // (4 bits) a chunk's scores are in units of its keys' reference and the head's queries: powers of two, never 0
            float unit[CH];
            int32_t v_ref[CH], new_ref = o_ref;
            if constexpr (FP4) {
              // the values' references are there with the values (whose next tile waits for this visit's weights)
              ok &= wait(full_v(n % kRingV), n / kRingV & 1, abort, &err);
              const float qu = q_unit[seg & 3][x];
              const int4 all = *(const int4*)refs[n % kAhead][1];
              new_ref = max(max(max(all.x, all.y), max(all.z, all.w)), o_ref);
              float best = kNegInf;
#pragma unroll
              for (int k = 0; k < CH; ++k) {
                unit[k] = fmaxf(fminf(fp4::pow2_of(refs[n % kAhead][0][c0 + k] - 12) * qu, 0x1p127f), 0x1p-126f);
                v_ref[k] = refs[n % kAhead][1][c0 + k];
                top = kNegInf, top2 = kNegInf;
                look(k, r[k]);
                best = fmaxf(best, fmaxf(top, top2) * unit[k]);
              }
              top = best, top2 = kNegInf;
            } else {
#pragma unroll
              for (int k = 0; k < CH; ++k) look(k, r[k]);
            }
            // of the whole row: the other warpgroup's thread has seen the other positions
            top = fmaxf(top, top2);
            row_max[b][g][x] = top;
            bar_sync(pair, 64);
            top = fmaxf(top, row_max[b][g ^ 1][x]);
            // does its weights' reference have to follow?
            if (__any_sync(~0u, exponent(top, ref, p.scale_log2) > kRaise<MB> || new_ref != o_ref)) {   // (false where both are -infinity)
              const float raised = fmaxf(ref, top);
              float f = raised == ref ? 1.f : ex2(exponent(ref, raised, p.scale_log2));
              ref = raised;
#pragma unroll
              for (int i = 0; i < 4; ++i) sum[i] *= f;
              if constexpr (FP4) f *= fp4::pow2_of(127 + o_ref - new_ref), o_ref = new_ref;
              if (had_a || had_b) {
                ok &= wait(done_pv(b ^ 1), (n - 1) >> 1 & 1, abort, &err);   // the last visit that added to them
                tc_fence_after();
                // a half of the columns each
                if constexpr (FP4 && SPLIT) {
                  // 16 at a time: a unit of 1024 slots has 8 visits, and the reference follows in most of them.
                  // 8192 rows of 1024 slots: 633 us, with 8 at a time 736, with 32 (which spills) 719.
                  const Two ff = two(f, f);
#pragma unroll 1
                  for (int y = 0; y < 64; y += 16) {
                    uint32_t a[16];
                    tmem_ld16(out_a + g * 64 + y, a);
                    tmem_wait_ld16(a);
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                      const float2 c = both(mul2(two(__uint_as_float(a[i]), __uint_as_float(a[i + 1])), ff));
                      a[i] = __float_as_uint(c.x), a[i + 1] = __float_as_uint(c.y);
                    }
                    tmem_st16(out_a + g * 64 + y, a);
                  }
                } else
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
              if constexpr (FP4) {
                // the weights count in the chunk's values' reference, their sum does not (values 2^-40 below the largest are
                // taken for 2^-40 of it)
                const int32_t down = max(v_ref[k] - o_ref, -40);
                Two part[2] = {two(0.f, 0.f), two(0.f, 0.f)};
                const float up = kShift<MB> + (float)down;
                const Two shift = two(up, up), uu = two(unit[k], unit[k]), minus = two(base, base), cc = two(p.scale_log2, p.scale_log2);
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                  const float2 d = both(fma2(fma2(two(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), uu, minus), cc, shift));
                  const float e0 = ex2(d.x), e1 = ex2(d.y);
                  part[i / 2 & 1] = idxk::add2(part[i / 2 & 1], two(e0, e1));
                  w[i / 2] = pack2<MB>(e0, e1);
                }
                const float2 all = both(idxk::add2(part[0], part[1]));
                const float back = fp4::pow2_of(127 - down);
                sum[0] = fmaf(all.x, back, sum[0]), sum[1] = fmaf(all.y, back, sum[1]);
              } else {
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                  float d0 = __uint_as_float(r[i]), d1 = __uint_as_float(r[i + 1]);
                  exponent2(d0, d1, base, p.scale_log2, kShift<BF16>);
                  const float e0 = ex2(d0), e1 = ex2(d1);
                  add2(sum[i & 2], sum[(i & 2) + 1], e0, e1);
                  w[i / 2] = pack2<BF16>(e0, e1);
                }
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
        ++seg;
        // the last visit of each tile of scores that this segment (or one before it) had
        auto last_products = [&]() {
          if (n > 0) ok &= wait(done_pv((n - 1) & 1), (n - 1) >> 1 & 1, abort, &err);
          if (n > 1) ok &= wait(done_pv(n & 1), (n - 2) >> 1 & 1, abort, &err);
          tc_fence_after();
        };
        if constexpr (!FP4) last_products();
        float l = (sum[0] + sum[1]) + (sum[2] + sum[3]);
        if constexpr (FP4) l *= kShiftUp<BF16> / kShiftUp<MB>;   // to the shift that the join expects
        // of the whole row
        row_sum[g][x] = (had_a || had_b) && (!SLOTS || seen) ? l : -1.f;
        bar_sync(pair, 64);
        const float l0 = row_sum[0][x], l1 = row_sum[1][x];
        const bool has = l0 != -1.f || l1 != -1.f;
        l = (l0 != -1.f ? l0 : 0.f) + (l1 != -1.f ? l1 : 0.f);
        if (SPLIT && g == 0) half_ml[part_of][x & (kCols - 1)] = make_float2(ref, has ? l : -1.f);
        // every softmax thread votes on the waits so far, so that all leave together
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
        if constexpr (FP4) f *= fp4::pow2_of(o_ref - 12) * (kShiftUp<BF16> / kShiftUp<MB>);
        T* out = (T*)p.out + row * p.out_row + (int64_t)qh * p.out_head;
        float* po = p.part_o + part * kHead;
        auto emit = [&](int c, const float (&z)[8]) {   // 8 columns of the thread's row
          if (!live || !ok) return;
          if (whole) {
            uint4 u;
            u.x = pack2<BF16>(z[0], z[1]), u.y = pack2<BF16>(z[2], z[3]);
            u.z = pack2<BF16>(z[4], z[5]), u.w = pack2<BF16>(z[6], z[7]);
            *(uint4*)(out + c) = u;
          } else if (any) {
            store32(po + c, z);
          }
        };
        // (4 bits) all of this beside the last products, and on to the next segment: `at` is its from here on.  8192 rows of
        // 1024 slots 629 -> 616 us, 32 requests x 2 rows of 64 heads on 1 120 -> 117; in 16 bits 529 -> 537
        if constexpr (FP4) more = next_segment(), last_products();
        if constexpr (SPLIT) {
          // each half finishes 64 columns, 32 a thread; the other half's share of them comes through shared
          // memory, some at a time
          constexpr int kSome = M::kStageCols;
          float* stage = (float*)(raw + (smem - smem_addr(raw)) + M::kStage);
          float* give = stage + ((part_of * 2 + g) * kCols + col) * M::kStageRow;
          const float* take = stage + (((part_of ^ 1) * 2 + g) * kCols + col) * M::kStageRow;
          if constexpr (FP4) {
#pragma unroll 1
            for (int at_col = 0; at_col < 32; at_col += kSome) {
              uint32_t theirs[16], ours[16];
              static_assert(kSome == 16, "columns of a round");
              tmem_ld16(out_a + (part_of ^ 1) * 64 + g * 32 + at_col, theirs);
              tmem_ld16(out_a + part_of * 64 + g * 32 + at_col, ours);
              tmem_wait_ld16(theirs, ours);
#pragma unroll
              for (int c = 0; c < kSome; ++c) give[c] = has ? __uint_as_float(theirs[c]) * f : 0.f;
              bar_sync(kAll, kSoft);
#pragma unroll
              for (int c = 0; c < kSome; c += 8) {
                float r[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) r[i] = (has ? __uint_as_float(ours[c + i]) * f : 0.f) + take[c + i];
                emit((int)part_of * 64 + g * 32 + at_col + c, r);
              }
              bar_sync(kAll, kSoft);
            }
          } else
#pragma unroll 1
          for (int at_col = 0; at_col < 32; at_col += kSome) {
#pragma unroll 1
            for (int c = 0; c < kSome; c += 8) {
              float r[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
              if (has) tmem_load8(out_a + (part_of ^ 1) * 64 + g * 32 + at_col + c, r);
#pragma unroll
              for (int i = 0; i < 8; ++i) give[c + i] = has ? r[i] * f : 0.f;
            }
            bar_sync(kAll, kSoft);
#pragma unroll 1
            for (int c = 0; c < kSome; c += 8) {
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
        if constexpr (!FP4) more = next_segment();
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
      constexpr int64_t kPiece = FP4 ? 16 : 8;   // elements, or bytes of codes
      const uint32_t page16 = (uint32_t)(s_page / kPiece), slot16 = (uint32_t)(s_slot / kPiece);
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
      if constexpr (SLOTS && !FP4) ask(p.slots + (int64_t)at.row0 * p.n_slots, at.s);
      bool more = true;
      if constexpr (FP4) {
        // Codes are unpacked on their way: 32 positions a warp, a lane 32 elements (a block) of one of 8 positions at a
        // time.  Each warp copies its positions' codes and scales into a small ring of its own, two visits ahead, over the
        // ends of segments, and unpacks them, times their scales over the largest of the 32 positions (attn_fp4.cuh), into
        // the tile, and publish the reference beside it.  Positions that the rows do not see have the scale 0 and the
        // codes of some other position: their scores are not used and their weights are 0.
        const uint8_t* codes = (const uint8_t*)cache;
        const int block = lane >> 3, in8 = lane & 7;
        const uint32_t scale_page = (uint32_t)(values ? p.vs_page : p.ks_page), scale_slot = (uint32_t)(values ? p.vs_slot : p.ks_slot);
        constexpr uint32_t kRaw = M::kRaw, kRawDepth = M::kRawDepth, kRawStage = M::kRawStage;
        const uint32_t mine = smem + kRaw + (uint32_t)(warp - 8) * (kRawDepth * kRawStage);
        uint32_t to[4];                    // places of a block's four 16-byte pieces, in a tile
#pragma unroll
        for (int y = 0; y < 4; ++y)
          to[y] = (uint32_t)(block >> 1) * kHalfTile + (uint32_t)(quarter * 32 + in8) * 128 +
                  ((uint32_t)(((block & 1) * 4 + y) ^ in8) << 4);
        // position i * 8 + r of the ring: 64 bytes, pieces swizzled so that 8 positions' same piece meets no bank twice
        const uint32_t copy_to = (uint32_t)(lane >> 2) * 64 + (((uint32_t)lane ^ (uint32_t)(lane >> 3)) & 3u) * 16;
        const uint32_t take_from = (uint32_t)in8 * 64 + (uint32_t)(block ^ (in8 >> 1)) * 16;
        // ---- copies: a walk of their own, ahead of the unpacking ----
        Place& ask_at = asking[warp - 8];
        if (lane == 0) ask_at = places[warp];
        __syncwarp();
        Steps<NB, SLOTS> ahead;            // the visit whose entry is asked for
        int32_t ask_v, ask_left;           // its number in its segment, and the visits from it to the end; 0: all done
        const int32_t* list;
        const uint8_t *base, *scale_head;  // of the head
        auto begin_asking = [&]() {
          const Walk<NB, SLOTS>& f = ask_at.at;
          ask_v = f.s;
          ask_left = (int32_t)min((int64_t)f.nsub, ask_at.end) - f.s;
          base = codes + f.kv * s_head + (lane & 3) * 16;
          scale_head = values ? p.v_scale + f.kv * p.vs_head : p.k_scale + f.kv * p.ks_head;
          if constexpr (SLOTS) {
            list = p.slots + (int64_t)f.row0 * p.n_slots;
            if (warp == 12 && f.row0 + 1 < p.rows)
              for (int32_t i = lane * 32; i < p.n_slots; i += 32 * 32)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(list + p.n_slots + i));
          } else {
            list = p.page_table + (int64_t)f.req * p.max_pages;
          }
          ahead.start(f, ask_v);
          ask(list, ahead.tile);
        };
        begin_asking();
        // the visit whose entry is there, into stage x of the ring; on to the next entry
        auto fetch = [&](uint32_t x) {
          if (ask_left > 0) {
            bool on;
            uint32_t page, off;
            if constexpr (SLOTS) {
              on = entry >= 0 && entry < p.num_pages * kPage;
              if (!on && entry != -1) bad = max(bad, (uint32_t)kErrInvalidPage);
              page = (uint32_t)entry / kPage, off = (uint32_t)entry % kPage;
            } else {
              int32_t lo = 0, hi = INT32_MAX;   // seen by every row of the visit
              const int32_t first = ahead.tile * kPos + quarter * 32;
              if (NB == 1 || ahead.rows != 3) {
#pragma unroll
                for (int j = 0; j < NB; ++j)
                  if (ahead.rows >> j & 1) lo = max(lo, ask_at.at.a[j]), hi = min(hi, ask_at.at.b[j]);
              }
              const bool any = first < hi && first + 32 > lo, there = entry >= 0 && entry < p.num_pages;
              if (any && !there) bad = max(bad, (uint32_t)kErrInvalidPage);
              on = there && first + lane >= lo && first + lane < hi;
              page = (uint32_t)entry, off = (uint32_t)((quarter & 1) * 32 + lane);
            }
            const uint32_t dst = mine + x * kRawStage, from = on ? page * page16 + off * slot16 : 0u;
            copy4(dst + 2048 + lane * 4, scale_head + (on ? page * scale_page + off * scale_slot : 0u), on ? 4u : 0u);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              copy16(dst + copy_to + i * 512, base + (uint64_t)__shfl_sync(~0u, from, i * 8 + (lane >> 2)) * 16, 16u);
            if (--ask_left > 0) {
              ahead.next(ask_at.at, ++ask_v);
              ask(list, ahead.tile);
            } else {
              __syncwarp();
              const int64_t rest = ask_at.end - ask_at.at.nsub - kUnitCost;
              __syncwarp();
              if (lane == 0) {
                ask_at.end = rest;
                if (rest > 0) ask_at.at.next_unit(p, meta);
              }
              __syncwarp();
              if (rest > 0) begin_asking();
            }
          }
          copy_commit();
        };
#pragma unroll
        for (uint32_t x = 0; x < kRawDepth; ++x) fetch(x);
        // ---- unpacking ----
        while (more) {
          const int32_t v1 = segment_end();
          for (int32_t v = at.s; v < v1; ++v) {
            copy_wait<kRawDepth - 1>();
            __syncwarp();
            const uint32_t x = n % kRawDepth, src = mine + x * kRawStage;
            const uint32_t scales = fp4::lds32(src + 2048 + lane * 4);
            const uint32_t ref = max(__reduce_max_sync(~0u, fp4::largest_of(scales)), fp4::kLowest);
            if (ref > kMaxScaleByte) bad = max(bad, (uint32_t)kErrInvalidValue);
            const uint32_t slot = n % depth;
            ok = __all_sync(~0u, wait(values ? empty_v(slot) : empty_k(slot), (n / depth & 1) ^ 1, abort, &err));
            if (!ok) break;
            if (lane == 0) refs[n % kAhead][values][quarter] = (int32_t)ref;
            const uint32_t dst = ring + slot * kTileBytes;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint4 u = fp4::lds128(src + take_from + i * 512);
              const uint32_t fac = fp4::factor2(__shfl_sync(~0u, scales, i * 8 + in8) >> (8 * block) & 255u, ref);
              const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                uint32_t h[4];
                from_codes(w[y], h);
                fp4::sts128(dst + to[y] + i * 1024,
                            make_uint4(fp4::hmul2(h[0], fac), fp4::hmul2(h[1], fac), fp4::hmul2(h[2], fac), fp4::hmul2(h[3], fac)));
              }
            }
            // (the issuing warp orders these writes before the products' reads, as it does the copies')
            mbar_arrive(values ? full_v(slot) : full_k(slot));
            __syncwarp();   // every lane has read the stage
            fetch(x);
            ++n;
          }
          if (!ok) break;
          more = next_segment();
        }
      } else
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
      constexpr uint32_t kQK = idesc_f16<MB>(128, kPos, false);
      const uint64_t q = desc128(smem + kQueries, 16, 1024);
      uint32_t n = 0, seg = 0;
      bool ok = true, more = true;
      while (more) {
        const int32_t v1 = segment_end();
        if constexpr (FP4) {
          ok = __all_sync(~0u, wait(full_q, seg++ & 1, abort, &err));
          if (!ok) break;
        }
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
            // (4 bits) what the copying warps left beside the tile reaches the softmax by this arrival
            if constexpr (FP4) mbar_arrive(full_s(b));
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
      constexpr uint32_t kPV = idesc_f16<MB>(128, kHead, true);
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
      } else if constexpr (FP4) {
      // ------------------------------------- queries, a segment ahead of the products ----
      // 16 lanes a row, brought to fp16's range; one row's stand in both halves
      // (converted before the tile is free; q_unit's place of this segment was read four segments ago, by a visit whose
      // products are done, as those of the segment before the last are)
      constexpr int kQRows = SPLIT ? kCols : 128, U = 8;
      const int t = threadIdx.x & 63;
      uint32_t seg = 0;
      bool ok = true, more = true;
      while (more) {
        const int32_t h0 = at.kv * p.group + at.chunk * p.chunk_heads;
        const int32_t heads = min(p.chunk_heads, p.group - at.chunk * p.chunk_heads);
        // piece y of rows r0 + 4 x, a batch of U of them
#pragma unroll 1
        for (int r0 = t / 16; r0 < kQRows; r0 += 4 * U) {
          const int y = t % 16, j = SPLIT ? 0 : r0 / kCols;
          const T* src = (const T*)p.q + (int64_t)(at.row0 + j) * p.q_row + (int64_t)(h0 + r0 % kCols) * p.q_head + y * 8;
          const int some = at.b[j] > at.a[j] ? heads - r0 % kCols : 0;
          uint4 u[U];
#pragma unroll
          for (int x = 0; x < U; ++x, src += 4 * p.q_head) u[x] = 4 * x < some ? *(const uint4*)src : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int x = 0; x < U; ++x) {
            float by_unit = 1.f;
            if constexpr (BF16) fp4::to_f16(u[x], by_unit);
            if (y == 0) {
              q_unit[seg & 3][r0 + 4 * x] = by_unit;
              if (SPLIT) q_unit[seg & 3][kCols + r0 + 4 * x] = by_unit;
            }
          }
          if (r0 < 4) ok = __all_sync(~0u, wait(empty_q, (seg & 1) ^ 1, abort, &err));
          if (!ok) break;
          // (r0 is less than 4 over a multiple of 8: 4 x shows in a row's third bit alone)
          const uint32_t dst = smem + kQueries + (y / 8) * kHalfTile + r0 * 128 + (((y & 7) ^ (r0 & 7)) << 4);
#pragma unroll
          for (int x = 0; x < U; ++x) {
            const uint32_t to = (dst ^ (x % 2 * 64)) + x * 512;
            fp4::sts128(to, u[x]);
            if (SPLIT) fp4::sts128(to + kCols * 128, u[x]);
          }
        }
        if (!ok) break;
        mbar_arrive(full_q);
        ++seg;
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

template <bool BF16, int NB, bool SLOTS, bool FP4>
cudaError_t launch(const AttnParams& p, int sm_count, cudaStream_t stream) {
  auto* kernel = attn_tc_kernel<BF16, NB, SLOTS, FP4>;
  static std::atomic<bool> done[64];
  cudaError_t e = set_smem_once(kernel, Memory<FP4>::kBytes, done);
  if (e != cudaSuccess) return e;
  kernel<<<sm_count, kThreads, Memory<FP4>::kBytes, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace tc
}  // namespace attn
}  // namespace idxk
