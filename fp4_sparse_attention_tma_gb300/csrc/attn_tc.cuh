// The attention kernel for many query heads on one key-value head (17 to 64 a chunk,
// head dimension 128), on the fifth-generation tensor cores.
//
// With that many heads the products, not the copies, bound warps that load every key and
// value once per 16 heads.  Here one CTA takes a tile of 128 positions for all 64 columns
// (query heads) of a row, in the transposed form, in which nothing is padded:
//
//   S^T [128 positions x 64] = K Q^T          (keys K-major, queries K-major)
//   O^T [128 (the head dimension) x 64] += V^T P^T   (both operands MN-major: the values as
//                                              they lie in the cache, P^T as a thread writes it)
//
// A tensor memory lane is a position in the first product and an output column in the second.
// A thread owns one position: its sums of 2^(s - m) stay in registers and are added up over
// the lanes once, at the segment's end.  The reference m of a column is not its running
// maximum: the segment's first tile sets it (to the tile's maximum; in bf16, whose range allows
// it, to the score of the first position), and a tile raises it when a weight would exceed
// 2^kRaise.  Only then are the sums and the accumulator in tensor memory scaled.  Columns are 64 a row; with two rows of one request both use the tiles
// that both see in full, and the tiles at the windows' edges are visited row by row, so that
// what one row does not see is zero for it.
//
// Roles: two warpgroups of softmax (for one row 32 columns each, for two a row each), two
// warps that copy keys (and the queries), two that copy values (16-byte asynchronous copies
// into the 128-byte swizzle, any stride, page or slot), one warp that issues the scores'
// products and one the outputs'.  Every wait is bounded.
#pragma once

#include "attn_common.cuh"
#include "idx_device.cuh"

namespace idxk {
namespace attn {
namespace tc {

constexpr int kPos = 128;                 // positions of a tile
constexpr int kCols = 64;                 // columns of a row
constexpr int kHead = 128;                // head dimension
constexpr uint32_t kHalfTile = kPos * 128;      // 64 of the dimension's elements of 128 positions
constexpr uint32_t kTileBytes = 2 * kHalfTile;  // a tile of keys or of values
constexpr uint32_t kQHalf = kCols * 128;
constexpr uint32_t kQBytes = 2 * kQHalf;        // a row's queries
constexpr uint32_t kPBytes = kPos * 128;        // a row's weights
constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kLoaders = 64;              // threads that copy keys (and as many values)
// A column's reference is raised when a weight exceeds 2^kRaise: fp16 weights have to stay
// below 2^16, bf16 ones far enough below the largest value for their product with any value.
template <bool BF16>
constexpr float kRaise = BF16 ? 16.f : 8.f;

template <int NB>
struct Smem {
  static constexpr int kRingK = NB == 1 ? 3 : 2;
  static constexpr int kRingV = 2;
  static constexpr int kQ = NB == 1 ? 2 : 1;
  static constexpr uint32_t k = 0;
  static constexpr uint32_t v = k + kRingK * kTileBytes;
  static constexpr uint32_t q = v + kRingV * kTileBytes;
  static constexpr uint32_t p = q + kQ * NB * kQBytes;
  static constexpr uint32_t total = p + NB * kPBytes;
  static constexpr int bytes = (int)total + 1024;   // the base is aligned to 1024 by hand
};

__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
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

// Instruction descriptor, kind::f16 with fp32 accumulation; `mn` : both operands MN-major.
template <bool BF16>
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t M, uint32_t N, bool mn) {
  return (1u << 4) | ((BF16 ? 1u : 0u) << 7) | ((BF16 ? 1u : 0u) << 10) | ((mn ? 1u : 0u) << 15) |
         ((mn ? 1u : 0u) << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
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
    return visits(a, b, c0, c1);
  }
  __device__ static int32_t row_count(const AttnParams& p) { return hi(p.n_slots); }

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
      int32_t x = v;
      const bool both = c1 > c0;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int32_t n = (both ? c0 : hi(b[j])) - lo(a[j]);
        if (x < n) {
          tile = lo(a[j]) + x;
          rows = 1u << j;
          return;
        }
        x -= n;
      }
      if (x < c1 - c0) {
        tile = c0 + x;
        rows = 3;
        return;
      }
      x -= c1 - c0;
      const int32_t n = hi(b[0]) - c1;
      rows = x < n ? 1u : 2u;
      tile = c1 + (x < n ? x : x - n);
    }
  }
};

// Lane i of the result: the sum (or maximum) over the lanes of x[i].  x is used up.
template <bool MAX>
__device__ __forceinline__ float over_lanes(float (&x)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 16; n; n >>= 1) {
    const bool up = lane & n;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = up ? x[i] : x[i + n];
      const float keep = up ? x[i + n] : x[i];
      const float got = __shfl_xor_sync(~0u, give, n);
      x[i] = MAX ? fmaxf(keep, got) : keep + got;
    }
  }
  return x[0];
}

// Two fp32 operations in one instruction, and a maximum of three.
__device__ __forceinline__ void fma2(float& x, float& y, float a, float bx, float by) {
  asm("{\n\t.reg .b64 v, m, s;\n\t"
      "mov.b64 v, {%0, %1};\n\tmov.b64 m, {%2, %2};\n\tmov.b64 s, {%3, %4};\n\t"
      "fma.rn.f32x2 v, v, m, s;\n\tmov.b64 {%0, %1}, v;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(bx), "f"(by));
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
  using L = Smem<NB>;
  constexpr int kSoft = NB == 1 ? 256 : 128;      // softmax threads of a row
  constexpr int kMine = NB == 1 ? 32 : 64;        // columns of a softmax thread
  constexpr uint32_t kTmemCols = NB == 1 ? 256 : 512;
  constexpr uint32_t kO = NB * 128;               // first column of the outputs

  extern __shared__ unsigned char raw[];
  __shared__ uint32_t err, tmem_base;
  __shared__ int abort_flag;
  __shared__ __align__(8) uint64_t bars[2 * L::kRingK + 2 * L::kRingV + L::kQ + NB * 6 + 1];
  __shared__ __align__(16) float ref[2][kMine];    // columns' references, negated, in units of log2
  __shared__ __align__(16) float raise[2][32];     // what they were raised by
  __shared__ __align__(16) float red[2][4][32];
  __shared__ uint32_t valid[2][4];                 // lanes whose position is one
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t smem = (smem_addr(raw) + 1023u) & ~1023u;
  const uint32_t bar0 = smem_addr(bars);
  auto full_k = [&](uint32_t i) { return bar0 + 8 * i; };
  auto empty_k = [&](uint32_t i) { return bar0 + 8 * (L::kRingK + i); };
  auto full_v = [&](uint32_t i) { return bar0 + 8 * (2 * L::kRingK + i); };
  auto empty_v = [&](uint32_t i) { return bar0 + 8 * (2 * L::kRingK + L::kRingV + i); };
  auto empty_q = [&](uint32_t i) { return bar0 + 8 * (2 * L::kRingK + 2 * L::kRingV + i); };
  constexpr uint32_t kRow = 2 * L::kRingK + 2 * L::kRingV + L::kQ;
  auto full_s = [&](uint32_t j, uint32_t i) { return bar0 + 8 * (kRow + j * 6 + i); };
  auto empty_s = [&](uint32_t j, uint32_t i) { return bar0 + 8 * (kRow + j * 6 + 2 + i); };
  auto full_p = [&](uint32_t j) { return bar0 + 8 * (kRow + j * 6 + 4); };
  auto done_pv = [&](uint32_t j) { return bar0 + 8 * (kRow + j * 6 + 5); };
  const uint32_t drain = bar0 + 8 * (kRow + NB * 6);

  allow_launch_after();
  if (threadIdx.x == 0) {
    err = kOk;
    abort_flag = 0;
    for (int i = 0; i < L::kRingK; ++i) mbar_init(full_k(i), kLoaders), mbar_init(empty_k(i), 1);
    for (int i = 0; i < L::kRingV; ++i) mbar_init(full_v(i), kLoaders), mbar_init(empty_v(i), 1);
    for (int i = 0; i < L::kQ; ++i) mbar_init(empty_q(i), 1);
    for (int j = 0; j < NB; ++j) {
      for (int i = 0; i < 2; ++i) mbar_init(full_s(j, i), 1), mbar_init(empty_s(j, i), kSoft);
      mbar_init(full_p(j), kSoft);
      mbar_init(done_pv(j), 1);
    }
    mbar_init(drain, 2);
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(smem_addr(&tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  volatile int* abort = &abort_flag;

  Split sp;
  Walk<NB, SLOTS> at;
  Rows meta{};
  const bool work = find_range<Walk<NB, SLOTS>, SLOTS, kWarps>(p, meta, sp, at, blockIdx.x, &err);
  if (threadIdx.x == 0) {
    if (work) p.open_row[blockIdx.x] = -1;
    if (blockIdx.x == 0) *p.active = sp.active;
  }
  if (work) {
    // A role walks over its segments (the part of a unit in the CTA's range) and a segment's visits.
    int64_t here = sp.first(blockIdx.x);                  // flat index of the segment's first visit
    const int64_t stop = sp.first(blockIdx.x + 1);
    // registers: 512 threads are launched with 128 each; two warpgroups of 152 and two of 104 are as many
    if (warp < 8) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
      // ------------------------------------------------------------ softmax ----
      const int wg = warp >> 2, x = threadIdx.x & 127;      // warpgroup, tensor memory lane
      const uint32_t bar_id = 1 + wg;
      const uint32_t j = NB == 1 ? 0 : wg;                  // row of the group
      const uint32_t col0 = NB == 1 ? wg * 32 : 0;          // first column
      const uint32_t lanes = (uint32_t)(warp & 3) << 21;    // this warp's 32 lanes
      const uint32_t p_row = smem + L::p + j * kPBytes + (uint32_t)x * 128;
      const float c = p.scale_log2;
      float sum[kMine];
      float mine_ref[kMine / 32];    // lane i: the reference of column 32 h + i, -inf if unset
      bool unset[kMine / 32];
      uint32_t n = 0;                // visits of this row so far
      bool ok = true, dead = false;
      // (slots) the slot of this thread's position of the next visit, asked for a visit ahead
      int32_t slot = -1;
      if constexpr (SLOTS) {
        const int32_t pos = at.s * kPos + x;
        if (pos < p.n_slots) slot = p.slots[(int64_t)at.row0 * p.n_slots + pos];
      }
      while (here < stop && !dead) {
        const int32_t v0 = at.s, v1 = (int32_t)min((int64_t)at.nsub, v0 + (stop - here));
        const bool cut_front = v0 > 0;
        const int32_t h0 = at.kv * p.group + at.chunk * p.chunk_heads;   // first query head
        const int32_t heads = min(p.chunk_heads, p.group - at.chunk * p.chunk_heads);
        int32_t win_a = at.a[0], win_b = at.b[0];                        // this row's window
        if (NB == 2 && j == 1) win_a = at.a[NB - 1], win_b = at.b[NB - 1];
        const bool live = win_b > win_a;
        bool visited = false, seen = false;
#pragma unroll
        for (int i = 0; i < kMine; ++i) sum[i] = 0.f;
#pragma unroll
        for (int h = 0; h < kMine / 32; ++h) mine_ref[h] = kNegInf, unset[h] = true;
        const int32_t* list = nullptr;
        if constexpr (SLOTS) list = p.slots + (int64_t)at.row0 * p.n_slots;
        for (int32_t v = v0; v < v1; ++v) {
          int32_t tile;
          uint32_t rows;
          at.visit(v, tile, rows);
          if (NB == 2 && !(rows >> j & 1)) continue;
          const int32_t pos = tile * kPos + x;
          bool on;
          if constexpr (SLOTS) {
            on = slot >= 0 && slot < p.num_pages * kPage;
            slot = -1;
            if (v + 1 < v1) {
              if (pos + kPos < p.n_slots) slot = list[pos + kPos];
            } else if (here + (v1 - v0) < stop) {
              // the next unit's first: of this row, or of the next
              if (at.chunk + 1 == p.chunks && at.kv + 1 == p.kv_heads) list += p.n_slots;
              if (x < p.n_slots) slot = list[x];
            }
          } else {
            on = pos >= win_a && pos < win_b;
          }
          const bool had = visited;   // the segment's output of this row has been begun
          visited = true;
          seen |= on;
          const uint32_t lanes_on = __ballot_sync(~0u, on);
          ok &= wait(full_s(j, n & 1), n >> 1 & 1, abort, &err);
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < kMine / 32; ++h) {
            uint32_t rs[32];
            tmem_ld32(tmem + lanes + (j * 2 + (n & 1)) * kCols + col0 + h * 32, rs);
            tmem_wait_ld32(rs);
            if (h == kMine / 32 - 1) {
              tc_fence_before();
              mbar_arrive(empty_s(j, n & 1));
            }
            float d[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) d[i] = __uint_as_float(rs[i]);
            if (lanes_on != ~0u) {
#pragma unroll
              for (int i = 0; i < 32; ++i) d[i] = on ? d[i] : kNegInf;
            }
            if constexpr (!SLOTS) {
              if (p.logits && on) {
                const int64_t width = (int64_t)p.max_pages * kPage;
                float* dst = p.logits + ((int64_t)(at.row0 + j) * p.q_heads + h0 + col0 + h * 32) * width + pos;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if ((int)col0 + h * 32 + i < heads) dst[i * width] = d[i];
              }
            }
            float top = kNegInf, top2 = kNegInf;
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
              if (!unset[h]) r = *(const float4*)&ref[wg][h * 32 + i];   // the negated references
              fma2(d[i], d[i + 1], c, r.x, r.y);
              fma2(d[i + 2], d[i + 3], c, r.z, r.w);
              top = max3(top, d[i], d[i + 1]);
              top2 = max3(top2, d[i + 2], d[i + 3]);
            }
            top = fmaxf(top, top2);
            for (int attempt = 0; attempt < 2; ++attempt) {
              if (!bar_red_or(bar_id, 128, unset[h] || top > kRaise<BF16> || !ok)) break;
              // a reference is to be set or raised (or a wait gave up): in bf16 first to the first
              // position's score, and where that leaves too large a weight, as always in fp16, to the maximum
              if (had) {
                ok &= wait(done_pv(j), (n - 1) & 1, abort, &err);
                tc_fence_after();
              }
              // lane i of every warp: what column i is compared with
              const bool first = BF16 && attempt == 0 && unset[h];
              if (lane == 0) valid[wg][warp & 3] = lanes_on;
              if (first) {
                if (lane == __ffs(lanes_on) - 1) {
#pragma unroll
                  for (int i = 0; i < 32; i += 4)
                    *(float4*)&red[wg][warp & 3][i] = make_float4(d[i], d[i + 1], d[i + 2], d[i + 3]);
                }
              } else {
                float t[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) t[i] = d[i];
                red[wg][warp & 3][lane] = over_lanes<true>(t);
              }
              if (bar_red_or(bar_id, 128, !ok)) {
                dead = true;
                break;
              }
              float m = kNegInf;
#pragma unroll
              for (int i = 3; i >= 0; --i) {
                const float y = red[wg][i][lane];
                if (valid[wg][i]) m = first ? y : fmaxf(m, y);
              }
              const bool was = mine_ref[h] != kNegInf;
              const float base = was ? mine_ref[h] : 0.f;
              // never lowered; set at the first finite score
              const bool set = m != kNegInf && (m > 0.f || !was);
              const float raised = set ? base + m : base;
              if (set) mine_ref[h] = raised;
              if ((warp & 3) == 0) {
                ref[wg][h * 32 + lane] = mine_ref[h] == kNegInf ? 0.f : -mine_ref[h];
                raise[wg][lane] = __fsub_rn(raised, base);
              }
              unset[h] = __any_sync(~0u, mine_ref[h] == kNegInf);
              bar_sync(bar_id, 128);
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                uint32_t r[16];
                const uint32_t o = tmem + lanes + kO + j * kCols + col0 + h * 32 + y * 16;
                if (had) {
                  tmem_ld16(o, r);
                  tmem_wait_ld16(r);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const float by = raise[wg][y * 16 + i];
                  d[y * 16 + i] -= by;
                  top = y + i == 0 ? d[0] : fmaxf(top, d[y * 16 + i]);
                  if (had) {
                    const float f = ex2(-by);
                    sum[h * 32 + y * 16 + i] *= f;
                    r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
                  }
                }
                if (had) tmem_st16(o, r);
              }
              if (had) tmem_wait_st();
              if (!first) break;
            }
            if (dead) break;   // a wait gave up: the whole warpgroup has voted
            if (h == 0 && n > 0) ok &= wait(done_pv(j), (n - 1) & 1, abort, &err);
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint32_t w[4];
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const float e0 = ex2(d[i + 2 * y]), e1 = ex2(d[i + 2 * y + 1]);
                add2(sum[h * 32 + i + 2 * y], sum[h * 32 + i + 2 * y + 1], e0, e1);
                w[y] = pack2<BF16>(e0, e1);
              }
              const uint32_t piece = (col0 + h * 32 + i) / 8;
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(p_row + ((piece ^ (x & 7)) << 4)), "r"(w[0]),
                           "r"(w[1]), "r"(w[2]), "r"(w[3])
                           : "memory");
            }
          }
          if (dead) break;
          fence_proxy_async_smem();
          tc_fence_before();
          mbar_arrive(full_p(j));
          ++n;
        }
        here += v1 - v0;
        if (!dead) {
          const bool unit_end = v1 == at.nsub;
          const bool whole = unit_end && !cut_front;
          const int which = cut_front ? 0 : 1;
          if (!unit_end && !cut_front && threadIdx.x == 0) {
            p.open_row[blockIdx.x] = at.row0;
            p.open_info[blockIdx.x] =
                make_int4(at.nrows, at.kv * p.chunks + at.chunk, sp.holder(here + (at.nsub - v1) - 1), 0);
          }
          if (visited) ok &= wait(done_pv(j), (n - 1) & 1, abort, &err);
          tc_fence_after();
          if constexpr (SLOTS) seen = bar_red_or(bar_id, 128, seen);
          const int64_t row = at.row0 + j;
#pragma unroll
          for (int h = 0; h < kMine / 32; ++h) {
            float t[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) t[i] = sum[h * 32 + i];
            red[wg][warp & 3][lane] = over_lanes<false>(t);
            if (bar_red_or(bar_id, 128, !ok)) {
              dead = true;
              break;
            }
            const float l = (red[wg][0][lane] + red[wg][1][lane]) + (red[wg][2][lane] + red[wg][3][lane]);
            const int32_t first = col0 + h * 32;
            const int32_t cols = min(32, heads - first);
            const float inv = SLOTS && !seen ? 0.f : 1.f / l;
            if ((warp & 3) == 0) raise[wg][lane] = whole ? inv : 1.f;
            bar_sync(bar_id, 128);
            const int64_t part = ((int64_t)blockIdx.x * 2 + which) * (NB * kCols) + j * kCols + first;
            if ((warp & 3) == 0 && lane < cols && live) {
              const float m = mine_ref[h];
              if (!whole) {
                p.part_ml[part + lane] = make_float2(m, !visited || (SLOTS && !seen) ? -1.f : l);
              } else {
                const int64_t i = row * p.q_heads + h0 + first + lane;
                if (p.lse) p.lse[i] = (m + log2f(l)) * 0.6931471805599453f;
                if (p.row_stat) p.row_stat[i] = make_float2(m == kNegInf ? 0.f : m, inv);
              }
            }
            if (live && (whole || visited)) {
              const uint32_t o = tmem + lanes + kO + j * kCols + first;
              uint32_t r[32];
              tmem_ld32(o, r);
              tmem_wait_ld32(r);
              if (whole) {
                T* out = (T*)p.out + row * p.out_row + (int64_t)(h0 + first) * p.out_head + x;
#pragma unroll
                for (int i = 0; i < 32; ++i, out += p.out_head)
                  if (i < cols) *out = (T)(__uint_as_float(r[i]) * raise[wg][i]);
              } else {
                float* po = p.part_o + part * kHead + x;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (i < cols) po[i * kHead] = __uint_as_float(r[i]);
              }
            }
            bar_sync(bar_id, 128);   // red is free again
          }
          tc_fence_before();
        }
        if (here < stop && !dead) at.next_unit(p, meta);
      }
    } else if (warp < 12) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
      // ------------------------------------------------------------- copies ----
      const bool values = warp >= 10;
      const int half = (warp - 8) & 1, t = threadIdx.x & (kLoaders - 1);
      const uint32_t depth = values ? L::kRingV : L::kRingK;
      const uint32_t ring = smem + (values ? L::v : L::k);
      const T* cache = (const T*)(values ? p.v : p.k);
      const int64_t s_page = values ? p.v_page : p.k_page, s_slot = values ? p.v_slot : p.k_slot,
                    s_head = values ? p.v_head : p.k_head;
      // Offsets are in units of 16 bytes (the caches span less than 64 GB).
      const uint32_t page16 = (uint32_t)(s_page / 8), slot16 = (uint32_t)(s_slot / 8);
      const int x = lane & 15, r0 = lane / 16;   // this lane's piece of a head, and its rows r0 + 2 i of the warp's 64
      uint32_t n = 0, seg = 0;                   // tiles, segments
      bool ok = true;
      uint32_t bad = kOk;
      // the slots of this thread's two positions, or the page of the warp's 64, of the next visit: asked
      // for a visit ahead (and a row's slots brought to L2 a row ahead)
      int32_t entry[2];
      auto ask = [&](const int32_t* list, int32_t tile) {
        if constexpr (SLOTS) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int32_t pos = tile * kPos + half * 64 + e * 32 + lane;
            entry[e] = pos < p.n_slots ? list[pos] : -1;
          }
        } else {
          const int32_t i = tile * 2 + half;
          entry[0] = i < p.max_pages ? list[i] : -1;
        }
      };
      const int32_t* list = nullptr;
      if constexpr (SLOTS) ask(p.slots + (int64_t)at.row0 * p.n_slots, at.s);
      while (here < stop && ok) {
        const int32_t v0 = at.s, v1 = (int32_t)min((int64_t)at.nsub, v0 + (stop - here));
        here += v1 - v0;
        int32_t tile;
        uint32_t rows;
        if constexpr (SLOTS) {
          list = p.slots + (int64_t)at.row0 * p.n_slots;
          if (warp == 10 && at.row0 + 1 < p.rows)
            for (int32_t i = lane * 32; i < p.n_slots; i += 32 * 32)
              asm volatile("prefetch.global.L2 [%0];" ::"l"(list + p.n_slots + i));
        } else {
          list = p.page_table + (int64_t)at.req * p.max_pages;
          at.visit(v0, tile, rows);
          ask(list, tile);
        }
        if (!values) {
          // the queries, with the segment's first tile of keys
          const uint32_t b = seg % L::kQ;
          ok = __all_sync(~0u, wait(empty_q(b), (seg / L::kQ & 1) ^ 1, abort, &err));
          if (!ok) break;
          const int32_t h0 = at.kv * p.group + at.chunk * p.chunk_heads;
          const int32_t heads = min(p.chunk_heads, p.group - at.chunk * p.chunk_heads);
          const uint32_t dst = smem + L::q + b * (NB * kQBytes);
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            const bool live = at.b[j] > at.a[j];
            const T* q = (const T*)p.q + (int64_t)(at.row0 + (live ? j : 0)) * p.q_row + (int64_t)h0 * p.q_head;
#pragma unroll 4
            for (int i = t; i < kCols * 16; i += kLoaders) {
              const int r = i / 16, y = i % 16;
              const bool in = live && r < heads;
              copy16(dst + j * kQBytes + (y / 8) * kQHalf + r * 128 + (((y & 7) ^ (r & 7)) << 4),
                     q + (in ? (int64_t)r * p.q_head : 0) + y * 8, in ? 16u : 0u);
            }
          }
          ++seg;
        }
        const char* base = (const char*)(cache + at.kv * s_head + x * 8);
        for (int32_t v = v0; v < v1; ++v) {
          at.visit(v, tile, rows);
          // where the warp's 64 positions lie; `all`: every one of them is read
          uint32_t from[2];
          bool all = true;
          if constexpr (SLOTS) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const bool on = entry[e] >= 0 && entry[e] < p.num_pages * kPage;
              if (!on && entry[e] != -1) bad = kErrInvalidPage;
              from[e] = on ? (uint32_t)(entry[e] / kPage) * page16 + (uint32_t)(entry[e] % kPage) * slot16 : ~0u;
              all &= on;
            }
            if (v + 1 < v1) {
              ask(list, v + 1);
            } else if (here < stop) {
              // the next unit's first: of this row, or of the next
              ask(list + (at.chunk + 1 == p.chunks && at.kv + 1 == p.kv_heads ? p.n_slots : 0), 0);
            }
          } else {
            int32_t lo = 0, hi = INT32_MAX;   // seen by every row of the visit
#pragma unroll
            for (int j = 0; j < NB; ++j)
              if (rows >> j & 1) lo = max(lo, at.a[j]), hi = min(hi, at.b[j]);
            const int32_t first = tile * kPos + half * 64;
            const bool any = first < hi && first + 64 > lo, there = entry[0] >= 0 && entry[0] < p.num_pages;
            if (any && !there) bad = kErrInvalidPage;
            const uint32_t page = there ? (uint32_t)entry[0] * page16 : 0u;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int32_t pos = first + e * 32 + lane;
              const bool on = there && pos >= lo && pos < hi;
              from[e] = on ? page + (uint32_t)(e * 32 + lane) * slot16 : ~0u;
              all &= on;
            }
            if (v + 1 < v1) {
              int32_t next_tile;
              uint32_t next_rows;
              at.visit(v + 1, next_tile, next_rows);
              ask(list, next_tile);
            }
          }
          all = __all_sync(~0u, all);
          const uint32_t slot = n % depth;
          ok = __all_sync(~0u, wait(values ? empty_v(slot) : empty_k(slot), (n / depth & 1) ^ 1, abort, &err));
          if (!ok) break;
          const uint32_t dst = ring + slot * kTileBytes + (x / 8) * kHalfTile + (uint32_t)half * (64 * 128);
          uint32_t to[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) to[i] = dst + (2 * i + r0) * 128 + (((x & 7) ^ (2 * i + r0)) << 4);
          if (!SLOTS && all) {
            const char* src = base + (uint64_t)__shfl_sync(~0u, from[0], 0) * 16 + (int64_t)r0 * s_slot * 2;
#pragma unroll
            for (int i = 0; i < 32; ++i, src += 4 * s_slot) copy16(to[i & 3] + (i >> 2) * 1024, src, 16u);
          } else if (all) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              copy16(to[i & 3] + (i >> 2) * 1024,
                     base + (uint64_t)__shfl_sync(~0u, from[i / 16], (2 * i + r0) & 31) * 16, 16u);
          } else {
#pragma unroll 8
            for (int i = 0; i < 32; ++i) {
              const uint32_t o = __shfl_sync(~0u, i < 16 ? from[0] : from[1], (2 * i + r0) & 31);
              const bool in = o != ~0u;
              copy16(to[i & 3] + (i >> 2) * 1024, base + (uint64_t)(in ? o : 0u) * 16, in ? 16u : 0u);
            }
          }
          arrive_when_copied(values ? full_v(slot) : full_k(slot));
          ++n;
        }
        if (here < stop && ok) at.next_unit(p, meta);
      }
      copy_wait_all();
      bad = __reduce_max_sync(~0u, bad);
      if (lane == 0 && bad != kOk) atomicMax(&err, bad);
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
      // ----------------------------------------------------------- products ----
      // One warp issues the scores' products and one the outputs', each its own waits in order; the
      // other two warps have no work.
      bool ok = true;
      uint32_t n = 0;                   // visits
      if (warp == 12) {
        constexpr uint32_t kQK = idesc_f16<BF16>(128, kCols, false);
        uint32_t seg = 0, ns[NB];       // segments; visits of each row
#pragma unroll
        for (int j = 0; j < NB; ++j) ns[j] = 0;
        while (here < stop && ok) {
          const int32_t v0 = at.s, v1 = (int32_t)min((int64_t)at.nsub, v0 + (stop - here));
          here += v1 - v0;
          const uint32_t qb = seg % L::kQ;
          const uint64_t q = desc128(smem + L::q + qb * (NB * kQBytes), 16, 1024);
          for (int32_t v = v0; v < v1; ++v) {
            int32_t tile;
            uint32_t rows;
            at.visit(v, tile, rows);
            const uint32_t slot = n % L::kRingK;
            ok = __all_sync(~0u, wait(full_k(slot), n / L::kRingK & 1, abort, &err));
            fence_proxy_async_smem();   // the copies' writes before the products' reads
            const uint64_t a = desc128(smem + L::k + slot * kTileBytes, 16, 1024);
#pragma unroll
            for (int j = 0; j < NB; ++j) {
              if (!(rows >> j & 1)) continue;
              const uint32_t b = ns[j] & 1;
              ok = ok && __all_sync(~0u, wait(empty_s(j, b), (ns[j] >> 1 & 1) ^ 1, abort, &err));
              tc_fence_after();
              if (ok && elect_one()) {
#pragma unroll
                for (int k = 0; k < kHead / 16; ++k)   // 16 elements: 32 bytes of a row
                  mma_f16(tmem + (j * 2 + b) * kCols, a + (k / 4) * (kHalfTile >> 4) + (k % 4) * 2,
                          q + j * (kQBytes >> 4) + (k / 4) * (kQHalf >> 4) + (k % 4) * 2, kQK, k > 0);
                tc_commit(full_s(j, b));
              }
              __syncwarp();
              ++ns[j];
            }
            if (!ok) break;
            if (elect_one()) tc_commit(empty_k(slot));
            __syncwarp();
            ++n;
          }
          if (ok && elect_one()) tc_commit(empty_q(qb));
          __syncwarp();
          ++seg;
          if (here < stop && ok) at.next_unit(p, meta);
        }
      } else if (warp == 13) {
        constexpr uint32_t kPV = idesc_f16<BF16>(128, kCols, true);
        uint32_t np[NB];                // visits of each row
        bool fresh[NB];                 // the row's output is to be begun anew
#pragma unroll
        for (int j = 0; j < NB; ++j) np[j] = 0, fresh[j] = true;
        while (here < stop && ok) {
          const int32_t v0 = at.s, v1 = (int32_t)min((int64_t)at.nsub, v0 + (stop - here));
          here += v1 - v0;
#pragma unroll
          for (int j = 0; j < NB; ++j) fresh[j] = true;
          for (int32_t v = v0; v < v1; ++v) {
            int32_t tile;
            uint32_t rows;
            at.visit(v, tile, rows);
            const uint32_t slot = n % L::kRingV;
            ok = __all_sync(~0u, wait(full_v(slot), n / L::kRingV & 1, abort, &err));
            fence_proxy_async_smem();   // the copies' writes before the products' reads
            const uint64_t a = desc128(smem + L::v + slot * kTileBytes, kHalfTile, 1024);
#pragma unroll
            for (int j = 0; j < NB; ++j) {
              if (!(rows >> j & 1)) continue;
              ok = ok && __all_sync(~0u, wait(full_p(j), np[j] & 1, abort, &err));
              tc_fence_after();
              if (ok && elect_one()) {
                const uint64_t b = desc128(smem + L::p + j * kPBytes, 1024, 1024);
#pragma unroll
                for (int k = 0; k < kPos / 16; ++k)   // 16 positions: 2048 bytes of either
                  mma_f16(tmem + kO + j * kCols, a + k * (2048 >> 4), b + k * (2048 >> 4), kPV, !fresh[j] || k > 0);
                tc_commit(done_pv(j));
              }
              __syncwarp();
              fresh[j] = false;
              ++np[j];
            }
            if (!ok) break;
            if (elect_one()) tc_commit(empty_v(slot));
            __syncwarp();
            ++n;
          }
          if (here < stop && ok) at.next_unit(p, meta);
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
  if (warp == 12 || warp == 13) {
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
  if (warp == 12) tmem_dealloc(tmem, kTmemCols);
}

template <bool BF16, int NB, bool SLOTS>
cudaError_t launch(const AttnParams& p, int sm_count, cudaStream_t stream) {
  auto* kernel = attn_tc_kernel<BF16, NB, SLOTS>;
  static std::atomic<bool> done[64];
  cudaError_t e = set_smem_once(kernel, Smem<NB>::bytes, done);
  if (e != cudaSuccess) return e;
  kernel<<<sm_count, kThreads, Smem<NB>::bytes, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace tc
}  // namespace attn
}  // namespace idxk
