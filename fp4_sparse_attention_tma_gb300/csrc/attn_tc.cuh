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
// maximum but one that a tile raises when it exceeds it by more than 2^8 (the first tile sets
// it): the sums stay exact in fp32, P stays below 2^8, and the accumulator in tensor memory is
// scaled only then.  Columns are 64 a row; with two rows of one request both use the tiles
// that both see in full, and the tiles at the windows' edges are visited row by row, so that
// what one row does not see is zero for it.
//
// Roles: two warpgroups of softmax (for one row 32 columns each, for two a row each), two
// warps that copy keys (and the queries), two that copy values (16-byte asynchronous copies
// into the 128-byte swizzle, any stride, page or slot), one that issues the products.  Every
// wait is bounded.
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
constexpr float kRaise = 8.f;             // a column's reference is raised when exceeded by 2^8

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
  int32_t u, s;

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
  __device__ static int32_t count(const AttnParams& p, int32_t r) {
    if (!starts_group(p, r)) return 0;
    int32_t a[NB], b[NB], c0, c1;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int32_t i = r + j;
      const bool in = i < p.rows && (j == 0 || (i % p.group_rows != 0 && p.row_req[i] == p.row_req[r]));
      a[j] = in ? p.row_start[i] : 0;
      b[j] = in ? p.row_end[i] : 0;
    }
    return visits(a, b, c0, c1);
  }
  __device__ static int32_t row_count(const AttnParams& p) { return hi(p.n_slots); }

  __device__ void load(const AttnParams& p, int32_t row) {
    row0 = row;
    req = 0;
    nrows = 1;
    if constexpr (SLOTS) {
      a[0] = 0;
      b[0] = p.n_slots;
    } else {
      req = p.row_req[row];
      if constexpr (NB == 2)
        if (row + 1 < p.rows && (row + 1) % p.group_rows != 0 && p.row_req[row + 1] == req) nrows = 2;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        a[j] = j < nrows ? p.row_start[row + j] : 0;
        b[j] = j < nrows ? p.row_end[row + j] : 0;
        if (b[j] <= a[j]) a[j] = b[j] = 0;
      }
    }
    nsub = visits(a, b, c0, c1);
  }
  __device__ void next(const AttnParams& p) {
    if (++s < nsub) return;
    s = 0;
    if (++u < p.kv_heads * p.chunks) return;
    u = 0;
    do {
      load(p, row0 + nrows);
    } while (nsub == 0);
  }
  // The visit: its tile and its rows (bit j).
  __device__ void visit(int32_t& tile, uint32_t& rows) const {
    if constexpr (NB == 1) {
      tile = lo(a[0]) + s;
      rows = 1;
    } else {
      int32_t x = s;
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

// A bounded wait: false when it gave up (after kWaitLimitNs, or because another role did).
__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort, uint32_t* err) {
  const uint64_t t0 = global_timer_ns();
  for (uint32_t i = 0;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 63u) {
      if (*abort) return false;
      if (global_timer_ns() - t0 > kWaitLimitNs) {
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
  __shared__ __align__(16) float ref[2][kMine];    // columns' references, in units of log2
  __shared__ float red[2][4][32];
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

  if (threadIdx.x == 0) {
    err = kOk;
    abort_flag = 0;
    p.open_row[blockIdx.x] = -1;
    for (int i = 0; i < L::kRingK; ++i) mbar_init(full_k(i), kLoaders), mbar_init(empty_k(i), 1);
    for (int i = 0; i < L::kRingV; ++i) mbar_init(full_v(i), kLoaders), mbar_init(empty_v(i), 1);
    for (int i = 0; i < L::kQ; ++i) mbar_init(empty_q(i), 1);
    for (int j = 0; j < NB; ++j) {
      for (int i = 0; i < 2; ++i) mbar_init(full_s(j, i), 1), mbar_init(empty_s(j, i), kSoft);
      mbar_init(full_p(j), kSoft);
      mbar_init(done_pv(j), 1);
    }
    mbar_init(drain, 1);
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
  const bool work = find_range<Walk<NB, SLOTS>, SLOTS, kWarps>(p, sp, at, blockIdx.x, &err);
  if (work) {
    int64_t here = sp.first(blockIdx.x);
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
      bool ok = true, begin = true, cut_front = false, visited = false, seen = false;
      while (here < stop) {
        if (begin) {
          begin = false;
          cut_front = at.s > 0;
          visited = seen = false;
#pragma unroll
          for (int i = 0; i < kMine; ++i) sum[i] = 0.f;
#pragma unroll
          for (int h = 0; h < kMine / 32; ++h) mine_ref[h] = kNegInf, unset[h] = true;
        }
        int32_t tile;
        uint32_t rows;
        at.visit(tile, rows);
        const int32_t chunk = at.u % p.chunks;
        const int32_t h0 = (at.u / p.chunks) * p.group + chunk * p.chunk_heads;   // first query head
        const int32_t heads = min(p.chunk_heads, p.group - chunk * p.chunk_heads);
        if (rows >> j & 1) {
          const int32_t pos = tile * kPos + x;
          bool on;
          if constexpr (SLOTS) {
            const int32_t slot = pos < p.n_slots ? p.slots[(int64_t)at.row0 * p.n_slots + pos] : -1;
            on = slot >= 0 && slot < p.num_pages * kPage;
          } else {
            on = pos >= at.a[j] && pos < at.b[j];
          }
          const bool had = visited;   // the segment's output of this row has been begun
          visited = true;
          seen |= on;
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
            for (int i = 0; i < 32; ++i) d[i] = on ? __uint_as_float(rs[i]) : kNegInf;
            if constexpr (!SLOTS) {
              if (p.logits && on) {
                const int64_t width = (int64_t)p.max_pages * kPage;
                float* dst = p.logits + ((int64_t)(at.row0 + j) * p.q_heads + h0 + col0 + h * 32) * width + pos;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if ((int)col0 + h * 32 + i < heads) dst[i * width] = d[i];
              }
            }
            float top = kNegInf;
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
              if (!unset[h]) r = *(const float4*)&ref[wg][h * 32 + i];
              d[i] = fmaf(d[i], c, -r.x);
              d[i + 1] = fmaf(d[i + 1], c, -r.y);
              d[i + 2] = fmaf(d[i + 2], c, -r.z);
              d[i + 3] = fmaf(d[i + 3], c, -r.w);
              top = fmaxf(top, fmaxf(fmaxf(d[i], d[i + 1]), fmaxf(d[i + 2], d[i + 3])));
            }
            if (bar_red_or(bar_id, 128, unset[h] || top > kRaise || !ok)) {
              // a reference is to be set or raised (or a wait gave up)
              if (n > 0) ok &= wait(done_pv(j), (n - 1) & 1, abort, &err);
              tc_fence_after();
              float t[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) t[i] = d[i];
              red[wg][warp & 3][lane] = over_lanes<true>(t);
              if (bar_red_or(bar_id, 128, !ok)) break;
              const float m = fmaxf(fmaxf(red[wg][0][lane], red[wg][1][lane]), fmaxf(red[wg][2][lane], red[wg][3][lane]));
              const bool was = mine_ref[h] != kNegInf;
              const float base = was ? mine_ref[h] : 0.f;
              // never lowered; set at the first finite score
              const bool set = m != kNegInf && (m > 0.f || !was);
              const float raised = set ? base + m : base;
              const float adj = __fsub_rn(raised, base);
              if (set) mine_ref[h] = raised;
              const float f = ex2(-adj);
              const bool moved = __any_sync(~0u, set);
              if (moved) {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  d[i] -= __shfl_sync(~0u, adj, i);
                  sum[h * 32 + i] *= __shfl_sync(~0u, f, i);
                }
                if (had) {
                  const uint32_t o = tmem + lanes + kO + j * kCols + col0 + h * 32;
#pragma unroll
                  for (int y = 0; y < 2; ++y) {
                    uint32_t r[16];
                    tmem_ld16(o + y * 16, r);
                    tmem_wait_ld16(r);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                      r[i] = __float_as_uint(__uint_as_float(r[i]) * __shfl_sync(~0u, f, y * 16 + i));
                    tmem_st16(o + y * 16, r);
                  }
                  tmem_wait_st();
                }
              }
              if ((warp & 3) == 0) ref[wg][h * 32 + lane] = mine_ref[h] == kNegInf ? 0.f : mine_ref[h];
              unset[h] = __any_sync(~0u, mine_ref[h] == kNegInf);
              bar_sync(bar_id, 128);
            }
            if (h == 0 && n > 0) ok &= wait(done_pv(j), (n - 1) & 1, abort, &err);
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint32_t w[4];
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const float e0 = ex2(d[i + 2 * y]), e1 = ex2(d[i + 2 * y + 1]);
                sum[h * 32 + i + 2 * y] += e0;
                sum[h * 32 + i + 2 * y + 1] += e1;
                w[y] = pack2<BF16>(e0, e1);
              }
              const uint32_t piece = (col0 + h * 32 + i) / 8;
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(p_row + ((piece ^ (x & 7)) << 4)), "r"(w[0]),
                           "r"(w[1]), "r"(w[2]), "r"(w[3])
                           : "memory");
            }
          }
          fence_proxy_async_smem();
          tc_fence_before();
          mbar_arrive(full_p(j));
          ++n;
        }
        ++here;
        const bool unit_end = at.s + 1 == at.nsub;
        if (unit_end || here == stop) {
          begin = true;
          const bool whole = unit_end && !cut_front;
          const int which = cut_front ? 0 : 1;
          if (!unit_end && !cut_front && threadIdx.x == 0) {
            p.open_row[blockIdx.x] = at.row0;
            p.open_info[blockIdx.x] = make_int4(at.nrows, at.u, sp.holder(here + (at.nsub - at.s) - 2), 0);
          }
          if (visited) ok &= wait(done_pv(j), (n - 1) & 1, abort, &err);
          tc_fence_after();
          if constexpr (SLOTS) seen = bar_red_or(bar_id, 128, seen);
          const bool live = at.b[j] > at.a[j];
          const int64_t row = at.row0 + j;
#pragma unroll
          for (int h = 0; h < kMine / 32; ++h) {
            float t[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) t[i] = sum[h * 32 + i];
            red[wg][warp & 3][lane] = over_lanes<false>(t);
            if (bar_red_or(bar_id, 128, !ok)) break;
            const float l = (red[wg][0][lane] + red[wg][1][lane]) + (red[wg][2][lane] + red[wg][3][lane]);
            const int32_t first = col0 + h * 32;
            const int32_t cols = min(32, heads - first);
            const float inv = SLOTS && !seen ? 0.f : 1.f / l;
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
              T* out = (T*)p.out + row * p.out_row + (int64_t)(h0 + first) * p.out_head + x;
              float* po = p.part_o + part * kHead + x;
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                uint32_t r[16];
                tmem_ld16(o + y * 16, r);
                tmem_wait_ld16(r);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const float scale = __shfl_sync(~0u, inv, y * 16 + i);
                  if (y * 16 + i < cols) {
                    if (whole)
                      out[(int64_t)(y * 16 + i) * p.out_head] = (T)(__uint_as_float(r[i]) * scale);
                    else
                      po[(y * 16 + i) * kHead] = __uint_as_float(r[i]);
                  }
                }
              }
            }
            bar_sync(bar_id, 128);   // red is free again
          }
          tc_fence_before();
        }
        // a wait that gave up ends the role, for the whole warpgroup at once
        if (bar_red_or(bar_id, 128, !ok)) break;
        if (here < stop) at.next(p);
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
      uint32_t n = 0, handed = 0, seg = 0;   // tiles asked for, tiles handed over, segments
      bool begin = true, ok = true;
      uint32_t bad = kOk;
      auto hand_over = [&]() {               // the oldest, which has arrived
        fence_proxy_async_smem();
        mbar_arrive(values ? full_v(handed % depth) : full_k(handed % depth));
        ++handed;
      };
      while (here < stop) {
        const int32_t chunk = at.u % p.chunks, kv = at.u / p.chunks;
        int32_t tile;
        uint32_t rows;
        at.visit(tile, rows);
        // positions 64 half + lane and + 32 of the tile: where they lie, and whether they are read
        const T* from[2];
        bool on[2];
        {
          int32_t lo = 0, hi = INT32_MAX;   // seen by every row of the visit
          if constexpr (!SLOTS) {
#pragma unroll
            for (int j = 0; j < NB; ++j)
              if (rows >> j & 1) lo = max(lo, at.a[j]), hi = min(hi, at.b[j]);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int32_t pos = tile * kPos + half * 64 + e * 32 + lane;
            int64_t page = 0;
            int32_t off = 0;
            if constexpr (SLOTS) {
              const int32_t slot = pos < p.n_slots ? p.slots[(int64_t)at.row0 * p.n_slots + pos] : -1;
              on[e] = slot >= 0 && slot < p.num_pages * kPage;
              if (!on[e] && slot != -1) bad = kErrInvalidPage;
              if (on[e]) page = slot / kPage, off = slot % kPage;
            } else {
              on[e] = pos >= lo && pos < hi;
              if (on[e]) {
                page = p.page_table[(int64_t)at.req * p.max_pages + pos / kPage];
                off = pos % kPage;
                if (page < 0 || page >= p.num_pages) bad = kErrInvalidPage, on[e] = false, page = 0;
              }
            }
            from[e] = cache + page * s_page + off * s_slot + kv * s_head;
          }
        }
        if (begin && !values) {
          // the queries, with the segment's first tile of keys
          const uint32_t b = seg % L::kQ;
          if (L::kQ == 1 && handed < n) {
            // the products that free the queries' place wait for the last tile
            copy_wait<0>();
            hand_over();
          }
          ok = __all_sync(~0u, wait(empty_q(b), (seg / L::kQ & 1) ^ 1, abort, &err));
          if (!ok) break;
          const int32_t h0 = kv * p.group + chunk * p.chunk_heads;
          const int32_t heads = min(p.chunk_heads, p.group - chunk * p.chunk_heads);
          const uint32_t dst = smem + L::q + b * (NB * kQBytes);
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            const bool live = at.b[j] > at.a[j];
            const T* q = (const T*)p.q + (int64_t)(at.row0 + (live ? j : 0)) * p.q_row + (int64_t)h0 * p.q_head;
            for (int i = t; i < kCols * 16; i += kLoaders) {
              const int r = i / 16, x = i % 16;
              const bool in = live && r < heads;
              copy16(dst + j * kQBytes + (x / 8) * kQHalf + r * 128 + (((x & 7) ^ (r & 7)) << 4),
                     q + (in ? (int64_t)r * p.q_head : 0) + x * 8, in ? 16u : 0u);
            }
          }
          ++seg;
        }
        begin = at.s + 1 == at.nsub;
        const uint32_t slot = n % depth;
        ok = __all_sync(~0u, wait(values ? empty_v(slot) : empty_k(slot), (n / depth & 1) ^ 1, abort, &err));
        if (!ok) break;
        {
          const int x = lane & 15;
          const uint32_t dst = ring + slot * kTileBytes + (x / 8) * kHalfTile + (uint32_t)half * (64 * 128);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int r = i * 2 + lane / 16;   // of this warp's 64 positions
            const unsigned long long base = __shfl_sync(~0u, (unsigned long long)from[i / 16], r & 31);
            const bool in = __shfl_sync(~0u, (int)on[i / 16], r & 31);
            copy16(dst + r * 128 + (((x & 7) ^ (r & 7)) << 4), (const T*)base + x * 8, in ? 16u : 0u);
          }
        }
        copy_commit();
        ++n;
        if (handed + 1 < n) {
          copy_wait<1>();   // the tile before this one
          hand_over();
        }
        if (++here < stop) at.next(p);
      }
      copy_wait<0>();
      if (ok && handed < n) hand_over();
      bad = __reduce_max_sync(~0u, bad);
      if (lane == 0 && bad != kOk) atomicMax(&err, bad);
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
      // ----------------------------------------------------------- products ----
      constexpr uint32_t kQK = idesc_f16<BF16>(128, kCols, false), kPV = idesc_f16<BF16>(128, kCols, true);
      uint32_t n = 0, seg = 0;          // visits, segments
      uint32_t ns[NB], np[NB];          // visits of each row: scores issued, outputs issued
      bool fresh[NB];                   // the row's output is to be begun anew
#pragma unroll
      for (int j = 0; j < NB; ++j) ns[j] = np[j] = 0, fresh[j] = true;
      uint32_t last_rows = 0;           // rows of the visit before, whose outputs are still to be issued
      bool last_end = false;            // it was its segment's last
      bool ok = true, begin = true;
      auto outputs = [&](uint32_t visit) {
        const uint32_t slot = visit % L::kRingV;
        ok = ok && __all_sync(~0u, wait(full_v(slot), visit / L::kRingV & 1, abort, &err));
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          if (!(last_rows >> j & 1)) continue;
          ok = ok && __all_sync(~0u, wait(full_p(j), np[j] & 1, abort, &err));
          tc_fence_after();
          if (ok && lane == 0) {
            const uint32_t a = smem + L::v + slot * kTileBytes, b = smem + L::p + j * kPBytes;
#pragma unroll
            for (int k = 0; k < kPos / 16; ++k)
              mma_f16(tmem + kO + j * kCols, desc128(a + k * 2048, kHalfTile, 1024), desc128(b + k * 2048, 1024, 1024), kPV,
                      !fresh[j] || k > 0);
            tc_commit(done_pv(j));
          }
          __syncwarp();
          fresh[j] = false;
          ++np[j];
        }
        if (ok && lane == 0) tc_commit(empty_v(slot));
        __syncwarp();
        if (last_end) {
#pragma unroll
          for (int j = 0; j < NB; ++j) fresh[j] = true;
        }
      };
      while (warp == 12 && here < stop && ok) {   // the warps beside it have no work
        int32_t tile;
        uint32_t rows;
        at.visit(tile, rows);
        if (begin && n > 0) ++seg;
        const uint32_t slot = n % L::kRingK;
        ok = __all_sync(~0u, wait(full_k(slot), n / L::kRingK & 1, abort, &err));
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          if (!(rows >> j & 1)) continue;
          const uint32_t b = ns[j] & 1;
          ok = ok && __all_sync(~0u, wait(empty_s(j, b), (ns[j] >> 1 & 1) ^ 1, abort, &err));
          tc_fence_after();
          if (ok && lane == 0) {
            const uint32_t a = smem + L::k + slot * kTileBytes,
                           q = smem + L::q + (seg % L::kQ) * (NB * kQBytes) + j * kQBytes;
#pragma unroll
            for (int k = 0; k < kHead / 16; ++k)
              mma_f16(tmem + (j * 2 + b) * kCols, desc128(a + (k / 4) * kHalfTile + (k % 4) * 32, 16, 1024),
                      desc128(q + (k / 4) * kQHalf + (k % 4) * 32, 16, 1024), kQK, k > 0);
            tc_commit(full_s(j, b));
          }
          __syncwarp();
          ++ns[j];
        }
        ++here;
        const bool end = at.s + 1 == at.nsub || here == stop;
        if (ok && lane == 0) {
          tc_commit(empty_k(slot));
          if (end) tc_commit(empty_q(seg % L::kQ));
        }
        __syncwarp();
        begin = end;
        if (n > 0 && ok) outputs(n - 1);
        last_rows = rows;
        last_end = end;
        ++n;
        if (here < stop) at.next(p);
      }
      if (n > 0 && ok) outputs(n - 1);
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
  if (warp == 12) {
    __syncwarp();
    if (lane == 0) tc_commit(drain);
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
