// Writing a paged cache: new tokens' queries and keys normed head by head and rotated by their
// positions, keys and values put into their requests' pages, in 16 bits or in the 4-bit form;
// and reading listed slots of a 4-bit cache back.
//
// For a head x of D elements, with the norm's weight w and the angles' cosines and sines c, s:
//   y = (x / sqrt(mean x^2 + eps)) * w,   (a, b) -> (a c - b s, b c + a s)  for each pair (a, b),
// a and b either neighbours or half of the rotated dimensions apart.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "append.h"
#include "fp4.cuh"
#include "idx_launch.h"
#include "pairs.cuh"

namespace idxk {
namespace {

constexpr int kMostBits = 15;                        // of the words of the table or bitmap that finds slots named twice
constexpr int kTableBytes = 4 << kMostBits;
constexpr int kGatherThreads = 256;

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*(const __half2*)&w[i]);
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      const __nv_bfloat162 t = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *(const uint32_t*)&t;
    } else {
      const __half2 t = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *(const uint32_t*)&t;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16-byte asynchronous copy; bytes = 0 writes zeros and reads nothing.
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void commit_async() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_async() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A sum held as a rounded part and what the roundings left (TwoSum, Knuth): the sum of a head's squares
// does not depend on the order then, up to its one final rounding, and so neither do the codes of a key
// that lies next to a border between two of them.
__device__ __forceinline__ void add_exactly(float& s, float& rest, float x) {
  const float t = __fadd_rn(s, x), b = __fsub_rn(t, s);
  rest = __fadd_rn(rest, __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(x, b)));
  s = t;
}

// The same for two sums at once (a - b as b * -1 + a, which rounds alike).  x is a square that fp32 holds exactly, so that
// it makes no difference whether the sums that take it are fused with its product.
__device__ __forceinline__ void add_exactly(Two& s, Two& rest, Two x) {
  const Two minus = two(-1.f, -1.f);
  const Two t = add2(s, x), b = fma2(s, minus, t);
  rest = add2(rest, add2(fma2(fma2(b, minus, t), minus, s), fma2(b, minus, x)));
  s = t;
}
// The larger magnitude; NaN if one is.
__device__ __forceinline__ float larger(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

constexpr int kChecked = 8;

// Checks every row of the call, so that all CTAs agree on whether anything is written: rows in range,
// pages in range, no slot named twice.  Returns the error (kOk: none) to every thread.
__device__ uint32_t check_rows(const AppendParams& p, uint32_t* table) {
  __shared__ uint32_t err;
  const int tid = threadIdx.x, n = blockDim.x;
  if (tid == 0) err = kOk;
  const bool bitmap = p.bitmap;
  const uint32_t entries = 1u << p.table_bits;
  const int64_t slots = (int64_t)p.num_pages * kPage;
  // the bitmap holds a part of the slots at a time; neighbours in different words, as rows of a prompt follow one another
  const int64_t span = bitmap ? (int64_t)entries * 32 : slots;
  for (int64_t s0 = 0; s0 < slots; s0 += span) {
    const uint32_t none = bitmap ? 0u : ~0u;
    for (uint32_t i = tid; i < entries / 4; i += n) ((uint4*)table)[i] = make_uint4(none, none, none, none);
    __syncthreads();
    // Some rows a thread at once, so that their loads wait for one another only by kind (8208 rows to
    // 4 bits: 8 at once 40 us a call, 4 at once 42, one 48, not looking 33).
    for (int32_t r0 = tid; r0 < p.rows; r0 += n * kChecked) {
      int32_t pos[kChecked], req[kChecked], page[kChecked];
#pragma unroll
      for (int k = 0; k < kChecked; ++k) {
        const int64_t r = r0 + (int64_t)k * n;
        pos[k] = -1;
        if (k * n >= p.rows) continue;      // (the same for all)
        pos[k] = r < p.rows ? p.row_pos[r] : -1;
        req[k] = r < p.rows ? p.row_req[r] : 0;
      }
      uint32_t e = kOk;
#pragma unroll
      for (int k = 0; k < kChecked; ++k) {
        page[k] = -1;
        if (k * n >= p.rows || pos[k] == -1) continue;
        if (pos[k] < 0 || req[k] < 0 || req[k] >= p.num_req || pos[k] / kPage >= p.max_pages ||
            (p.rope && pos[k] >= p.rope_rows)) {
          e = max(e, (uint32_t)kErrInvalidMetadata);
          pos[k] = -1;
        } else {
          page[k] = p.page_table[(int64_t)req[k] * p.max_pages + pos[k] / kPage];
        }
      }
#pragma unroll
      for (int k = 0; k < kChecked; ++k) {
        if (k * n >= p.rows || pos[k] == -1) continue;
        if (page[k] < 0 || page[k] >= p.num_pages) {
          e = max(e, (uint32_t)kErrInvalidPage);
          continue;
        }
        const int64_t slot = (int64_t)page[k] * kPage + pos[k] % kPage;
        if (bitmap) {
          if (slot >= s0 && slot < s0 + span) {
            const uint32_t x = (uint32_t)(slot - s0), bit = 1u << (x >> p.table_bits);
            if (atomicOr(&table[x & (entries - 1)], bit) & bit) e = max(e, (uint32_t)kErrInvalidPage);
          }
        } else {
          // open addressing: at most half of the entries are taken
          const uint32_t key = (uint32_t)slot;
          uint32_t at = (key * 2654435769u) >> (32 - p.table_bits);
          for (uint32_t i = 0; i < entries; ++i) {
            const uint32_t old = atomicCAS(&table[at], ~0u, key);
            if (old == ~0u) break;
            if (old == key) {
              e = max(e, (uint32_t)kErrInvalidPage);
              break;
            }
            at = (at + 1) & (entries - 1);
          }
        }
      }
      if (e != kOk) atomicMax(&err, e);
    }
    __syncthreads();
  }
  __syncthreads();
  return err;
}

// The lane's dimensions of a head: two groups of 4, at pa and pb.  A head that stays in 16 bits and is rotated half by half:
// a group of either half, so that the pairs lie within the lane; else 8 in a row (the 4-bit form's blocks are 4 lanes).
struct Dims {
  int pa, pb, j;        // j: the first of the lane's 4 angles, -1: none
  __device__ Dims(int in, int rot, int first, bool halves) {
    const int d0 = in * 8;
    pa = d0, pb = d0 + 4, j = -1;
    if (rot == 0) return;
    if (!halves) {
      if (d0 >= first && d0 < first + rot) j = (d0 - first) / 2;
    } else if (in < rot / 8) {
      pa = first + in * 4, pb = pa + rot / 2, j = in * 4;
    } else {
      pa = d0 - rot, pa += pa < first ? 0 : rot, pb = pa + 4;
    }
  }
};

template <bool BF16>
__device__ __forceinline__ void unpack4(const uint2& u, float* x) {
  const uint32_t w[2] = {u.x, u.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (BF16) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*(const __half2*)&w[i]);
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
}

// A warp takes U x 32 / (D / 8) heads of a row at a time: 16 bytes of a head a lane, D / 8 lanes a head.
// Bound by HBM in 16 bits where rows are many (8192 rows, 64 heads of 128 on 8: 336 MB in 63 us, 5.3 TB/s with
// the check of the rows, 4 us, before it; 131072 rows: 930 us, 5.8 TB/s); to 4 bits by the instructions between and the
// check (24000 rows, 8 heads of 128 of each kind, without norm and rotation: 223 MB in 65 us, of them 15 for the check; half
// of the issue slots used); by the chain position, page entry, store and one launch where rows are few (one row 3 us of device time).
template <bool FP4, int U>
constexpr int kMaxThreads = FP4 || U == 1 ? 512 : 768;   // of a CTA
template <int U>
constexpr int kStages = U == 1 ? 1 : 2;                  // chunks that a warp has on their way
template <bool FP4, int U>
constexpr int kRingBytes = kMaxThreads<FP4, U> / 32 * kStages<U> * U * 512;

template <bool BF16, int D, bool FP4, int U>
__global__ void __launch_bounds__(kMaxThreads<FP4, U>, 1) append_kernel(const __grid_constant__ AppendParams p) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr int L = D / 8;            // lanes of a head
  constexpr int H = 32 / L;           // heads that the warp has in its lanes
  constexpr int HEADS = U * H;        // of a chunk
  constexpr int STAGES = kStages<U>;
  // A warp's chunks follow one another, row by row.  To 4 bits, where they are many, the warp takes the first and every
  // per_row-th after it, then the second and those after it, and so on: what depends on a chunk's kind and heads is set up
  // when they change, and rows are looked up ahead.  (96000 rows of 3 x 8 heads of 128: 462 -> 430 us.)
  constexpr bool BY_KIND = FP4 && U > 1;
  extern __shared__ __align__(128) unsigned char shared[];
  const int lane = threadIdx.x & 31, in = lane % L, sub = lane / L;
  const int warps = blockDim.x >> 5;
  const int32_t qc = p.q.data ? (p.q_heads + HEADS - 1) / HEADS : 0, kc = (p.kv_heads + HEADS - 1) / HEADS;
  const int32_t per_row = qc + kc + (p.v.data ? kc : 0);
  const uint32_t chunks = (uint32_t)p.rows * per_row, workers = gridDim.x * warps;   // (below 2^31 and 2^13)
  const bool halves = p.rope && !p.pairs;
  const Dims wide(in, p.rot, p.first, halves), flat(in, p.rot, p.first, false);

  // Chunk `i` of a row, its heads h0 .. of kind 0 query, 1 key, 2 value.
  struct Chunk {
    int32_t row, i;
    uint32_t x, lap;     // (by kind) its number in the call, and how often the warp began anew
  };
  uint32_t first = 0, end = 0;   // the warp's chunks
  auto kind_of = [&](const Chunk& x) { return x.i < qc ? 0 : x.i < qc + kc ? 1 : 2; };
  auto first_head = [&](const Chunk& x, int kind) { return (x.i - (kind == 0 ? 0 : kind == 1 ? qc : qc + kc)) * HEADS; };
  auto advance = [&](Chunk& x) {
    if constexpr (BY_KIND) {
      ++x.row, x.x += per_row;
      if (x.x < end) return;
      x.x = first + ++x.lap;
      x.row = (int32_t)(x.x / (uint32_t)per_row), x.i = (int32_t)x.x - x.row * per_row;
    } else {
      if (++x.i == per_row) x.i = 0, ++x.row;
    }
  };
  // The warp's ring: a chunk's heads one after another as they are.
  unsigned char* ring = shared + (size_t)p.table_bytes + (threadIdx.x >> 5) * (STAGES * U * 512);
  const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
  uint32_t to_fetch = 0, left = 0;   // chunks
  Chunk ahead{}, at_chunk{};
  // this lane's first piece of a row's chunk, how far rows and its pieces are apart, and the heads from it on
  const T* from = nullptr;
  int64_t from_row = 0, from_step = 0;
  int32_t from_heads = 0;
  auto aim = [&]() {
    const int kind = kind_of(ahead);
    const int32_t h = first_head(ahead, kind) + sub;
    const HeadsIn& x = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
    from_heads = (kind == 0 ? p.q_heads : p.kv_heads) - h;
    from = (const T*)x.data + h * x.head + in * 8;
    from_row = x.row, from_step = H * x.head;
  };
  auto fetch = [&](int stage) {
    if (to_fetch > 0) {
      // every lane has read the stage: what is rotated half by half is read from pieces that other lanes copy
      __syncwarp();
      --to_fetch;
      if (!BY_KIND) aim();
      const T* at = from + ahead.row * from_row;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool on = u * H < from_heads;
        copy_async(ring_at + (uint32_t)((stage * U + u) * 512 + lane * 16), on ? at + u * from_step : (const T*)p.k.data, on ? 16u : 0u);
      }
      const uint32_t lap = ahead.lap;
      advance(ahead);
      if (BY_KIND && ahead.lap != lap) aim();
    }
    commit_async();
  };
  {
    // consecutive warps on different SMs
    const uint32_t w = (threadIdx.x >> 5) * gridDim.x + blockIdx.x, per = chunks / workers, more = chunks - per * workers;
    const uint32_t c = w * per + min(w, more);
    left = to_fetch = per + (w < more ? 1 : 0);
    first = c, end = c + left;
    ahead.row = (int32_t)(c / (uint32_t)per_row);
    ahead.i = (int32_t)c - ahead.row * per_row;
    ahead.x = c;
    at_chunk = ahead;
    if (BY_KIND && left > 0) aim();
  }
#pragma unroll
  for (int i = 0; i < STAGES; ++i) fetch(i);
  int32_t pos = -1, next_pos = -1, next_req = 0;
  if (left > 0) next_pos = p.row_pos[at_chunk.row], next_req = p.row_req[at_chunk.row];
  const uint32_t err = check_rows(p, (uint32_t*)shared);
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status_out = err;
  if (err != kOk) {
    // nothing was written; queries that have a place of their own become NaN
    wait_async<0>();
    if (!p.out_q || p.q_in_place) return;
    const int64_t n = (int64_t)p.rows * p.q_heads;
    for (int64_t i = (int64_t)blockIdx.x * warps + (threadIdx.x >> 5); i < n; i += workers) {
      const int64_t r = i / p.q_heads, h = i - r * p.q_heads;
      if (p.out_q_scale) {
        for (int j = lane; j < D / 2; j += 32) ((uint8_t*)p.out_q)[r * p.oq_row + h * p.oq_head + j] = 0;
        if (lane < D / kFp4Block) p.out_q_scale[r * p.oqs_row + h * p.oqs_head + lane] = 255;
      } else {
        for (int j = lane; j < D; j += 32) ((T*)p.out_q)[r * p.oq_row + h * p.oq_head + j] = (T)__uint_as_float(0x7FC00000u);
      }
    }
    return;
  }

  // what the chunk's kind and heads decide
  int kind = 0, pa = 0, pb = 0, j = -1;
  int32_t h0 = 0, heads = 0;
  bool four = false, apart = false;                          // becomes codes; is rotated half by half
  const void* weight = nullptr;
  char* to0 = nullptr;                                       // its first place in row 0 (queries) or slot 0 of page 0
  uint8_t* st0 = nullptr;
  int64_t by_page = 0, by_slot = 0, s_by_page = 0, s_by_slot = 0, head = 0, s_head = 0;   // (bytes, bytes; elements or bytes)
  float w4[FP4 ? 8 : 1];
  auto set_up = [&](const Chunk& chunk) {
    kind = kind_of(chunk);
    h0 = first_head(chunk, kind), heads = kind == 0 ? p.q_heads : p.kv_heads;
    four = FP4 && (kind > 0 || p.out_q_scale);
    weight = kind == 0 ? p.q_weight : kind == 1 ? p.k_weight : nullptr;
    apart = halves && kind < 2 && !four;
    pa = apart ? wide.pa : flat.pa, pb = apart ? wide.pb : flat.pb, j = apart ? wide.j : flat.j;
    const PagedOut& dst = kind == 1 ? p.k_dst : p.v_dst;
    const int64_t size = four ? 1 : sizeof(T);
    head = kind == 0 ? p.oq_head : dst.head;
    to0 = (char*)(kind == 0 ? p.out_q : dst.data) + (h0 + sub) * head * size;
    by_page = (kind == 0 ? p.oq_row : dst.page) * size, by_slot = kind == 0 ? 0 : dst.slot * size;
    if constexpr (FP4) {
      s_head = kind == 0 ? p.oqs_head : dst.s_head;
      st0 = (kind == 0 ? p.out_q_scale : dst.scale) + (h0 + sub) * s_head + in / 4;
      s_by_page = kind == 0 ? p.oqs_row : dst.s_page, s_by_slot = kind == 0 ? 0 : dst.s_slot;
      if (four && weight) {
        if (p.weight_f32) {
          *(float4*)&w4[0] = *(const float4*)((const float*)weight + pa);
          *(float4*)&w4[4] = *(const float4*)((const float*)weight + pb);
        } else {
          unpack4<BF16>(*(const uint2*)((const T*)weight + pa), &w4[0]);
          unpack4<BF16>(*(const uint2*)((const T*)weight + pb), &w4[4]);
        }
      }
    }
  };
  auto page_of = [&](int32_t pos, int32_t req) { return pos >= 0 ? p.page_table[(int64_t)req * p.max_pages + pos / kPage] : 0; };
  // (a position is asked for two chunks before it is used, its page one)
  int32_t after_pos = -1, after_req = 0;
  auto look_after = [&](Chunk x, uint32_t behind) {
    advance(x);
    if (left > behind) after_pos = p.row_pos[x.row], after_req = p.row_req[x.row];
  };
  int stage = 0;
  int32_t page = 0, next_page = 0;
  if constexpr (BY_KIND) {
    if (left > 0) next_page = page_of(next_pos, next_req), look_after(at_chunk, 1);
  }
  for (bool fresh = true; left > 0; --left, fetch(stage), stage = stage == STAGES - 1 ? 0 : stage + 1) {
    const Chunk chunk = at_chunk;
    advance(at_chunk);
    const int32_t row = chunk.row;
    if constexpr (BY_KIND) {
      if (fresh) set_up(chunk);
      fresh = at_chunk.lap != chunk.lap;
      pos = next_pos, page = next_page, next_pos = after_pos, next_req = after_req;
      if (left > 1) next_page = page_of(next_pos, next_req);
      look_after(at_chunk, 2);
    } else {
      if (fresh) {
        pos = next_pos, page = page_of(next_pos, next_req);
        if (row + 1 < p.rows) next_pos = p.row_pos[row + 1], next_req = p.row_req[row + 1];
      }
      fresh = at_chunk.i == 0;
      set_up(chunk);
    }
    wait_async<STAGES - 1>();
    __syncwarp();
    if (pos < 0) continue;            // a row that is not there
    // this lane's elements of the chunk's heads
    const unsigned char* mine = ring + stage * (U * 512) + sub * (L * 16);
    const int64_t at = kind == 0 ? row : page;
    const int32_t off = pos % kPage;
    char* const to_row = to0 + at * by_page + off * by_slot;
    if (!four) {
      // ---- 16 bits: sums in fp32, one rounding at the end ----
      T *ta = (T*)to_row + pa, *tb = (T*)to_row + pb;
      const int64_t step = H * head;
      if (kind == 2) {                // a copy
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (h0 + u * H + sub < heads) *(uint4*)(ta + u * step) = *(const uint4*)(mine + u * 512 + pa * 2);
        continue;
      }
      // Pairs: of dimensions that are turned alike, (0, 1), (2, 3) and their partners (4, 5), (6, 7) where those lie in the
      // other group, else (0, 2) and (1, 3), (4, 6) and (5, 7).
      auto pairs = [&](const float (&x)[8], Two (&t)[4]) {
        if (apart) {
          t[0] = two(x[0], x[1]), t[1] = two(x[2], x[3]), t[2] = two(x[4], x[5]), t[3] = two(x[6], x[7]);
        } else {
          t[0] = two(x[0], x[2]), t[1] = two(x[4], x[6]), t[2] = two(x[1], x[3]), t[3] = two(x[5], x[7]);
        }
      };
      Two w[4], co[2], si[2], minus[2];
      if (weight) {
        float y[8];
        if (p.weight_f32) {
          *(float4*)&y[0] = *(const float4*)((const float*)weight + pa);
          *(float4*)&y[4] = *(const float4*)((const float*)weight + pb);
        } else {
          unpack4<BF16>(*(const uint2*)((const T*)weight + pa), &y[0]);
          unpack4<BF16>(*(const uint2*)((const T*)weight + pb), &y[4]);
        }
        pairs(y, w);
      }
      if (j >= 0) {
        const float* t = p.rope + (int64_t)pos * p.rot + j;
        const float4 x = *(const float4*)t, y = *(const float4*)(t + p.rot / 2);
        co[0] = two(x.x, x.y), co[1] = two(x.z, x.w), si[0] = two(y.x, y.y), si[1] = two(y.z, y.w);
        minus[0] = two(-y.x, -y.y), minus[1] = two(-y.z, -y.w);
      }
      // (the branches outside the loop over the heads)
      auto heads_of = [&](auto normed, auto lies_apart, auto full) {
        constexpr bool NORM = decltype(normed)::value, APART = decltype(lies_apart)::value, FULL = decltype(full)::value;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (!FULL && h0 + u * H >= heads) break;   // (the same for the whole warp)
          Two t[4];
          {
            float x[8];
            if (APART) {
              unpack4<BF16>(*(const uint2*)(mine + u * 512 + pa * 2), &x[0]);
              unpack4<BF16>(*(const uint2*)(mine + u * 512 + pb * 2), &x[4]);
              t[0] = two(x[0], x[1]), t[1] = two(x[2], x[3]), t[2] = two(x[4], x[5]), t[3] = two(x[6], x[7]);
            } else {
              unpack8<BF16>(*(const uint4*)(mine + u * 512 + pa * 2), x);
              t[0] = two(x[0], x[2]), t[1] = two(x[4], x[6]), t[2] = two(x[1], x[3]), t[3] = two(x[5], x[7]);
            }
          }
          if constexpr (NORM) {
            const float2 q = both(fma2(t[3], t[3], fma2(t[2], t[2], fma2(t[1], t[1], mul2(t[0], t[0])))));
            float s = q.x + q.y;
#pragma unroll
            for (int o = 1; o < L; o <<= 1) s += __shfl_xor_sync(~0u, s, o);
            const float r = rsqrtf(fmaf(s, 1.f / D, p.eps));
            const Two rr = two(r, r);
#pragma unroll
            for (int i = 0; i < 4; ++i) t[i] = mul2(mul2(t[i], rr), w[i]);
          }
          if (j >= 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const Two a = t[i], b = t[i + 2];
              t[i] = fma2(a, co[i], mul2(b, minus[i]));
              t[i + 2] = fma2(b, co[i], mul2(a, si[i]));
            }
          }
          if (FULL || h0 + u * H + sub < heads) {
            const float2 a = both(t[0]), b = both(t[1]), c = both(t[2]), d = both(t[3]);
            if (APART) {
              const float x[8] = {a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
              const uint4 o = pack8<BF16>(x);
              *(uint2*)(ta + u * step) = make_uint2(o.x, o.y);
              *(uint2*)(tb + u * step) = make_uint2(o.z, o.w);
            } else {
              const float x[8] = {a.x, c.x, a.y, c.y, b.x, d.x, b.y, d.y};
              *(uint4*)(ta + u * step) = pack8<BF16>(x);
            }
          }
        }
      };
      auto by_fill = [&](auto normed, auto lies_apart) {
        if (h0 + HEADS <= heads)
          heads_of(normed, lies_apart, std::true_type{});
        else
          heads_of(normed, lies_apart, std::false_type{});
      };
      if (weight && apart)
        by_fill(std::true_type{}, std::true_type{});
      else if (weight)
        by_fill(std::true_type{}, std::false_type{});
      else if (apart)
        by_fill(std::false_type{}, std::true_type{});
      else
        by_fill(std::false_type{}, std::false_type{});
      continue;
    }
    // ---- 4 bits: every rounding in the documented order ----
    if constexpr (FP4) {
      const bool turn = p.rope && kind < 2, turned = turn && flat.j >= 0;
      // the angles of this lane's dimensions: 4 pairs of neighbours, or 8 of a half whose partners another lane has
      bool upper = false;
      int partner = lane;
      float co[8], si[8];                // (halves: the sines with the sign that the lane's half has)
      if (turned) {
        const float* t = p.rope + (int64_t)pos * p.rot;
        if (p.pairs) {
          *(float4*)&co[0] = *(const float4*)(t + flat.j);
          *(float4*)&si[0] = *(const float4*)(t + p.rot / 2 + flat.j);
        } else {
          int j = 2 * flat.j;
          upper = j >= p.rot / 2;
          partner = upper ? lane - p.rot / 16 : lane + p.rot / 16;
          if (upper) j -= p.rot / 2;
#pragma unroll
          for (int i = 0; i < 8; i += 4) {
            *(float4*)&co[i] = *(const float4*)(t + j + i);
            *(float4*)&si[i] = *(const float4*)(t + p.rot / 2 + j + i);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) si[i] = upper ? si[i] : -si[i];
        }
      }
      uint8_t* to = (uint8_t*)to_row + in * 4;
      uint8_t* st = st0 + at * s_by_page + off * s_by_slot;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (h0 + u * H >= heads) break;   // (the same for the whole warp)
        float x[8];
        unpack8<BF16>(*(const uint4*)(mine + u * 512 + pa * 2), x);
        if (weight) {
          // squares of 16-bit numbers are exact in fp32
          Two s2 = two(x[0], x[1]), rest2 = two(0.f, 0.f);
          s2 = mul2(s2, s2);
#pragma unroll
          for (int i = 2; i < 8; i += 2) {
            const Two t = two(x[i], x[i + 1]);
            add_exactly(s2, rest2, mul2(t, t));
          }
          const float2 ss = both(s2), rr = both(rest2);
          float s = ss.x, rest = __fadd_rn(rr.x, rr.y), less = 0.f;
          add_exactly(s, less, ss.y);
          rest = __fadd_rn(rest, less);
#pragma unroll
          for (int o = 1; o < L; o <<= 1) {
            const float s1 = __shfl_xor_sync(~0u, s, o), r1 = __shfl_xor_sync(~0u, rest, o);
            rest = __fadd_rn(rest, r1);
            float r2 = 0.f;
            add_exactly(s, r2, s1);
            rest = __fadd_rn(rest, r2);
          }
          const float sum = fabsf(s) < INFINITY ? __fadd_rn(s, rest) : s;
          const float r = __fdiv_rn(1.f, __fsqrt_rn(__fadd_rn(sum / D, p.eps)));
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float2 y = both(mul2(mul2(two(x[i], x[i + 1]), two(r, r)), two(w4[i], w4[i + 1])));
            x[i] = y.x, x[i + 1] = y.y;
          }
        }
        if (turn) {
          if (p.pairs) {
            if (turned) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float a = x[2 * i], b = x[2 * i + 1];
                x[2 * i] = __fsub_rn(__fmul_rn(a, co[i]), __fmul_rn(b, si[i]));
                x[2 * i + 1] = __fadd_rn(__fmul_rn(b, co[i]), __fmul_rn(a, si[i]));
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              const float o0 = __shfl_sync(~0u, x[i], partner), o1 = __shfl_sync(~0u, x[i + 1], partner);
              if (turned) {
                // (one by one: a packed sum and a packed product that it takes may become one operation, of one rounding)
                x[i] = __fadd_rn(__fmul_rn(x[i], co[i]), __fmul_rn(o0, si[i]));
                x[i + 1] = __fadd_rn(__fmul_rn(x[i + 1], co[i + 1]), __fmul_rn(o1, si[i + 1]));
              }
            }
          }
        }
        // (as integers from here on: a NaN counts as the largest)
        uint32_t top = __float_as_uint(larger(larger(larger(x[0], x[1]), larger(x[2], x[3])),
                                              larger(larger(x[4], x[5]), larger(x[6], x[7]))));
        top = max(top, __shfl_xor_sync(~0u, top, 1));
        top = max(top, __shfl_xor_sync(~0u, top, 2));
        const uint32_t e = scale_byte(top), codes = to_codes(x, e);
        if (h0 + u * H + sub < heads) {
          *(uint32_t*)(to + u * (H * head)) = codes;
          if (in % 4 == 0) st[u * (H * s_head)] = (uint8_t)e;
        }
      }
    }
  }
}

// 32 bytes to a 32-byte boundary.
__device__ __forceinline__ void store32(void* a, const uint4& x, const uint4& y) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(a), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w),
               "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w)
               : "memory");
}

// Listed slots of a 4-bit cache as 16-bit rows, rounded once (exact unless beyond the type's range or below its
// last place): 8 bytes of codes, 16 elements, a thread.  Bound by HBM: 0.53 bytes read and 2 written an element.
// The last CTA only looks for slots that are none.
template <bool BF16, int D, int U>
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const __grid_constant__ GatherParams p) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr int L = D / 16;             // threads of a head
  const int32_t most = p.num_pages * kPage;
  if (blockIdx.x == gridDim.x - 1) {
    bool bad = false;
#pragma unroll 8
    for (int32_t i = threadIdx.x; i < p.n; i += kGatherThreads) bad |= p.slots[i] < -1 || p.slots[i] >= most;
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *p.status_out = bad ? kErrInvalidPage : kOk;
    return;
  }
  const uint32_t j = threadIdx.x % L;
  const int32_t step = (int32_t)(gridDim.x - 1) * (kGatherThreads / L);   // heads from one of a thread's to its next
  const int32_t dr = step / p.kv_heads, dh = step - dr * p.kv_heads;
  const int32_t v0 = (int32_t)blockIdx.x * (kGatherThreads / L) + (int32_t)threadIdx.x / L;
  int32_t r = v0 / p.kv_heads, h = v0 - r * p.kv_heads;
  while (r < p.n) {
    int32_t rs[U], hs[U], slots[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rs[u] = r, hs[u] = h;
      slots[u] = r < p.n ? p.slots[r] : -1;
      r += dr, h += dh;
      if (h >= p.kv_heads) h -= p.kv_heads, ++r;
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const GatherParams::From& f = p.t[t];
      if (!f.codes) continue;
      uint2 codes[U];
      uint32_t e[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        codes[u] = make_uint2(0, 0), e[u] = slots[u] == -1 ? 127u : 255u;   // what is no slot becomes NaN
        if (slots[u] < 0 || slots[u] >= most) continue;
        const uint32_t page = (uint32_t)slots[u] / kPage, off = (uint32_t)slots[u] % kPage, head = (uint32_t)hs[u];
        if (p.far) {
          codes[u] = *(const uint2*)(f.codes + (page * f.page + off * f.slot + head * f.head) + j * 8);
          e[u] = f.scale[page * f.s_page + off * f.s_slot + head * f.s_head + j / 2];
        } else {
          const uint32_t at16 = page * (uint32_t)(f.page / 16) + off * (uint32_t)(f.slot / 16) + head * (uint32_t)(f.head / 16);
          codes[u] = *(const uint2*)(f.codes + (uint64_t)at16 * 16 + j * 8);
          e[u] = f.scale[page * (uint32_t)f.s_page + off * (uint32_t)f.s_slot + head * (uint32_t)f.s_head + j / 2];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (rs[u] >= p.n) break;
        const float s = scale_of(e[u]);
        uint4 out[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t w[4];
          from_codes(x ? codes[u].y : codes[u].x, w);
          float y[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 z = __half22float2(*(const __half2*)&w[k]);
            y[2 * k] = z.x * s, y[2 * k + 1] = z.y * s;
          }
          out[x] = pack8<BF16>(y);
        }
        T* to = (T*)f.out + rs[u] * f.row + hs[u] * f.out_head + j * 16;
        if (p.wide) {   // (65535 slots x 8 heads 72 us, in halves 85)
          store32(to, out[0], out[1]);
        } else {
          *(uint4*)to = out[0], *(uint4*)(to + 8) = out[1];
        }
      }
    }
  }
}

template <bool BF16, int D, bool FP4, int U>
cudaError_t launch_append_u(const AppendParams& p, int threads, int grid, cudaStream_t stream) {
  auto* kernel = append_kernel<BF16, D, FP4, U>;
  static std::atomic<bool> done[64];
  cudaError_t e = set_smem_once(kernel, kTableBytes + kRingBytes<FP4, U>, done);
  if (e != cudaSuccess) return e;
  kernel<<<grid, threads, p.table_bytes + threads / 32 * kStages<U> * U * 512, stream>>>(p);
  return cudaGetLastError();
}

template <bool BF16, int D, bool FP4>
cudaError_t launch_append_as(AppendParams p, int sm, cudaStream_t stream) {
  constexpr int H = 32 / (D / 8);
  auto chunks = [&](int heads) {
    const int64_t q = p.q.data ? (p.q_heads + heads - 1) / heads : 0, k = (p.kv_heads + heads - 1) / heads;
    return p.rows * (q + k * (p.v.data ? 2 : 1));
  };
  // Few chunks: one head's worth a lane, small CTAs on as many SMs as there are.  Many: four in flight a lane, one CTA an SM
  // (every CTA looks over all rows).  Measured (us between events; one head, four), 128 elements, 64 heads on 8:
  // to 4 bits, 4 chunks an SM 13, 17, 8 chunks 15, 15, 16 chunks 15, 17, 26 chunks 19, 17, 45 chunks 23, 19; in
  // 16 bits, up to 16 chunks 9, 9, 26 chunks 11, 11, 45 chunks 15, 11.
  // The slots named twice are found in a table with room for twice the rows.  Past 2^14 rows it would not fit, and a bitmap
  // does it, which takes a walk over the rows for every 2^20 slots (one walk: as fast as the table, 8208 rows 37.5 us with
  // either; bits of neighbouring slots in one word instead: 96000 rows 418 -> 430).  So the cost grows with the pool: 32768
  // rows of one head of 64, keys only, pools of 2^18 and 2^20 slots 40 us, 2^22 91, 2^24 298, 2^26 1117.  A table that is
  // nearly half full takes longer than the bitmap's one walk: 16384 such rows 48 to 76 us, 24000 with the bitmap 31.
  const int64_t slots = (int64_t)p.num_pages * kPage;
  int table = 0, map = 6;
  for (int b = 6; b <= kMostBits && !table; ++b)
    if ((int64_t)1 << b >= 2 * (int64_t)p.rows) table = b;
  while (map < kMostBits && (int64_t)32 << map < slots) ++map;
  p.bitmap = !table;
  p.table_bits = p.bitmap ? map : table;
  p.table_bytes = 4 << p.table_bits;
  if (chunks(H) <= (int64_t)sm * 16) {
    const int64_t n = chunks(H);
    const int64_t want = (n + sm - 1) / sm;      // warps an SM
    const int warps = want <= 4 ? 4 : want <= 8 ? 8 : 16;
    const int64_t grid = (n + warps - 1) / warps;
    return launch_append_u<BF16, D, FP4, 1>(p, warps * 32, (int)(grid < 1 ? 1 : grid), stream);
  }
  return launch_append_u<BF16, D, FP4, 4>(p, kMaxThreads<FP4, 4>, sm, stream);
}

template <bool BF16>
cudaError_t launch_append_dim(const AppendParams& p, int dim, bool fp4, int sm, cudaStream_t stream) {
  if (fp4) {
    if (dim == 64) return launch_append_as<BF16, 64, true>(p, sm, stream);
    if (dim == 128) return launch_append_as<BF16, 128, true>(p, sm, stream);
    return launch_append_as<BF16, 256, true>(p, sm, stream);
  }
  if (dim == 64) return launch_append_as<BF16, 64, false>(p, sm, stream);
  if (dim == 128) return launch_append_as<BF16, 128, false>(p, sm, stream);
  return launch_append_as<BF16, 256, false>(p, sm, stream);
}

template <bool BF16, int D>
cudaError_t launch_gather_as(const GatherParams& p, int sm, cudaStream_t stream) {
  // One head a thread where that is a few waves of CTAs, else four at a time.  Measured (us between events; one, four),
  // 128 elements: 512 slots x 1 head 7, 9; x 8 heads: 1000 slots 9, 9, 4000 13, 13, 8000 17, 19, 16000 25, 27, 65535 79, 72.
  const int64_t ctas = ((int64_t)p.n * p.kv_heads * (D / 16) + kGatherThreads - 1) / kGatherThreads;
  if (ctas <= 32 * (int64_t)sm)
    gather_kernel<BF16, D, 1><<<(int)ctas + 1, kGatherThreads, 0, stream>>>(p);
  else
    gather_kernel<BF16, D, 4><<<sm * 4 + 1, kGatherThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <bool BF16>
cudaError_t launch_gather_dim(const GatherParams& p, int dim, int sm, cudaStream_t stream) {
  if (dim == 64) return launch_gather_as<BF16, 64>(p, sm, stream);
  if (dim == 128) return launch_gather_as<BF16, 128>(p, sm, stream);
  return launch_gather_as<BF16, 256>(p, sm, stream);
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, bool bf16, int dim, bool fp4, int sm_count, cudaStream_t stream) {
  return bf16 ? launch_append_dim<true>(p, dim, fp4, sm_count, stream)
              : launch_append_dim<false>(p, dim, fp4, sm_count, stream);
}

cudaError_t launch_gather(const GatherParams& p, bool bf16, int dim, int sm_count, cudaStream_t stream) {
  return bf16 ? launch_gather_dim<true>(p, dim, sm_count, stream) : launch_gather_dim<false>(p, dim, sm_count, stream);
}

}  // namespace idxk
