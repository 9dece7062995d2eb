// What follows the attention kernel: the join of the units that were cut, and the
// accumulated weights.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "attn.h"
#include "idx_launch.h"

namespace idxk {

cudaError_t launch_attn_pages(const AttnParams& p, bool bf16, int sm_count, cudaStream_t stream);
cudaError_t launch_attn_slots(const AttnParams& p, bool bf16, int sm_count, cudaStream_t stream);
cudaError_t launch_attn_tc(const AttnParams& p, bool bf16, int sm_count, cudaStream_t stream);
cudaError_t launch_attn_tc_fp4(const AttnParams& p, bool bf16, int sm_count, cudaStream_t stream);
cudaError_t launch_attn_fp4_pages(const AttnParams& p, bool bf16, int sm_count, cudaStream_t stream);
cudaError_t launch_attn_fp4_slots(const AttnParams& p, bool bf16, int sm_count, cudaStream_t stream);

cudaError_t launch_attn(const AttnParams& p, bool bf16, int sm_count, cudaStream_t stream) {
  if (p.k_scale && p.tensor_core) return launch_attn_tc_fp4(p, bf16, sm_count, stream);
  if (p.k_scale)
    return p.slots ? launch_attn_fp4_slots(p, bf16, sm_count, stream) : launch_attn_fp4_pages(p, bf16, sm_count, stream);
  if (p.tensor_core) return launch_attn_tc(p, bf16, sm_count, stream);
  return p.slots ? launch_attn_slots(p, bf16, sm_count, stream) : launch_attn_pages(p, bf16, sm_count, stream);
}

namespace {

__device__ __forceinline__ float pow2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// First error of the CTAs of the attention kernel, seen by every thread.
__device__ uint32_t call_status(const AttnParams& p) {
  uint32_t e = kOk;
  for (int i = threadIdx.x; i < p.n_cta; i += blockDim.x) e = max(e, p.cta_status[i]);
  for (int o = 16; o; o >>= 1) e = max(e, __shfl_xor_sync(~0u, e, o));
  __shared__ uint32_t all;
  if (threadIdx.x == 0) all = kOk;
  __syncthreads();
  if ((threadIdx.x & 31) == 0 && e != kOk) atomicMax(&all, e);
  __syncthreads();
  return all;
}

// Units of at most so many parts are joined by one warp a tile row (32 requests x 2 rows x 64 heads on one:
// 116 us with 4, 110 with 8, 107 with 16, 106 with 32).
constexpr int kFewParts = 16;
constexpr int kLooks = 5;   // ranges that a thread looks at together

struct OpenUnit {
  uint16_t w0, n;               // first worker and parts
  int32_t row0;                 // its group's first row
  uint32_t nrows : 8, u : 24;   // its group's rows and its index in the group
};

// Parts i0, i0 + step, ... of a tile row added up by one warp; a lane has D / 32 columns.
template <int D>
__device__ __forceinline__ void join_parts(const AttnParams& p, const OpenUnit& un, int m, int i0, int step, float& M,
                                           float& l, float (&acc)[D / 32], bool& seen) {
  constexpr int V = D / 32, U = 4;   // U parts in flight
  const int lane = threadIdx.x & 31;
  M = -INFINITY, l = 0.f, seen = false;
#pragma unroll
  for (int x = 0; x < V; ++x) acc[x] = 0.f;
  for (; i0 < un.n; i0 += step * U) {
    float2 ml[U];
    float o[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * step;
      ml[u] = make_float2(-INFINITY, -1.f);
#pragma unroll
      for (int x = 0; x < V; ++x) o[u][x] = 0.f;
      if (i < un.n) {
        const int64_t part = ((int64_t)(un.w0 + i) * 2 + (i == 0 ? 1 : 0)) * p.tile + m;
        ml[u] = p.part_ml[part];
        const float* src = p.part_o + part * D + lane * V;
#pragma unroll
        for (int x = 0; x < V; x += 2) {
          const float2 t = *(const float2*)(src + x);
          o[u][x] = t.x, o[u][x + 1] = t.y;
        }
      }
    }
    // a sum of -1: the part saw no position (its values mean nothing)
    float top = M;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (ml[u].y != -1.f) top = fmaxf(top, ml[u].x);
    const float base = reference(top);
    const float a = pow2(exponent(M, base, p.scale_log2));
    l *= a;
#pragma unroll
    for (int x = 0; x < V; ++x) acc[x] *= a;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (ml[u].y == -1.f) continue;
      seen = true;
      const float e = pow2(exponent(ml[u].x, base, p.scale_log2));
      l += ml[u].y * e;
#pragma unroll
      for (int x = 0; x < V; ++x) acc[x] += o[u][x] * e;
    }
    M = top;
  }
}

// One tile row (query head x row) of one cut unit at a time: its parts lie with the worker
// that opened the unit (part 1) and the workers after it (part 0), and
//   M = max m_i, l = sum l_i 2^(c (m_i - M)), out = sum o_i 2^(c (m_i - M)) / l.
// Where a unit has few parts, each warp joins a row by itself; where it has many (few rows
// over a long context), the warps of a CTA take the row's parts in turn, in a fixed order,
// and their sums are joined in the same way.  Bound by the latency of a chain of loads: the ranges' ends,
// the parts.  CTAs of 16 warps look over the 1216 ranges and more of attn.cuh, CTAs of 8 the one an SM of
// attn_tc.cuh (48 requests x 3 rows x 16 heads: 61 us with 16 warps, 64 with 8; 32 requests x 2 rows x 64
// heads on one: 115 and 113).
template <bool BF16, int D, int kJoinWarps>
__global__ void __launch_bounds__(kJoinWarps * 32, 32 / kJoinWarps) attn_join_kernel(const __grid_constant__ AttnParams p) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr int V = D / 32;   // columns of a lane
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  extern __shared__ OpenUnit open[];   // [workers]: units of few parts from the front, others from the back
  __shared__ uint32_t warp_n[kLooks][kJoinWarps];
  __shared__ float wm[kJoinWarps], wl[kJoinWarps];
  __shared__ float wo[kJoinWarps][D];
  allow_launch_after();
  wait_for_launch_before();
  // the first ranges' ends (what lies beyond the workers that had a range is read too, and means nothing)
  constexpr int N = kJoinWarps * 32;
  int n[kLooks];
#pragma unroll
  for (int i = 0; i < kLooks; ++i) n[i] = (int)threadIdx.x + i * N < p.workers ? p.open_parts[threadIdx.x + i * N] : 0;
  int4 info = (int)threadIdx.x < p.workers ? p.open_info[threadIdx.x] : make_int4(0, 0, 0, 0);
  const int active = p.n_cta > 0 ? *p.active : 0;
  const uint32_t status = call_status(p);
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.status_out) *p.status_out = status;
  if (status != kOk) {
    const float nan = __uint_as_float(0x7FC00000u);
    const int64_t n = (int64_t)p.rows * p.q_heads;
    for (int64_t i = (int64_t)blockIdx.x * kJoinWarps + warp; i < n; i += (int64_t)gridDim.x * kJoinWarps) {
      const int64_t r = i / p.q_heads, h = i - r * p.q_heads;
      T* o = (T*)p.out + r * p.out_row + h * p.out_head;
      for (int j = lane; j < D; j += 32) o[j] = (T)nan;
      if (p.lse && lane == 0) p.lse[i] = nan;
    }
    return;
  }
  // the cut units, in the same order in every CTA
  uint32_t below[kLooks][2];
#pragma unroll
  for (int i = 0; i < kLooks; ++i) {
    if ((int)threadIdx.x + i * N >= active) n[i] = 0;
    const uint32_t bf = __ballot_sync(~0u, n[i] > 0 && n[i] <= kFewParts), bm = __ballot_sync(~0u, n[i] > kFewParts);
    if (lane == 0) warp_n[i][warp] = (uint32_t)__popc(bf) | (uint32_t)__popc(bm) << 16;
    below[i][0] = __popc(bf & ((1u << lane) - 1)), below[i][1] = __popc(bm & ((1u << lane) - 1));
  }
  __syncthreads();
  uint32_t all = 0;   // few, and 65536 times the others
#pragma unroll
  for (int i = 0; i < kLooks; ++i) {
    if (i * N >= active) break;
    uint32_t before = all;
#pragma unroll
    for (int x = 0; x < kJoinWarps; ++x) {
      const uint32_t c = warp_n[i][x];
      if (x < warp) before += c;
      all += c;
    }
    if (n[i] == 0) continue;
    const int w = (int)threadIdx.x + i * N;
    if (i > 0) info = p.open_info[w];
    OpenUnit un;
    un.w0 = (uint16_t)w, un.n = (uint16_t)n[i], un.row0 = info.x, un.nrows = info.y, un.u = info.z;
    open[n[i] <= kFewParts ? (before & 0xFFFF) + below[i][0] : p.workers - 1 - (before >> 16) - below[i][1]] = un;
  }
  __syncthreads();
  const int few = all & 0xFFFF, many = all >> 16;
  // the output row of tile row m: false where it is none, or sees nothing
  auto row_of = [&](const OpenUnit& un, int m, int64_t& row, int& qh) {
    const int j = m / p.row_cols, h = m - j * p.row_cols;
    const int in_group = un.u % p.chunks * p.chunk_heads + h;
    row = un.row0 + j;
    qh = un.u / p.chunks * p.group + in_group;
    return j < un.nrows && h < p.chunk_heads && in_group < p.group;
  };
  for (int job = blockIdx.x * kJoinWarps + warp; job < few * p.tile; job += gridDim.x * kJoinWarps) {
    const int m = job / few;   // (a group's first rows first: its last are often not there)
    const OpenUnit un = open[job - m * few];
    int64_t row;
    int qh;
    if (!row_of(un, m, row, qh)) continue;
    const int32_t a = p.slots ? 0 : p.row_start[row], b = p.slots ? 1 : p.row_end[row];
    float M, l, acc[V];
    bool seen;
    join_parts<D>(p, un, m, 0, 1, M, l, acc, seen);
    if (b <= a) continue;   // the row sees nothing, and its parts mean nothing
    const float inv = seen ? 1.f / l : 0.f;
    T* dst = (T*)p.out + row * p.out_row + (int64_t)qh * p.out_head + lane * V;
#pragma unroll
    for (int x = 0; x < V; ++x) dst[x] = (T)(acc[x] * inv);
    if (lane == 0) {
      const int64_t at = row * p.q_heads + qh;
      if (p.lse) p.lse[at] = log_sum_exp<BF16>(M, l, p.scale_log2);
      if (p.row_stat) p.row_stat[at] = make_float2(M == -INFINITY ? 0.f : M, inv * kShiftUp<BF16>);
    }
  }
  for (int job = blockIdx.x; job < many * p.tile; job += gridDim.x) {
    const int m = job / many;
    const OpenUnit un = open[p.workers - 1 - (job - m * many)];
    int64_t row;
    int qh;
    // the same for the whole CTA
    if (!row_of(un, m, row, qh) || (!p.slots && p.row_end[row] <= p.row_start[row])) continue;
    float M, l, acc[V];
    bool seen;
    join_parts<D>(p, un, m, warp, kJoinWarps, M, l, acc, seen);
    if (lane == 0) wm[warp] = M, wl[warp] = seen ? l : -1.f;
#pragma unroll
    for (int x = 0; x < V; ++x) wo[warp][lane * V + x] = acc[x];
    __syncthreads();
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kJoinWarps; ++i) top = fmaxf(top, wm[i]);
    const float base = reference(top);
    float total = 0.f;
    bool any = false;
#pragma unroll
    for (int i = 0; i < kJoinWarps; ++i)
      if (wl[i] != -1.f) any = true, total += wl[i] * pow2(exponent(wm[i], base, p.scale_log2));
    const float inv = any ? 1.f / total : 0.f;
    T* dst = (T*)p.out + row * p.out_row + (int64_t)qh * p.out_head;
    for (int x = threadIdx.x; x < D; x += kJoinWarps * 32) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kJoinWarps; ++i)
        if (wl[i] != -1.f) sum += wo[i][x] * pow2(exponent(wm[i], base, p.scale_log2));
      dst[x] = (T)(sum * inv);
    }
    if (threadIdx.x == 0) {
      const int64_t at = row * p.q_heads + qh;
      if (p.lse) p.lse[at] = log_sum_exp<BF16>(top, total, p.scale_log2);
      if (p.row_stat) p.row_stat[at] = make_float2(top == -INFINITY ? 0.f : top, inv * kShiftUp<BF16>);
    }
    __syncthreads();
  }
}

// weight_out[i, s] = weight_in[i, s] + the sum over request i's rows (in order) and
// query heads of 2^(c (logit - M)) / l.  Reads every logit once; a thread owns 4
// positions and a quarter of the heads, and the quarters are added up in order, so
// the sum's order is fixed.  Bound by the logits' traffic and, with few requests, the
// latency of a thread's loads (16 requests x 32 heads of up to 32768 positions: a call of 213 us,
// 5 us more with all heads in one thread).
constexpr int kWeightPos = 128;                       // threads that share a quarter of the heads
constexpr int kWeightParts = 4;
constexpr int kWeightThreads = kWeightPos * kWeightParts;
constexpr int kRowList = 2 * kWeightThreads;

__global__ void __launch_bounds__(kWeightThreads) attn_weights_kernel(const __grid_constant__ AttnParams p) {
  const int64_t width = (int64_t)p.max_pages * kPage;
  const int part = threadIdx.x / kWeightPos, at_pos = threadIdx.x % kWeightPos;
  const int h0 = p.q_heads * part / kWeightParts, h1 = p.q_heads * (part + 1) / kWeightParts;
  const int64_t pos = ((int64_t)blockIdx.x * kWeightPos + at_pos) * 4;
  const bool in = pos < width;
  wait_for_launch_before();
  const bool failed = call_status(p) != kOk;
  __shared__ int32_t list[kRowList];
  __shared__ int32_t warp_n[kWeightThreads / 32];
  __shared__ float4 sums[kWeightParts - 1][kWeightPos];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float c = p.scale_log2;
  for (int32_t req = blockIdx.y; req < p.num_req; req += gridDim.y) {
    const int64_t at = (int64_t)req * width + pos;
    if (failed) {
      // totals kept in place stay as they were
      const float nan = __uint_as_float(0x7FC00000u);
      if (in && part == 0 && p.weight_in != p.weight_out) *(float4*)(p.weight_out + at) = make_float4(nan, nan, nan, nan);
      continue;
    }
    float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in && part == 0 && p.weight_in) w = *(const float4*)(p.weight_in + at);
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    const int64_t b0 = (int64_t)blockIdx.x * kWeightPos * 4, b1 = b0 + kWeightPos * 4;
    int n = 0;
    auto flush = [&]() {
      for (int i = 0; i < n; ++i) {
        const int32_t r = list[i];
        const int32_t a = p.row_start[r], b = p.row_end[r];
        if (!in || pos + 4 <= a || pos >= b) continue;
        const float* lg = p.logits + (int64_t)r * p.q_heads * width + pos;
        const float2* st = p.row_stat + (int64_t)r * p.q_heads;
        const bool m0 = pos >= a, m1 = pos + 1 >= a && pos + 1 < b, m2 = pos + 2 >= a && pos + 2 < b, m3 = pos + 3 < b;
#pragma unroll 8
        for (int h = h0; h < h1; ++h) {
          const float4 x = __ldcs((const float4*)(lg + h * width));
          const float2 s = st[h];
          if (m0) sum.x += pow2(exponent(x.x, s.x, c)) * s.y;
          if (m1) sum.y += pow2(exponent(x.y, s.x, c)) * s.y;
          if (m2) sum.z += pow2(exponent(x.z, s.x, c)) * s.y;
          if (m3) sum.w += pow2(exponent(x.w, s.x, c)) * s.y;
        }
      }
    };
    for (int32_t r0 = 0; r0 < p.rows; r0 += kWeightThreads) {
      const int32_t r = r0 + (int32_t)threadIdx.x;
      const bool on = r < p.rows && p.row_req[r] == req && p.row_end[r] > b0 && p.row_start[r] < b1;
      const uint32_t b = __ballot_sync(~0u, on);
      if (lane == 0) warp_n[warp] = __popc(b);
      __syncthreads();
      int before = n, all = 0;
#pragma unroll
      for (int i = 0; i < kWeightThreads / 32; ++i) {
        if (i < warp) before += warp_n[i];
        all += warp_n[i];
      }
      if (on) list[before + __popc(b & ((1u << lane) - 1))] = r;
      n += all;
      __syncthreads();
      if (n + kWeightThreads > kRowList) {
        flush();
        n = 0;
        __syncthreads();
      }
    }
    flush();
    if (part > 0) sums[part - 1][at_pos] = sum;
    __syncthreads();
    if (part == 0 && in) {
#pragma unroll
      for (int i = 0; i < kWeightParts - 1; ++i) {
        const float4 s = sums[i][at_pos];
        sum.x += s.x, sum.y += s.y, sum.z += s.z, sum.w += s.w;
      }
      *(float4*)(p.weight_out + at) = make_float4(w.x + sum.x, w.y + sum.y, w.z + sum.z, w.w + sum.w);
    }
    __syncthreads();
  }
}

}  // namespace

template <bool BF16, int D, int WARPS>
static cudaError_t launch_join(const AttnParams& p, int sm_count, cudaStream_t stream) {
  if (p.workers > kLooks * WARPS * 32) return cudaErrorInvalidValue;
  return launch_overlapped(attn_join_kernel<BF16, D, WARPS>, dim3(sm_count * (32 / WARPS)), dim3(WARPS * 32),
                           (size_t)p.workers * sizeof(OpenUnit), stream, p);
}

template <bool BF16>
static cudaError_t pick_join(const AttnParams& p, int sm_count, cudaStream_t stream) {
  if (p.tensor_core) return launch_join<BF16, 128, 8>(p, sm_count, stream);
  if (p.dim == 64) return launch_join<BF16, 64, 16>(p, sm_count, stream);
  if (p.dim == 128) return launch_join<BF16, 128, 16>(p, sm_count, stream);
  return launch_join<BF16, 256, 16>(p, sm_count, stream);
}

cudaError_t launch_attn_join(const AttnParams& p, bool bf16, int sm_count, cudaStream_t stream) {
  return bf16 ? pick_join<true>(p, sm_count, stream) : pick_join<false>(p, sm_count, stream);
}

cudaError_t launch_attn_weights(const AttnParams& p, cudaStream_t stream) {
  const int64_t per = kWeightPos * 4;
  const int64_t x = ((int64_t)p.max_pages * kPage + per - 1) / per;
  const dim3 grid((unsigned)x, (unsigned)(p.num_req < 65535 ? p.num_req : 65535));
  return launch_overlapped(attn_weights_kernel, grid, dim3(kWeightThreads), 0, stream, p);
}

}  // namespace idxk
