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

namespace idxk {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kBitmapBytes = 128 * 1024;
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

// A sum held as a rounded part and what the roundings left (TwoSum, Knuth): the sum of a head's squares
// does not depend on the order then, up to its one final rounding, and so neither do the codes of a key
// that lies next to a border between two of them.
__device__ __forceinline__ void add_exactly(float& s, float& rest, float x) {
  const float t = __fadd_rn(s, x), b = __fsub_rn(t, s);
  rest = __fadd_rn(rest, __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(x, b)));
  s = t;
}

// Checks every row of the call, so that all CTAs agree on whether anything is written: rows in range,
// pages in range, no slot named twice.  Returns the error (kOk: none) to every thread.
__device__ uint32_t check_rows(const AppendParams& p, uint32_t* table) {
  __shared__ uint32_t err;
  const int tid = threadIdx.x, n = blockDim.x;
  if (tid == 0) err = kOk;
  const bool bitmap = p.table_bits == 0;
  const uint32_t entries = bitmap ? kBitmapBytes / 4 : 1u << p.table_bits;
  const int64_t slots = (int64_t)p.num_pages * kPage;
  // the bitmap holds a part of the slots at a time
  const int64_t span = bitmap ? (int64_t)entries * 32 : slots;
  for (int64_t s0 = 0; s0 < slots; s0 += span) {
    for (uint32_t i = tid; i < entries; i += n) table[i] = bitmap ? 0u : ~0u;
    __syncthreads();
    for (int32_t r = tid; r < p.rows; r += n) {
      const int32_t pos = p.row_pos[r];
      if (pos == -1) continue;
      const int32_t req = p.row_req[r];
      uint32_t e = kOk;
      int32_t page = 0;
      if (pos < 0 || req < 0 || req >= p.num_req || pos / kPage >= p.max_pages || (p.rope && pos >= p.rope_rows)) {
        e = kErrInvalidMetadata;
      } else {
        page = p.page_table[(int64_t)req * p.max_pages + pos / kPage];
        if (page < 0 || page >= p.num_pages) e = kErrInvalidPage;
      }
      if (e == kOk) {
        const int64_t slot = (int64_t)page * kPage + pos % kPage;
        if (bitmap) {
          if (slot >= s0 && slot < s0 + span) {
            const uint32_t bit = 1u << (slot & 31);
            if (atomicOr(&table[(slot - s0) >> 5], bit) & bit) e = kErrInvalidPage;
          }
        } else {
          // open addressing: at most half of the entries are taken
          const uint32_t key = (uint32_t)slot;
          uint32_t at = (key * 2654435769u) >> (32 - p.table_bits);
          for (uint32_t i = 0; i < entries; ++i) {
            const uint32_t old = atomicCAS(&table[at], ~0u, key);
            if (old == ~0u) break;
            if (old == key) {
              e = kErrInvalidPage;
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

// A warp takes U x 32 / (D / 8) heads of a row at a time: 16 bytes of a head a lane, D / 8 lanes a head.
// Bound by HBM where rows are many, by the chain position, page entry, store and one launch where they are
// few.
template <bool BF16, int D, bool FP4, int U>
__global__ void __launch_bounds__(kMaxThreads) append_kernel(const __grid_constant__ AppendParams p) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr int L = D / 8;            // lanes of a head
  constexpr int H = 32 / L;           // heads that the warp has in its lanes
  constexpr int HEADS = U * H;        // of a chunk
  extern __shared__ uint32_t table[];
  const int lane = threadIdx.x & 31, in = lane % L, sub = lane / L;
  const int warps = blockDim.x >> 5;
  const int32_t qc = p.q.data ? (p.q_heads + HEADS - 1) / HEADS : 0, kc = (p.kv_heads + HEADS - 1) / HEADS;
  const int32_t per_row = qc + kc + (p.v.data ? kc : 0);
  const uint32_t chunks = (uint32_t)p.rows * per_row, stride = gridDim.x * warps;   // (below 2^31 and 2^13)
  const int d0 = in * 8;

  uint32_t c = (threadIdx.x >> 5) * gridDim.x + blockIdx.x;
  int32_t row = 0, h0 = 0, heads = 0, pos = -1;
  int kind = 0;                       // 0 query, 1 key, 2 value
  uint4 raw[U];
  auto fetch = [&]() {
    if (c >= chunks) return;
    row = (int32_t)(c / (uint32_t)per_row);
    int32_t i = (int32_t)c - row * per_row;
    kind = i < qc ? 0 : i < qc + kc ? 1 : 2;
    i -= kind == 0 ? 0 : kind == 1 ? qc : qc + kc;
    h0 = i * HEADS;
    heads = kind == 0 ? p.q_heads : p.kv_heads;
    const HeadsIn& x = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
    pos = p.row_pos[row];
    const T* from = (const T*)x.data + row * x.row + d0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int32_t h = h0 + u * H + sub;
      raw[u] = h < heads ? __ldcs((const uint4*)(from + h * x.head)) : make_uint4(0, 0, 0, 0);
    }
  };
  fetch();
  const uint32_t err = check_rows(p, table);
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status_out = err;
  if (err != kOk) {
    // nothing was written; queries that have a place of their own become NaN
    if (!p.out_q || p.q_in_place) return;
    const int64_t n = (int64_t)p.rows * p.q_heads;
    for (int64_t i = (int64_t)blockIdx.x * warps + (threadIdx.x >> 5); i < n; i += stride) {
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

  for (; c < chunks; c += stride, fetch()) {
    if (pos < 0) continue;            // a row that is not there
    const void* weight = kind == 0 ? p.q_weight : kind == 1 ? p.k_weight : nullptr;
    float w[8];
    if (weight) {
      if (p.weight_f32) {
        *(float4*)&w[0] = *(const float4*)((const float*)weight + d0);
        *(float4*)&w[4] = *(const float4*)((const float*)weight + d0 + 4);
      } else {
        unpack8<BF16>(*(const uint4*)((const T*)weight + d0), w);
      }
    }
    // the angles of this lane's dimensions: 4 pairs of neighbours, or 8 of a half
    const bool turn = p.rope && kind < 2, mine = turn && d0 >= p.first && d0 < p.first + p.rot;
    const int half = p.rot / 2;
    bool upper = false;
    int partner = lane;
    float co[8], si[8];
    if (mine) {
      const float* t = p.rope + (int64_t)pos * p.rot;
      int j = d0 - p.first;
      if (p.pairs) {
        j /= 2;
        *(float4*)&co[0] = *(const float4*)(t + j);
        *(float4*)&si[0] = *(const float4*)(t + half + j);
      } else {
        upper = j >= half;
        partner = upper ? lane - half / 8 : lane + half / 8;
        if (upper) j -= half;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          *(float4*)&co[i] = *(const float4*)(t + j + i);
          *(float4*)&si[i] = *(const float4*)(t + half + j + i);
        }
      }
    }
    const PagedOut& dst = kind == 1 ? p.k_dst : p.v_dst;
    int64_t at = 0, s_at = 0;
    if (kind == 0) {
      at = row * p.oq_row, s_at = row * p.oqs_row;
    } else {
      const int64_t page = p.page_table[(int64_t)p.row_req[row] * p.max_pages + pos / kPage];
      at = page * dst.page + pos % kPage * dst.slot;
      s_at = page * dst.s_page + pos % kPage * dst.s_slot;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int32_t h = h0 + u * H + sub;
      const bool on = h < heads;
      if (h0 + u * H >= heads) break;   // (the same for the whole warp)
      if (!FP4 && kind == 2) {          // a copy
        if (on) *(uint4*)((T*)dst.data + at + h * dst.head + d0) = raw[u];
        continue;
      }
      float x[8];
      unpack8<BF16>(raw[u], x);
      if (weight) {
        float s = 0.f, rest = 0.f;      // squares of 16-bit numbers are exact in fp32
#pragma unroll
        for (int i = 0; i < 8; ++i) add_exactly(s, rest, __fmul_rn(x[i], x[i]));
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
        for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(__fmul_rn(x[i], r), w[i]);
      }
      if (turn) {
        if (p.pairs) {
          if (mine) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a = x[2 * i], b = x[2 * i + 1];
              x[2 * i] = __fsub_rn(__fmul_rn(a, co[i]), __fmul_rn(b, si[i]));
              x[2 * i + 1] = __fadd_rn(__fmul_rn(b, co[i]), __fmul_rn(a, si[i]));
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float o = __shfl_sync(~0u, x[i], partner);
            if (mine) {
              const float cross = __fmul_rn(o, si[i]), own = __fmul_rn(x[i], co[i]);
              x[i] = upper ? __fadd_rn(own, cross) : __fsub_rn(own, cross);
            }
          }
        }
      }
      if (kind == 0 ? p.out_q_scale != nullptr : FP4) {
        uint32_t top = 0;               // as integers: a NaN counts as the largest
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
        top = max(top, __shfl_xor_sync(~0u, top, 1));
        top = max(top, __shfl_xor_sync(~0u, top, 2));
        const uint32_t e = scale_byte(top), codes = to_codes(x, e);
        if (on) {
          uint8_t* to = (kind == 0 ? (uint8_t*)p.out_q + h * p.oq_head : (uint8_t*)dst.data + h * dst.head) + at;
          uint8_t* st = (kind == 0 ? p.out_q_scale + h * p.oqs_head : dst.scale + h * dst.s_head) + s_at;
          *(uint32_t*)(to + in * 4) = codes;
          if (in % 4 == 0) st[in / 4] = (uint8_t)e;
        }
      } else if (on) {
        T* to = (kind == 0 ? (T*)p.out_q + h * p.oq_head : (T*)dst.data + h * dst.head) + at;
        *(uint4*)(to + d0) = pack8<BF16>(x);
      }
    }
  }
}

// Listed slots of a 4-bit cache as 16-bit rows, rounded once (exact unless beyond the type's range or below its
// last place): 4 bytes of codes, 8 elements, a thread.  Bound by HBM: 0.53 bytes read and 2 written an element.
// The last CTA only looks for slots that are none.
template <bool BF16, int D, int U>
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const __grid_constant__ GatherParams p) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr int L = D / 8;              // threads of a head
  const int32_t most = p.num_pages * kPage;
  if (blockIdx.x == gridDim.x - 1) {
    bool bad = false;
#pragma unroll 8
    for (int32_t i = threadIdx.x; i < p.n; i += kGatherThreads) bad |= p.slots[i] < -1 || p.slots[i] >= most;
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *p.status_out = bad ? kErrInvalidPage : kOk;
    return;
  }
  const int j = threadIdx.x % L;
  const int32_t step = (int32_t)(gridDim.x - 1) * (kGatherThreads / L);   // heads from one of a thread's to its next
  const int32_t dr = step / p.kv_heads, dh = step - dr * p.kv_heads;
  const int32_t v0 = (int32_t)blockIdx.x * (kGatherThreads / L) + (int32_t)threadIdx.x / L;
  int32_t r = v0 / p.kv_heads, h = v0 - r * p.kv_heads;
  while (r < p.n) {
    int32_t rs[U], hs[U];
    uint32_t codes[2][U], e[2][U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rs[u] = r, hs[u] = h;
      const int32_t slot = r < p.n ? p.slots[r] : -1;
      const bool on = slot >= 0 && slot < most;
      const int64_t page = slot / kPage, off = slot % kPage;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const GatherParams::From& f = p.t[t];
        codes[t][u] = 0, e[t][u] = slot == -1 ? 127u : 255u;   // what is no slot becomes NaN
        if (!on || !f.codes) continue;
        codes[t][u] = *(const uint32_t*)(f.codes + page * f.page + off * f.slot + h * f.head + j * 4);
        e[t][u] = f.scale[page * f.s_page + off * f.s_slot + h * f.s_head + j / 4];
      }
      r += dr, h += dh;
      if (h >= p.kv_heads) h -= p.kv_heads, ++r;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (rs[u] >= p.n) break;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const GatherParams::From& f = p.t[t];
        if (!f.codes) continue;
        uint32_t w[4];
        from_codes(codes[t][u], w);
        const float s = scale_of(e[t][u]);
        float x[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 y = __half22float2(*(const __half2*)&w[k]);
          x[2 * k] = y.x * s, x[2 * k + 1] = y.y * s;
        }
        __stcs((uint4*)((T*)f.out + rs[u] * f.row + hs[u] * f.out_head + j * 8), pack8<BF16>(x));
      }
    }
  }
}

template <bool BF16, int D, bool FP4, int U>
cudaError_t launch_append_u(const AppendParams& p, int threads, int grid, size_t smem, cudaStream_t stream) {
  auto* kernel = append_kernel<BF16, D, FP4, U>;
  static std::atomic<bool> done[64];
  cudaError_t e = set_smem_once(kernel, kBitmapBytes, done);
  if (e != cudaSuccess) return e;
  kernel<<<grid, threads, smem, stream>>>(p);
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
  // (every CTA looks over all rows).
  p.table_bits = 0;
  for (int b = 6; b <= 15 && !p.table_bits; ++b)
    if ((int64_t)1 << b >= 2 * (int64_t)p.rows) p.table_bits = b;
  const size_t smem = p.table_bits ? (size_t)4 << p.table_bits : kBitmapBytes;
  if (chunks(H) <= (int64_t)sm * 16) {
    const int64_t n = chunks(H);
    const int64_t want = (n + sm - 1) / sm;      // warps an SM
    const int warps = want <= 4 ? 4 : want <= 8 ? 8 : 16;
    const int64_t grid = (n + warps - 1) / warps;
    return launch_append_u<BF16, D, FP4, 1>(p, warps * 32, (int)(grid < 1 ? 1 : grid), smem, stream);
  }
  return launch_append_u<BF16, D, FP4, 4>(p, kMaxThreads, sm, smem, stream);
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
  const int64_t ctas = ((int64_t)p.n * p.kv_heads * (D / 8) + kGatherThreads - 1) / kGatherThreads;
  if (ctas <= 2 * sm)
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
