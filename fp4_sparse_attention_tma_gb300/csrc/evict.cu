// Eviction from a paged cache by accumulated weight.  A request longer than the budget
// keeps its first keep_first and last keep_last positions and, of those between, the
// heaviest: an exact selection by the order key of the TopK (weight descending, +0 above
// -0, NaN below every number, lower position first).  What is kept moves, in order of
// position, into fresh pages.
//
// Three kernels: the check of the destination pages, the selection (one cluster per
// request), and the copy, which waits for all checks, so that a call that fails has moved
// nothing.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "attn.h"
#include "idx_device.cuh"
#include "idx_launch.h"

namespace idxk {
namespace {

namespace cg = cooperative_groups;

constexpr int kPrepThreads = 1024;
constexpr int kSelThreads = 1024;
constexpr int kCopyThreads = 256;

__device__ __forceinline__ void raise(uint32_t* status, uint32_t code) { atomicCAS(status, (uint32_t)kOk, code); }

__device__ __forceinline__ bool bad_length(const EvictParams& p, int32_t n) {
  return n < 0 || (int64_t)n > (int64_t)p.max_pages * kPage;
}

// Lengths, and the destination pages: each inside the pool and named once.  One CTA.
__global__ void __launch_bounds__(kPrepThreads) evict_check_kernel(const __grid_constant__ EvictParams p) {
  allow_launch_after();
  __shared__ uint32_t err;
  if (threadIdx.x == 0) err = kOk;
  const int32_t words = (p.dst_pages + 31) / 32;
  for (int32_t i = threadIdx.x; i < words; i += kPrepThreads) p.dst_mark[i] = 0;
  __syncthreads();
  const int32_t used = (p.budget + kPage - 1) / kPage;   // pages of a request that was cut
  for (int32_t r = threadIdx.x; r < p.num_req; r += kPrepThreads)
    if (bad_length(p, p.seq_len[r])) atomicMax(&err, (uint32_t)kErrInvalidMetadata);
  for (int64_t i = threadIdx.x; i < (int64_t)p.num_req * used; i += kPrepThreads) {
    const int32_t r = (int32_t)(i / used), j = (int32_t)(i - (int64_t)r * used);
    const int32_t n = p.seq_len[r];
    if (n <= p.budget || bad_length(p, n)) continue;
    const int32_t page = p.dst_table[(int64_t)r * p.dst_width + j];
    if (page < 0 || page >= p.dst_pages ||
        (atomicOr(&p.dst_mark[page / 32], 1u << (page % 32)) >> (page % 32) & 1u))
      atomicMax(&err, (uint32_t)kErrInvalidPage);
  }
  __syncthreads();
  if (threadIdx.x == 0) *p.hdr_status = err;
}

// The selection.  Every CTA of a request's cluster holds a slice of its positions (their
// keys in shared memory where they fit); four passes over 8 bits of the key each count the
// slice's keys by digit, add the counts up over the cluster and keep the digit that holds
// the last key to be kept.  Then every warp counts what it keeps of its part of the slice,
// the counts are added up in order, and the positions go to their ranks.  Deterministic:
// the counts do not depend on the order of the additions.  Bound by latency (the barriers
// of the passes), not by the weights' bytes.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const __grid_constant__ EvictParams p) {
  allow_launch_after();
  wait_for_launch_before();
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int32_t req = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = kSelThreads / 32;
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t hist[2][256];   // counts of a pass, read by the cluster
  __shared__ uint32_t total[256];
  __shared__ uint32_t picked[2];      // digit, keys above it
  __shared__ uint32_t warp_gt[kWarps], warp_eq[kWarps];
  __shared__ uint32_t cta_cnt[2];     // this CTA's kept above the threshold, and at it

  const int64_t width = (int64_t)p.max_pages * kPage;
  int32_t n = p.seq_len[req];
  if (bad_length(p, n)) n = 0;        // an error: nothing is written that stays
  const bool cut = n > p.budget;
  const int32_t new_len = cut ? p.budget : n;
  const int64_t gtid = (int64_t)rank * kSelThreads + tid, gthreads = (int64_t)C * kSelThreads;

  // the pages of the request, and its new table
  const int32_t pages = (n + kPage - 1) / kPage;
  for (int64_t i = gtid; i < p.max_pages; i += gthreads) {
    const int32_t page = p.page_table[(int64_t)req * p.max_pages + i];
    if (i < pages) {
      if (page < 0 || page >= p.num_pages)
        raise(p.hdr_status, kErrInvalidPage);
      else if (p.same_pool && (p.dst_mark[page / 32] >> (page % 32) & 1u))
        raise(p.hdr_status, kErrInvalidPage);
    }
    p.new_table[(int64_t)req * p.max_pages + i] =
        !cut ? page : i < p.dst_width ? p.dst_table[(int64_t)req * p.dst_width + i] : -1;
  }
  if (rank == 0 && tid == 0) p.new_len[req] = new_len;
  const float* weight = p.weight + (int64_t)req * width;
  float* new_weight = p.new_weight + (int64_t)req * width;
  int32_t* keep = p.keep + (int64_t)req * p.budget;
  for (int64_t i = new_len + gtid; i < width; i += gthreads) new_weight[i] = 0.f;
  for (int64_t i = new_len + gtid; i < p.budget; i += gthreads) keep[i] = -1;
  if (!cut) {
    for (int64_t i = gtid; i < n; i += gthreads) {
      new_weight[i] = weight[i];
      keep[i] = (int32_t)i;
    }
    return;   // the whole cluster
  }

  // positions [lo, hi) compete for `want` places
  const int32_t lo = p.keep_first, hi = n - p.keep_last;
  uint32_t want = (uint32_t)(p.budget - p.keep_first - p.keep_last);
  const int32_t slice = ((n + C - 1) / C + 31) / 32 * 32;
  const int32_t s0 = min((int64_t)n, (int64_t)rank * slice), s1 = min((int64_t)n, (int64_t)s0 + slice);
  const bool held = slice <= p.slice_cap;
  if (held)
    for (int32_t i = s0 + tid; i < s1; i += kSelThreads) keys[i - s0] = score_key(weight[i]);
  auto key_at = [&](int32_t i) { return held ? keys[i - s0] : score_key(weight[i]); };

  // the threshold: of the competing keys, `want` are kept, all above `thr` and `want` (as it
  // is then) of those equal to it.  Nothing competes for no place: then thr stays the top.
  uint32_t thr = 0xFFFFFFFFu;
  if (want > 0) {
    uint32_t prefix = 0;
    for (int pass = 0; pass < 4; ++pass) {
      const int shift = 24 - 8 * pass, buf = pass & 1;
      if (tid < 256) hist[buf][tid] = 0;
      __syncthreads();
      const uint32_t mask = pass == 0 ? 0u : 0xFFFFFFFFu << (shift + 8);
      for (int32_t i = max(s0, lo) + tid; i < min(s1, hi); i += kSelThreads) {
        const uint32_t k = key_at(i);
        if ((k & mask) == prefix) atomicAdd(&hist[buf][k >> shift & 255u], 1u);
      }
      cluster.sync();
      if (tid < 256) {
        uint32_t t = 0;
        for (int i = 0; i < C; ++i) t += cluster.map_shared_rank(&hist[buf][0], i)[tid];
        total[tid] = t;
      }
      __syncthreads();
      if (warp == 0) {
        // lane l: digits 255 - 8l .. 248 - 8l, from the top
        uint32_t sum = 0;
        for (int i = 0; i < 8; ++i) sum += total[255 - 8 * lane - i];
        uint32_t inc = sum;
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t x = __shfl_up_sync(~0u, inc, o);
          if (lane >= o) inc += x;
        }
        uint32_t above = inc - sum;
        if (above < want && inc >= want) {
          int d = 255 - 8 * lane;
          while (above + total[d] < want) above += total[d--];
          picked[0] = (uint32_t)d;
          picked[1] = above;
        }
      }
      __syncthreads();
      prefix |= picked[0] << shift;
      want -= picked[1];
    }
    thr = prefix;
  } else {
    __syncthreads();   // the keys
  }

  // what every warp keeps of its part of the slice
  const int32_t part = (slice / 32 + kWarps - 1) / kWarps * 32;
  const int32_t w0 = min(s1, s0 + warp * part), w1 = min(s1, w0 + part);
  const uint32_t take = want;   // of the keys equal to thr
  auto classify = [&](int32_t i, bool& gt, bool& eq) {
    gt = eq = false;
    if (i >= w1) return;
    if (i < lo || i >= hi) {
      gt = true;
    } else if (p.budget > p.keep_first + p.keep_last) {
      const uint32_t k = key_at(i);
      gt = k > thr;
      eq = k == thr;
    }
  };
  uint32_t n_gt = 0, n_eq = 0;
  for (int32_t i0 = w0; i0 < w1; i0 += 32) {
    bool gt, eq;
    classify(i0 + lane, gt, eq);
    n_gt += __popc(__ballot_sync(~0u, gt));
    n_eq += __popc(__ballot_sync(~0u, eq));
  }
  if (lane == 0) warp_gt[warp] = n_gt, warp_eq[warp] = n_eq;
  __syncthreads();
  if (tid == 0) {
    uint32_t a = 0, b = 0;
    for (int i = 0; i < kWarps; ++i) a += warp_gt[i], b += warp_eq[i];
    cta_cnt[0] = a, cta_cnt[1] = b;
  }
  cluster.sync();
  uint32_t gt0 = 0, eq0 = 0;   // before this warp's part
  for (int i = 0; i < rank; ++i) {
    const uint32_t* c = cluster.map_shared_rank(&cta_cnt[0], i);
    gt0 += c[0], eq0 += c[1];
  }
  for (int i = 0; i < warp; ++i) gt0 += warp_gt[i], eq0 += warp_eq[i];
  for (int32_t i0 = w0; i0 < w1; i0 += 32) {
    bool gt, eq;
    classify(i0 + lane, gt, eq);
    const uint32_t bg = __ballot_sync(~0u, gt), be = __ballot_sync(~0u, eq);
    const uint32_t below = (1u << lane) - 1;
    const uint32_t e = eq0 + __popc(be & below);
    if (gt || (eq && e < take)) {
      const uint32_t at = gt0 + __popc(bg & below) + min(e, take);
      keep[at] = i0 + lane;
      new_weight[at] = weight[i0 + lane];
    }
    gt0 += __popc(bg);
    eq0 += __popc(be);
  }
  cluster.sync();   // no CTA leaves while another reads its counts
}

// Moves the kept keys and values, 16 bytes a thread at a time, one destination page of
// keys or of values per CTA; the last kernel of the call, so it also publishes the status
// and, after an error, fills the outputs.  Bound by HBM: every kept byte read and written
// once.
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(const __grid_constant__ EvictParams p) {
  wait_for_launch_before();
  const uint32_t status = *p.hdr_status;
  const int32_t used = (p.budget + kPage - 1) / kPage;
  const int64_t job = blockIdx.x;
  if (job == 0 && threadIdx.x == 0) *p.status_out = status;
  if (status != kOk) {
    const int64_t width = (int64_t)p.max_pages * kPage;
    const int64_t t = job * kCopyThreads + threadIdx.x, step = (int64_t)gridDim.x * kCopyThreads;
    const float nan = __uint_as_float(0x7FC00000u);
    for (int64_t i = t; i < p.num_req * (int64_t)p.budget; i += step) p.keep[i] = -1;
    for (int64_t i = t; i < p.num_req; i += step) p.new_len[i] = -1;
    for (int64_t i = t; i < p.num_req * (int64_t)p.max_pages; i += step) p.new_table[i] = -1;
    for (int64_t i = t; i < p.num_req * width; i += step) p.new_weight[i] = nan;
    return;
  }
  const bool values = job & 1;
  const int64_t at = job >> 1;
  const int32_t req = (int32_t)(at / used), j = (int32_t)(at - (int64_t)req * used);
  if (req >= p.num_req || p.seq_len[req] <= p.budget) return;
  __shared__ int64_t from[kPage];
  const int32_t rows = min(kPage, p.budget - j * kPage);
  if ((int)threadIdx.x < rows) {
    const int32_t pos = p.keep[(int64_t)req * p.budget + j * kPage + threadIdx.x];
    const int64_t page = p.page_table[(int64_t)req * p.max_pages + pos / kPage];
    from[threadIdx.x] = page * (values ? p.v_page : p.k_page) + pos % kPage * (values ? p.v_slot : p.k_slot);
  }
  __syncthreads();
  const char* src = (const char*)(values ? p.v : p.k);
  const int64_t page = p.dst_table[(int64_t)req * p.dst_width + j];
  char* dst = (char*)(values ? p.v_dst : p.k_dst) + page * (values ? p.vd_page : p.kd_page);
  const int64_t sh = values ? p.v_head : p.k_head, dh = values ? p.vd_head : p.kd_head;
  const int64_t ds = values ? p.vd_slot : p.kd_slot;
  const int32_t pieces = p.head_bytes / 16;   // a power of two
  const int32_t n = rows * p.kv_heads * pieces;
  // the faster index over pieces and then over what lies closer together in the source
  const bool slots_inner = sh > (values ? p.v_slot : p.k_slot);
#pragma unroll 4
  for (int32_t i = threadIdx.x; i < n; i += kCopyThreads) {
    const int32_t x = i % pieces, y = i / pieces;
    const int32_t h = slots_inner ? y / rows : y % p.kv_heads, r = slots_inner ? y % rows : y / p.kv_heads;
    const uint4 t = __ldcs((const uint4*)(src + from[r] + h * sh + x * 16));
    __stcs((uint4*)(dst + r * ds + h * dh + x * 16), t);
  }
}

}  // namespace

cudaError_t launch_evict(EvictParams p, cudaStream_t stream) {
  // one CTA of a cluster for 8192 positions of the widest request, at most 8
  int C = 1;
  const int64_t width = (int64_t)p.max_pages * kPage;
  while (C < 8 && (int64_t)C * 8192 < width) C *= 2;
  const int64_t slice = ((width + C - 1) / C + 31) / 32 * 32;
  constexpr int64_t kMost = 48 * 1024;   // keys of a slice in shared memory
  p.slice_cap = (int32_t)(slice < kMost ? slice : kMost);
  const int smem = p.slice_cap * 4;
  static std::atomic<bool> done[64];
  cudaError_t e = set_smem_once(evict_select_kernel, (int)kMost * 4, done);
  if (e != cudaSuccess) return e;
  evict_check_kernel<<<1, kPrepThreads, 0, stream>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(p.num_req * C));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 2;
  if ((e = cudaLaunchKernelEx(&cfg, evict_select_kernel, (const EvictParams)p)) != cudaSuccess) return e;
  const int64_t used = (p.budget + kPage - 1) / kPage;
  // a budget above every length moves nothing
  const int64_t jobs = p.budget >= width ? 1 : p.num_req * used * 2;
  return launch_overlapped(evict_copy_kernel, dim3((unsigned)jobs), dim3(kCopyThreads), 0, stream, p);
}

}  // namespace idxk
