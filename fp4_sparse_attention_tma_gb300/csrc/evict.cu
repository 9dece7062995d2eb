// Eviction from a paged cache by accumulated weight.  A request longer than the budget
// keeps its first keep_first and last keep_last positions and, of those between, the
// heaviest: an exact selection by the order key of the TopK (weight descending, +0 above
// -0, NaN below every number, lower position first).  What is kept moves, in order of
// position, into fresh pages.
//
// Two kernels: the selection (one cluster per request, and one that checks the fresh pages
// meanwhile), and the copy, which sees what all of them found before it moves anything.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "attn.h"
#include "idx_device.cuh"
#include "idx_launch.h"

namespace idxk {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kBins = 2048;          // digits of 11, 11 and 10 bits of the key
constexpr int64_t kSliceKeys = 48 * 1024;          // keys of a CTA's slice that fit its shared memory
constexpr int64_t kMarkBytes = kSliceKeys * 4;     // and the bitmap of the destination pages

// First error of a cluster: the CTAs' own words are gathered at its end.
__device__ __forceinline__ void note(uint32_t* err, uint32_t code) { atomicMax(err, code); }

__device__ __forceinline__ bool bad_length(const EvictParams& p, int32_t n) {
  return n < 0 || (int64_t)n > (int64_t)p.max_pages * kPage;
}

// The check of the fresh pages, by the cluster after the requests': each inside the pool and
// named once and, where the pool is the cache itself, under no request's positions.  Every CTA
// marks all fresh pages (in shared memory, or in its own part of the workspace where they do
// not fit) and looks at its share of the pages in use.
__device__ void check_fresh(const EvictParams& p, int C, int rank, uint32_t* shared, uint32_t* err) {
  const int tid = threadIdx.x;
  const int32_t words = (p.dst_pages + 31) / 32;
  uint32_t* mark = p.mark_shared ? shared : p.dst_mark + (int64_t)rank * words;
  for (int32_t i = tid; i < words; i += kSelThreads) mark[i] = 0;
  __syncthreads();
  const int32_t used = (p.budget + kPage - 1) / kPage;   // pages of a request that was cut
#pragma unroll 4
  for (int64_t i = tid; i < (int64_t)p.num_req * used; i += kSelThreads) {
    const int32_t r = (int32_t)(i / used), j = (int32_t)(i - (int64_t)r * used);
    const int32_t n = p.seq_len[r];
    if (n <= p.budget || bad_length(p, n)) continue;
    const int32_t page = p.dst_table[(int64_t)r * p.dst_width + j];
    if (page < 0 || page >= p.dst_pages || (atomicOr(&mark[page / 32], 1u << (page % 32)) >> (page % 32) & 1u))
      note(err, kErrInvalidPage);
  }
  __syncthreads();
  if (!p.same_pool) return;
#pragma unroll 4
  for (int64_t i = (int64_t)rank * kSelThreads + tid; i < (int64_t)p.num_req * p.max_pages; i += (int64_t)C * kSelThreads) {
    const int32_t r = (int32_t)(i / p.max_pages), j = (int32_t)(i - (int64_t)r * p.max_pages);
    const int32_t n = p.seq_len[r], page = p.page_table[i];
    if (bad_length(p, n) || j >= (n + kPage - 1) / kPage || page < 0 || page >= p.num_pages) continue;
    if (mark[page / 32] >> (page % 32) & 1u) note(err, kErrInvalidPage);
  }
}

__device__ __forceinline__ uint4 keys_of(float4 w) {
  return make_uint4(score_key(w.x), score_key(w.y), score_key(w.z), score_key(w.w));
}

// Barrier of the cluster (of the CTA, where that is all of it).
__device__ __forceinline__ void sync_all(cooperative_groups::cluster_group& cluster, int C) {
  if (C == 1)
    __syncthreads();
  else
    cluster.sync();
}

// The selection.  Every CTA of a request's cluster holds a slice of its positions (their
// keys in shared memory where they fit); three passes over 11, 11 and 10 bits of the key
// each count the slice's keys by digit, find in the whole cluster's counts (first by groups of
// 64 digits, then in one group) the digit that holds the last key to be kept, and go on with
// the keys of that digit.  (Of the first 11 bits 9 are sign and exponent: fewer bits would send
// most keys to a handful of counters.  Where all weights are equal every key goes to one: 8 requests of up to
// 262144 positions, 91 us a call for 84.)  Then every warp counts what it keeps of its part of the
// slice, the counts are added up in order, and the positions go to their ranks.
// Deterministic: the counts do not depend on the order of the additions.  Bound by latency
// (2 to 3 us a pass, half of it barriers and reads of the other CTAs' counts) and, where a CTA
// has 32768 positions, by the instructions that look at each of them five times: 10 us for one
// request of 5001 positions, 25 us for 8 of up to 262144.
__device__ void select(const EvictParams& p, cooperative_groups::cluster_group& cluster, int32_t req, uint32_t* bits,
                       uint32_t* err) {
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = kSelThreads / 32;
  static_assert(kWarps == 32 && kBins == 64 * 32, "one group of 64 digits per warp");
  __shared__ __align__(16) uint32_t hist[2][kBins];   // counts of a pass, read by the cluster two at a time
  __shared__ uint32_t group[2][32];     // counts of 64 digits each
  __shared__ uint32_t picked[2];        // digit, keys above it
  __shared__ uint32_t warp_gt[kWarps], warp_eq[kWarps];
  __shared__ uint32_t cta_cnt[2];       // this CTA's kept above the threshold, and at it

  const int64_t width = (int64_t)p.max_pages * kPage;
  int32_t n = p.seq_len[req];
  // this thread's entry of the two page tables (most requests have no more than the cluster has threads)
  const int32_t g = rank * kSelThreads + tid, all_threads = C * kSelThreads;
  const int32_t* table = p.page_table + (int64_t)req * p.max_pages;
  const int32_t* fresh = p.dst_table + (int64_t)req * p.dst_width;
  int32_t page = g < p.max_pages ? table[g] : -1, fresh_page = g < p.dst_width ? fresh[g] : -1;
  if (bad_length(p, n)) {
    if (tid == 0) note(err, kErrInvalidMetadata);
    n = 0;
  }
  const bool cut = n > p.budget;
  const int32_t new_len = cut ? p.budget : n;
  const float* weight = p.weight + (int64_t)req * width;
  float* new_weight = p.new_weight + (int64_t)req * width;
  int32_t* keep = p.keep + (int64_t)req * p.budget;

  // positions [lo, hi) compete for `want` places
  const int32_t lo = p.keep_first, hi = n - p.keep_last;
  uint32_t want = (uint32_t)(p.budget - p.keep_first - p.keep_last);
  const int32_t slice = ((n + C - 1) / C + 31) / 32 * 32;
  const int32_t s0 = min((int64_t)n, (int64_t)rank * slice), s1 = min((int64_t)n, (int64_t)s0 + slice);
  const bool held = slice <= p.slice_cap;
  if (cut && held) {
    const int32_t fours = (s1 - s0) / 4;   // (a request's weights, 256 bytes a page, begin at 16-byte boundaries)
#pragma unroll 8
    for (int32_t i = tid; i < fours; i += kSelThreads) ((uint4*)bits)[i] = keys_of(((const float4*)(weight + s0))[i]);
#pragma unroll 8
    for (int32_t i = s0 + 4 * fours + tid; i < s1; i += kSelThreads) bits[i - s0] = score_key(weight[i]);
  }
  // the keys of positions i .. i + 3 (i - s0 a multiple of 4; what lies behind the slice means nothing)
  auto keys_at = [&](int32_t i) {
    if (held) return *(const uint4*)(bits + (i - s0));
    return keys_of(make_float4(weight[i], i + 1 < s1 ? weight[i + 1] : 0.f, i + 2 < s1 ? weight[i + 2] : 0.f,
                               i + 3 < s1 ? weight[i + 3] : 0.f));
  };
  for (int i = tid; i < 2 * kBins; i += kSelThreads) hist[0][i] = 0;

  // the pages of the request, its new table, and what lies behind the kept positions
  const int32_t pages = (n + kPage - 1) / kPage;
  for (int32_t i = g; i < p.max_pages; i += all_threads) {
    if (i != g) page = table[i], fresh_page = i < p.dst_width ? fresh[i] : -1;
    if (i < pages && (page < 0 || page >= p.num_pages)) note(err, kErrInvalidPage);
    p.new_table[(int64_t)req * p.max_pages + i] = cut ? fresh_page : page;
  }
  if (g == 0) p.new_len[req] = new_len;
  for (int64_t i = (int64_t)new_len + g; i < width; i += all_threads) new_weight[i] = 0.f;
  for (int64_t i = (int64_t)new_len + g; i < p.budget; i += all_threads) keep[i] = -1;
  if (!cut) {
    for (int64_t i = g; i < n; i += all_threads) {
      new_weight[i] = weight[i];
      keep[i] = (int32_t)i;
    }
    return;   // the whole cluster
  }
  __syncthreads();

  // the threshold: of the competing keys, `want` are kept, all above `thr` and `want` (as it
  // is then) of those equal to it.  Nothing competes for no place: then thr stays the top.
  uint32_t thr = 0xFFFFFFFFu;
  if (want > 0) {
    uint32_t prefix = 0;
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, buf = pass & 1;
      const uint32_t digits = pass == 2 ? 1024u : (uint32_t)kBins;
      const uint32_t mask = pass == 0 ? 0u : pass == 1 ? 0xFFFFFFFFu << 21 : 0xFFFFFFFFu << 10;
      const int32_t x0 = max(s0, lo), x1 = min(s1, hi);
#pragma unroll 2
      for (int32_t i = s0 + 4 * tid; i < x1; i += 4 * kSelThreads) {
        const uint4 k4 = keys_at(i);
        const uint32_t four[4] = {k4.x, k4.y, k4.z, k4.w};
        const bool inside = i >= x0 && i + 4 <= x1;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t k = four[j];
          if ((k & mask) == prefix && (inside || (i + j >= x0 && i + j < x1)))
            atomicAdd(&hist[buf][k >> shift & (digits - 1)], 1u);
        }
      }
      __syncthreads();
      const uint2 mine = ((const uint2*)&hist[buf][warp * 64])[lane];
      const uint32_t sum = __reduce_add_sync(~0u, mine.x + mine.y);
      if (lane == 0) group[buf][warp] = sum;
      sync_all(cluster, C);
      if (warp == 0) {
        // lane l: group 31 - l, so that a scan counts from the top
        uint32_t cnt = 0;
        for (int i = 0; i < C; ++i) cnt += cluster.map_shared_rank(&group[buf][0], i)[31 - lane];
        uint32_t inc = cnt;
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(~0u, inc, o);
          if (lane >= o) inc += y;
        }
        const uint32_t at = __ballot_sync(~0u, inc >= want);
        const int l = __ffs(at) - 1;   // the competing keys are at least `want`
        uint32_t above = __shfl_sync(~0u, inc - cnt, l);
        // its digits 63 - 2 lane and 62 - 2 lane
        uint32_t hi_n = 0, lo_n = 0;
        for (int i = 0; i < C; ++i) {
          const uint2 two = ((const uint2*)(cluster.map_shared_rank(&hist[buf][0], i) + (31 - l) * 64))[31 - lane];
          lo_n += two.x, hi_n += two.y;
        }
        inc = hi_n + lo_n;
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(~0u, inc, o);
          if (lane >= o) inc += y;
        }
        above += inc - hi_n - lo_n;
        if (above < want && above + hi_n + lo_n >= want) {
          const bool low = above + hi_n < want;
          picked[0] = (31 - l) * 64 + 63 - 2 * lane - (low ? 1 : 0);
          picked[1] = above + (low ? hi_n : 0);
        }
      } else if (pass == 1) {
        // the counters of the third pass: those of the first, which every CTA has read by now
        for (int i = tid - 32; i < kBins; i += kSelThreads - 32) hist[0][i] = 0;
      }
      __syncthreads();
      prefix |= picked[0] << shift;
      want -= picked[1];
    }
    thr = prefix;
  }

  // what every warp keeps of its part of the slice, four positions a lane at a time
  const int32_t part = (slice + kWarps * 128 - 1) / (kWarps * 128) * 128;
  const int32_t w0 = min(s1, s0 + warp * part), w1 = min(s1, w0 + part);
  const uint32_t take = want;   // of the keys equal to thr
  const bool some = p.budget > p.keep_first + p.keep_last;
  // positions i .. i + 3: bit j of gt, of eq
  auto classify = [&](int32_t i, uint32_t (&four)[4], uint32_t& gt, uint32_t& eq) {
    gt = eq = 0;
    if (i >= w1) return;
    const uint4 k4 = keys_at(i);
    four[0] = k4.x, four[1] = k4.y, four[2] = k4.z, four[3] = k4.w;
    if (some && i >= lo && i + 4 <= min(hi, w1)) {
#pragma unroll
      for (int j = 0; j < 4; ++j) gt |= (four[j] > thr) << j, eq |= (four[j] == thr) << j;
      return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t k = four[j];
      const bool in = i + j < w1, always = i + j < lo || i + j >= hi;
      if (in && (always || (some && k > thr))) gt |= 1u << j;
      if (in && !always && some && k == thr) eq |= 1u << j;
    }
  };
  uint32_t n_gt = 0, n_eq = 0;
#pragma unroll 2
  for (int32_t i0 = w0; i0 < w1; i0 += 128) {
    uint32_t gt, eq;
    uint32_t four[4];
    classify(i0 + 4 * lane, four, gt, eq);
    n_gt += __popc(gt);
    n_eq += __popc(eq);
  }
  n_gt = __reduce_add_sync(~0u, n_gt);
  n_eq = __reduce_add_sync(~0u, n_eq);
  if (lane == 0) warp_gt[warp] = n_gt, warp_eq[warp] = n_eq;
  __syncthreads();
  if (warp == 0) {
    const uint32_t a = __reduce_add_sync(~0u, warp_gt[lane]), b = __reduce_add_sync(~0u, warp_eq[lane]);
    if (lane == 0) cta_cnt[0] = a, cta_cnt[1] = b;
  }
  sync_all(cluster, C);
  // before this warp's part
  uint32_t gt0 = lane < warp ? warp_gt[lane] : 0u, eq0 = lane < warp ? warp_eq[lane] : 0u;
  if (lane < rank) {
    const uint32_t* c = cluster.map_shared_rank(&cta_cnt[0], lane);
    gt0 += c[0], eq0 += c[1];
  }
  gt0 = __reduce_add_sync(~0u, gt0);
  eq0 = __reduce_add_sync(~0u, eq0);
#pragma unroll 2
  for (int32_t i0 = w0; i0 < w1; i0 += 128) {
    uint32_t gt, eq;
    uint32_t four[4];
    classify(i0 + 4 * lane, four, gt, eq);
    const uint32_t mine = __popc(gt) | __popc(eq) << 16;   // at most 128 of each in a warp
    uint32_t inc = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(~0u, inc, o);
      if (lane >= o) inc += y;
    }
    const uint32_t all = __shfl_sync(~0u, inc, 31);
    inc -= mine;
    uint32_t g0 = gt0 + (inc & 0xFFFF), e0 = eq0 + (inc >> 16);   // before this position
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool is_gt = gt >> j & 1, is_eq = eq >> j & 1;
      if (is_gt || (is_eq && e0 < take)) {
        const uint32_t at = g0 + min(e0, take);
        keep[at] = i0 + 4 * lane + j;
        new_weight[at] = four[j] ? key_score((uint64_t)four[j] << 32) : weight[i0 + 4 * lane + j];   // (0: some NaN, as it was)
      }
      g0 += is_gt;
      e0 += is_eq;
    }
    gt0 += all & 0xFFFF;
    eq0 += all >> 16;
  }
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const __grid_constant__ EvictParams p) {
  allow_launch_after();
  cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int32_t req = blockIdx.x / C;
  extern __shared__ __align__(16) uint32_t room[];
  __shared__ uint32_t err;
  if (threadIdx.x == 0) err = kOk;
  __syncthreads();
  if (req < p.num_req)
    select(p, cluster, req, room, &err);
  else
    check_fresh(p, C, rank, room, &err);
  sync_all(cluster, C);
  if (rank == 0 && threadIdx.x == 0) {
    uint32_t all = kOk;
    for (int i = 0; i < C; ++i) all = max(all, *cluster.map_shared_rank(&err, i));
    p.part_status[req] = all;
  }
  sync_all(cluster, C);   // no CTA leaves while another reads its words
}

// Moves the kept keys and values, 16 bytes a thread at a time, some rows of a destination page
// of keys or of values per CTA; the last kernel of the call, so it also publishes the status
// and, after an error, fills the outputs.  Bound by HBM: every kept byte read and written
// once (32 requests to 8192 positions, 8 heads: 1.96 GB in 327 us with the selection, 6.0 TB/s;
// single heads of 256 bytes, 8 requests to 30001 positions: 246 MB in 47 us, 5.2 TB/s).
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(const __grid_constant__ EvictParams p) {
  wait_for_launch_before();
  uint32_t status = kOk;
  {
    __shared__ uint32_t all;
    if (threadIdx.x == 0) all = kOk;
    __syncthreads();
    for (int32_t i = threadIdx.x; i <= p.num_req; i += kCopyThreads) status = max(status, p.part_status[i]);
    if (status != kOk) atomicMax(&all, status);
    __syncthreads();
    status = all;
  }
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
  const int32_t per_page = kPage / p.copy_rows;
  const int64_t at = (job >> 1) / per_page;
  const int32_t part = (int32_t)((job >> 1) - at * per_page);
  const int32_t req = (int32_t)(at / used), j = (int32_t)(at - (int64_t)req * used);
  if (req >= p.num_req || p.seq_len[req] <= p.budget) return;
  __shared__ int64_t from[kPage];
  const int32_t first = j * kPage + part * p.copy_rows;   // rank of the CTA's first row
  const int32_t rows = min(p.copy_rows, p.budget - first);
  if (rows <= 0) return;
  if ((int)threadIdx.x < rows) {
    const int32_t pos = p.keep[(int64_t)req * p.budget + first + threadIdx.x];
    const int64_t page = p.page_table[(int64_t)req * p.max_pages + pos / kPage];
    from[threadIdx.x] = page * (values ? p.v_page : p.k_page) + pos % kPage * (values ? p.v_slot : p.k_slot);
  }
  __syncthreads();
  const char* src = (const char*)(values ? p.v : p.k);
  const int64_t page = p.dst_table[(int64_t)req * p.dst_width + j];
  const int64_t sh = values ? p.v_head : p.k_head, dh = values ? p.vd_head : p.kd_head;
  const int64_t ds = values ? p.vd_slot : p.kd_slot;
  char* dst = (char*)(values ? p.v_dst : p.k_dst) + page * (values ? p.vd_page : p.kd_page) + part * p.copy_rows * ds;
  const uint32_t pieces = (uint32_t)p.head_bytes / 16;   // a power of two
  const uint32_t shift = 31 - __clz(pieces);
  const uint32_t n = (uint32_t)rows * p.kv_heads * pieces;
  // the faster index over pieces and then over what lies closer together in the source
  const bool slots_inner = sh > (values ? p.v_slot : p.k_slot);
  const uint32_t inner = slots_inner ? rows : p.kv_heads;
#pragma unroll 8
  for (uint32_t i = threadIdx.x; i < n; i += kCopyThreads) {
    const uint32_t x = i & (pieces - 1), y = i >> shift, a = y / inner, b = y - a * inner;
    const uint32_t h = slots_inner ? a : b, r = slots_inner ? b : a;
    const uint4 t = __ldcs((const uint4*)(src + from[r] + h * sh + x * 16));
    __stcs((uint4*)(dst + r * ds + h * dh + x * 16), t);
  }
}

}  // namespace

int evict_cluster(int64_t num_req, int64_t max_pages, int sm_count) {
  // one CTA for 8192 positions of the widest request, at most 8, and no more than a wave of
  // them (a CTA fills an SM): 32 requests of up to 65,536 positions, one head, take 70 us, and
  // 83 with clusters of 8 in two waves
  int C = 1;
  while (C < 8 && (int64_t)C * 8192 < max_pages * kPage && (num_req + 1) * 2 * C <= sm_count) C *= 2;
  return C;
}

bool evict_mark_shared(int64_t dst_pages) { return (dst_pages + 31) / 32 * 4 <= kMarkBytes; }

cudaError_t launch_evict(EvictParams p, int sm_count, cudaStream_t stream) {
  const int C = evict_cluster(p.num_req, p.max_pages, sm_count);
  const int64_t width = (int64_t)p.max_pages * kPage;
  const int64_t slice = ((width + C - 1) / C + 31) / 32 * 32;
  p.slice_cap = (int32_t)(slice < kSliceKeys ? slice : kSliceKeys);
  p.mark_shared = evict_mark_shared(p.dst_pages);
  int smem = p.slice_cap * 4;
  const int mark = (int)((p.dst_pages + 31) / 32 * 4);
  if (p.mark_shared && mark > smem) smem = mark;
  static std::atomic<bool> done[64];
  cudaError_t e = set_smem_once(evict_select_kernel, (int)kMarkBytes, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((p.num_req + 1) * C));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, evict_select_kernel, (const EvictParams)p)) != cudaSuccess) return e;
  // a CTA of the copy moves up to 32 KB: short rows a page at a time, long ones some of a page's (32
  // requests to 8192 positions, 8 heads of 256 bytes: 328 us, 330 with whole pages)
  p.copy_rows = kPage;
  while (p.copy_rows > 4 && (int64_t)p.copy_rows * p.kv_heads * p.head_bytes > 32 * 1024) p.copy_rows /= 2;
  const int64_t used = (p.budget + kPage - 1) / kPage;
  // a budget above every length moves nothing
  const int64_t jobs = p.budget >= width ? 1 : p.num_req * used * 2 * (kPage / p.copy_rows);
  return launch_overlapped(evict_copy_kernel, dim3((unsigned)jobs), dim3(kCopyThreads), 0, stream, p);
}

}  // namespace idxk
