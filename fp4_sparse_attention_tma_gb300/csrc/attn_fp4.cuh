// The attention kernel over a cache in 4 bits (fp4.cuh): one pass over the cached positions with the
// running maximum and sum of the softmax, as in attn.cuh, whose division of the work it shares.
//
// Codes are exact in fp16, and so are their products with a power of two: keys and values are unpacked
// in registers, on their way from shared memory to the matrix instructions, times their scales over a
// reference that keeps them within fp16: of keys the largest scale of the subtile, of values the largest
// so far of the unit (the weighted values are scaled when it grows, as with the softmax's maximum).
//   k' = code * 2^(12 + e - E),  s = 2^(E - 139) q . k'   (e, E: scale bytes)
// is exact for e >= E - 26; smaller blocks count as 0, an error of 6 * 2^(E - 127 - 27) at most, below
// fp32's place of the sum with a key of the largest scale.  bf16 queries are brought to fp16's range by a
// power of two for each head (elements below 2^-38 of the head's largest lose bits); softmax weights are
// rounded to fp16 (kShift in attn.h) whatever the queries' type is.
//
// A quad of lanes holds a position's codes, each lane a contiguous quarter, so that a lane's 16 bytes share
// a scale and no element is moved between lanes: the first product sums over the head's elements in
// whatever order the quarters give, and the queries are laid out alike.  For the second product, two
// positions' codes are paired nibble by nibble before they are unpacked.
#pragma once

#include "attn_common.cuh"
#include "fp4.cuh"
#include "pairs.cuh"

namespace idxk {
namespace attn {
namespace fp4 {

constexpr int kSub4 = 32;                 // cached positions per subtile
constexpr uint32_t kLowest = 26;          // no reference is below this byte: no scale is below 2^-26 of it then
constexpr uint32_t kF16Shift = 10;        // weights are 2^kF16Shift times what they stand for
constexpr float kRaise = 5.f;             // and at most 2^(kRaise + kF16Shift)

// 2^(12 + e - E) as an fp16 number in both halves of a word (0 where e < E - 26).
__device__ __forceinline__ uint32_t factor2(uint32_t e, uint32_t E) {
  const int32_t d = max((int32_t)e - (int32_t)E + 27, 0);
  return (uint32_t)d * 0x04000400u;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*(const __half2*)&a, *(const __half2*)&b);
  return *(const uint32_t*)&r;
}
// 8 codes each of two positions -> 8 pairs (first, second), by element.
__device__ __forceinline__ void from_pairs(uint32_t a, uint32_t b, uint32_t (&h)[8]) {
  const uint32_t even = (a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u), odd = ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
  uint32_t x[4], y[4];
  from_codes(even, x);
  from_codes(odd, y);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[2 * i] = x[i], h[2 * i + 1] = y[i];
}

// D / 32 scale bytes of a position.
template <int NB>
struct Scales {
  uint32_t w[NB == 8 ? 2 : 1];
  __device__ __forceinline__ void load(const uint8_t* a) {
    if constexpr (NB == 2) w[0] = *(const uint16_t*)a;
    if constexpr (NB == 4) w[0] = *(const uint32_t*)a;
    if constexpr (NB == 8) {
      const uint2 u = *(const uint2*)a;
      w[0] = u.x, w[1] = u.y;
    }
  }
  __device__ __forceinline__ void clear() {
    w[0] = 0;
    if constexpr (NB == 8) w[1] = 0;
  }
  __device__ __forceinline__ uint32_t get(int b) const { return (w[b / 4] >> (8 * (b % 4))) & 255u; }
  __device__ __forceinline__ uint32_t largest() const {
    uint32_t m = get(0);
#pragma unroll
    for (int b = 1; b < NB; ++b) m = max(m, get(b));
    return m;
  }
};

template <int D>
struct Shape {
  static constexpr int NB = D / 32;                 // scale blocks
  static constexpr int CH = D / 32;                 // 16-byte pieces of a position's codes
  static constexpr uint32_t kRow = D / 2;           // bytes of a position
  static constexpr uint32_t kCodes = kSub4 * kRow;  // of a stage's keys (and of its values)
  static constexpr int H = D == 256 ? 2 : 1;        // blocks of a lane's quarter of a key
  // a stage: keys, values, keys' factors [8][4][H][4] words, values' factors [NB][4][4] words, references
  static constexpr uint32_t kV = kCodes, kKf = 2 * kCodes, kVf = kKf + 8 * 4 * H * 4 * 4, kRef = kVf + NB * 4 * 4 * 4,
                            kStage = kRef + 16;
  // where the 16-byte piece `c` of position p lies.  Keys: rows in the order of the score matrix's columns
  // (column 2 c + x of tile t: position 8 t + c + 4 x)
  __device__ static uint32_t key_at(int p, int c) {
    const int r = (p & ~7) | ((p & 3) << 1) | ((p >> 2) & 1);
    return (uint32_t)r * kRow + (uint32_t)((D == 256 ? c ^ (r & 1) : c) << 4);
  }
  __device__ static uint32_t value_swizzle(int p) { return D == 64 ? 0 : D == 128 ? ((uint32_t)p & 2u) : ((uint32_t)p & 3u) << 1; }
  __device__ static uint32_t value_at(int p, int c) {
    return kV + (uint32_t)p * kRow + (((uint32_t)c ^ value_swizzle(p)) << 4);
  }
};

__device__ __forceinline__ float pow2_of(int32_t e) { return __uint_as_float((uint32_t)max(e, 0) << 23); }   // 2^(e - 127)

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// The largest byte of a word.
__device__ __forceinline__ uint32_t largest_of(uint32_t w) {
  return max(max(w & 255u, w >> 8 & 255u), max(w >> 16 & 255u, w >> 24));
}
// 8 bf16 elements, of a head that 16 lanes hold, to fp16 with the head's largest element in [2^14, 2^15): exact, but for
// what is below 2^-24 then.  `unit`: what they were divided by.
__device__ __forceinline__ void to_f16(uint4& u, float& unit) {
  uint32_t w[4] = {u.x, u.y, u.z, u.w}, top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) top = max(top, __shfl_xor_sync(~0u, top, o));
  const int32_t by = min(268 - (int32_t)(top >> 7), 253);
  const float up = pow2_of(by);
  unit = pow2_of(254 - by);
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack2<false>(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xFFFF0000u) * up);
  u = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) { asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory"); }
__device__ __forceinline__ void sts16(uint32_t a, uint32_t v) {
  asm volatile("{\n\t.reg .u16 t;\n\tcvt.u16.u32 t, %1;\n\tst.shared.u16 [%0], t;\n\t}" ::"r"(a), "r"(v) : "memory");
}

__device__ __forceinline__ void mma_from_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

template <bool BF16, int D, int TILE, int WARPS, int STAGES, bool SLOTS>
__global__ void __launch_bounds__(WARPS * 32, 1) attn_fp4_kernel(const __grid_constant__ AttnParams p) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  using S = Shape<D>;
  using Place = Cursor<SLOTS, kSub4>;
  constexpr int MT = TILE / 16;          // matrix tiles of 16 query heads x rows
  constexpr int KS = D / 16;             // steps of the first product
  constexpr int NT = D / 8;              // output columns of a lane pair, and tiles of 8 columns
  constexpr int CH = S::CH;
  static_assert(STAGES >= 3, "scales are stored one fetch after their codes");

  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ uint32_t err;
  // What only a unit's or segment's ends need lies in shared memory: in registers it would push the loops' own
  // values out to local memory.
  struct Walks {
    Place fetch, at;
    int64_t end;                         // of the worker's range, counted from at's unit's first subtile
    int64_t f_end;                       // the same of fetch's
  };
  __shared__ Walks walks[WARPS];
  __shared__ Split split;
  __shared__ Rows meta;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int quad = lane & 3, col = lane >> 2;
  // a team's warps have the same range, each with a key-value head of its own
  const int32_t member = warp % p.team, team = warp / p.team * gridDim.x + blockIdx.x;
  Walks& w = walks[warp];
  allow_launch_after();
  if (threadIdx.x == 0) err = kOk;
  __syncthreads();

  bool work;
  {
    Split sp;
    Place at;
    Rows rows{};
    int64_t end;
    work = find_range<Place, SLOTS, WARPS>(p, rows, sp, at, end, team, ring, &err);
    // the parts of a head's units lie one after another
    if (team < sp.active && lane == 0) p.open_parts[member * sp.active + team] = 0;
    if (threadIdx.x == 0) {
      if (blockIdx.x == 0) *p.active = sp.active * p.team;
      split = sp;
      meta = rows;
    }
    if (lane == 0) w.fetch = w.at = at, w.end = w.f_end = end;
  }
  __syncthreads();
  uint32_t warp_err = kOk;
  if (work) {
    const int32_t worker = member * split.active + team;
    const uint32_t my_ring = smem_addr(ring) + (uint32_t)warp * (STAGES * S::kStage);

    // ---- fetching side: runs STAGES - 1 subtiles ahead, over the ends of segments ----
    constexpr int ROWS = 32 / CH;                     // positions that one copy of the warp covers
    constexpr int COPIES = kSub4 / ROWS;
    const int piece = lane % CH, row_in = lane / CH;
    // (offsets in 32 bits; where a tensor spans 4 GB or more, `far`, in 64)
    const uint32_t kp = (uint32_t)p.k_page, ks = (uint32_t)p.k_slot, vp = (uint32_t)p.v_page, vs = (uint32_t)p.v_slot;
    const uint32_t ksp = (uint32_t)p.ks_page, kss = (uint32_t)p.ks_slot, vsp = (uint32_t)p.vs_page, vss = (uint32_t)p.vs_slot;
    int32_t f_left;                                   // subtiles of the segment that are still to be fetched; 0: all done
    int32_t f_sub;                                    // the next subtile, counted from position 0
    int32_t f_lo, f_hi;                               // what the group's rows see of it
    uint32_t f_k, f_v, f_ks, f_vs;                    // the head: this lane's first copy and scales in a page (slots: the head)
    const int32_t* f_list;                            // the request's pages, or the row's slots
    bool f_first;                                     // the next subtile fetched is a segment's first
    int32_t entry;                                    // page of the next subtile, or slot of its position `lane`
    uint32_t shown[STAGES];                           // (slots) which positions of the stages are one
    // the scales of this lane's position of the subtile fetched last: on their way from memory
    Scales<S::NB> sk, sv;
    bool pend = false, pend_first = false;
    uint32_t ref = kLowest;                           // largest scale of values so far of the segment
    auto look_up = [&]() {
      if constexpr (SLOTS) {
        const int32_t j = f_sub * kSub4 + lane;
        entry = j < p.n_slots ? f_list[j] : -1;
      } else {
        entry = f_list[f_sub / (kPage / kSub4)];
      }
    };
    auto begin_fetch = [&]() {
      const Place& f = w.fetch;
      f_left = (int32_t)min((int64_t)f.nsub, w.f_end) - f.s;
      f_sub = f.base + f.s;
      f_lo = f.lo, f_hi = f.hi;
      f_first = true;
      const int32_t kv = f.kv * p.team + member;
      f_k = (uint32_t)(kv * p.k_head) + piece * 16, f_v = (uint32_t)(kv * p.v_head) + piece * 16;
      f_ks = (uint32_t)(kv * p.ks_head), f_vs = (uint32_t)(kv * p.vs_head);
      if constexpr (!SLOTS) f_k += row_in * ks, f_v += row_in * vs, f_ks += lane * kss, f_vs += lane * vss;
      f_list = SLOTS ? p.slots + (int64_t)f.row0 * p.n_slots : p.page_table + (int64_t)f.req * p.max_pages;
      look_up();
    };
    begin_fetch();
    // factors of the subtile fetched last, into its stage
    const uint32_t kf_to = S::kKf + (uint32_t)((2 * quad + (col & 1)) * 16 * S::H + (lane >> 3)) * 4;
    const uint32_t vf_to = S::kVf + (uint32_t)(quad * 4 + (lane >> 3)) * 4 + (col & 1) * 2;
    auto put_scales = [&](int stage) {
      if (!pend) return;
      const uint32_t to = my_ring + (uint32_t)stage * S::kStage;
      const uint32_t ek = max(__reduce_max_sync(~0u, sk.largest()), kLowest), ev = __reduce_max_sync(~0u, sv.largest());
      if (max(ek, ev) > kMaxScaleByte) warp_err = kErrInvalidValue;
      ref = max(pend_first ? kLowest : ref, ev);
#pragma unroll
      for (int i = 0; i < 4 * S::H; ++i)              // quarter i / H, its block i % H
        sts32(to + kf_to + (uint32_t)i * 16, factor2(sk.get(D == 64 ? i / 2 : i), ek));
#pragma unroll
      for (int b = 0; b < S::NB; ++b) sts16(to + vf_to + (uint32_t)b * 64, factor2(sv.get(b), ref));
      if (lane == 0) sts32(to + S::kRef, ek), sts32(to + S::kRef + 4, ref);
    };
    // where this lane's pieces go: copy i, from the first one's place (keys of head dimension 256: every second copy
    // is swizzled the other way)
    const uint32_t key0 = S::key_at(row_in, piece), value0 = S::value_at(row_in, piece);
    const uint32_t key1 = D == 256 ? S::key_at(row_in + 4, piece) : 0;
    static_assert(ROWS % (D == 256 ? 4 : 8) == 0, "the copies of a lane lie alike");
    auto key_to = [&](uint32_t dst, int i) {
      return dst + (D == 256 ? (i & 1 ? key1 : key0) + (uint32_t)(i >> 1) * 8 * S::kRow : key0 + (uint32_t)(i * ROWS) * S::kRow);
    };
    auto fetch = [&](int stage, int stage_before) {
      put_scales(stage_before);
      pend = f_left > 0;
      if (f_left > 0) {
        const uint32_t dst = my_ring + (uint32_t)stage * S::kStage, dv = dst + value0;
        auto to_v = [&](int i) { return dv + (uint32_t)(i * ROWS) * S::kRow; };
        // where a tensor is far, from its first byte: the head's
        auto far_head = [&](int64_t head) { return (w.fetch.kv * p.team + member) * head; };
        if constexpr (SLOTS) {
          const bool on = entry >= 0 && entry < p.num_pages * kPage;
          if (!on && entry != -1) warp_err = kErrInvalidPage;
          const uint32_t mask = __ballot_sync(~0u, on);
#pragma unroll
          for (int i = 0; i < STAGES; ++i)
            if (i == stage) shown[i] = mask;
          const uint32_t page = on ? (uint32_t)entry / kPage : 0, off = on ? (uint32_t)entry % kPage : 0;
          sk.clear(), sv.clear();
          if (!p.far) {
            if (on) sk.load(p.k_scale + (f_ks + page * ksp + off * kss)), sv.load(p.v_scale + (f_vs + page * vsp + off * vss));
            const uint32_t ok = page * kp + off * ks, ov = page * vp + off * vs;
#pragma unroll
            for (int i = 0; i < COPIES; ++i) {
              const int r = i * ROWS + row_in;
              const uint32_t bytes = mask >> r & 1u ? 16u : 0u;
              copy16(key_to(dst, i), (const uint8_t*)p.k + (__shfl_sync(~0u, ok, r) + f_k), bytes);
              copy16(to_v(i), (const uint8_t*)p.v + (__shfl_sync(~0u, ov, r) + f_v), bytes);
            }
          } else {
            if (on) {
              sk.load(p.k_scale + far_head(p.ks_head) + page * p.ks_page + off * p.ks_slot);
              sv.load(p.v_scale + far_head(p.vs_head) + page * p.vs_page + off * p.vs_slot);
            }
            const unsigned long long ok = page * p.k_page + off * p.k_slot, ov = page * p.v_page + off * p.v_slot;
            const uint8_t *k = (const uint8_t*)p.k + far_head(p.k_head) + piece * 16, *v = (const uint8_t*)p.v + far_head(p.v_head) + piece * 16;
#pragma unroll
            for (int i = 0; i < COPIES; ++i) {
              const int r = i * ROWS + row_in;
              const uint32_t bytes = mask >> r & 1u ? 16u : 0u;
              copy16(key_to(dst, i), k + __shfl_sync(~0u, ok, r), bytes);
              copy16(to_v(i), v + __shfl_sync(~0u, ov, r), bytes);
            }
          }
        } else {
          const bool there = entry >= 0 && entry < p.num_pages;
          const int32_t pos0 = f_sub * kSub4;
          const uint32_t page = (uint32_t)entry;
          if (!p.far && there && pos0 >= f_lo && pos0 + kSub4 <= f_hi) {
            const bool second = f_sub & 1;            // of the page's halves
            sk.load(p.k_scale + (f_ks + page * ksp + (second ? kSub4 * kss : 0u)));
            sv.load(p.v_scale + (f_vs + page * vsp + (second ? kSub4 * vss : 0u)));
            uint32_t k = f_k + page * kp + (second ? kSub4 * ks : 0u), v = f_v + page * vp + (second ? kSub4 * vs : 0u);
#pragma unroll
            for (int i = 0; i < COPIES; ++i, k += ROWS * ks, v += ROWS * vs) {
              copy16(key_to(dst, i), (const uint8_t*)p.k + k, 16u);
              copy16(to_v(i), (const uint8_t*)p.v + v, 16u);
            }
          } else {
            if (!there) warp_err = kErrInvalidPage;
            const int64_t at = there ? entry : 0;
            const int32_t off = pos0 % kPage;
            sk.clear(), sv.clear();
            if (there && pos0 + lane >= f_lo && pos0 + lane < f_hi) {
              sk.load(p.k_scale + far_head(p.ks_head) + at * p.ks_page + (off + lane) * p.ks_slot);
              sv.load(p.v_scale + far_head(p.vs_head) + at * p.vs_page + (off + lane) * p.vs_slot);
            }
            const uint8_t* k = (const uint8_t*)p.k + far_head(p.k_head) + piece * 16 + at * p.k_page + (off + row_in) * p.k_slot;
            const uint8_t* v = (const uint8_t*)p.v + far_head(p.v_head) + piece * 16 + at * p.v_page + (off + row_in) * p.v_slot;
#pragma unroll
            for (int i = 0; i < COPIES; ++i, k += ROWS * p.k_slot, v += ROWS * p.v_slot) {
              const int32_t pos = pos0 + i * ROWS + row_in;
              const bool on = there && pos >= f_lo && pos < f_hi;
              copy16(key_to(dst, i), on ? k : (const uint8_t*)p.k, on ? 16u : 0u);
              copy16(to_v(i), on ? v : (const uint8_t*)p.v, on ? 16u : 0u);
            }
          }
        }
        pend_first = f_first;
        f_first = false;
        ++f_sub;
        if (--f_left > 0) {
          look_up();
        } else {
          Place f = w.fetch;
          const int64_t left = w.f_end - f.nsub - kUnitCost;
          if (left > 0) f.next_unit(p, meta);
          __syncwarp();
          if (lane == 0) w.fetch = f, w.f_end = left;
          __syncwarp();
          if (left > 0) begin_fetch();
        }
      }
      copy_commit();
    };
#pragma unroll
    for (int i = 0; i < STAGES; ++i) shown[i] = 0;
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) fetch(i, i - 1);

    // ---- computing side ----
    int stage = 0;
    const float c = p.scale_log2;
    const Two cc = two(c, c), shift = two((float)kF16Shift, (float)kF16Shift);
    for (bool more = true; more;) {
      int32_t left, sub;                  // subtiles of the segment to go, and the next one
      uint32_t qf[MT][KS][4];
      float o[MT][NT][4];
      float mx[MT][2], unit[MT][2];       // the weights' reference; what the queries were divided by
      Two sum[MT][2];
      uint32_t live = 0;                  // bit 2t + e: the thread's tile row is a row that sees something
      bool seen = false;                  // (slots) some slot of the segment was one
      uint32_t o_ref = kLowest;           // the weighted values' reference
      int32_t full_lo = 0, full_hi = INT32_MAX;   // positions that every row of the group sees
      // tile row m: row m / chunk_heads of the group, head h0 + m % chunk_heads
      {
        const Place at = w.at;
        const Rows rows = meta;
        const int32_t h0 = (at.kv * p.team + member) * p.group + at.chunk * p.chunk_heads;
        const int32_t heads = min(p.chunk_heads, p.group - at.chunk * p.chunk_heads);
        left = (int32_t)min((int64_t)at.nsub, w.end) - at.s;
        sub = at.base + at.s;
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int m = t * 16 + e * 8 + col;
            const int j = m / p.chunk_heads, h = m - j * p.chunk_heads;
            bool on = j < at.nrows && h < heads;
            int32_t a = at.lo, b = at.hi;
            if constexpr (!SLOTS) {
              if (on) {
                a = rows.start[at.row0 + j], b = rows.end[at.row0 + j];
                if (b <= a) on = false, a = at.lo, b = at.hi;
              }
            }
            if (on) live |= 1u << (2 * t + e);
            full_lo = max(full_lo, a), full_hi = min(full_hi, b);
            mx[t][e] = kNegInf, sum[t][e] = two(0.f, 0.f), unit[t][e] = 1.f;
            // this lane's quarter of the head
            const uint2* src = (const uint2*)((const T*)p.q + (int64_t)(at.row0 + j) * p.q_row + (int64_t)(h0 + h) * p.q_head +
                                              quad * (D / 4));
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              const uint2 u = on ? src[k] : make_uint2(0, 0);
              qf[t][k][e] = u.x;
              qf[t][k][2 + e] = u.y;
              if constexpr (BF16) {
                top = max(top, max(u.x & 0x7FFFu, (u.x >> 16) & 0x7FFFu));
                top = max(top, max(u.y & 0x7FFFu, (u.y >> 16) & 0x7FFFu));
              }
            }
            if constexpr (BF16) {
              // to a largest element in [2^14, 2^15): exact, but for what is below 2^-24 then
              top = max(top, __shfl_xor_sync(~0u, top, 1));
              top = max(top, __shfl_xor_sync(~0u, top, 2));
              const int32_t by = min(268 - (int32_t)(top >> 7), 253);
              const float up = pow2_of(by);
              unit[t][e] = pow2_of(254 - by);
#pragma unroll
              for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int x = 0; x < 4; x += 2) {
                  const uint32_t u = qf[t][k][x + e];
                  qf[t][k][x + e] = pack2<false>(__uint_as_float(u << 16) * up, __uint_as_float(u & 0xFFFF0000u) * up);
                }
            }
          }
      }
      full_lo = __reduce_max_sync(~0u, full_lo);
      full_hi = __reduce_min_sync(~0u, full_hi);
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) o[t][n][x] = 0.f;

      for (; left > 0; --left, ++sub) {
        // the next stage goes where the last one computed was
        copy_wait<STAGES - 2>();
        uint32_t on = ~0u;
        if constexpr (SLOTS) {
#pragma unroll
          for (int i = 0; i < STAGES; ++i)
            if (i == stage) on = shown[i];
        }
        __syncwarp();
        {
          const int into = stage == 0 ? STAGES - 1 : stage - 1;
          fetch(into, into == 0 ? STAGES - 1 : into - 1);
        }
        const uint32_t st = my_ring + (uint32_t)stage * S::kStage;
        stage = stage == STAGES - 1 ? 0 : stage + 1;
        const uint2 refs = lds64(st + S::kRef);

        // scores of the subtile: four tiles of 8 positions, four chains of products
        float s[MT][4][4];
        {
#pragma unroll
          for (int i = 0; i < S::H; ++i) {            // a block's 16 bytes (8 at head dimension 64)
            uint32_t kw[4][4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              const uint32_t row = st + (uint32_t)(n * 8 + col) * S::kRow;
              if constexpr (D == 64) {
                const uint2 u = lds64(row + quad * 8);
                kw[n][0] = u.x, kw[n][1] = u.y;
              } else {
                const uint4 u = lds128(row + (uint32_t)((D == 256 ? (quad * 2 + i) ^ (col & 1) : quad) << 4));
                kw[n][0] = u.x, kw[n][1] = u.y, kw[n][2] = u.z, kw[n][3] = u.w;
              }
            }
            const uint4 kf = lds128(st + S::kKf + (uint32_t)((col * 4 + quad) * S::H + i) * 16);
#pragma unroll
            for (int k = 0; k < (D == 64 ? 2 : 4); ++k)
#pragma unroll
              for (int n = 0; n < 4; ++n) {
                uint32_t h[4];
                from_codes(kw[n][k], h);
#pragma unroll
                for (int x = 0; x < 4; ++x) h[x] = hmul2(h[x], n == 0 ? kf.x : n == 1 ? kf.y : n == 2 ? kf.z : kf.w);
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                  if (i == 0 && k == 0)
                    mma_from_zero(s[t][n], qf[t][0], h[0], h[1]);
                  else
                    mma16816<false>(s[t][n], qf[t][(i * 4 + k) * 2], h[0], h[1]);
                  mma16816<false>(s[t][n], qf[t][(i * 4 + k) * 2 + 1], h[2], h[3]);
                }
              }
          }
        }

        const int32_t pos0 = sub * kSub4;
        if constexpr (SLOTS) {
          seen |= on != 0;
          if (on != ~0u) {
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
              for (int x = 0; x < 2; ++x)
                if (!(on >> (n * 8 + quad + 4 * x) & 1)) {
#pragma unroll
                  for (int t = 0; t < MT; ++t) s[t][n][x] = s[t][n][2 + x] = kNegInf;
                }
          }
        } else if (pos0 < full_lo || pos0 + kSub4 > full_hi) {
          // (windows are looked up again: the loop has no registers for them)
          const Place& at = w.at;
#pragma unroll
          for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const bool there = live >> (2 * t + e) & 1;
              const int32_t row = at.row0 + (there ? (t * 16 + e * 8 + col) / p.chunk_heads : 0);
              const int32_t a = there ? meta.start[row] : 0, b = there ? meta.end[row] : 0;
#pragma unroll
              for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  const int32_t pos = pos0 + n * 8 + quad + 4 * x;
                  if (pos < a || pos >= b) s[t][n][2 * e + x] = kNegInf;
                }
            }
        }

        // The reference follows a maximum from 2^kRaise on: until then nothing is scaled, and the lanes of a row need not
        // know one another's maxima.
        const float k_unit = pow2_of((int32_t)refs.x - 12);
        float u[MT][2], top[MT][2];
        bool raise = refs.y != o_ref;
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float m = fmaxf(s[t][0][2 * e], s[t][0][2 * e + 1]);
#pragma unroll
            for (int n = 1; n < 4; ++n) m = fmaxf(m, fmaxf(s[t][n][2 * e], s[t][n][2 * e + 1]));
            // in true units (the factor a power of two, never 0: -infinity stays)
            u[t][e] = BF16 ? fmaxf(fminf(k_unit * unit[t][e], 0x1p127f), 0x1p-126f) : k_unit;
            top[t][e] = m * u[t][e];
            raise |= exponent(top[t][e], mx[t][e], c) > kRaise;   // (false where both are -infinity)
          }
        if (__any_sync(~0u, raise)) {
          const float down = pow2_of(127 + (int32_t)o_ref - (int32_t)refs.y);
          o_ref = refs.y;
#pragma unroll
          for (int t = 0; t < MT; ++t) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float m = top[t][e];
              m = fmaxf(m, __shfl_xor_sync(~0u, m, 1));
              m = fmaxf(m, __shfl_xor_sync(~0u, m, 2));
              const float raised = exponent(m, mx[t][e], c) > kRaise ? m : mx[t][e];
              const float alpha = raised == mx[t][e] ? 1.f : ex2(exponent(mx[t][e], raised, c));
              mx[t][e] = raised;
              sum[t][e] = mul2(sum[t][e], two(alpha, alpha));
              const float a = alpha * down;
              const Two aa = two(a, a);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                const float2 z = both(mul2(two(o[t][n][2 * e], o[t][n][2 * e + 1]), aa));
                o[t][n][2 * e] = z.x, o[t][n][2 * e + 1] = z.y;
              }
            }
          }
        }
        uint32_t pf[MT][2][4];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float base = reference(mx[t][e]);
            const Two uu = two(u[t][e], u[t][e]), minus = two(-base, -base);
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              // (the product with a power of two is exact: one rounding, that of the difference)
              const float2 d = both(fma2(fma2(two(s[t][n][2 * e], s[t][n][2 * e + 1]), uu, minus), cc, shift));
              const float a = ex2(d.x), b = ex2(d.y);
              sum[t][e] = add2(sum[t][e], two(a, b));
              pf[t][n / 2][(n & 1) * 2 + e] = pack2<false>(a, b);
            }
          }

        // the second product: 16 positions a step; this lane's D / 8 elements of four positions, all of one block
        const uint4 vf = lds128(st + S::kVf + (uint32_t)((col * (D / 8) / 32) * 4 + quad) * 16);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const uint32_t f0 = g ? vf.z : vf.x, f1 = g ? vf.w : vf.y;
          constexpr int W = D / 64;                  // words of a lane
          uint32_t vw[4][W];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int pos = g * 16 + i * 4 + quad;
            const uint32_t row = st + S::kV + (uint32_t)pos * S::kRow;
            const uint32_t sw = S::value_swizzle(quad);   // (the same for all four)
            if constexpr (D == 64) {
              vw[i][0] = lds32(row + col * 4);
            } else if constexpr (D == 128) {
              const uint2 x = lds64(row + ((((uint32_t)col >> 1) ^ sw) << 4) + (col & 1) * 8);
              vw[i][0] = x.x, vw[i][1] = x.y;
            } else {
              const uint4 x = lds128(row + (((uint32_t)col ^ sw) << 4));
              vw[i][0] = x.x, vw[i][1] = x.y, vw[i][2] = x.z, vw[i][3] = x.w;
            }
          }
#pragma unroll
          for (int i = 0; i < W; ++i) {
            uint32_t b0[8], b1[8];
            from_pairs(vw[0][i], vw[1][i], b0);
            from_pairs(vw[2][i], vw[3][i], b1);
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              const uint32_t y0 = hmul2(b0[x], f0), y1 = hmul2(b1[x], f1);
#pragma unroll
              for (int t = 0; t < MT; ++t) mma16816<false>(o[t][i * 8 + x], pf[t][g], y0, y1);
            }
          }
        }
      }

      // the segment ends: finish the unit, or leave its part
      {
        Place at = w.at;
        const int64_t end = w.end;
        const int32_t kv = at.kv * p.team + member, h0 = kv * p.group + at.chunk * p.chunk_heads;
        const bool unit_end = end >= at.nsub, cut_front = at.s > 0, whole = unit_end && !cut_front;
        const int which = cut_front ? 0 : 1;
        if (!unit_end && !cut_front && lane == 0) {
          p.open_parts[worker] = split.holder(split.first(team + 1) - end + at.nsub - 1) - team + 1;
          p.open_info[worker] = make_int4(at.row0, at.nrows, kv * p.chunks + at.chunk, 0);
        }
        const float o_unit = pow2_of((int32_t)o_ref - 12);
        constexpr float kBack = kShiftUp<BF16> / (float)(1 << kF16Shift);   // to the shift that the join expects
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 halves = both(sum[t][e]);
            float l = halves.x + halves.y;
            l += __shfl_xor_sync(~0u, l, 1);
            l += __shfl_xor_sync(~0u, l, 2);
            l *= kBack;
            const int m = t * 16 + e * 8 + col;
            const int j = m / p.chunk_heads, h = m - j * p.chunk_heads;
            if (!(live >> (2 * t + e) & 1)) continue;
            // the lane's elements: 2 NT of the head from quad * 2 NT on, o[n][x] is number x * NT + n
            if (!whole) {
              const int64_t at_part = ((int64_t)worker * 2 + which) * TILE + m;
              // a sum of -1: the part saw no position at all
              if (quad == 0) p.part_ml[at_part] = make_float2(mx[t][e], SLOTS && !seen ? -1.f : l);
              float4* dst = (float4*)(p.part_o + at_part * D + quad * (2 * NT));
              const float by = o_unit * kBack;
#pragma unroll
              for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int n = 0; n < NT; n += 4)
                  dst[(x * NT + n) / 4] = make_float4(o[t][n][2 * e + x] * by, o[t][n + 1][2 * e + x] * by,
                                                      o[t][n + 2][2 * e + x] * by, o[t][n + 3][2 * e + x] * by);
            } else {
              const int64_t row = at.row0 + j;
              const int32_t qh = h0 + h;
              const float by = SLOTS && !seen ? 0.f : o_unit * kBack / l;
              uint4* dst = (uint4*)((T*)p.out + row * p.out_row + (int64_t)qh * p.out_head + quad * (2 * NT));
#pragma unroll
              for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int n = 0; n < NT; n += 8) {
                  uint32_t u[4];
#pragma unroll
                  for (int i = 0; i < 4; ++i)
                    u[i] = pack2<BF16>(o[t][n + 2 * i][2 * e + x] * by, o[t][n + 2 * i + 1][2 * e + x] * by);
                  dst[(x * NT + n) / 8] = make_uint4(u[0], u[1], u[2], u[3]);
                }
              if (quad == 0 && p.lse) p.lse[row * p.q_heads + qh] = log_sum_exp<BF16>(mx[t][e], l, c);
            }
          }
        const int64_t rest = end - at.nsub - kUnitCost;
        more = rest > 0;
        if (more) at.next_unit(p, meta);
        __syncwarp();
        if (lane == 0) w.at = at, w.end = rest;
        __syncwarp();
      }
    }
    copy_wait<0>();
  }
  // rows that see nothing
  if constexpr (!SLOTS) {
    for (int64_t i = (int64_t)blockIdx.x * (WARPS * 32) + threadIdx.x; i < p.rows * (int64_t)p.q_heads;
         i += (int64_t)gridDim.x * (WARPS * 32)) {
      const int32_t r = (int32_t)(i / p.q_heads), h = (int32_t)(i - (int64_t)r * p.q_heads);
      if (p.row_end[r] > p.row_start[r]) continue;
      uint4* o = (uint4*)((T*)p.out + r * p.out_row + h * p.out_head);
      for (int j = 0; j < D / 8; ++j) o[j] = make_uint4(0, 0, 0, 0);
      if (p.lse) p.lse[i] = kNegInf;
    }
  }
  warp_err = __reduce_max_sync(~0u, warp_err);
  if (lane == 0 && warp_err != kOk) atomicMax(&err, warp_err);
  __syncthreads();
  if (threadIdx.x == 0) p.cta_status[blockIdx.x] = err;
}

template <bool BF16, int D, int TILE, int WARPS, int STAGES, bool SLOTS>
cudaError_t launch_one(const AttnParams& p, int sm_count, cudaStream_t stream) {
  auto* kernel = attn_fp4_kernel<BF16, D, TILE, WARPS, STAGES, SLOTS>;
  constexpr int smem = WARPS * STAGES * (int)Shape<D>::kStage;
  static_assert(smem >= WARPS * 32 * 8, "find_range's room");
  if (p.workers != sm_count * WARPS) return cudaErrorInvalidValue;
  static std::atomic<bool> done[64];
  cudaError_t e = set_smem_once(kernel, smem, done);
  if (e != cudaSuccess) return e;
  kernel<<<sm_count, WARPS * 32, smem, stream>>>(p);
  return cudaGetLastError();
}

template <bool BF16, bool SLOTS>
cudaError_t pick(const AttnParams& p, int sm_count, cudaStream_t stream) {
  if (p.dim == 64 && p.tile == 16) return launch_one<BF16, 64, 16, 12, 3, SLOTS>(p, sm_count, stream);
  if (p.dim == 64 && p.tile == 32) return launch_one<BF16, 64, 32, 8, 3, SLOTS>(p, sm_count, stream);
  if (p.dim == 128 && p.tile == 16) return launch_one<BF16, 128, 16, SLOTS ? 8 : 12, 3, SLOTS>(p, sm_count, stream);
  if (p.dim == 128 && p.tile == 32) return launch_one<BF16, 128, 32, 8, 3, SLOTS>(p, sm_count, stream);
  if (p.dim == 256 && p.tile == 16) return launch_one<BF16, 256, 16, 6, 3, SLOTS>(p, sm_count, stream);
  return cudaErrorInvalidValue;
}

}  // namespace fp4
}  // namespace attn
}  // namespace idxk
