/*
 * idxtopk.h -- C ABI of the GB300 (sm_103a) FP4 paged-MQA indexer prefill with
 * fused exact TopK.
 *
 * The operation (defined by "[FlyDSL] Add FP4 LiteTopK prefill operator",
 * ROCm/aiter#5309, Summary and Implementation, and "[FlyDSL][DSv4] Prototype
 * FP4 MQA streaming TopK", ROCm/aiter#5282, Changes and Scope):
 *
 *   for every query row r of request req = row_req[r] and window
 *   [start, end) = [row_start[r], row_end[r]) of logical C4 positions:
 *     logit[r,h,s] = sum_{d<128} q[r,h,d] * k[s,d]        (FP4 E2M1, UE8M0/32)
 *     score[r,s]   = sum_{h<64} w[r,h] * max(logit[r,h,s], 0)    (fp32)
 *     raw[r]       = the topk positions s in [start, end) ranked by score
 *                    descending, then position ascending; NaN ranks below
 *                    every number and +0 above -0 (aiter#5282 Changes).  When
 *                    end - start <= topk the row returns start..end-1 in
 *                    order, padded with -1 (short-row contract, aiter#5282
 *                    Changes).  The dense [rows, context] score matrix is
 *                    never materialised (aiter#5309 Summary).
 *     phys[r]      = page_table[req][raw / 64] * 64 + raw % 64; -1 stays -1
 *                    (aiter#5282 Changes: raw C4 positions mapped through the
 *                    page table; sglang#38101 Changes: physical slots and
 *                    optional raw indices written in place).
 *
 * Conventions for every entry point:
 *  - Tensors are passed as idx_tensor_t descriptors of DEVICE memory that the
 *    caller owns (idx_topk_fp4_prefill_host alone takes host memory); the
 *    library keeps no pointer after it returns.  All tensors
 *    of a call must live on one device; the call makes that device current for
 *    its duration and restores the caller's current device before returning
 *    (aiter#5309 Implementation: caller device/stream ownership).
 *  - Work is enqueued on the caller's `stream` only (never the legacy default
 *    stream); the call returns after that stream has reached the end of the
 *    call's work, because the status is read back to the host.  Scratch is
 *    allocated stream-ordered on that stream from a library-owned pool and is
 *    bounded by rows, topk and the SM count -- never by the context length
 *    (aiter#5282 Changes, last paragraph).
 *  - Every tensor must be C-contiguous with a 16-byte-aligned base address
 *    (the 16-bit tensors of the attention and eviction operators may have
 *    strides, see there).
 *  - Offsets are computed in 64 bits (aiter#5309 Implementation).
 *  - Fail closed (aiter#5309 Implementation): any error returns a nonzero
 *    code, and, when the output descriptors themselves are valid, the outputs
 *    are filled with -1 -- except while the stream is being captured into a
 *    CUDA graph, where nothing is enqueued and IDX_ERR_UNSUPPORTED is returned
 *    (aiter#5282 Scope: graph capture is rejected explicitly).
 */
#ifndef IDXTOPK_H_
#define IDXTOPK_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t / CUstream. */
typedef struct CUstream_st* idx_stream_t;

typedef enum {
  IDX_OK = 0,
  IDX_ERR_INVALID_ARGUMENT = 1, /* null/misaligned/non-contiguous tensor, wrong dtype/rank/shape,
                                   tensors on different devices */
  IDX_ERR_UNSUPPORTED = 2,      /* topk not in {512, 1024}; H != 64, D != 128, page != 64;
                                   stream capture active; device is not sm_103 */
  IDX_ERR_INVALID_METADATA = 3, /* row_req out of [0, num_req), start < 0, end < start,
                                   end > max_pages * 64 */
  IDX_ERR_INVALID_PAGE = 4,     /* a page-table entry covering some row's window is outside
                                   [0, num_pages) */
  IDX_ERR_OVERFLOW = 5,         /* num_pages * 64 or max_pages * 64 exceeds INT32_MAX, or a
                                   size product overflows 64 bits */
  IDX_ERR_CUDA = 6,             /* a CUDA runtime/driver call failed */
  IDX_ERR_INTERNAL = 7,         /* selector failure: a scored row produced fewer than topk
                                   candidates, or a plan bound was exceeded */
  IDX_ERR_TIMEOUT = 8,          /* a bounded device-side wait expired (the kernel returned
                                   instead of hanging) */
  IDX_ERR_SCRATCH_LIMIT = 9,    /* idx_topk_fp4_prefill_noalloc only: the call needs more
                                   scratch than IDX_NOALLOC_SCRATCH_BYTES */
  IDX_ERR_INVALID_VALUE = 10    /* an input value outside the accepted domain (see
                                   IDX_MAX_SCALE_BYTE and IDX_MAX_ABS_WEIGHT): a scale byte
                                   above 167 in the query block of a scored row or in a K page
                                   that a window covers, or a weight of a scored row that is not
                                   finite or exceeds 2^24 in magnitude; attention over a 4-bit
                                   cache: a scale byte above 167 of a position that a row sees */
} idx_status_t;

/*
 * Accepted value domain (aiter#5309 Implementation: the operator fails closed
 * rather than produce nonfinite scores).  Every UE8M0 scale byte the scorer
 * reads -- the query block of each row it scores, and every K page under a
 * scored window -- must be at most IDX_MAX_SCALE_BYTE (scale exponent at most
 * +40; the NaN byte 255 is above it), and every weight of a scored row must be
 * finite with magnitude at most IDX_MAX_ABS_WEIGHT.  A per-head logit is then
 * below 2^93 in magnitude (at most 4 blocks x 32 products of E2M1 magnitudes
 * <= 6, i.e. < 2^13, times 2^(40+40)) and a score below 64 * 2^24 * 2^93 =
 * 2^123, so every score is finite.  A call that reads a value outside the
 * domain returns IDX_ERR_INVALID_VALUE with -1 outputs.  Bytes the scorer never
 * reads (pages outside every window, query blocks and weights of rows of
 * length <= topk) are not checked.
 */
#define IDX_MAX_SCALE_BYTE 167
#define IDX_MAX_ABS_WEIGHT 16777216.0f

typedef enum { IDX_U8 = 1, IDX_I32 = 2, IDX_F32 = 3, IDX_BF16 = 4, IDX_F16 = 5 } idx_dtype_t;

/* Descriptor of one device tensor.  shape/stride are in elements; only the
 * first ndim entries are read. */
typedef struct {
  void* data;
  int32_t dtype; /* idx_dtype_t */
  int32_t ndim;
  int64_t shape[4];
  int64_t stride[4];
} idx_tensor_t;

/*
 * Fused FP4 paged-MQA scoring + exact TopK + page mapping (the hot path).
 *
 *   q_fp4        u8  [R, 64, 64]   FP4 E2M1 codes of the 64x128 query block of each row,
 *                                  two per byte, even element of D in the low nibble
 *   q_scale      u8  [R, 64, 4]    UE8M0 scale per 32 elements of D (2^(byte-127))
 *   k_cache_fp4  u8  [NP, 64, 64]  C4 K cache, page size 64, same encoding
 *   k_scale      u8  [NP, 64, 4]   UE8M0 scales of the K cache
 *   weights      f32 [R, 64]       per-head weights
 *   page_table   i32 [NR, MP]      physical page of logical page p of request i
 *   row_req      i32 [R]           request of each row
 *   row_start    i32 [R]           window start (logical C4 position, inclusive)
 *   row_end      i32 [R]           window end (exclusive)
 *   topk         512 or 1024
 *   out_phys_slot i32 [R, topk]    physical C4 slot (page * 64 + offset) or -1
 *   out_raw_idx   i32 [R, topk]    logical C4 position or -1; may be NULL
 *
 * Rows whose window is longer than topk are ordered by (score desc, position asc).
 * Scale bytes and weights must lie in the accepted domain above (else
 * IDX_ERR_INVALID_VALUE).  The operation is the one
 * defined at the top of this file (aiter#5309 Summary and Implementation;
 * aiter#5282 Changes and Scope).
 */
int idx_topk_fp4_prefill(const idx_tensor_t* q_fp4, const idx_tensor_t* q_scale,
                         const idx_tensor_t* k_cache_fp4, const idx_tensor_t* k_scale,
                         const idx_tensor_t* weights, const idx_tensor_t* page_table,
                         const idx_tensor_t* row_req, const idx_tensor_t* row_start,
                         const idx_tensor_t* row_end, int32_t topk,
                         const idx_tensor_t* out_phys_slot, const idx_tensor_t* out_raw_idx,
                         idx_stream_t stream);

/*
 * idx_topk_fp4_prefill for a page-interleaved K cache (a consumer layout named
 * as follow-up work in "[FlyDSL][DSv4] Prototype FP4 MQA streaming TopK",
 * ROCm/aiter#5282, Scope): each physical page holds its codes and then its
 * scales, so one page is one contiguous 4352-byte record.
 *   k_pages u8 [NP, 4352]   bytes [0, 4096): 64 slots x 64 B of E2M1 codes
 *                           (as k_cache_fp4[page]); bytes [4096, 4352): 64
 *                           slots x 4 UE8M0 scales (as k_scale[page]).
 * Every other argument, the results and the error behaviour are those of
 * idx_topk_fp4_prefill; the outputs are identical for the same data.
 */
int idx_topk_fp4_prefill_paged(const idx_tensor_t* q_fp4, const idx_tensor_t* q_scale,
                               const idx_tensor_t* k_pages, const idx_tensor_t* weights,
                               const idx_tensor_t* page_table, const idx_tensor_t* row_req,
                               const idx_tensor_t* row_start, const idx_tensor_t* row_end,
                               int32_t topk, const idx_tensor_t* out_phys_slot,
                               const idx_tensor_t* out_raw_idx, idx_stream_t stream);

/*
 * idx_topk_fp4_prefill with the K cache's scales pre-arranged in the order in
 * which the block-scaled MMA's scale copy reads them (the pre-shuffled scale
 * input named as follow-up work in "[FlyDSL][DSv4] Prototype FP4 MQA streaming
 * TopK", ROCm/aiter#5282, Scope; here the layout of sm_103a's 32x128b scale
 * copy into tensor memory instead of the AMD matrix-core layout):
 *   k_scale_mma u8 [NP, 256]  byte 8*j + 4*h + b of page p = scale b (D
 *                             elements 32b .. 32b+31) of slot 32*h + j of page
 *                             p, for j < 32, h < 2, b < 4; i.e. the page's
 *                             slot words reordered j, 32+j, j+1, 33+j, ...
 * A cache writer that stores its scales this way spares the scorer the
 * rearrangement; each producer lane then reads one 8-byte word per page.
 * Every other argument, the value domain, the results and the errors are those
 * of idx_topk_fp4_prefill; the outputs are identical for the same data.
 */
int idx_topk_fp4_prefill_mma_scales(const idx_tensor_t* q_fp4, const idx_tensor_t* q_scale,
                                    const idx_tensor_t* k_cache_fp4,
                                    const idx_tensor_t* k_scale_mma, const idx_tensor_t* weights,
                                    const idx_tensor_t* page_table, const idx_tensor_t* row_req,
                                    const idx_tensor_t* row_start, const idx_tensor_t* row_end,
                                    int32_t topk, const idx_tensor_t* out_phys_slot,
                                    const idx_tensor_t* out_raw_idx, idx_stream_t stream);

/*
 * idx_topk_fp4_prefill on tensors in host memory (no counterpart on the
 * pages: it serves callers whose query block, K cache and metadata sit
 * in host memory, and it is the end-to-end form of the operation, host copies
 * included).
 *   device  the GPU to run on (0 .. count-1); stream must belong to it or be NULL.
 * Every descriptor points to host memory: pinned memory (cudaHostAlloc or
 * cudaHostRegister) makes the copies asynchronous DMA; pageable memory also
 * works, at host-copy speed.  Shapes, dtypes and results are those of
 * idx_topk_fp4_prefill; host buffers need no particular alignment.  The call
 * takes one block of device memory from the library's stream-ordered pool,
 * copies each input into it (one cudaMemcpyAsync per tensor on `stream`), runs
 * the fused path there, copies the outputs back, returns the block to the pool
 * and returns once `stream` has completed.  It keeps no pointer.  Error codes
 * are those of idx_topk_fp4_prefill; a descriptor that points to device memory
 * or a device index out of range is IDX_ERR_INVALID_ARGUMENT.  On any error
 * after the output descriptors are validated, the host outputs are filled
 * with -1.
 */
int idx_topk_fp4_prefill_host(const idx_tensor_t* q_fp4, const idx_tensor_t* q_scale,
                              const idx_tensor_t* k_cache_fp4, const idx_tensor_t* k_scale,
                              const idx_tensor_t* weights, const idx_tensor_t* page_table,
                              const idx_tensor_t* row_req, const idx_tensor_t* row_start,
                              const idx_tensor_t* row_end, int32_t topk,
                              const idx_tensor_t* out_phys_slot, const idx_tensor_t* out_raw_idx,
                              int32_t device, idx_stream_t stream);

/*
 * Stream-ordered variant of idx_topk_fp4_prefill for decode loops and CUDA
 * graphs: the same operation and outputs, with no allocation and no host
 * synchronisation, so a call may be captured into a graph and replayed.  The
 * pages keep decode and graph capture on their previous path and name it as
 * follow-up work ("[FlyDSL][DSv4] Prototype FP4 MQA streaming TopK",
 * ROCm/aiter#5282, Scope); this entry point is that follow-up.
 *   workspace        device memory on the tensors' device, 256-byte aligned,
 *                    at least idx_topk_fp4_scratch_bytes(rows, topk) bytes;
 *                    caller-owned, must not be used by another call that runs
 *                    at the same time.
 *   status           one device uint32 (4-byte aligned) on the same device;
 *                    after the call's work completes on `stream` it holds
 *                    IDX_OK or the device-detected error (invalid metadata,
 *                    invalid page, internal, timeout), and on such an error
 *                    every output entry is -1.
 * Returns IDX_OK when the work was enqueued on `stream` (whether or not the
 * stream is being captured).  Argument errors found on the host (descriptors,
 * shapes, topk, device, workspace size or alignment) return their code with
 * nothing enqueued, the outputs and *status untouched; IDX_ERR_CUDA means a
 * launch failed and *status is not written.  While `stream` is being
 * captured, pointer and stream-device queries are not allowed, so the call
 * uses the current device and does not check that the stream and the tensors
 * belong to it; make one call outside the capture first (it checks them and
 * performs the library's per-device setup).  Graph
 * replays reuse the pointers and sizes seen at capture (a new shape needs a
 * new capture).
 */
int idx_topk_fp4_prefill_async(const idx_tensor_t* q_fp4, const idx_tensor_t* q_scale,
                               const idx_tensor_t* k_cache_fp4, const idx_tensor_t* k_scale,
                               const idx_tensor_t* weights, const idx_tensor_t* page_table,
                               const idx_tensor_t* row_req, const idx_tensor_t* row_start,
                               const idx_tensor_t* row_end, int32_t topk,
                               const idx_tensor_t* out_phys_slot, const idx_tensor_t* out_raw_idx,
                               void* workspace, uint64_t workspace_bytes, uint32_t* status,
                               idx_stream_t stream);

/*
 * Allocation-free variant of idx_topk_fp4_prefill (no counterpart on the
 * pages; it exists for callers that must not allocate device memory
 * during a call: a serving process that has handed all free HBM to its own
 * caches and allocator, so a new reservation would fail or evict; or a caller
 * that cannot afford the device synchronisation and driver work that growing
 * a memory pool may cost inside a latency-bound loop).
 *
 * Arguments, layouts, results, ownership and error behaviour are those of
 * idx_topk_fp4_prefill, with one difference: the scratch comes from a fixed
 * buffer of IDX_NOALLOC_SCRATCH_BYTES per device that is part of the
 * library's device image, so the call makes no cudaMalloc/cudaFree, pool or
 * event allocation.  Its size need is idx_topk_fp4_scratch_bytes(rows, topk):
 * (rows + 3 * SMs) * topk * 8 bytes plus a few KB; a call that needs more
 * returns IDX_ERR_SCRATCH_LIMIT (outputs filled with -1) without running.
 * At 152 SMs that admits up to about 5,640 rows at topk 1024 and 11,630 at 512.
 *
 *  - The buffer is reserved on a device when the library's device code is
 *    loaded there: under CUDA's default lazy module loading that happens at
 *    the first call of this function on the device (which also looks up the
 *    buffer's address, with the device made current); under eager loading
 *    (CUDA_MODULE_LOADING=EAGER) it happens when the process creates its
 *    context on the device, whether or not this function is ever called.
 *    Make the first call before any stream capture begins, and before the
 *    caller hands the device's remaining memory to its own allocator (the
 *    reservation can fail with IDX_ERR_CUDA when no memory is left).
 *  - A device index of 64 or more is rejected with IDX_ERR_INVALID_ARGUMENT
 *    before anything is enqueued.
 *  - All calls on one device share the one buffer.  The call returns only
 *    after its work on `stream` has completed, and a per-device lock held for
 *    the whole call makes concurrent calls from several host threads run one
 *    after another, so calls never overlap on the buffer (other streams of
 *    the same process included; each process has its own buffer).
 */
#define IDX_NOALLOC_SCRATCH_BYTES (48u * 1024u * 1024u)
int idx_topk_fp4_prefill_noalloc(const idx_tensor_t* q_fp4, const idx_tensor_t* q_scale,
                                 const idx_tensor_t* k_cache_fp4, const idx_tensor_t* k_scale,
                                 const idx_tensor_t* weights, const idx_tensor_t* page_table,
                                 const idx_tensor_t* row_req, const idx_tensor_t* row_start,
                                 const idx_tensor_t* row_end, int32_t topk,
                                 const idx_tensor_t* out_phys_slot,
                                 const idx_tensor_t* out_raw_idx, idx_stream_t stream);

/* The supported topk values, {512, 1024} (aiter#5309 Implementation: explicit
 * supported-K contract).  *ks points to static storage.  Always IDX_OK unless
 * an argument is NULL (IDX_ERR_INVALID_ARGUMENT). */
int idx_topk_supported_k(const int32_t** ks, int32_t* n);

/* Static, human-readable name of a status code (the fail-closed status
 * contract of aiter#5309 Implementation). */
const char* idx_topk_status_string(int code);

/* Scratch bytes that idx_topk_fp4_prefill allocates for `rows` rows and
 * `topk`, on `device` (its SM count bounds the work units).  Independent of
 * the context length (aiter#5282 Changes, last paragraph; sglang#38101 Memory
 * geometry).  Returns IDX_ERR_UNSUPPORTED for an unsupported topk,
 * IDX_ERR_CUDA if the device cannot be queried. */
int idx_topk_fp4_scratch_bytes(int32_t rows, int32_t topk, int32_t device, uint64_t* bytes);

/* Diagnostic of the device-side failure detection (no counterpart on the
 * pages).  One CTA on `device` waits, through the same bounded mbarrier wait
 * every kernel of the library uses, on a phase that its own thread completes
 * (never_completes == 0) or that nothing completes (never_completes != 0).
 * Returns the status the kernel recorded: IDX_OK, or IDX_ERR_TIMEOUT once the
 * wait has given up after its 2 s limit -- the kernel then returns with
 * nothing in flight and the CUDA context stays usable.  Synchronises
 * `stream`; IDX_ERR_UNSUPPORTED while the stream is being captured;
 * IDX_ERR_INVALID_ARGUMENT for a bad device index or a stream of another
 * device. */
int idx_debug_bounded_wait(int32_t device, int32_t never_completes, idx_stream_t stream);

/* Peak bytes ever reserved by the library's scratch pool on `device` in this
 * process (the pool's reserved-memory high-water mark).  Measurement support
 * with no counterpart on the pages; it evidences the context-independent
 * scratch bound of aiter#5282 Changes. */
int idx_topk_scratch_high_water(int32_t device, uint64_t* bytes);

/* Measurement support (no counterpart on the pages): when enabled, each call
 * of the calling thread records CUDA events on its stream around the kernel
 * phases; idx_topk_last_timings then returns, in milliseconds, {planning,
 * scoring kernel, finishing kernel, whole kernel sequence} of
 * that thread's last completed call.  Process-wide switch; default off. */
int idx_topk_set_timing(int32_t enable);
int idx_topk_last_timings(float* ms4);

/*
 * Context-parallel pieces ("[AMD][DSv4] Add experimental AITER FP4 streaming
 * TopK", sglang#38101, Changes: context-parallel paths; "[FlyDSL][DSv4]
 * Prototype FP4 MQA streaming TopK", ROCm/aiter#5282, Changes: merge split
 * candidates exactly).  A context partition [c_0, c_1), [c_1, c_2), ... of the
 * logical C4 positions is scored one shard at a time (each call may run where
 * that shard's K pages live); the shards' lists, gathered into one
 * [S, R, topk] pair of tensors by the caller, are merged exactly.  The merged
 * outputs equal those of idx_topk_fp4_prefill on the same data, bit for bit.
 *
 * idx_topk_fp4_prefill_shard: every row whose whole window [start, end) is
 * longer than topk is scored against the part of it inside [ctx_begin,
 * ctx_end) only -- however short that part -- and emits that part's exact
 * TopK, ordered by (score desc, position asc):
 *   out_score    f32 [R, topk]  the scores (as the fused path computes them),
 *                               NaN after the part's last position
 *   out_raw_idx  i32 [R, topk]  logical C4 positions, -1 after the last one
 * Rows whose whole window is at most topk long emit only -1 / NaN (the merge
 * gives them the closed form).  Inputs, value domain and errors as
 * idx_topk_fp4_prefill; ctx_begin < 0 or ctx_end < ctx_begin is
 * IDX_ERR_INVALID_ARGUMENT.  Only the page entries and K pages under the
 * clipped windows are read and checked.  On error out_raw_idx is -1 and
 * out_score NaN.
 */
int idx_topk_fp4_prefill_shard(const idx_tensor_t* q_fp4, const idx_tensor_t* q_scale,
                               const idx_tensor_t* k_cache_fp4, const idx_tensor_t* k_scale,
                               const idx_tensor_t* weights, const idx_tensor_t* page_table,
                               const idx_tensor_t* row_req, const idx_tensor_t* row_start,
                               const idx_tensor_t* row_end, int32_t ctx_begin, int32_t ctx_end,
                               int32_t topk, const idx_tensor_t* out_score,
                               const idx_tensor_t* out_raw_idx, idx_stream_t stream);

/*
 * idx_topk_merge_shards: the exact TopK of each row over the union of its S
 * shard lists (aiter#5282 Changes: exact merge of split candidates), then the
 * short-row contract and the page mapping of idx_topk_fp4_prefill.
 *   shard_score  f32 [S, R, topk]  shard s's out_score (S >= 1)
 *   shard_raw    i32 [S, R, topk]  shard s's out_raw_idx (-1 = empty entry)
 *   page_table, row_req, row_start, row_end  as for idx_topk_fp4_prefill
 *   out_phys_slot, out_raw_idx (nullable)   as for idx_topk_fp4_prefill
 * The shards must cover every window and be disjoint.  A listed position
 * outside its row's window, a position listed twice among the emitted TopK, or
 * a row whose lists hold fewer than topk positions although its window is
 * longer than topk returns IDX_ERR_INVALID_METADATA (as do bad row metadata);
 * a negative page-table entry read by the mapping returns IDX_ERR_INVALID_PAGE
 * (the K cache is not an argument, so entries are not compared with its page
 * count here: the shard calls checked every entry under their windows);
 * unsupported topk IDX_ERR_UNSUPPORTED; outputs -1 on every error.  Scratch:
 * one status word.
 */
int idx_topk_merge_shards(const idx_tensor_t* shard_score, const idx_tensor_t* shard_raw,
                          const idx_tensor_t* page_table, const idx_tensor_t* row_req,
                          const idx_tensor_t* row_start, const idx_tensor_t* row_end,
                          int32_t topk, const idx_tensor_t* out_phys_slot,
                          const idx_tensor_t* out_raw_idx, idx_stream_t stream);

/*
 * Context-tiled comparison path (an ablation of the fused design: "[FlyDSL]
 * [DSv4] Prototype FP4 MQA streaming TopK", ROCm/aiter#5282, Changes, names a
 * bounded context-tiled fallback).  The same operation and outputs as
 * idx_topk_fp4_prefill, computed by scoring `context_tile` logical positions
 * at a time into a materialised fp32 buffer [rows, context_tile] and folding
 * each chunk into every row's running TopK.  Scratch is bounded by rows *
 * (context_tile * 4 + topk * 8) bytes plus the plan, not by the context.
 *   context_tile  positions per chunk, a multiple of 128 and >= 1024.
 * Errors and ownership as idx_topk_fp4_prefill (a bad context_tile returns
 * IDX_ERR_INVALID_ARGUMENT).
 */
int idx_tiled_topk_fp4_prefill(const idx_tensor_t* q_fp4, const idx_tensor_t* q_scale,
                               const idx_tensor_t* k_cache_fp4, const idx_tensor_t* k_scale,
                               const idx_tensor_t* weights, const idx_tensor_t* page_table,
                               const idx_tensor_t* row_req, const idx_tensor_t* row_start,
                               const idx_tensor_t* row_end, int32_t topk, int32_t context_tile,
                               const idx_tensor_t* out_phys_slot, const idx_tensor_t* out_raw_idx,
                               idx_stream_t stream);

/*
 * Debug / dense scorer: the same scoring kernel as the fused path, writing the
 * fp32 scores instead of selecting (no counterpart on the pages; it exposes
 * the scores and per-head logits that the parity tests compare).
 *   out_scores f32 [R, S]      score[r, s] written for every s in [start_r, end_r)
 *                              of every row with a non-empty window; other entries are
 *                              left untouched.  S >= max(row_end) is required and
 *                              checked on the device (IDX_ERR_INVALID_METADATA).
 *   out_logits f32 [R, 64, S2] optional (may be NULL): per-head logits
 *                              logit[r, h, s] for the same (r, s).
 * Other arguments as for idx_topk_fp4_prefill (no topk, no outputs).
 */
int idx_fp4_debug_scores(const idx_tensor_t* q_fp4, const idx_tensor_t* q_scale,
                         const idx_tensor_t* k_cache_fp4, const idx_tensor_t* k_scale,
                         const idx_tensor_t* weights, const idx_tensor_t* page_table,
                         const idx_tensor_t* row_req, const idx_tensor_t* row_start,
                         const idx_tensor_t* row_end, const idx_tensor_t* out_scores,
                         const idx_tensor_t* out_logits, idx_stream_t stream);

/*
 * Exact TopK of a materialised fp32 score matrix under the same total order and
 * short-row contract (aiter#5282 Changes: the order key, NaN below every
 * number, +0 above -0, ties to the lower position; the selection half of the
 * dense comparison path, and the entry that pins that ordering on crafted
 * matrices).
 *   scores      f32 [R, S]   row r's candidates are scores[r, start_r .. end_r)
 *   row_start, row_end i32 [R]
 *   out_raw_idx i32 [R, topk]   positions (absolute within the row) or -1
 * Requires end_r <= S (checked on the device, IDX_ERR_INVALID_METADATA).
 */
int idx_topk_select_scores(const idx_tensor_t* scores, const idx_tensor_t* row_start,
                           const idx_tensor_t* row_end, int32_t topk,
                           const idx_tensor_t* out_raw_idx, idx_stream_t stream);

/*
 * Dense comparison path: materialises fp32 scores [R, score_stride] (rows with
 * window longer than topk), then runs the separate TopK and the page mapping
 * (aiter#5309 Validation: the dense-scores-then-TopK baseline the pages time
 * the fused operator against).
 * Same arguments and outputs as idx_topk_fp4_prefill plus:
 *   score_workspace f32 [R, S_ws], S_ws >= max(row_end), caller-owned; may be
 *                   NULL, in which case R * MP * 64 * 4 bytes are allocated
 *                   stream-ordered for the call.
 */
int idx_dense_topk_fp4_prefill(const idx_tensor_t* q_fp4, const idx_tensor_t* q_scale,
                               const idx_tensor_t* k_cache_fp4, const idx_tensor_t* k_scale,
                               const idx_tensor_t* weights, const idx_tensor_t* page_table,
                               const idx_tensor_t* row_req, const idx_tensor_t* row_start,
                               const idx_tensor_t* row_end, int32_t topk,
                               const idx_tensor_t* out_phys_slot,
                               const idx_tensor_t* out_raw_idx,
                               const idx_tensor_t* score_workspace, idx_stream_t stream);

/*
 * Attention over the cache, and its eviction.
 *
 * The operators below serve the layers that the indexer works for: attention of
 * new tokens over all cached positions of their request (idx_attn_paged), over
 * the slots that the indexer chose (idx_attn_selected), and the eviction of what
 * received little attention (idx_cache_evict).  They have no counterpart on the
 * pages.
 *
 * Common to all of them:
 *   q        [R, Hq, D]        queries of R rows
 *   k_cache  [NP, 64, Hk, D]   keys, physical page by page (page size 64)
 *   v_cache  [NP, 64, Hk, D]   values
 * of one type, IDX_BF16 or IDX_F16; D 64, 128 or 256; Hq a multiple of Hk (query
 * head h reads key-value head h / (Hq / Hk)).  These tensors and `out` may have
 * any strides whose last dimension is contiguous and whose others are
 * non-negative multiples of 8 elements (a cache laid out head by head, keys and
 * values in one allocation, a slice of a fused projection); base addresses are
 * 16-byte aligned.  All other tensors are contiguous.  Outputs must lie apart
 * from the inputs and from each other (their address ranges), except where a
 * function says otherwise.
 *
 * Each has a synchronous form, with the conventions at the top of this file, and
 * a stream-ordered one (_async) that allocates and synchronises nothing and may be
 * captured into a CUDA graph: `workspace` is device memory, 256-byte aligned, of
 * at least the bytes that the _scratch_bytes function gives for the sizes, not
 * used by another call at the same time; `status` is a device uint32 that holds
 * the call's status once its work is done.  Errors that the host finds return
 * their code with nothing enqueued and the outputs untouched.  After an error that
 * the device finds (IDX_ERR_INVALID_METADATA, IDX_ERR_INVALID_PAGE) floating
 * outputs are NaN and integer outputs -1.  Sums, maxima and weights are held in
 * fp32; outputs are rounded once, and the softmax weights p are rounded to the
 * inputs' type for their product with the values: an error of u sum p |v| at most
 * (u 2^-8 or 2^-11; fp16 weights below 2^-24 of a row's largest lose more, n of them
 * n 2^-35 max |v|).  Values are weighted before the division by the sum of up to n
 * weights, so |v| from 2^119 / n on (bf16) can overflow.  Results do not depend on the
 * stream, on timing, or on other calls.  More than INT32_MAX - 65536 positions or
 * slots of a request or row, or NP * 64 above INT32_MAX, are IDX_ERR_OVERFLOW.
 */

/*
 * Attention of new tokens over a paged cache (no counterpart on the pages).  Row r
 * attends over the logical positions [row_start, row_end) of request row_req:
 *   s_hj = scale * q[r, h] . k[j],  out[r, h] = sum_j softmax_j(s_hj) v[j],
 *   out_lse[r, h] = log sum_j exp(s_hj).
 * A row whose window is empty gets out 0 and out_lse -infinity.  Positions
 * outside a row's window never reach its outputs, whatever their keys and values
 * hold, and page entries under no window may be anything; within it infinities and
 * NaN propagate as in the formula.  Rows of one request that follow one another may
 * read the cache together (which of them do depends on their place among the call's
 * rows and on the page table's height; it changes the time a call takes).
 *   page_table i32 [NR, MP], row_req / row_start / row_end i32 [R] as above
 *   scale      above 0, and finite also when multiplied by log2(e)
 *   out        [R, Hq, D], q's type
 *   out_lse    f32 [R, Hq] or NULL
 *   weight_in, weight_out  f32 [NR, MP * 64] or NULL: weight_out[i, s] =
 *              weight_in[i, s] (0 where it is NULL) + the softmax weights that
 *              logical position s of request i received, summed over the
 *              request's rows and query heads in a fixed order.  weight_out may be
 *              weight_in itself; after a device error it then keeps its values.
 *              The workspace then holds R * Hq * MP * 64 fp32 logits.
 * Errors: metadata out of range IDX_ERR_INVALID_METADATA, a page entry under a
 * window outside [0, NP) IDX_ERR_INVALID_PAGE.
 */
int idx_attn_paged(const idx_tensor_t* q, const idx_tensor_t* k_cache, const idx_tensor_t* v_cache,
                   const idx_tensor_t* page_table, const idx_tensor_t* row_req,
                   const idx_tensor_t* row_start, const idx_tensor_t* row_end, float scale,
                   const idx_tensor_t* out, const idx_tensor_t* out_lse,
                   const idx_tensor_t* weight_in, const idx_tensor_t* weight_out,
                   idx_stream_t stream);

/* Stream-ordered idx_attn_paged (no counterpart on the pages). */
int idx_attn_paged_async(const idx_tensor_t* q, const idx_tensor_t* k_cache,
                         const idx_tensor_t* v_cache, const idx_tensor_t* page_table,
                         const idx_tensor_t* row_req, const idx_tensor_t* row_start,
                         const idx_tensor_t* row_end, float scale, const idx_tensor_t* out,
                         const idx_tensor_t* out_lse, const idx_tensor_t* weight_in,
                         const idx_tensor_t* weight_out, void* workspace, uint64_t workspace_bytes,
                         uint32_t* status, idx_stream_t stream);

/* Workspace of idx_attn_paged_async for these sizes on `device` (no counterpart on
 * the pages); without weights it does not depend on the context. */
int idx_attn_paged_scratch_bytes(int32_t rows, int32_t q_heads, int32_t kv_heads,
                                 int32_t head_dim, int32_t num_req, int32_t max_pages,
                                 int32_t with_weights, int32_t device, uint64_t* bytes);

/*
 * Attention of each row over its own list of physical slots, as the TopK writes
 * them to out_phys_slot (no counterpart on the pages: what the indexer's selection
 * is for).
 *   slots  i32 [R, N], N >= 1: physical slot (page * 64 + offset), or -1 for no
 *          position; in any order, empty entries anywhere; a slot listed twice
 *          counts twice.  Row r attends over its slots as idx_attn_paged over a
 *          window; a row without slots gets out 0 and out_lse -infinity.
 * A slot below -1 or at or above NP * 64 is IDX_ERR_INVALID_PAGE.
 */
int idx_attn_selected(const idx_tensor_t* q, const idx_tensor_t* k_cache,
                      const idx_tensor_t* v_cache, const idx_tensor_t* slots, float scale,
                      const idx_tensor_t* out, const idx_tensor_t* out_lse, idx_stream_t stream);

/* Stream-ordered idx_attn_selected (no counterpart on the pages). */
int idx_attn_selected_async(const idx_tensor_t* q, const idx_tensor_t* k_cache,
                            const idx_tensor_t* v_cache, const idx_tensor_t* slots, float scale,
                            const idx_tensor_t* out, const idx_tensor_t* out_lse, void* workspace,
                            uint64_t workspace_bytes, uint32_t* status, idx_stream_t stream);

/* Workspace of idx_attn_selected_async for these sizes on `device` (no counterpart
 * on the pages). */
int idx_attn_selected_scratch_bytes(int32_t rows, int32_t q_heads, int32_t kv_heads,
                                    int32_t head_dim, int32_t selected, int32_t device,
                                    uint64_t* bytes);

/*
 * Eviction of a paged cache by accumulated weight (no counterpart on the pages).  A
 * request of seq_len > budget keeps exactly `budget` positions: its first
 * keep_first, its last keep_last and, of those between, the heaviest (weight
 * descending, +0 above -0, NaN below every number, lower position first: the
 * TopK's order).  Their keys and values are copied, in order of position, to
 * positions 0 .. budget - 1 of the pages that dst_page_table names; the pages that
 * they came from are left as they are, for the caller to free.  A request within
 * the budget keeps its pages, and nothing of it moves.
 *   page_table     i32 [NR, MP], seq_len i32 [NR], weight f32 [NR, MP * 64]
 *   budget >= 1, keep_first >= 0, keep_last >= 0, keep_first + keep_last <= budget
 *   k_dst, v_dst   [DN, 64, Hk, D]: the caches themselves (same address and strides),
 *                  or tensors that lie apart from them.  The two may interleave in one
 *                  allocation, but share no element; only where keys and values of a
 *                  position share elements in the caches (two views of one latent cache)
 *                  may they share the same ones of a position here.
 *   dst_page_table i32 [NR, DP]: fresh pages, DP <= MP, DP * 64 >= min(budget, MP * 64)
 *   out_keep_idx   i32 [NR, budget]  kept positions, ascending, then -1
 *   out_len        i32 [NR]          min(seq_len, budget)
 *   out_page_table i32 [NR, MP]      a cut request's row of dst_page_table, then -1;
 *                                    another's row of page_table
 *   out_weight     f32 [NR, MP * 64] the kept positions' weights at their new
 *                                    positions, then 0
 * Errors: a length outside [0, MP * 64] IDX_ERR_INVALID_METADATA; a page entry under
 * a request's positions outside [0, NP), a fresh page of a cut request outside
 * [0, DN), named twice, or (the caches themselves) under any request's positions
 * IDX_ERR_INVALID_PAGE.  On an error no key or value has moved.
 */
int idx_cache_evict(const idx_tensor_t* k_cache, const idx_tensor_t* v_cache,
                    const idx_tensor_t* page_table, const idx_tensor_t* seq_len,
                    const idx_tensor_t* weight, int32_t budget, int32_t keep_first,
                    int32_t keep_last, const idx_tensor_t* k_dst, const idx_tensor_t* v_dst,
                    const idx_tensor_t* dst_page_table, const idx_tensor_t* out_keep_idx,
                    const idx_tensor_t* out_len, const idx_tensor_t* out_page_table,
                    const idx_tensor_t* out_weight, idx_stream_t stream);

/* Stream-ordered idx_cache_evict (no counterpart on the pages). */
int idx_cache_evict_async(const idx_tensor_t* k_cache, const idx_tensor_t* v_cache,
                          const idx_tensor_t* page_table, const idx_tensor_t* seq_len,
                          const idx_tensor_t* weight, int32_t budget, int32_t keep_first,
                          int32_t keep_last, const idx_tensor_t* k_dst, const idx_tensor_t* v_dst,
                          const idx_tensor_t* dst_page_table, const idx_tensor_t* out_keep_idx,
                          const idx_tensor_t* out_len, const idx_tensor_t* out_page_table,
                          const idx_tensor_t* out_weight, void* workspace,
                          uint64_t workspace_bytes, uint32_t* status, idx_stream_t stream);

/* Workspace of idx_cache_evict_async for these sizes (no counterpart on the pages). */
int idx_cache_evict_scratch_bytes(int32_t num_req, int32_t max_pages, int32_t dst_pages,
                                  int32_t budget, int32_t device, uint64_t* bytes);

/*
 * Writing a paged cache (no counterpart on the pages).  For every row r with a position
 * pos = row_pos[r] >= 0 of request row_req[r]:
 *   y = (x / sqrt(mean x^2 + eps)) * weight   head by head, of q with q_weight and of k with
 *       k_weight (NULL: x as it is);
 *   (a, b) -> (a cos - b sin, b cos + a sin)  for each pair of the rotated dimensions
 *       rope_first .. rope_first + rot - 1 of y, angle i of position pos: neighbours
 *       (rope_pairs 1: dimensions rope_first + 2 i and + 2 i + 1) or halves (0: + i and
 *       + i + rot / 2); NULL: nothing is rotated;
 *   out_q[r] = q's result; k's result and v[r] become slot pos % 64 of page
 *       page_table[row_req[r], pos / 64].
 * A row with position -1 is not there (padding): nothing of it is written.  Rows may
 * come in any order.  All in fp32; results are rounded once to the output's type.
 *   q [R, Hq, D] or NULL (then out_q is too), k [R, Hk, D], v [R, Hk, D] or NULL (then v_cache
 *              is too); strides as above
 *   q_weight, k_weight [D] or NULL, in q's type or IDX_F32 (both alike); eps >= 0, finite
 *   rope       f32 [P, 2, rot / 2] or NULL: the cosines, then the sines of position p's
 *              angles; rot <= D a multiple of 16, rope_first a multiple of 8 (0 without rope)
 *   out_q      [R, Hq, D]; may be q itself
 *   k_cache, v_cache [NP, 64, Hk, D]; they may interleave, but share no element
 * Errors: a position below -1, at or above MP * 64 or (with rope) P, or a request out of range
 * IDX_ERR_INVALID_METADATA; a page outside [0, NP), or a slot named by two rows
 * IDX_ERR_INVALID_PAGE.  After an error that the device finds the caches, and queries in place,
 * are as they were, and out_q is NaN.  (Every call looks for such rows before it writes; with more
 * than 2^14 rows, padding among them, that takes a walk over the rows for every 2^20 slots of
 * the pool.)
 */
int idx_cache_append(const idx_tensor_t* q, const idx_tensor_t* k, const idx_tensor_t* v,
                     const idx_tensor_t* page_table, const idx_tensor_t* row_req,
                     const idx_tensor_t* row_pos, const idx_tensor_t* q_weight,
                     const idx_tensor_t* k_weight, float eps, const idx_tensor_t* rope,
                     int32_t rope_first, int32_t rope_pairs, const idx_tensor_t* out_q,
                     const idx_tensor_t* k_cache, const idx_tensor_t* v_cache,
                     idx_stream_t stream);

/* Stream-ordered idx_cache_append (no counterpart on the pages); it needs no workspace. */
int idx_cache_append_async(const idx_tensor_t* q, const idx_tensor_t* k, const idx_tensor_t* v,
                           const idx_tensor_t* page_table, const idx_tensor_t* row_req,
                           const idx_tensor_t* row_pos, const idx_tensor_t* q_weight,
                           const idx_tensor_t* k_weight, float eps, const idx_tensor_t* rope,
                           int32_t rope_first, int32_t rope_pairs, const idx_tensor_t* out_q,
                           const idx_tensor_t* k_cache, const idx_tensor_t* v_cache,
                           uint32_t* status, idx_stream_t stream);

/*
 * A cache in 4 bits (no counterpart on the pages; the format is the indexer's): E2M1 codes
 * u8 [NP, 64, Hk, D / 2], the even element in the low half of a byte, with one UE8M0 scale e
 * for 32 elements, u8 [NP, 64, Hk, D / 32], which stand for code * 2^(e - 127).  Codes may have
 * any strides whose last dimension is contiguous and whose others are multiples of 16 bytes,
 * scales of D / 32 bytes.  With Hk 1 and D 128 keys in it are the indexer's k_cache_fp4 and
 * k_scale.
 *
 * idx_cache_append_fp4 is idx_cache_append into such a cache: of the normed and rotated key in
 * fp32, and of the value, e is the smallest of 0 .. 254 such that no element of the block
 * exceeds 6 * 2^(e - 127), and an element becomes the nearest code, ties to the even one.  A
 * block with a NaN or an infinity gets e = 255, and codes 0.  Bytes above IDX_MAX_SCALE_BYTE
 * (these, and magnitudes above 6 * 2^40) are written like others and are no error here, but the
 * indexer and attention refuse a call of which a row sees one, with all its rows: a caller whose
 * requests share calls finds the request by its scales.  What becomes codes is computed in
 * the order written, x * (1 / sqrt(mean + eps)) * weight, each operation rounded by itself and
 * the sum of squares as if it were rounded once: the codes do not depend on how the work is
 * divided.
 *   out_q, out_q_scale  out_q [R, Hq, D] in q's type with out_q_scale NULL, or in 4 bits: codes
 *                       u8 [R, Hq, D / 2] with scales u8 [R, Hq, D / 32] (after a device error
 *                       codes 0 and scales 255)
 * No element of the four (or two) cache tensors is shared; codes and scales may interleave page
 * by page.
 */
int idx_cache_append_fp4(const idx_tensor_t* q, const idx_tensor_t* k, const idx_tensor_t* v,
                         const idx_tensor_t* page_table, const idx_tensor_t* row_req,
                         const idx_tensor_t* row_pos, const idx_tensor_t* q_weight,
                         const idx_tensor_t* k_weight, float eps, const idx_tensor_t* rope,
                         int32_t rope_first, int32_t rope_pairs, const idx_tensor_t* out_q,
                         const idx_tensor_t* out_q_scale, const idx_tensor_t* k_codes,
                         const idx_tensor_t* k_scale, const idx_tensor_t* v_codes,
                         const idx_tensor_t* v_scale, idx_stream_t stream);

/* Stream-ordered idx_cache_append_fp4 (no counterpart on the pages); it needs no workspace. */
int idx_cache_append_fp4_async(const idx_tensor_t* q, const idx_tensor_t* k,
                               const idx_tensor_t* v, const idx_tensor_t* page_table,
                               const idx_tensor_t* row_req, const idx_tensor_t* row_pos,
                               const idx_tensor_t* q_weight, const idx_tensor_t* k_weight,
                               float eps, const idx_tensor_t* rope, int32_t rope_first,
                               int32_t rope_pairs, const idx_tensor_t* out_q,
                               const idx_tensor_t* out_q_scale, const idx_tensor_t* k_codes,
                               const idx_tensor_t* k_scale, const idx_tensor_t* v_codes,
                               const idx_tensor_t* v_scale, uint32_t* status,
                               idx_stream_t stream);

/*
 * Listed slots of a 4-bit cache as 16-bit rows (no counterpart on the pages): what the codes
 * stand for, rounded once to the outputs' type.
 *   slots  i32 [N]: physical slots (page * 64 + offset) in any order, also several times; -1
 *          gives zeros
 *   out_k, out_v  [N, Hk, D], IDX_BF16 or IDX_F16, strides as above; v_codes, v_scale and out_v
 *          may be NULL together
 * A slot below -1 or at or above NP * 64 is IDX_ERR_INVALID_PAGE; its row becomes NaN, the
 * others are as they should be.  A scale of 255 gives NaN.
 */
int idx_cache_gather_fp4(const idx_tensor_t* k_codes, const idx_tensor_t* k_scale,
                         const idx_tensor_t* v_codes, const idx_tensor_t* v_scale,
                         const idx_tensor_t* slots, const idx_tensor_t* out_k,
                         const idx_tensor_t* out_v, idx_stream_t stream);

/* Stream-ordered idx_cache_gather_fp4 (no counterpart on the pages); it needs no workspace. */
int idx_cache_gather_fp4_async(const idx_tensor_t* k_codes, const idx_tensor_t* k_scale,
                               const idx_tensor_t* v_codes, const idx_tensor_t* v_scale,
                               const idx_tensor_t* slots, const idx_tensor_t* out_k,
                               const idx_tensor_t* out_v, uint32_t* status, idx_stream_t stream);

/*
 * idx_attn_paged and idx_attn_selected over a cache in 4 bits (no counterpart on the pages):
 * k[j] and v[j] are what the codes and scales of position j stand for, tensors as for
 * idx_cache_append_fp4 (keys and values may share elements here).  Rows, windows, slots, empty
 * rows, outputs and errors as there, and:
 *   a scale byte above IDX_MAX_SCALE_BYTE of a position that a row sees (NaN included) is
 *   IDX_ERR_INVALID_VALUE: as after every error all rows are NaN, of other requests too (in 16
 *   bits a NaN reaches the rows that see it).  idx_cache_append_fp4 writes such bytes.
 * Sums, maxima and weights are held in fp32; softmax weights are rounded to fp16 for their
 * product with the values, for queries of either type: an error of 2^-11 sum p |v| at most, n
 * weights below 2^-24 of a row's largest lose n 2^-35 max |v|.  Of keys, blocks whose scale is
 * below 2^-26 of the largest within 128 positions, and of values, blocks below 2^-26 of the
 * largest that the head has in the request or list, may count as 0 (their elements are below
 * 2^-24 of what the largest block can hold); bf16 queries' elements below 2^-38 of the head's
 * largest lose bits, and that largest (2^x or more), times the largest 2^(e - 127) of keys near
 * (e 26 or more), is taken for 2^153 at most and 2^-100 at least: scores beyond are held there.
 */
int idx_attn_paged_fp4(const idx_tensor_t* q, const idx_tensor_t* k_codes,
                       const idx_tensor_t* k_scale, const idx_tensor_t* v_codes,
                       const idx_tensor_t* v_scale, const idx_tensor_t* page_table,
                       const idx_tensor_t* row_req, const idx_tensor_t* row_start,
                       const idx_tensor_t* row_end, float scale, const idx_tensor_t* out,
                       const idx_tensor_t* out_lse, idx_stream_t stream);

/* Stream-ordered idx_attn_paged_fp4 (no counterpart on the pages). */
int idx_attn_paged_fp4_async(const idx_tensor_t* q, const idx_tensor_t* k_codes,
                             const idx_tensor_t* k_scale, const idx_tensor_t* v_codes,
                             const idx_tensor_t* v_scale, const idx_tensor_t* page_table,
                             const idx_tensor_t* row_req, const idx_tensor_t* row_start,
                             const idx_tensor_t* row_end, float scale, const idx_tensor_t* out,
                             const idx_tensor_t* out_lse, void* workspace,
                             uint64_t workspace_bytes, uint32_t* status, idx_stream_t stream);

/* Workspace of idx_attn_paged_fp4_async for these sizes on `device` (no counterpart on the
 * pages); it does not depend on the context. */
int idx_attn_paged_fp4_scratch_bytes(int32_t rows, int32_t q_heads, int32_t kv_heads,
                                     int32_t head_dim, int32_t num_req, int32_t max_pages,
                                     int32_t device, uint64_t* bytes);

/* The same over each row's list of slots (no counterpart on the pages). */
int idx_attn_selected_fp4(const idx_tensor_t* q, const idx_tensor_t* k_codes,
                          const idx_tensor_t* k_scale, const idx_tensor_t* v_codes,
                          const idx_tensor_t* v_scale, const idx_tensor_t* slots, float scale,
                          const idx_tensor_t* out, const idx_tensor_t* out_lse,
                          idx_stream_t stream);

/* Stream-ordered idx_attn_selected_fp4 (no counterpart on the pages). */
int idx_attn_selected_fp4_async(const idx_tensor_t* q, const idx_tensor_t* k_codes,
                                const idx_tensor_t* k_scale, const idx_tensor_t* v_codes,
                                const idx_tensor_t* v_scale, const idx_tensor_t* slots,
                                float scale, const idx_tensor_t* out,
                                const idx_tensor_t* out_lse, void* workspace,
                                uint64_t workspace_bytes, uint32_t* status, idx_stream_t stream);

/* Workspace of idx_attn_selected_fp4_async for these sizes on `device` (no counterpart on the
 * pages). */
int idx_attn_selected_fp4_scratch_bytes(int32_t rows, int32_t q_heads, int32_t kv_heads,
                                        int32_t head_dim, int32_t selected, int32_t device,
                                        uint64_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* IDXTOPK_H_ */
