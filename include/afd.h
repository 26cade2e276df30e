/*
 * afd.h -- MoE token dispatch and combine between Attention sources and FFN
 * expert workers, on one GPU (C ABI of libafd.so).
 *
 * The calls follow the afdEP-comm "API contract" page (sections "Roles and
 * tensors" and "Graphs, streams and lifetime"): source_dispatch,
 * worker_receive, worker_reply, source_collect. On one GPU the A sources and
 * F workers are logical partitions of the same HBM: nothing crosses a device
 * or process boundary, and a call's "rank" is an index argument.
 *
 * One exchange:
 *   1. afd_source_dispatch(s) for every source s (any order). The last one
 *      enqueues the layout and scatter kernels.
 *   2. afd_worker_receive(f) for every worker f: expert-major rows, their
 *      weights, the device prefix sums ends[] and an opaque receipt.
 *   3. the caller's expert computes BF16 replies, then afd_worker_reply(f)
 *      with the receipt, for every worker.
 *   4. afd_source_collect(s) for every source: BF16 [T,H] summed over the
 *      selected experts, in original token order.
 * A context holds at most one exchange in flight; the next dispatch waits
 * (host-side check) until every source has collected the previous one.
 *
 * Conventions for every call:
 *   - Device pointers are addresses on the context's device; host pointers
 *     are noted as such. Every array is dense row-major unless a stride says
 *     otherwise.
 *   - Wherever a buffer argument below says "device", the call also takes
 *     managed memory and page-locked host memory (cudaHostAlloc /
 *     cudaHostRegister; the kernels then read or write it over the host link
 *     through its mapped device address, with no copy). Pageable host memory,
 *     memory of another device and pointers CUDA does not know are refused
 *     with AFD_ERR_ARG before anything is enqueued.
 *   - `stream` is a cudaStream_t of the context's device (NULL = the legacy
 *     default stream). Work is enqueued, never waited for, unless a call says
 *     it synchronizes. When a call uses a different stream from the previous
 *     call on the context, it first makes its stream wait for the previous
 *     call's work (an event), so roles may run on separate streams. No such
 *     wait crosses a stream-capture boundary: around a capture the caller
 *     orders the work (e.g. synchronizes before capturing).
 *   - Host-detected errors return at once and enqueue nothing.
 *   - The caller owns every pointer it passes; each must stay valid and
 *     unchanged until the GPU work that reads or writes it has completed.
 *   - The context owns the receive arenas, the receipts, the single-worker
 *     view inboxes and the pinned host counts; pointers it returns stay
 *     valid until afd_destroy, and their contents until the exchange's rules
 *     below say.
 *   - All calls are host-thread-unsafe on one context: serialize them.
 */
#ifndef AFD_H
#define AFD_H

#include <stdint.h>

#if defined(__GNUC__)
#define AFD_API __attribute__((visibility("default")))
#else
#define AFD_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st;
typedef struct CUstream_st* afd_stream; /* a cudaStream_t */

typedef struct afd_ctx afd_ctx; /* opaque, owned by the library */

typedef enum afd_status {
  AFD_OK = 0,
  AFD_ERR_ARG = 1,          /* null pointer, size, shape or stride outside the contract */
  AFD_ERR_STATE = 2,        /* call out of exchange order, or repeated */
  AFD_ERR_BUCKET = 3,       /* T > bucket, bucket > capacity, or roles disagree on
                               bucket / read_host_counts within one exchange */
  AFD_ERR_RECEIPT = 4,      /* reply receipt, worker or row count differs from the receive */
  AFD_ERR_ROUTE_RANGE = 5,  /* device-detected top-k ID outside [-1, num_experts) */
  AFD_ERR_ROUTE_DUP = 6,    /* device-detected repeated ID within one token */
  AFD_ERR_CUDA = 7,         /* a CUDA runtime call failed (see afd_error_detail) */
  AFD_ERR_OOM = 8,          /* device or pinned allocation failed at create */
  AFD_ERR_CAPTURING = 9,    /* a host-synchronizing request on a capturing stream */
  AFD_ERR_UNSUPPORTED = 10, /* configuration outside what this build implements */
  AFD_ERR_TIMEOUT = 11      /* a bounded device-side wait gave up (reported like a route
                               error, through afd_get_error; the outputs are unspecified) */
} afd_status;

enum { AFD_BF16 = 0, AFD_FP8_E4M3 = 1, AFD_FP32 = 2 /* router logits only */ };

/* How the combine sums a token's reply rows (afd_config.combine_mode).
 * FUSED: one FP32 fused multiply-add chain over the routes in ascending k,
 *   one rounding to BF16.
 * TWO_STAGE: the pages' two-stage reduction (afdEP-comm design page,
 *   sections 6 and 19): each worker's routes give a BF16 partial (FMA chain
 *   in ascending k, one rounding); the partials are added in FP32 in the
 *   order of each worker's last route and rounded once. Equal to FUSED when
 *   F == 1.
 * TWO_STAGE_FP8: as TWO_STAGE, with each partial carried as E4M3 values and
 *   a shared power-of-two factor 2^e for every block of 128 of them (e the
 *   smallest integer >= -117 with amax <= 448 * 2^e): the lossy reply format
 *   of section 19. Each decoded value q * 2^e is rounded to FP32 before it is
 *   added, so a block whose amax is 248 * 2^120 or more decodes to infinity.
 * The two-stage modes need top_k <= 8. */
enum { AFD_COMBINE_FUSED = 0, AFD_COMBINE_TWO_STAGE = 1, AFD_COMBINE_TWO_STAGE_FP8 = 2 };

/* Fixed per context. "API contract", Roles and tensors: H divisible by 256,
 * top-k at most 32 and at most E, experts divide evenly over the workers (worker f owns
 * experts [f*E/F, (f+1)*E/F)). Limits of this build: A <= 64, F <= 64,
 * E <= 1024, and a worker arena below 2^24 rows. */
typedef struct afd_config {
  int32_t num_sources;      /* A >= 1 Attention sources */
  int32_t num_workers;      /* F >= 1 FFN workers */
  int32_t num_experts;      /* E, a multiple of F */
  int32_t top_k;            /* K, 1 <= K <= min(32, E) */
  int32_t hidden;           /* H, a multiple of 256 */
  int32_t capacity;         /* max tokens per source in one exchange (sizes the arenas) */
  int32_t expert_alignment; /* alpha >= 1: each expert's first row is a multiple of alpha */
  int32_t dtype;            /* AFD_BF16, or AFD_FP8_E4M3 (E4M3 rows + FP32 block-128 scales) */
  int32_t num_sms;          /* cap on the SMs the kernels spread over; 0 = every SM */
  int32_t combine_mode;     /* AFD_COMBINE_FUSED (0), _TWO_STAGE or _TWO_STAGE_FP8 */
} afd_config;

/* Creates a context on `device` and allocates its device arenas:
 *   rows      F x R_arena x row_bytes   (row_bytes = 2H for BF16, H for FP8)
 *   scales    F x R_arena x H/128 FP32  (FP8 only)
 *   inboxes   A x capacity x H BF16     (F == 1 only; see afd_source_collect)
 * with R_arena = align_up(A*capacity*min(K, E/F) + (E/F)*(alpha-1), alpha).
 * Returns AFD_ERR_ARG / AFD_ERR_UNSUPPORTED for a bad config, AFD_ERR_OOM if
 * an allocation fails (nothing is leaked), AFD_ERR_CUDA for a bad device.
 * "API contract": Buffer(group, config). */
AFD_API afd_status afd_create(const afd_config* config, int32_t device, afd_ctx** out);

/* Waits for the context's outstanding work, frees everything it owns.
 * NULL is accepted. Counterpart of Buffer.close() in the "API contract"
 * (Graphs, streams and lifetime). CUDA graphs that captured calls on this
 * context must be destroyed before it. */
AFD_API afd_status afd_destroy(afd_ctx* ctx);

/* Stages source `source` for the current exchange. "API contract", Roles and
 * tensors: source_dispatch(x, ids, weights, x_scale=None, *, bucket,
 * read_host_counts=False).
 *   x          device, [num_tokens, H]: BF16, or E4M3 bytes for AFD_FP8_E4M3
 *   ids        device int64 [num_tokens, K]; each ID in [0, E) or -1 (skip),
 *              unique within a token
 *   weights    device FP32 [num_tokens, K]; weight of the matching ID
 *   x_scale    device FP32 scales (FP8 only, else NULL): the scale of token t,
 *              128-column block b is x_scale[t*scale_stride_t +
 *              b*scale_stride_b] (strided views, e.g. a transposed [H/128, T]
 *              tensor, are allowed); strides are in elements
 *   num_tokens T, 0 <= T <= bucket (T = 0 sources are valid and contribute
 *              nothing; x/ids/weights may then be NULL)
 *   bucket     bucket <= capacity; every call of one exchange passes the same
 *   read_host_counts  0 or 1; every call of one exchange passes the same
 * When every source has staged, this call enqueues the exchange's layout and
 * scatter kernels on `stream`. Route checks run on the GPU: an invalid ID
 * makes the exchange's outputs unspecified and sets the context's sticky
 * route error (afd_get_error); it never traps the device.
 * Errors: AFD_ERR_STATE (source already staged, or the previous exchange is
 * not collected), AFD_ERR_BUCKET, AFD_ERR_ARG, AFD_ERR_CAPTURING
 * (read_host_counts on a capturing stream), AFD_ERR_CUDA. */
AFD_API afd_status afd_source_dispatch(afd_ctx* ctx, int32_t source, const void* x, const int64_t* ids,
                               const float* weights, const float* x_scale,
                               int64_t scale_stride_t, int64_t scale_stride_b,
                               int32_t num_tokens, int32_t bucket, int32_t read_host_counts,
                               afd_stream stream);

/* Dispatch that reuses the routing of the last exchange (its IDs, layout and
 * receipts) and moves only the rows: the decode-time routing reuse of
 * "DeepEP V2 ElasticBuffer first principles", section 4 (cached dispatch
 * skips the layout and any host synchronization). Every source of the
 * exchange must use this call (no mixing with afd_source_dispatch), with the
 * same num_tokens and bucket as in the last exchange whose dispatch ran the
 * layout; ends[], host counts, row_src and the receipts stay as they were.
 *   x, x_scale, strides, read_host_counts: as in afd_source_dispatch
 *   weights    device FP32 [num_tokens, K] new routing weights for the same
 *              IDs, or NULL to keep the previous exchange's weights
 * Errors: AFD_ERR_STATE (no layout to reuse, a different num_tokens/bucket,
 * or an exchange that mixes the two dispatch calls), plus those of
 * afd_source_dispatch. */
AFD_API afd_status afd_source_dispatch_cached(afd_ctx* ctx, int32_t source, const void* x,
                                              const float* weights, const float* x_scale,
                                              int64_t scale_stride_t, int64_t scale_stride_b,
                                              int32_t num_tokens, int32_t bucket,
                                              int32_t read_host_counts, afd_stream stream);

/* What a worker receives. Rows of local expert l (0 <= l < E/F) are
 * [align_up(ends[l-1], alpha), ends[l]) with ends[-1] = 0 ("API contract",
 * Roles and tensors). Inside an expert, rows follow source ascending, then
 * token ascending. Padding rows below align_up(ends[E/F-1], alpha) have
 * row_src -1 and weight +0; rows from there up to num_rows are unspecified,
 * and so are the bytes of every padding row. A consumer must treat only the
 * rows inside some [start, ends[l]) range as tokens. */
typedef struct afd_recv {
  void* rows;                 /* device [num_rows, H] BF16 or E4M3 bytes (context-owned) */
  float* row_scales;          /* device FP32 [num_rows, H/128] (FP8), else NULL */
  const float* weights;       /* device FP32 [num_rows]: routing weight of each row */
  const int32_t* row_src;     /* device int32 [num_rows]: (s*bucket + t)*K + k, or -1 */
  const int32_t* ends;        /* device int32 [E/F] receive prefix sums */
  const int32_t* host_counts; /* pinned host int32 [E/F] aligned counts
                                 align_up(count[l], alpha), or NULL */
  int64_t num_rows;           /* receive shape to hand back to afd_worker_reply */
  uint64_t receipt;           /* opaque; pass unchanged to afd_worker_reply */
} afd_recv;

/* Returns worker `worker`'s part of the current exchange. Launches no kernel.
 * read_host_counts = 0: num_rows is the conservative capacity
 * align_up(A*bucket*min(K, E/F) + (E/F)*(alpha-1), alpha) and the device
 * ends[] identify live rows; host_counts is NULL. read_host_counts = 1:
 * synchronizes `stream`, copies the aligned counts to pinned host memory and
 * sets num_rows to their sum (the exact receive shape); it then reports a
 * pending route error as AFD_ERR_ROUTE_*. This is the host-synchronizing
 * mode of the "API contract" (Graphs, streams and lifetime), meant for eager
 * callers that size their expert buffers exactly. Rows stay valid until the
 * next exchange's last afd_source_dispatch is enqueued.
 * Errors: AFD_ERR_STATE (no dispatched exchange, or worker already received),
 * AFD_ERR_BUCKET, AFD_ERR_CAPTURING, AFD_ERR_ARG, AFD_ERR_CUDA. */
AFD_API afd_status afd_worker_receive(afd_ctx* ctx, int32_t worker, int32_t bucket,
                              int32_t read_host_counts, afd_stream stream, afd_recv* out);

/* Hands worker `worker`'s BF16 replies back ("API contract": worker_reply).
 * The reply covers the whole receive shape, row for row; only rows that hold
 * a route are read.
 *   rows      device BF16 [num_rows, H], unweighted expert outputs; row r
 *             answers received row r. Padding rows are never read. It may be
 *             the received rows themselves (an identity expert, BF16 only).
 *             The library reads it until the combine of the exchange's last
 *             collected source has completed; it must stay unchanged until
 *             then.
 *   num_rows  must equal the afd_recv.num_rows of this worker's receive
 *   receipt   must equal the afd_recv.receipt of this worker's receive
 * The library applies each routing weight exactly once, in the combine,
 * which runs in afd_source_collect (one launch per source) or
 * afd_source_collect_all (one launch for all sources), for every F. This call
 * launches no kernel.
 * Errors: AFD_ERR_STATE, AFD_ERR_RECEIPT, AFD_ERR_ARG, AFD_ERR_CUDA. */
AFD_API afd_status afd_worker_reply(afd_ctx* ctx, int32_t worker, const void* rows, int64_t num_rows,
                            uint64_t receipt, afd_stream stream);

/* A view handed out by afd_source_collect. */
typedef struct afd_view {
  const void* data;   /* device BF16 [num_tokens, H] with row stride `row_stride` */
  int64_t row_stride; /* in elements */
  int32_t num_tokens;
  int32_t is_view;    /* 1: `data` is the context's inbox; 0: the result is in `out` */
} afd_view;

/* Source `source`'s result: out[t][h] = bf16(sum over k ascending of
 * w[t][k] * reply(k)[h]) accumulated with FP32 fused multiply-adds from +0
 * and rounded once to nearest-even; skipped (-1) routes add nothing; a token
 * with no valid route gives +0. Rows come back in the source's own token
 * order. Counterpart of source_collect(*, view=False) in the "API contract".
 *   out   device BF16 [T, H] (contiguous), T = the source's num_tokens; may be
 *         NULL only when view = 1 and F == 1
 *   view  1 asks for the single-worker view: with F == 1 the combine writes
 *         the context's inbox instead of `out`, and `view_out` points at it,
 *         read-only and valid until the next afd_source_dispatch on this
 *         context ("13. Single-FFN collect view" of the design page). With
 *         F > 1 the ordinary result is written to `out` and
 *         view_out->is_view = 0.
 *   view_out  host; filled on success (may be NULL when view = 0)
 * When the previous call on this context was a collect of the same exchange
 * that launched a combine on the same stream, and no other call of this
 * library has enqueued kernels there since, this call's combine starts
 * without waiting for that one (both only read the replies) and completes
 * after it, so stream order still holds for whatever follows. Work that the
 * caller enqueues on the stream between the two calls must therefore not
 * write the reply rows or this source's `out`, and work that lets its
 * dependents start before it has finished (a programmatic trigger in a kernel
 * of the caller's own) must not read this source's `out` either. Calls of
 * this library in between may read and write either: the combine then waits
 * for them (a graph replayed in between has ended before the combine starts),
 * as it does where its `out` shares memory with that of a source
 * collected before it.
 * Errors: AFD_ERR_STATE (replies missing, or source already collected),
 * AFD_ERR_ARG, AFD_ERR_CUDA. */
AFD_API afd_status afd_source_collect(afd_ctx* ctx, int32_t source, void* out, int32_t view,
                              afd_stream stream, afd_view* view_out);

/* Every source's result at once: for each source s the same as
 * afd_source_collect(s, outs[s], view, ...), with one combine launch for all
 * sources (on one GPU the sources' combines are independent, so they can
 * share a launch). Every source must still be uncollected.
 *   outs   host array of A device pointers, BF16 [T_s, H] each; an entry may
 *          be NULL for a source with T = 0, or when view = 1 and F == 1
 *   view   as in afd_source_collect
 *   views  host array of A afd_view, filled on success; may be NULL
 * Errors: as afd_source_collect (nothing is enqueued on an error). */
AFD_API afd_status afd_source_collect_all(afd_ctx* ctx, void* const* outs, int32_t view,
                                          afd_stream stream, afd_view* views);

/* The sticky error found on the GPU. Synchronizes the context's device work
 * first. code = AFD_OK, AFD_ERR_ROUTE_RANGE or AFD_ERR_ROUTE_DUP (for these,
 * (source, token, k) is the invalid route that comes first in (source,
 * token, k) order among all exchanges since the last afd_clear_error), or
 * AFD_ERR_TIMEOUT (a bounded wait of the scatter's bulk copies gave up at
 * (source, token); k = 0; see afd_set_wait_limit). Any pointer may be NULL.
 * Not allowed while the context's last stream is capturing
 * (AFD_ERR_CAPTURING). */
AFD_API afd_status afd_get_error(afd_ctx* ctx, int32_t* code, int32_t* source, int32_t* token,
                         int32_t* k);

/* Sets how many times the scatter polls for each source row's bulk load
 * before it gives up (default 4,194,304, each poll possibly suspending the
 * thread for a while). A load that does not complete in time is reported
 * through afd_get_error as AFD_ERR_TIMEOUT at that row's (source, token); the
 * warp that gave up waits for the load still in flight (up to 2 s of GPU
 * time), moves no more rows but still writes every receipt, so the rest of
 * the exchange runs and its outputs are unspecified. 0 makes every first
 * wait give up at once: a way to exercise that error path. Applies to
 * dispatches enqueued after the call (a captured graph keeps the value it
 * was captured with).
 * Errors: AFD_ERR_ARG (polls < 0). */
AFD_API afd_status afd_set_wait_limit(afd_ctx* ctx, int32_t polls);

/* For benchmarks that start every step with a cold L2: writes the first half
 * of `scratch` and then reads the second half, 16 bytes at a time, both with
 * an L2 evict-last policy (the one the scatter's row stores use, which
 * ordinary writes and reads cannot evict). Afterwards L2 holds only clean
 * lines of the second half: every earlier line, whatever its priority, has
 * been evicted and, if dirty, written back. Enqueued on `stream`.
 *   scratch  device memory of `bytes` bytes, 16-byte aligned; its contents
 *            are overwritten
 *   bytes    a multiple of 32, at least twice the L2 size for a full flush
 * Errors: AFD_ERR_ARG (alignment or size), AFD_ERR_CUDA. */
AFD_API afd_status afd_l2_flush(void* scratch, int64_t bytes, afd_stream stream);

/* Diagnostic: the phase stamps of a library built with -DAFD_PHASE_TIMERS=1
 * (%globaltimer, ns). Synchronizes the device, then copies the stamps to
 * `host` as uint64 [4][4096][8]: [kind][block][point], 0 where nothing was
 * recorded; clear = 1 also zeroes them. Kinds: 0 the exchange's first
 * dispatch kernel (points 0 start, 1 dependency wait passed, 2 first IDs
 * marked, 3 counted, 4 cluster barrier passed, 5 counts of all CTAs read,
 * 6 scan done, 7 route codes written; the one-kernel dispatches record 0, 1
 * and 7), 1 the scatter (0 start, 1 wait passed, 2 first row in shared
 * memory, 3 all stores issued, 4 stores complete, 5 end), 2 a combine that
 * waits first and 3 an early-started combine (0 start, 1 wait passed or
 * ready to load, 2 sums stored, 3 end). The stamps are global to the process;
 * the last launch of a kind overwrites the earlier ones; blocks past 4096
 * are not recorded.
 *   host   host uint64 array of `count` >= 131072 elements
 * Errors: AFD_ERR_UNSUPPORTED when built without phase timers (whatever the
 * arguments), AFD_ERR_ARG, AFD_ERR_CUDA. */
AFD_API afd_status afd_phase_stamps(afd_ctx* ctx, uint64_t* host, int64_t count, int32_t clear);

/* Clears the sticky route error (enqueued on `stream`). */
AFD_API afd_status afd_clear_error(afd_ctx* ctx, afd_stream stream);

/* Abandons the current exchange (host state only; enqueued GPU work still
 * runs). Lets a caller recover after a failed call mid-exchange. */
AFD_API afd_status afd_reset_exchange(afd_ctx* ctx);

/* Static text for a status. */
AFD_API const char* afd_status_string(afd_status status);

/* Text of the last failure on this context (host check or CUDA error). */
AFD_API const char* afd_error_detail(const afd_ctx* ctx);

/* Receive arena rows per worker (R_arena above), for sizing reply buffers. */
AFD_API int64_t afd_arena_rows(const afd_ctx* ctx);

/* Receive shape for `bucket` with read_host_counts = 0. */
AFD_API int64_t afd_recv_rows_for_bucket(const afd_ctx* ctx, int32_t bucket);

/* Routing layout without allocation (no counterpart in the pages). Some
 * callers cannot call cudaMalloc: code that runs inside another framework's
 * memory pool or allocator hook, or a process whose device memory is fully
 * reserved up front. This call allocates nothing, through the CUDA runtime or
 * any library: its scratch (384 KiB) is a fixed device array inside
 * libafd, which every GPU that loads the library holds until the process
 * exits. It computes, for one source's routing, what the dispatch layout
 * computes: route checks, per-worker ends[] with expert_alignment padding,
 * and the row of every valid route (expert-major; inside an expert, token
 * order), without moving any payload.
 *   ids        device int64 [num_tokens, top_k]; IDs in [0, num_experts) or -1
 *   ends       device int32 [num_experts] out: per worker f, ends[f*E/F + l]
 *              is local expert l's end (same convention as afd_recv.ends)
 *   slots      device int32 [num_tokens, top_k] out: the route's row inside
 *              its worker (worker = ID / (E/F)), or -1 (skipped or invalid)
 *   error      device int32 [3] out: {code, token, k} of the first invalid
 *              route in (token, k) order (code AFD_ERR_ROUTE_RANGE or
 *              AFD_ERR_ROUTE_DUP), or {AFD_OK, -1, -1}
 * Limits: num_tokens <= 8192, top_k <= 32, num_tokens * top_k <= 65536,
 * num_experts <= 1024, and align_up(num_tokens * top_k + (E/F) *
 * (expert_alignment - 1), expert_alignment) <= INT32_MAX (the largest row
 * index of a worker must fit an int32); larger sizes return
 * AFD_ERR_UNSUPPORTED and enqueue nothing. Every buffer must be reachable from the current device (its
 * device memory, managed memory, or page-locked host memory); pageable host
 * memory or another device's memory returns AFD_ERR_ARG and enqueues
 * nothing. Work is enqueued on `stream` (the current device's).
 * The first call on a device looks up the scratch array's device address
 * (and sets a kernel attribute); make that first call before any stream
 * capture on that device. All calls on a device share the one scratch array:
 * calls whose GPU work overlaps (different streams without ordering) race and
 * give wrong results; order them. */
AFD_API afd_status afd_route_layout_noalloc(const int64_t* ids, int32_t num_tokens, int32_t top_k,
                                            int32_t num_experts, int32_t num_workers,
                                            int32_t expert_alignment, int32_t* ends,
                                            int32_t* slots, int32_t* error, afd_stream stream);

/* The experts' side of an exchange: the router that makes a dispatch's IDs
 * and weights, and the products a worker computes between worker_receive and
 * worker_reply. These calls take no context and keep no state (but for
 * afd_set_product_wait_limit's limit): they allocate
 * nothing, never synchronize, and may run at the same time on any streams, in
 * any number of captured graphs, as long as their buffers do not overlap.
 * Work is enqueued on `stream`, a stream of the current device, on which
 * every buffer must be reachable (a buffer of another device returns
 * AFD_ERR_ARG and enqueues nothing). They take at most 2^31 - 2^20 - 1 rows
 * or tokens (less expert_alignment where there is one) and 2^24 features. */

/* How afd_route_topk scores an expert. */
enum { AFD_SCORE_SOFTMAX = 0, AFD_SCORE_SIGMOID = 1 };

/* Router: the top_k experts of every token, in the form afd_source_dispatch
 * takes (no counterpart in the pages, which start from given IDs).
 *   score_e = softmax(logits)_e over all experts, or sigmoid(logits_e)
 *   key_e   = score_e + bias_e (bias given), else logits_e
 * The experts with the largest keys are selected, in descending order, a tie
 * going to the lowest index; bias moves the selection only. Keys are compared
 * as if in 64 bits. Then
 *   weight = scale * score                          (renormalize = 0)
 *   weight = scale * score / sum of selected scores (renormalize = 1; the
 *            scores' common factor cancels before it can underflow)
 * An expert whose logit (or bias) is NaN or -infinity is never selected and
 * adds nothing to the softmax; +infinity counts as the largest finite value.
 * A slot for which no expert is left gets ID -1 and weight 0, which a
 * dispatch skips.
 *   logits       device [num_tokens, num_experts], BF16 or FP32 (logits_dtype),
 *                row t at logits + t * row_stride elements
 *   bias         device FP32 [num_experts], or NULL
 *   live_tokens  device int32 [1], or NULL: tokens t >= *live_tokens (a
 *                bucket's padding) get IDs -1 and weights 0; their logits are
 *                not read
 *   ids, weights device int64 / FP32 [num_tokens, top_k] out
 * Limits: top_k <= min(32, num_experts), num_experts <= 1024.
 * Buffers may be device, managed or page-locked host memory.
 * Errors: AFD_ERR_ARG, AFD_ERR_UNSUPPORTED (num_experts, num_tokens),
 * AFD_ERR_CUDA. */
AFD_API afd_status afd_route_topk(const void* logits, int32_t logits_dtype, int64_t row_stride,
                                  const float* bias, const int32_t* live_tokens, int32_t num_tokens,
                                  int32_t num_experts, int32_t top_k, int32_t scoring,
                                  int32_t renormalize, float scale, int64_t* ids, float* weights,
                                  afd_stream stream);

/* The experts' matrix product over received rows: for every row r of expert l
 * (rows [align_up(ends[l-1], expert_alignment), ends[l]), as afd_recv gives
 * them)
 *   y[r][n] = sum over k of x[r][k] * weight[l][n][k]
 *   out[r]  = y[r]                              (gated = 0)
 *   out[r][n] = silu(y[r][n]) * y[r][N + n]     (gated = 1, N = out_features;
 *               weight then has 2N rows per expert, the gate's first)
 * with FP32 sums and one rounding to BF16. FP8: x and weight are E4M3 with
 * FP32 scales for blocks of 128, and the sum is that of (x_scale[r][k/128] *
 * weight_scale[l][n/128][k/128]) * (the block's sum of x * weight). The two
 * scales' product is rounded to FP32 first, so it has to lie in that type's
 * normal range (2^-126 to 2^128) or be zero: below it a block's part loses
 * digits or is lost, above it the part is infinite, or NaN where the block's
 * sum is zero. The scales by themselves may be any FP32 numbers.
 * Rows of `out` outside every expert's range are left as they were; rows of
 * `x` there are never used for a result, whatever they hold. Ends beyond
 * num_rows are taken as num_rows.
 *   x             device [num_rows, in_features] BF16 or E4M3 (dtype), row r at
 *                 x + r * x_stride elements
 *   x_scale       device FP32 [num_rows, in_features/128] (FP8), else NULL
 *   weight        device [num_groups, N or 2N, in_features], contiguous
 *   weight_scale  device FP32 [num_groups, (N or 2N)/128, in_features/128]
 *                 (FP8), else NULL
 *   ends          device int32 [num_groups], non-decreasing
 *   out           device BF16 [num_rows, out_features], row r at out + r *
 *                 out_stride elements; must not overlap the inputs
 *   error         device int32 [1], or NULL: set to AFD_ERR_TIMEOUT if a
 *                 bounded wait of the kernel gave up (the rows of `out` are
 *                 then unspecified), else left as it was. Without it nothing
 *                 tells of a wait that gave up.
 * Buffers are device memory of the current device (the rows and weights move
 * by bulk copies). x, weight, x_stride and the rows of weight are multiples
 * of 16 bytes; FP8 takes in_features and out_features that are multiples of
 * 128. num_groups <= 1024, and at most 2^30 tiles of 256 weight rows by 256
 * rows.
 * Errors: AFD_ERR_ARG, AFD_ERR_UNSUPPORTED (sizes or alignments above),
 * AFD_ERR_CUDA. */
AFD_API afd_status afd_grouped_linear(const void* x, int64_t x_stride, const float* x_scale,
                                      const void* weight, const float* weight_scale,
                                      const int32_t* ends, int32_t num_groups,
                                      int32_t expert_alignment, int64_t num_rows,
                                      int32_t in_features, int32_t out_features, int32_t dtype,
                                      int32_t gated, void* out, int64_t out_stride, int32_t* error,
                                      afd_stream stream);

/* Sets the most clocks of an SM for which a wait inside afd_grouped_linear's
 * kernel lasts before the kernel gives up (default 4,000,000,000, about two
 * seconds; see `error` there). It holds for the process's calls from then on;
 * what was captured before keeps its own. 0: the kernel gives up at once,
 * without a wait or a product: a way to exercise that path.
 * Errors: AFD_ERR_ARG (negative). */
AFD_API afd_status afd_set_product_wait_limit(int64_t cycles);

/* The gated activation over received rows, for products whose activation
 * cannot be part of them (afd_adapter_add between the two): for every row r
 * of an expert's range (as in afd_grouped_linear)
 *   out[r][n] = silu(h[r][n]) * h[r][features + n]
 * computed in FP32 and rounded once. Other rows are left as they were.
 *   h    device BF16 [num_rows, 2 * features], row r at h + r * h_stride
 *   out  device BF16 [num_rows, features], row r at out + r * out_stride; may
 *        be the first half of h itself
 * Buffers may be device, managed or page-locked host memory.
 * Errors: AFD_ERR_ARG, AFD_ERR_UNSUPPORTED (num_groups > 1024, sizes),
 * AFD_ERR_CUDA. */
AFD_API afd_status afd_gated_rows(const void* h, int64_t h_stride, const int32_t* ends,
                                  int32_t num_groups, int32_t expert_alignment, int64_t num_rows,
                                  int32_t features, void* out, int64_t out_stride,
                                  afd_stream stream);

/* Low-rank adapters of many requests beside a shared projection: row r of the
 * request whose adapter is a gets
 *   out[r] = base[r] + scales[a] * up[a] (down[a] x[r])
 * in FP32 with one rounding to BF16 (the low-rank product scales[a] down[a]
 * x[r] is kept to at least 16 bits of precision between the two, or to
 * 2^-134 where that is more).
 * The adapter of a row: a = token_slots[t], where t = row_src[r] / top_k for
 * received rows (row_src as afd_recv gives it), or t = r without row_src. A
 * slot outside [0, num_slots) means no adapter: out[r] = base[r].
 * With row_src, rows r >= ends[num_groups-1] and rows whose row_src is
 * negative or names a token outside [0, num_tokens) are left as they were.
 *   base, out    device BF16 [num_rows, out_features], row strides
 *                base_stride / out_stride; out may be base (in place), and must
 *                not overlap the inputs in any other way
 *   x            device [num_rows, in_features], row stride x_stride elements:
 *                BF16, or E4M3 with x_scale
 *   x_scale      device FP32 [num_rows, in_features/128], or NULL (BF16)
 *   down         device BF16 [num_slots, rank, in_features], contiguous
 *   up           device BF16 [num_slots, out_features, rank], contiguous
 *   token_slots  device int32 [num_tokens]
 *   scales       device FP32 [num_slots]
 *   row_src      device int32 [num_rows] with ends, or NULL (then num_tokens
 *                >= num_rows, and ends may be NULL)
 *   workspace    device, workspace_bytes >= afd_adapter_workspace_bytes(...)
 *                bytes, 16-byte aligned (NULL where that is 0); its contents
 *                need not be set and mean nothing afterwards. Calls that may
 *                run at the same time (other streams, other captured graphs)
 *                need one each.
 * Limits: num_slots <= 1023; rank 8, 16, 32 or 64; in_features a multiple of
 * 16 (E4M3: of 128); out_features a multiple of 8; base, out, x, down, up and
 * the strides multiples of 16 bytes. Buffers may be device, managed or page-locked host memory.
 * Errors: AFD_ERR_ARG, AFD_ERR_UNSUPPORTED (limits), AFD_ERR_CUDA. */
AFD_API afd_status afd_adapter_add(const void* base, int64_t base_stride, const void* x,
                                   int64_t x_stride, const float* x_scale, const void* down,
                                   const void* up, const int32_t* token_slots,
                                   const float* scales, const int32_t* row_src,
                                   const int32_t* ends, int32_t num_groups, int32_t top_k,
                                   int64_t num_rows, int32_t num_tokens,
                                   int32_t num_slots, int32_t rank, int32_t in_features,
                                   int32_t out_features, void* out, int64_t out_stride,
                                   void* workspace, int64_t workspace_bytes, afd_stream stream);

/* Bytes of workspace for afd_adapter_add with these sizes (-1 for negative
 * ones; 0 where few rows can be live). top_k: 0 for calls without row_src. */
AFD_API int64_t afd_adapter_workspace_bytes(int64_t num_rows, int32_t num_tokens, int32_t top_k,
                                            int32_t num_slots, int32_t rank, int32_t in_features,
                                            int32_t out_features);

/* The Attention source's side of an exchange: what a source runs around its
 * attention before it dispatches, and the attention of a decode step itself.
 * As the experts' side, these calls take no context, keep no state, allocate
 * nothing, never synchronize, may run at the same time on any streams and in any
 * number of captured graphs as long as what they write does not overlap, and work
 * on a stream of the current device, on which every buffer must be reachable.
 * They take at most 2^31 - 2^20 - 1 rows or tokens.
 * Where values go to E4M3, a vector of them shares one FP32 scale,
 *   scale = max(max |v| / 448, 2^-100), value = e4m3(v / scale),
 * the scale to a step of FP32, the FP32 quotients rounded to nearest even; all of
 * a vector with an infinity or a NaN decodes to NaN. */

/* The rows a source dispatches, from its residual stream:
 *   r = x + residual                     residual_out = bf16(r)
 *   y = r / sqrt(mean(r^2) + eps) * weight        out = bf16(y)
 *   and y in E4M3 with a scale for each block of 128 columns, in the form
 *   afd_source_dispatch takes (fp8_out, scale_out)
 * in FP32, from the unrounded r; the sum of squares has to be finite in FP32,
 * and with eps = 0 a normal number or 0 (a row of zeros is NaN then).
 *   x             device BF16 [num_rows, features], row stride x_stride elements
 *   residual      device BF16 [num_rows, features], row stride residual_stride,
 *                 or NULL (then residual_out is NULL too)
 *   weight        device BF16 [features]
 *   residual_out  device BF16, or NULL; may be residual or x itself (the same
 *                 address and stride)
 *   out           device BF16, or NULL; may be x or residual itself
 *   fp8_out       device E4M3 [num_rows, features], contiguous, or NULL
 *   scale_out     device FP32 [num_rows, features/128], contiguous; with fp8_out
 * One output at least. Outputs must not overlap the inputs or each other in any
 * other way. fp8_out takes features that are multiples of 128, up to 32,768, and
 * rows of every array, and the weight, on 16-byte boundaries (fp8_out: 8).
 * Features are at most 2^24. Buffers may be device, managed or page-locked host
 * memory.
 * Errors: AFD_ERR_ARG, AFD_ERR_UNSUPPORTED (limits), AFD_ERR_CUDA. */
AFD_API afd_status afd_norm_rows(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                                 const void* weight, float eps, int64_t num_rows, int32_t features,
                                 void* residual_out, int64_t residual_out_stride, void* out, int64_t out_stride,
                                 void* fp8_out, float* scale_out, afd_stream stream);

/* A paged cache of keys and values. Token j of a sequence lies in the
 * sequence's page j / page_size at j % page_size; a page holds each KV head's
 * tokens one after another. */
typedef struct afd_cache {
  void* k;               /* device [num_pages][num_kv_heads][page_size][head_dim], BF16 or E4M3 bytes */
  void* v;               /* the same of the values */
  float* k_scale;        /* device FP32 [num_pages][num_kv_heads][page_size] (E4M3), else NULL */
  float* v_scale;        /* not negative; zero, or 2^-100 to 2^80: where a scale is above that (infinite), its head's
                            attention may come out infinite or NaN, its lse stays that of the scores */
  int64_t k_page_stride; /* elements from a page to the next (the rest is dense): keys and values may */
  int64_t v_page_stride; /*   be two halves of one allocation's pages; multiples of 64 bytes */
  int32_t num_pages;     /* num_pages * page stride at most 256 GB each, num_pages * page_size below 2^31 */
  int32_t page_size;     /* tokens of a page, any number; multiples of 16 are read fastest */
  int32_t num_kv_heads;
  int32_t head_dim;      /* 64 or 128 */
  int32_t dtype;         /* AFD_BF16 or AFD_FP8_E4M3 */
} afd_cache;

/* New tokens' rotary positions and their way into a cache: for every token t
 *   q_out[t] = rotated q[t];  the cache's row slots[t] = rotated k[t], and v[t]
 * Pair i < rotary_pairs of a head's columns, (i, rotary_pairs + i), or (2i, 2i + 1)
 * with interleaved = 1, becomes
 *   (a cos - b sin, b cos + a sin) * factor, angle = positions[t] * inv_freq[i]
 * with the angle and its remainder in 64 bits (positions to 2^53); the head's other
 * columns stay. A change of the frequencies for long contexts is in inv_freq and
 * factor. BF16 caches hold the rotated values rounded, E4M3 ones a scale for
 * each token and head, of the FP32 values.
 *   q          device BF16 [num_tokens, num_q_heads, head_dim], row stride
 *              q_stride elements; not used with num_q_heads = 0
 *   k, v       device BF16 [num_tokens, num_kv_heads, head_dim], row strides
 *   positions, inv_freq  device int64 [num_tokens] and FP32 [rotary_pairs]; not
 *              used with rotary_pairs = 0
 *   slots      device int64 [num_tokens]: page * page_size + place in the page.
 *              A token whose slot is negative or beyond the cache (a bucket's
 *              padding) leaves the cache as it is; its q_out is written. Two
 *              tokens with the same slot leave parts of either there.
 *   q_out      device BF16 [num_tokens, num_q_heads, head_dim], row stride
 *              q_out_stride; may be q itself (the same address and stride)
 * Limits: at most 1,024 heads of either kind; q, k, v, q_out, the caches
 * and the rows' strides multiples of 16 bytes.
 * Buffers may be device, managed or page-locked host memory.
 * Errors: AFD_ERR_ARG, AFD_ERR_UNSUPPORTED (limits), AFD_ERR_CUDA. */
AFD_API afd_status afd_cache_write(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                   const void* v, int64_t v_stride, const int64_t* positions,
                                   const int64_t* slots, const float* inv_freq, int32_t rotary_pairs,
                                   int32_t interleaved, float factor, int64_t num_tokens, int32_t num_q_heads,
                                   const afd_cache* cache, void* q_out, int64_t q_out_stride, afd_stream stream);

/* Attention of one new token a sequence over its cache: for every sequence b and
 * query head h, with KV head h / (num_q_heads / num_kv_heads),
 *   s_j = scale * q[b][h] . k_j,  p = softmax(s) over the tokens j that are seen,
 *   out[b][h] = sum over j of p_j v_j,  lse[b][h] = log(sum over j of exp(s_j))
 * Seen are j < lengths[b], and j >= lengths[b] - window where window > 0; the new
 * token's own key and value are in the cache (afd_cache_write) and counted. A
 * page number outside [0, num_pages) hides its tokens, a length beyond the
 * table's pages ends there. A sequence that sees nothing (a bucket's padding:
 * length 0) gets out = +0 and lse = -infinity. What the cache holds in places
 * that are not seen is not read.
 * Sums, maxima and exponentials are FP32. The probabilities are rounded for the
 * product with the values: BF16 caches, to two BF16 parts (16 bits); E4M3, to FP16
 * (11 bits), weighted by the values' scales first, and a token of less than 2^-32 of
 * the largest such weight (up to 2^-25 with scales below 2^-93) may be left out there. With
 * E4M3 caches the queries' columns are rounded to 2^-24 of their head's largest.
 * Which tokens are summed together depends on all lengths of the call, so the last
 * bits of a sequence's result may change with what it is batched with; the same
 * call gives the same bits.
 * A column with an infinity among the values that are seen may come out as NaN
 * (its weight's second part may be zero or negative). A head with a score of
 * +infinity or NaN gets NaN for out and lse; one whose scores are all -infinity is
 * one that sees nothing.
 *   q           device BF16 [num_seqs, num_q_heads, head_dim], row stride q_stride
 *   page_table  device int32 [num_seqs, max_pages], row stride table_stride
 *   lengths     device int32 [num_seqs]
 *   out         device BF16 [num_seqs, num_q_heads, head_dim], row stride
 *               out_stride; must not overlap the inputs
 *   lse         device FP32 [num_seqs, num_q_heads] (natural logarithm), or NULL
 *   workspace   device, workspace_bytes >= afd_decode_workspace_bytes(...), 16-byte
 *               aligned (NULL where that is 0); its contents need not be set and
 *               mean nothing afterwards. Calls that may run at the same time
 *               (other streams, other captured graphs) need one each.
 * Limits: num_q_heads a multiple of num_kv_heads, at most 1,024; max_pages *
 * page_size below 2^31 - 2^10; num_seqs * num_kv_heads below 2^31 - 2^20, counted
 * once for each 16 query heads of a KV head, and that times max_pages * page_size
 * below 2^44; q, out and their strides multiples of 16 bytes.
 * Buffers may be device, managed or page-locked host memory.
 * Errors: AFD_ERR_ARG, AFD_ERR_UNSUPPORTED (limits), AFD_ERR_CUDA. */
AFD_API afd_status afd_decode_attention(const void* q, int64_t q_stride, const afd_cache* cache,
                                        const int32_t* page_table, int64_t table_stride, int32_t max_pages,
                                        const int32_t* lengths, int32_t num_seqs, int32_t num_q_heads, float scale,
                                        int32_t window, void* out, int64_t out_stride, float* lse,
                                        void* workspace, int64_t workspace_bytes, afd_stream stream);

/* Bytes of workspace for afd_decode_attention with these sizes (-1 for ones it
 * does not take; 0 where nothing is split). */
AFD_API int64_t afd_decode_workspace_bytes(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                           int32_t head_dim, int32_t max_pages, int32_t page_size);

/* Library version, (major << 16) | minor. */
AFD_API int32_t afd_version(void);

#ifdef __cplusplus
}
#endif
#endif /* AFD_H */
