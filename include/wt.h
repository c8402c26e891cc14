/*
 * wt.h -- C ABI of the MI355X parameter-preparation library (libwt.so).
 *
 * The library implements the "parameter preparation" stage of an RL
 * weight-transfer pipeline ("Weight transfer for RL post-training in under 2
 * seconds", Perplexity, 2025; section "Task pipeline"): after a training step
 * it takes FSDP dim-0 row shards of BF16 weights, rebuilds each full tensor
 * (the full_tensor() step), fuses projections (e.g. q/k/v -> qkv,
 * gate/up -> gate_up), quantizes to FP8 and writes the bytes into a
 * registered destination region at offsets fixed ahead of time by the
 * controller's static schedule (section "Static schedule": the schedule is
 * computed once, each iteration replays it). The region stands in for the
 * remote inference GPU's memory that a one-sided RDMA WRITE would fill
 * (section "RDMA WRITE: one-sided transfers"); the destination side gets no
 * notification.
 *
 * Numerics of an FP8 output (the page lists quantization as a step but fixes
 * no format or rounding; this is the reading the library implements): OCP
 * FP8 E4M3 ("e4m3fn", max 448,
 * no infinity) with one fp32 scale per 128x128 tile of the fused tensor,
 * s = amax / 448 (s = 1 for an all-zero tile), each element
 * cast(fl32(x / s)) with IEEE-rounded fp32 division and round-to-nearest-even
 * with saturation. FP8 bytes are row-major [R x C]; scales are row-major
 * fp32 over the ceil(R/128) x ceil(C/128) tile grid. A WT_BF16_COPY output is
 * the fused BF16 bytes, unchanged.
 *
 * Conventions: every entry point returns a wt_status (no C++ exception ever
 * crosses the ABI). All pointers are plain host or device addresses; sizes
 * are in bytes unless a field says rows/cols. "stream" arguments are
 * hipStream_t values passed as void* (NULL = the null stream). Separate plans
 * are independent and may be used from different threads.
 */
#ifndef WT_H
#define WT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum wt_status {
  WT_OK = 0,
  WT_E_INVAL = 1,     /* malformed task table or argument */
  WT_E_RANGE = 2,     /* a data or scale range falls outside [0, dst_bytes) */
  WT_E_OVERLAP = 3,   /* two destination ranges overlap */
  WT_E_ALIGN = 4,     /* misaligned shard pointer, BF16 dst_offset or scale_offset */
  WT_E_NOMEM = 5,     /* host or device allocation failed */
  WT_E_HIP = 6,       /* HIP runtime error; text from wt_plan_last_error() */
  WT_E_WATERMARK = 7, /* watermark below the staging need of one output */
  WT_E_STATE = 8,     /* wt_prepare already running on this plan */
  WT_E_TIMEOUT = 9    /* wt_progress_wait: the word did not reach its target in time */
} wt_status;

/* Output data type of a task (and of its fusion group). */
enum { WT_FP8_E4M3FN_B128 = 0, WT_BF16_COPY = 1 };

/* Where shards or the destination region live. */
enum { WT_MEM_DEVICE = 0, WT_MEM_PINNED_HOST = 1 };

/* How prepared bytes reach the destination region (emulated RDMA WRITE). */
enum {
  WT_DST_ZERO_COPY = 0, /* the kernels store straight into the region */
  WT_DST_STAGED = 1     /* kernels store into device staging; a copy stage moves them */
};

/* One FSDP shard: `rows` consecutive rows (row length = the task's cols,
 * BF16, row-major, rows contiguous). rows may be 0 (ptr is then ignored).
 * ptr must be 2-byte aligned. */
typedef struct wt_shard {
  const void *ptr;
  int64_t rows;
} wt_shard;

/* One task = one source parameter tensor ("Task pipeline": each parameter
 * tensor transfer is a task), given as its shards in rank order. Its full
 * tensor is the dim-0 concatenation of the shards.
 *
 * fusion_group: -1 = the task is an output of its own. Tasks that share an
 * id >= 0 form ONE output, their full tensors concatenated along dim 0 in
 * table order (projection fusion); they must share cols, dtype and
 * shard_mem, and the output's dst_offset / scale_offset are taken from the
 * group's first task (the others' offsets are ignored).
 *
 * dst_offset: byte offset of the output's data in the destination region
 * (FP8: R*C bytes; BF16 copy: 2*R*C bytes, offset must be even).
 * scale_offset: byte offset of the fp32 scale grid (FP8 only; multiple of 4).
 * A 1-D tensor of n elements is described as rows = n, cols = 1. */
typedef struct wt_task {
  const wt_shard *shards;
  int32_t n_shards;
  int32_t shard_mem; /* WT_MEM_DEVICE or WT_MEM_PINNED_HOST */
  int64_t cols;
  int32_t dtype; /* WT_FP8_E4M3FN_B128 or WT_BF16_COPY */
  int32_t fusion_group;
  uint64_t dst_offset;
  uint64_t scale_offset;
} wt_task;

/* Plan options; wt_plan_options_init() fills the defaults. */
typedef struct wt_plan_options {
  /* Upper bound on temporary device memory held by tasks in flight (the
   * watermark of the weight-transfer page's section "GPU memory usage
   * control", under which tasks are admitted). Used for staging of
   * pinned-host shards and, in WT_DST_STAGED mode, of outputs.
   * Default 512 MiB (a staged pipeline into pinned host memory with one
   * 176 MB output per layer measured 39 ms per replay under 256 MiB, 34 ms
   * under 512 MiB). */
  uint64_t watermark_bytes;
  /* Target bytes of one pipeline chunk (outputs moved through the stages
   * together, one kernel launch each). 0 (default): about 1/16 of the bytes
   * that go through the pipeline, at least 32 MiB, at most watermark / 2
   * (watermark / 3 when both shards and outputs are staged, so that each of
   * the three stages can hold a slot of the ring).
   * Smaller chunks let the first parts of the destination region complete
   * sooner (see the completion counters); many more than a few dozen chunks
   * per replay cost throughput. */
  uint64_t chunk_bytes;
  int32_t dst_write_mode; /* WT_DST_ZERO_COPY (default) or WT_DST_STAGED */
  int32_t device;         /* HIP device ordinal; -1 (default) = current device */
  /* Cache hint for reading full 128 x 128 tiles: WT_LOAD_AUTO (default; the
   * library's choice, currently non-temporal loads), WT_LOAD_PLAIN, or
   * WT_LOAD_STREAM (non-temporal loads). Affects speed only, never results;
   * values above WT_LOAD_STREAM are WT_E_INVAL. */
  uint32_t load_hint;
  /* Host-side backpressure of pipelined plans: wt_prepare first waits on the
   * host until at most max_replays_in_flight - 1 earlier replays of the plan
   * are unfinished. 0 (default): 1, i.e. a call returns once the previous
   * replay has finished and this one is enqueued. Values above 8 are
   * WT_E_INVAL. Affects speed and host blocking, never results. */
  uint32_t max_replays_in_flight;
  /* Grouping of full 128 x 128 tiles on the aligned path: WT_GROUP_AUTO
   * (default: adjacent full tiles of a row band two to a workgroup, except in
   * a launch of at most 768 full tiles, which fits in one round of
   * workgroups and is latency-bound: one tile each), WT_GROUP_SINGLE or
   * WT_GROUP_PAIR. Affects speed only, never results; values above
   * WT_GROUP_PAIR are WT_E_INVAL. */
  uint32_t tile_group;
  uint32_t reserved[3];
} wt_plan_options;

enum { WT_GROUP_AUTO = 0, WT_GROUP_SINGLE = 1, WT_GROUP_PAIR = 2 };

enum { WT_LOAD_AUTO = 0, WT_LOAD_PLAIN = 1, WT_LOAD_STREAM = 2 };

/* Shape of a plan, filled by wt_plan_check / wt_plan_get_info. */
typedef struct wt_plan_info {
  int64_t n_tasks;
  int64_t n_outputs;
  int64_t n_fp8_outputs;
  int64_t n_copy_outputs;
  int64_t n_tiles;            /* 128x128 tiles over all FP8 outputs */
  int64_t input_bytes;        /* BF16 bytes read */
  int64_t output_bytes;       /* FP8 + scale + BF16 bytes written */
  int64_t n_launches;         /* kernel launches per wt_prepare */
  int64_t n_chunks;           /* pipeline chunks (0 when no stage needs staging) */
  int64_t n_h2d_copies;       /* host-to-device copies per wt_prepare */
  int64_t n_dst_copies;       /* staging-to-destination copies per wt_prepare */
  int64_t staging_bytes;      /* device staging allocated (<= watermark) */
  int64_t n_units;            /* completion units: the device-resident launch (if any), then each chunk */
  int64_t n_regular_items;    /* work items of full tiles on the aligned path (a pair of tiles is one item) */
  int64_t n_edge_tiles;       /* aligned-path tiles that are partial or draw rows from several shards */
  int64_t n_general_tiles;    /* tiles of outputs with ragged columns or unaligned addresses */
} wt_plan_info;

/* One operation of the replayed schedule, as listed by wt_plan_schedule. */
typedef struct wt_sched_op {
  int32_t stage;        /* 0 = host-to-device copy, 1 = prepare launch, 2 = destination copy */
  int32_t chunk;        /* chunk index (-1: the launch over device-resident outputs) */
  int32_t wait_chunk;   /* stage 0: chunk whose release this op waits for (-1: none) */
  int32_t reserved;
  int64_t bytes;        /* bytes moved (stages 0, 2) or prepared input bytes (stage 1) */
  int64_t staging_offset; /* start of the chunk's staging slot in the ring */
  int64_t staging_bytes;  /* size of the chunk's staging slot */
} wt_sched_op;

typedef struct wt_plan wt_plan;

/* Fills `opts` with the defaults. */
void wt_plan_options_init(wt_plan_options *opts);

/* Validates a task table exactly as wt_plan_create does and describes the
 * plan it would build, without touching any GPU (host only). opts may be
 * NULL (defaults). info may be NULL. */
wt_status wt_plan_check(const wt_task *tasks, size_t n_tasks, size_t dst_bytes, int32_t dst_kind,
                        const wt_plan_options *opts, wt_plan_info *info);

/* Lists the operations one wt_prepare would enqueue, in enqueue order, for
 * the plan wt_plan_check would build (host only). Writes at most max_ops
 * records to ops (may be NULL) and the total count to *n_ops. */
wt_status wt_plan_schedule(const wt_task *tasks, size_t n_tasks, size_t dst_bytes, int32_t dst_kind,
                           const wt_plan_options *opts, wt_sched_op *ops, size_t max_ops, size_t *n_ops);

/* Builds a plan: the static schedule of "Weight transfer for RL post-training
 * in under 2 seconds", section "Static schedule" (the transfer schedule is
 * computed once at initialisation and every training step replays it). It
 * validates the table,
 * builds the device descriptor tables (outputs, row segments, tile and copy
 * work lists), allocates staging within the watermark and creates the
 * plan's streams and events. The table is copied; the caller may free it on
 * return. Shard memory and the destination region stay owned by the caller
 * and must outlive the plan; their ADDRESSES are fixed in the plan, their
 * CONTENTS may change between wt_prepare calls.
 * dst: destination region base (device pointer, or pinned host pointer when
 * dst_kind is WT_MEM_PINNED_HOST), dst_bytes long. On failure *out is NULL. */
wt_status wt_plan_create(const wt_task *tasks, size_t n_tasks, void *dst, size_t dst_bytes, int32_t dst_kind,
                         const wt_plan_options *opts, wt_plan **out);

/* For callers that cannot allocate memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc): builds the same plan
 * as wt_plan_create, with the same arguments, validation and results, but
 * calls no hipMalloc, hipHostMalloc or hipFree (host-side bookkeeping uses
 * the C++ heap). Its device descriptor tables go into a static array of
 * WT_NOALLOC_TABLE_BYTES bytes that the library holds on every GPU it runs
 * on until the process ends; they are copied there synchronously before
 * the call returns. Limits:
 *  - one such plan per device at a time: while one is live on the device,
 *    another call returns WT_E_STATE (destroy the first with
 *    wt_plan_destroy, which waits for its latest wt_prepare launch);
 *  - tables larger than WT_NOALLOC_TABLE_BYTES (16 MiB): WT_E_NOMEM. A pair
 *    of full 128 x 128 tiles takes 32 bytes of tables, so 16 MiB holds, for
 *    example, a dense 7B-shaped model (about 6.5 MB of tables);
 *  - pinned-host shards or WT_DST_STAGED (they need staging memory):
 *    WT_E_INVAL.
 * Replays, progress words and destruction work as for any plan. A plan
 * created here shares the device's array with every later one: a graph that
 * captured its replays must not be launched after it is destroyed, and work
 * of an earlier plan that still reads the array when a new plan is created
 * (graph launches are not tracked) races with it. */
#define WT_NOALLOC_TABLE_BYTES 16777216u
wt_status wt_plan_create_noalloc(const wt_task *tasks, size_t n_tasks, void *dst, size_t dst_bytes,
                                 int32_t dst_kind, const wt_plan_options *opts, wt_plan **out);

/* Replays the plan (same page, section "Static schedule": each iteration
 * replays the schedule; section "Task pipeline": per task, the stages
 * parameter preparation -> RDMA transfer, each with its own FIFO queue, a
 * task moving to the next queue once its stage is done). Enqueues the whole
 * preparation so that it is ordered
 * after prior work on `stream` and completes before later work on `stream`.
 * With device-resident shards and WT_DST_ZERO_COPY this is one kernel launch
 * on `stream`. Pinned-host shards or WT_DST_STAGED run the three-stage
 * pipeline (host-to-device copy, prepare, destination copy) on the plan's own
 * streams, one in-order queue per stage, and join `stream` at the end.
 * Returns without waiting for the GPU, except that a pipelined plan keeps at
 * most max_replays_in_flight replays enqueued and unfinished: by default a
 * call first waits on the host for the plan's previous replay (deeper queues
 * of copies make the runtime block single copy submissions in lockstep with
 * the GPU and starve the copy engine). No validation or allocation
 * happens here. A plan without a pipeline may be replayed inside stream
 * capture (its launches, completion-word kernels and event record become
 * graph nodes; each graph replay is a replay of the plan); a pipelined plan
 * may not, since its backpressure waits on the host (WT_E_STATE, nothing
 * enqueued). A graph holding captured replays reads the plan's device
 * tables every time it is launched: it must not be launched after
 * wt_plan_destroy, and its launches must have finished before that call.
 * Returns WT_E_STATE if another wt_prepare on the same plan is
 * running in another thread, WT_E_HIP on a runtime error. */
wt_status wt_prepare(wt_plan *plan, void *stream);

/* Copies the plan's shape into *info. */
wt_status wt_plan_get_info(const wt_plan *plan, wt_plan_info *info);

/* Ends a plan. The staging it frees is the temporary memory that the
 * watermark bounds ("Weight transfer for RL post-training in under 2
 * seconds", section "GPU memory usage control"). Waits for the plan's work
 * already enqueued (its own streams, and for a plan without a pipeline the
 * latest wt_prepare launch on the caller's stream), then frees everything
 * the plan owns (device tables, staging, streams, events). Launches of a
 * captured graph are not waited for: every graph holding replays of this
 * plan must have finished, and must not be launched again, before this
 * call. Never frees shards or the destination region. NULL is ignored. */
void wt_plan_destroy(wt_plan *plan);

/* Static text for a status code. */
const char *wt_status_str(int status);

/* Text of the last error recorded on `plan`, or, for plan == NULL, of the
 * last failed wt_plan_create / wt_plan_check on the calling thread. */
const char *wt_plan_last_error(const wt_plan *plan);

/* ---- Element-function checks (exhaustive verification of the kernels' arithmetic) ----
 * These run the same device code the prepare kernel runs per tile and per
 * element, over complete input domains, so that the result can be compared
 * with an independent implementation. */

/* out[i * 65536 + x] = E4M3 byte that the prepare kernel writes for the BF16
 * pattern x in a tile whose amax is the BF16 pattern amax_bits[i] (the sign
 * bit of amax_bits is ignored; scale and division chosen exactly as in the
 * prepare kernel). path = 0: the element function of the aligned (fast) tile
 * path; path = 1: that of the general (any shape, any alignment) tile path.
 * amax_bits and out are device pointers; out holds n_amax * 65536 bytes;
 * 0 <= n_amax <= 2^20 (WT_E_INVAL otherwise). */
wt_status wt_quantize_domain(const uint16_t *amax_bits, int64_t n_amax, int32_t path, uint8_t *out, void *stream);

/* out[i] = the kernel's fp32 -> E4M3 cast of the fp32 bit pattern first + i
 * (wrapping modulo 2^32), for i < count. out is a device pointer. */
wt_status wt_cast_f32_range(uint32_t first, uint64_t count, uint8_t *out, void *stream);

/* ---- Static schedule builder (host only) ----
 * The controller's computation ("Weight transfer for RL post-training in
 * under 2 seconds", section "High-level workflow": collect parameter
 * metadata from training and inference, compute a static transfer schedule
 * that says which training GPU sends which parameter where and in what
 * order; section "Static schedule": computed once, replayed every step).
 * Input: the training side's parameters (unique names, full shapes, FSDP
 * dim-0 shard count and, optionally, shard addresses) and the inference
 * side's tensors (names, the training parameters fused into each, in fusion
 * order, and the output dtype). Output: destination offsets packed in the
 * order of the inference tensors (data, then the FP8 scale grid, each
 * aligned), the source GPU of every output (longest-processing-time-first
 * over BF16 input bytes; ties to the lower index), and the task table that
 * wt_plan_create takes, for all sources or one. Shards are the torch.chunk
 * split of the rows: ceil(rows / n) rows each, trailing shards smaller or
 * empty. */

typedef struct wt_param_meta {
  const char *name;              /* unique, NUL-terminated */
  int64_t rows, cols;            /* full shape; a 1-D tensor of n elements is rows = n, cols = 1 */
  int32_t n_shards;              /* FSDP dim-0 shards, >= 1 */
  int32_t shard_mem;             /* WT_MEM_DEVICE or WT_MEM_PINNED_HOST */
  const void *const *shard_ptrs; /* n_shards addresses, or NULL (tasks then carry NULL shard pointers) */
} wt_param_meta;

typedef struct wt_dst_meta {
  const char *name;              /* inference-side tensor name */
  const char *const *components; /* training parameter names, in fusion (dim-0 concatenation) order */
  int32_t n_components;          /* >= 1; all components must have the same cols */
  int32_t dtype;                 /* WT_FP8_E4M3FN_B128 or WT_BF16_COPY */
} wt_dst_meta;

typedef struct wt_schedule_options {
  uint64_t align;    /* destination offset alignment, a power of two >= 16; 0 = 256 */
  int32_t n_sources; /* source GPUs to balance outputs over; 0 = 1 */
  int32_t reserved[5];
} wt_schedule_options;

typedef struct wt_schedule wt_schedule;

/* Matches names, validates (unknown or duplicate names, cols that differ
 * inside a fusion group, rows < 1: WT_E_INVAL), packs offsets and assigns
 * sources. The inputs are copied. On failure *out is NULL and
 * wt_plan_last_error(NULL) says why. */
wt_status wt_schedule_build(const wt_param_meta *params, size_t n_params, const wt_dst_meta *dsts, size_t n_dsts,
                            const wt_schedule_options *opts, wt_schedule **out);

/* Totals: tasks (one per fusion component) and shard records over all
 * sources, the destination region size, and how many training parameters no
 * inference tensor uses. Any pointer may be NULL. */
wt_status wt_schedule_info(const wt_schedule *sch, size_t *n_tasks, size_t *n_shards, uint64_t *dst_bytes,
                           size_t *n_unused_params);

/* Placement of inference tensor i: data and scale offsets (scale_offset is
 * 0 for BF16 copies), its source GPU and its BF16 input bytes. */
wt_status wt_schedule_output(const wt_schedule *sch, size_t i, uint64_t *dst_offset, uint64_t *scale_offset,
                             int32_t *source, uint64_t *input_bytes);

/* Writes the task table of one source (source = -1: every source) in
 * inference-tensor order: tasks[0 .. *n_tasks) with their shard records in
 * shards[]; task.shards points into the caller's shards array. Fusion
 * groups are numbered by inference-tensor index. WT_E_RANGE if max_tasks or
 * max_shards is too small (*n_tasks and *n_shards_out then give the sizes
 * needed). */
wt_status wt_schedule_tasks(const wt_schedule *sch, int32_t source, wt_task *tasks, size_t max_tasks,
                            wt_shard *shards, size_t max_shards, size_t *n_tasks, size_t *n_shards_out);

/* Frees the schedule. NULL is ignored. */
void wt_schedule_destroy(wt_schedule *sch);

/* ---- Block-scaled FP8 quantization of token activations ----
 * The sender half of MoE dispatch quantizes token activations to FP8 with
 * block scales before writing them to peers ("Enabling trillion-parameter
 * models on AWS EFA", dispatch/combine evaluation: hidden size 7168, FP8
 * dispatch with block scales; the sender shuffles tokens into send buffers
 * so each peer receives one write). Blocks are 1 x 128: one token's 128
 * consecutive channels, the last block of a row holding cols % 128 channels
 * when cols is not a multiple of 128. Per block s = amax / 448 in IEEE fp32
 * (1 for an all-zero block) and q = E4M3(fl32(x / s)), round to nearest even,
 * saturating: the same arithmetic as the weight tiles.
 *
 * x: n_rows rows of BF16 on the device, x_row_stride elements apart (>= cols),
 *    2-byte aligned.
 * row_index: NULL, or n_out int32 input-row indices on the device: output
 *    row i quantizes input row row_index[i] (row i when NULL). Output rows
 *    whose index is outside [0, n_rows) are not written. Indices may repeat.
 * q: n_out rows of q_row_stride bytes (>= cols), device or pinned host; the
 *    first cols bytes of a row receive the FP8 codes, the rest is untouched.
 * scales: n_out rows of scale_row_stride bytes (>= 4 ceil(cols / 128)),
 *    4-byte aligned, device or pinned host; the row's block scales as fp32.
 *    q and scales may interleave (e.g. one send-buffer slot per token holding
 *    its codes, then its scales) as long as no two written ranges overlap.
 * Shapes with cols, x_row_stride and q_row_stride multiples of 8, x 16-byte
 * and q 8-byte aligned take the vector path; any other shape takes a general
 * path with the same results.
 * Enqueued on `stream` (a hipStream_t; NULL = the default stream); returns
 * without waiting. Errors: WT_E_INVAL for negative or inconsistent sizes,
 * NULL pointers with n_out > 0, n_out * ceil(cols / 128) >= 2^31 or
 * cols >= 2^31; WT_E_ALIGN for a misaligned x or scales; WT_E_HIP if the
 * launch fails. Pointer kinds and extents are not queried (that would cost a
 * runtime call per pointer per call on the dispatch path): the caller
 * guarantees that every range above lies in its allocation. n_out == 0 is a
 * no-op. */
wt_status wt_quantize_act_b128(const void *x, int64_t n_rows, int64_t cols, int64_t x_row_stride,
                               const int32_t *row_index, int64_t n_out, void *q, int64_t q_row_stride,
                               void *scales, int64_t scale_row_stride, void *stream);

/* Element types of gradients and router logits. */
enum { WT_DT_F32 = 0, WT_DT_BF16 = 1 };

/* ---- Expert router: selection, per-expert counts and the balance loss ----
 * What decides where a token's activations are dispatched ("Enabling
 * trillion-parameter models on AWS EFA", dispatch/combine evaluation: each
 * token goes to its top-k experts) and, in training, the loss that keeps the
 * experts evenly used, with the gradient of both.
 *
 * For token t with logits x_e (fp32 or BF16, computed in fp32; a score below
 * 2^-126 counts as 0):
 *   score s_e = 1 / (1 + exp(-x_e))   (WT_SCORE_SIGMOID)
 *             = exp(x_e) / sum_j exp(x_j)   (WT_SCORE_SOFTMAX)
 *   selected: the top_k experts by s_e + bias_e (by x_e without a bias), in
 *     falling order, ties to the lower index. Near-ties are decided in fp64.
 *   weight_k = scale s_k, with `normalize` scale s_k / (sum over the selected
 *     s + 1e-20). The bias takes part in the selection alone.
 *   probability p_e = s_e (softmax), s_e / (sum_j s_j + 1e-20) (sigmoid)
 * An expert whose logit (or bias) is -infinity or NaN is never selected (a way
 * to switch experts off; the lowest finite value only puts it last); where fewer than top_k are left, the remaining places hold
 * index -1 and weight 0. A token with no expert left has probabilities 0. A
 * NaN logit still reaches the loss as NaN, and with softmax the weights (with
 * softmax and a bias no key of such a token is a number, and none is selected).
 *
 * Sequences: seq_offsets holds n_seqs + 1 token numbers, rising from >= 0 to
 * <= n_tokens; sequence q is the tokens [seq_offsets[q], seq_offsets[q + 1]).
 * Tokens before the first and behind the last sequence are padding: index -1,
 * weight 0, gradient 0, counted nowhere. NULL: one sequence of all tokens
 * (n_seqs = 1). With T_q tokens and c_{q,e} selections of expert e in sequence q,
 *   loss = balance_coef / n_seqs * sum_q sum_e f_{q,e} P_{q,e},
 *   f_{q,e} = n_experts c_{q,e} / (top_k T_q), P_{q,e} = mean over q of p_e
 * (an empty sequence adds 0). Offsets that fall or leave [0, n_tokens] give
 * meaningless results but no access outside the arrays. Sums run in a fixed
 * order: a call repeats bit for bit. */
enum { WT_SCORE_SIGMOID = 0, WT_SCORE_SOFTMAX = 1 };

typedef struct wt_router_desc {
  int64_t n_tokens;       /* 0 .. 2^27, with n_tokens top_k < 2^31 */
  int32_t n_experts;      /* 1 .. 1024 */
  int32_t top_k;          /* 1 .. min(n_experts, 32) */
  const void *logits;     /* n_tokens rows, device */
  int64_t logits_stride;  /* elements from row to row, >= n_experts */
  int32_t logits_dtype;   /* WT_DT_F32 or WT_DT_BF16 */
  int32_t score;
  int32_t normalize;      /* 0 or 1 */
  float scale;            /* of the weights; finite */
  const float *bias;      /* n_experts, or NULL */
  const int32_t *seq_offsets; /* n_seqs + 1, or NULL */
  int32_t n_seqs;         /* 1 .. 2^20 */
  float balance_coef;     /* finite */
} wt_router_desc;

/* Zeroes, then top_k = n_seqs = 1 and scale = 1. */
void wt_router_desc_init(wt_router_desc *desc);

/* Bytes of workspace wt_router_forward needs (16-byte aligned device memory).
 * It need not be cleared; calls that may run at the same time need one each. */
wt_status wt_router_workspace_bytes(const wt_router_desc *desc, size_t *bytes);

/* index [n_tokens x top_k] int32 and weight [n_tokens x top_k] fp32 are dense;
 * counts [n_experts] and seq_counts [n_seqs x n_experts] int32 receive the
 * selections per expert over all sequences and per sequence; loss one fp32.
 * counts may be NULL. Errors as for wt_quantize_act_b128; WT_E_RANGE if the
 * workspace is too small. */
wt_status wt_router_forward(const wt_router_desc *desc, int32_t *index, float *weight, int32_t *counts,
                            int32_t *seq_counts, float *loss, void *workspace, size_t workspace_bytes, void *stream);

/* Gradient of <dweight, weight> + dloss * loss with respect to the logits
 * (counts and selection are constants of it). index and seq_counts as
 * wt_router_forward wrote them (an index outside [0, n_experts) counts as -1;
 * an expert in several places adds up, from the first place to the last); dweight [n_tokens x top_k] fp32, NULL: no
 * gradient of the weights; dloss one fp32 on the device, NULL: no gradient of
 * the loss (seq_counts may then be NULL). dlogits: n_tokens rows of n_experts
 * values of logits_dtype, dlogits_stride elements apart; it may be the logits'
 * own memory when the strides agree. */
wt_status wt_router_backward(const wt_router_desc *desc, const int32_t *index, const int32_t *seq_counts,
                             const float *dweight, const float *dloss, void *dlogits, int64_t dlogits_stride,
                             void *stream);

/* ---- Rows of a dispatch ----
 * Groups token copies by expert: the row_index that wt_quantize_act_b128
 * gathers by (same page: the sender shuffles tokens into send buffers so that
 * each peer receives one write), and where each copy went.
 *
 * index: [n_tokens x top_k] int32 experts as wt_router_forward writes them;
 *   values outside [0, n_experts) are no copy.
 * Expert e's copies take the rows [offsets[e], offsets[e] + counts[e]) in the
 * order of (token, place); offsets[e + 1] = offsets[e] + counts[e] rounded up
 * to a multiple of row_align, offsets[0] = 0.
 * row_token [n_rows] int32: the token of each row, -1 for rows that hold none
 *   (padding to row_align, and everything from offsets[n_experts] on). n_rows
 *   = n_tokens top_k + min(n_experts, n_tokens top_k) (row_align - 1) always
 *   suffices; copies whose row is >= n_rows are dropped.
 * pair_row [n_tokens x top_k] int32: each copy's row, -1 for none or dropped.
 * offsets [n_experts + 1] and counts [n_experts] int32 (not cut by n_rows).
 * row_token, pair_row and counts may be NULL. n_tokens top_k < 2^31 and the
 * last offset must stay below 2^31 (n_tokens top_k + n_experts (row_align - 1)
 * < 2^31); n_experts 1 .. 1024, row_align 1 .. 4096. */
wt_status wt_dispatch_workspace_bytes(int64_t n_tokens, int32_t top_k, int32_t n_experts, size_t *bytes);
wt_status wt_dispatch_rows(const int32_t *index, int64_t n_tokens, int32_t top_k, int32_t n_experts,
                           int32_t row_align, int64_t n_rows, int32_t *row_token, int32_t *pair_row,
                           int32_t *offsets, int32_t *counts, void *workspace, size_t workspace_bytes, void *stream);

/* ---- Experts: grouped products and the gated feed-forward block ----
 * What a token's copies go through between the row map and the way back ("Weight
 * transfer for RL post-training in under 2 seconds", section "Task pipeline":
 * gate and up projections are fused to gate_up; "Enabling trillion-parameter
 * models on AWS EFA": tokens reach their experts as groups of rows), forward and
 * backward, over the weights that wt_adamw_step updates and wt_prepare ships. A
 * dense layer is one expert that owns every row.
 *
 * Rows. Expert e owns the rows [offsets[e], offsets[e] + counts[e]) of a row
 * space of n_rows rows, as wt_dispatch_rows leaves them; offsets and counts stay
 * on the device. Other rows (padding, and what lies behind the last expert) are
 * neither read nor written. Offsets or counts that leave [0, n_rows] are cut to
 * it. Experts whose rows overlap are for TN only: in NT and NN a row of several experts
 * holds meaningless results, and if the experts' rows add up to more than n_rows, any
 * expert's results may be left unwritten in part (tiles are dealt for n_rows rows). Rows of
 * no expert stay as they were, and no access leaves the arrays.
 *
 * wt_expert_product, per expert e with rows r (BF16 operands, fp32 sums, rounded
 * once to out_dtype):
 *   WT_PRODUCT_NT: out[r, j] = sum_k a[r, k] b_e[j, k]    j < n: a projection, b_e [n x k]
 *   WT_PRODUCT_NN: out[r, j] = sum_k a[r, k] b_e[k, j]    j < n: its input's gradient, b_e [k x n]
 *   WT_PRODUCT_TN: out_e[i, j] = sum_r a[r, i] b[r, j]    i < m, j < n: its weights' gradient
 *     (zeros for an expert without rows; k is ignored)
 * row_index (may be NULL) makes row r of one operand row row_index[r] of an
 * array of n_index_rows rows: of a in NT and NN, of b in TN. Row numbers outside
 * of it stand for a row of zeros; the same row may be taken many times.
 *
 * wt_gated_forward (form NT, b_e [2n x k]: n gate rows, then n up rows, the order
 * of a fused gate_up): g = a[r] . b_e[j], u = a[r] . b_e[n + j],
 *   out[r, j] = act(g) u, rounded once to BF16; pre (may be NULL): pre[r, j] = g,
 *   pre[r, n + j] = u in BF16, what the backward pass reads.
 * wt_gated_backward (form NN, a = the gradient of the block's output, b_e = the
 * weights back, [k x n]): dh = a[r] . b_e[:, j], g and u from pre,
 *   out[r, j] = dh u act'(g), out[r, n + j] = dh act(g), in BF16 (out has 2n columns).
 *   Rounded, since it is an operand of the products below: the gradients of rows and gate_up weights
 *   differ from 64 bits by 0.0023 to 0.0024 of their norm, and by 0.0017 if it is kept in fp32.
 * The rest of the block's backward pass are products of `out`: NN with the
 * gate_up weights for the rows' gradient, TN with the rows for the weights'.
 *   act = WT_ACT_SILU: x / (1 + exp(-x)); WT_ACT_GELU: x / 2 (1 + tanh(sqrt(2 / pi)
 *   (x + 0.044715 x^3))); at an infinity their limits.
 *
 * A NaN or an infinity in an operand reaches exactly the results whose sum it is
 * part of. Sums run in an order that depends on sizes, strides and alignment alone (and
 * on whether offsets are given): a call repeats bit for bit, whichever rows the experts own.
 *
 * Speed. Arrays whose addresses, row and expert strides are even numbers of
 * elements, with even sizes (NT: k; NN: k and n; TN: m and n) and spans below
 * 2^31 bytes (512 rows of any operand, a gathered array as a whole, an expert's gate
 * and up rows) are copied to shared memory 16 bytes at a time; all others pass through
 * registers, with the same results to rounding (2001 rows, k = 4001, n = 777, us: NT 49
 * against 28 for 2000 rows, k = 4000, n = 776; NN 68 against 26; 4001 x 777 weights' gradient 56 against 21).
 *
 * out must not overlap an operand, with one exception: wt_gated_backward may write over
 * pre (out = pre, out_stride = pre_stride). No workspace; every call may be captured.
 * Calls on the same arrays must be ordered. */
enum { WT_PRODUCT_NT = 0, WT_PRODUCT_NN = 1, WT_PRODUCT_TN = 2 };
enum { WT_ACT_SILU = 0, WT_ACT_GELU = 1 };

typedef struct wt_product_desc {
  int64_t n_rows;          /* 0 .. 2^27 */
  int32_t n_experts;       /* 1 .. 1024 */
  int32_t form;
  const int32_t *offsets;  /* n_experts + 1, or NULL: one expert that owns every row */
  const int32_t *counts;   /* n_experts, or NULL: counts[e] = offsets[e + 1] - offsets[e] */
  const int32_t *row_index; /* n_rows, or NULL */
  int64_t n_index_rows;    /* 0 .. 2^31 - 1, with row_index */
  int64_t m, n, k;         /* 1 .. 2^24 where the form has them */
  const void *a;           /* rows, BF16 */
  int64_t a_stride;        /* elements from row to row, at least the row's length; likewise below */
  const void *b;           /* NT, NN: the weights; TN: rows */
  int64_t b_stride;
  int64_t b_expert_stride; /* NT, NN: elements from expert to expert (0: all share one) */
  void *out;               /* NT, NN: rows; TN: n_experts matrices */
  int64_t out_stride;
  int64_t out_expert_stride; /* TN: elements from expert to expert */
  int32_t out_dtype;       /* WT_DT_BF16 or WT_DT_F32 (gated calls: WT_DT_BF16) */
  int32_t act;             /* gated calls */
} wt_product_desc;

/* Zeroes, then n_experts = 1 and out_dtype = WT_DT_BF16. */
void wt_product_desc_init(wt_product_desc *desc);

/* Enqueued on `stream` (of the device that owns the arrays, whichever is
 * current; NULL: the current device's null stream); returns without waiting.
 * WT_E_INVAL: NULL pointers, sizes, strides or values out of range (a grid of
 * 2^31 tiles too); WT_E_ALIGN: an address that is no multiple of its element's
 * size; WT_E_HIP if a launch fails. n_rows = 0 is a no-op in NT and NN. */
wt_status wt_expert_product(const wt_product_desc *desc, void *stream);
wt_status wt_gated_forward(const wt_product_desc *desc, void *pre, int64_t pre_stride, void *stream);
wt_status wt_gated_backward(const wt_product_desc *desc, const void *pre, int64_t pre_stride, void *stream);

/* ---- MXFP4: 4-bit floating point with a scale to each 32 elements ----
 * The OCP microscaling format MXFP4, the narrower companion of the block-scaled
 * FP8 above: elements E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives: code =
 * sign 8 + index), scales E8M0 (byte c stands for 2^(c - 127), 255 for NaN), one
 * to each 32 consecutive elements of a row.
 *
 * Quantisation of a block with the largest magnitude amax:
 *   c = 127 + clamp(floor(log2 amax) - 2, -127, 125) (127 for a block of zeros),
 *   element = the value nearest to x / 2^(c - 127), of two equally near ones the
 *   even code, magnitudes beyond 6 become 6; the sign is kept, also of a zero.
 *   A block that holds a NaN or an infinity gets c = 255 and codes 0, so that all
 *   of it reads as NaN.
 * Element 2i of a row is the low half of byte i, element 2i + 1 the high half. A
 * row's codes take 16 ceil(cols / 32) bytes (the last block is filled with
 * codes 0), its scales ceil(cols / 32). */

/* x: n_rows rows of cols elements of `dtype`, x_row_stride elements apart.
 * row_index (may be NULL): output row i quantizes row row_index[i], as in
 * wt_quantize_act_b128; output rows whose index is outside of [0, n_rows) are not
 * written. codes: 4-byte aligned, code_row_stride bytes from row to row, a
 * multiple of 4 and >= 16 ceil(cols / 32); scales: scale_row_stride bytes >= ceil(cols /
 * 32). Bytes between the rows are left alone. For the operands of
 * wt_mxfp4_product see the alignments there. Weights are rows too: a matrix
 * [n x k] is quantized along k. Errors as for wt_quantize_act_b128 (with
 * ceil(cols / 32) for its ceil(cols / 128)). */
wt_status wt_mxfp4_quantize(const void *x, int32_t dtype, int64_t n_rows, int64_t cols, int64_t x_row_stride,
                            const int32_t *row_index, int64_t n_out, void *codes, int64_t code_row_stride,
                            void *scales, int64_t scale_row_stride, void *stream);

/* out (dtype WT_DT_BF16 or WT_DT_F32): the values that n_rows rows of codes stand
 * for. Every value but those that overflow (c > 252) is exact in both types. */
wt_status wt_mxfp4_dequantize(const void *codes, int64_t code_row_stride, const void *scales,
                              int64_t scale_row_stride, int64_t n_rows, int64_t cols, void *out, int32_t dtype,
                              int64_t out_row_stride, void *stream);

/* out[r, j] = sum_k a[r, k] b_e[j, k] over the values that the codes stand for, in
 * fp32 sums; gated = 1: out[r, j] = act(a[r] . b_e[j]) (a[r] . b_e[n + j]), b_e
 * then having 2n rows. Experts and rows as for wt_expert_product. The rows of a
 * are the expert's own (gather while quantizing). Strides of codes and scales are in bytes.
 * Codes: 16-byte aligned, strides multiples of 16 and rows >= 16 ceil(k / 32) bytes whose codes
 * beyond k are 0, as wt_mxfp4_quantize writes them; scales: 4-byte aligned,
 * strides multiples of 4, rows >= ceil(k / 32) (WT_E_ALIGN otherwise). Scales are read in
 * whole words of 4 bytes: up to 3 bytes behind a row's last scale are read and not used, so
 * that the allocation has to reach to the end of the last row's last word. */
typedef struct wt_mxfp4_product_desc {
  int64_t n_rows;          /* 0 .. 2^27 */
  int32_t n_experts;       /* 1 .. 1024 */
  int32_t gated;           /* 0 or 1 */
  const int32_t *offsets;  /* as in wt_product_desc */
  const int32_t *counts;
  int64_t n, k;            /* 1 .. 2^24 */
  const void *a;
  int64_t a_stride;
  const void *a_scales;
  int64_t a_scale_stride;
  const void *b;
  int64_t b_stride, b_expert_stride;
  const void *b_scales;
  int64_t b_scale_stride, b_scale_expert_stride;
  void *out;
  int64_t out_stride;      /* elements */
  int32_t out_dtype;       /* WT_DT_BF16 or WT_DT_F32 */
  int32_t act;             /* with gated */
} wt_mxfp4_product_desc;

/* Zeroes, then n_experts = 1 and out_dtype = WT_DT_BF16. */
void wt_mxfp4_product_desc_init(wt_mxfp4_product_desc *desc);
wt_status wt_mxfp4_product(const wt_mxfp4_product_desc *desc, void *stream);

/* ---- AdamW over many parameter shards ----
 * The optimizer step that produces what wt_prepare transfers ("Weight transfer
 * for RL post-training in under 2 seconds", section "High-level workflow":
 * after each training step the training GPUs send their parameters). One call
 * updates every shard of a rank in place, in one launch (three when the
 * gradients are clipped by their global norm), so a prepare enqueued behind it
 * on the same stream reads the new weights.
 *
 * Per element, with g = grad * grad_scale * clip and t = the step's number:
 *   m' = beta1 m + (1 - beta1) g        v' = beta2 v + (1 - beta2) g^2
 *   u  = (m' / (1 - beta1^t)) / (sqrt(v' / (1 - beta2^t)) + eps)
 *   p' = p - lr lr_mul (weight_decay p + u)
 * all in fp32. p is the fp32 master copy if the tensor has one (the BF16 shard
 * then receives p' rounded to nearest even), else the BF16 shard itself.
 * clip = min(1, max_norm / (norm + 1e-6)), norm = |grad_scale| sqrt(the sum of
 * grad^2 over every tensor); 1 when max_norm is 0. The squares are taken in
 * fp32 (added in 64 bits): a gradient beyond 1.8e19 makes the norm infinite,
 * one below 1e-23 counts as 0.
 *
 * Rounded states. Where fewer than 32 bits carry a value from step to step
 * (8-bit states, a BF16 shard without a master), rounding to nearest would
 * drop every change below half a step of the format and the state would stand
 * still; those values are rounded up or down with the probabilities that keep
 * their mean: x in units of its format becomes floor(|x| + rho), with 16
 * random bits rho = r / 65536. The bits come from `seed`, the step's number
 * and the element's place in the table, so a run repeats exactly.
 *
 * 8-bit states: m and sqrt(v) (the root halves the range of exponents) are
 * held as OCP E4M3 codes with one fp32 scale per 128 consecutive elements of
 * the tensor (the last block may be shorter): scale = amax / 448, code =
 * x / scale rounded as above. A block whose amax is below 2^-100 holds zeros
 * with scale 1. A positive sqrt(v) never rounds to zero (the smallest code
 * stands for it), which keeps u bounded. A value that is not finite is held as
 * the NaN code and takes no part in its block's amax, so it stays with its
 * element. States start as zeros (codes 0; the scales must be finite).
 * It is the root's mean that rounding keeps, so v's lies higher by the root's
 * variance: with beta2 = 0.999 and gradients of one size (20,000 steps of the
 * definition) v is 5 % high in the mean and between 0.49 and 2.0 times its
 * value from the 1st to the 99th percentile (fp32 states: 0.93 to 1.08), the
 * root 1.3 % high, and |u| 1.6 %.
 *
 * Random bits of element i of a tensor: block b = the tensor's first block +
 * i / 128 (blocks are numbered through the table, ceil(n / 128) per tensor),
 * j = i mod 128, and with mix(x): x ^= x >> 16; x *= 0x6A09E667; x ^= x >> 15;
 * x *= 0xBB67AE85; x ^= x >> 16 (32-bit),
 *   w = mix(mix(b ^ k0) + k1 + j * 0x9E3779B9);
 * m takes w's low 16 bits, sqrt(v) the high 16, a BF16 shard the high 16 of
 * w * 0x9E3779B9. (k0, k1) are the low and high half of z = seed +
 * t * 0x9E3779B97F4A7C15; z ^= z >> 32; z *= 0x6A09E667F3BCC909; z ^= z >> 29;
 * z *= 0xBB67AE8584CAA73B; z ^= z >> 32 (64-bit). */

/* One parameter shard: n consecutive elements (n may be 0). Device memory;
 * every range the step writes must be disjoint from every other range of the
 * table (two tensors may share a gradient). */
typedef struct wt_adamw_tensor {
  void *param;      /* BF16 shard, 2-byte aligned, or NULL (the fp32 master is then all there is) */
  float *master;    /* fp32 copy, or NULL (then param is the only copy) */
  const void *grad; /* grad_dtype */
  void *m;          /* first moment: fp32, or E4M3 codes */
  void *v;          /* second moment as fp32, or its root as E4M3 codes */
  float *m_scale;   /* 8-bit states: ceil(n / 128) scales; ignored otherwise */
  float *v_scale;
  int64_t n;
  int32_t grad_dtype;
  float lr_mul;       /* 0 .. 1e6; multiplies the step's learning rate */
  float weight_decay; /* 0 .. 1e6 */
  int32_t reserved;
} wt_adamw_tensor;

typedef struct wt_adamw_options {
  int32_t state_bits; /* 32 (default) or 8 */
  int32_t device;     /* HIP device ordinal; -1 (default) = current device */
  int32_t reserved[6];
} wt_adamw_options;

/* What one step takes. wt_adamw_hyper_init() fills the defaults. */
typedef struct wt_adamw_hyper {
  double lr;         /* 1e-3; 0 .. 1e6 */
  double beta1;      /* 0.9; 0 <= beta < 1 */
  double beta2;      /* 0.999 */
  double eps;        /* 1e-8; at least 1e-30 */
  double grad_scale; /* 1: every gradient is multiplied by it (1 / loss scale, 1 / accumulated steps) */
  double max_norm;   /* 0: no clipping; > 0: the norm the gradients are clipped to */
  int64_t step;      /* number of this step, from 1 */
  uint64_t seed;     /* of the random bits */
  /* Device memory, may be NULL. step_dev / lr_dev: the step's number and the
   * learning rate are read there when the step runs instead of from `step` and
   * `lr`, so that a captured step can be replayed with new ones. norm_out
   * receives the gradients' norm (before clipping). */
  const int64_t *step_dev;
  const float *lr_dev;
  float *norm_out;
} wt_adamw_hyper;

typedef struct wt_adamw_info {
  int64_t n_tensors;        /* with n > 0 */
  int64_t n_elements;
  int64_t n_blocks;         /* 128-element blocks */
  int64_t n_items;          /* work items of the launch */
  int64_t n_vector_tensors; /* tensors all of whose addresses allow 4-element accesses (16 bytes for fp32, 8 for BF16,
                               4 for codes); the others take 1.7 (32-bit states) to 2.3 times (8-bit) as long */
  int64_t table_bytes;      /* device memory the handle holds */
} wt_adamw_info;

typedef struct wt_adamw wt_adamw;

void wt_adamw_options_init(wt_adamw_options *opts);
void wt_adamw_hyper_init(wt_adamw_hyper *hyper);

/* Validates a table exactly as wt_adamw_create does and describes the handle,
 * without touching any GPU. opts (defaults) and info may be NULL. WT_E_INVAL:
 * NULL pointers, sizes or factors out of range; WT_E_ALIGN; WT_E_OVERLAP. */
wt_status wt_adamw_check(const wt_adamw_tensor *tensors, size_t n_tensors, const wt_adamw_options *opts,
                         wt_adamw_info *info);

/* Builds the step's device tables. The table is copied; the tensors stay the
 * caller's and must outlive the handle at the same addresses. Allocates and
 * copies, so not for use under stream capture: 0.13 ms for 96 tensors with
 * 32-bit states, 0.4 ms for 96 to 301 with 8-bit ones. No call changes an
 * address afterwards: keep the gradients in the same buffers from step to step,
 * since gradients that are allocated anew need a new handle. On failure *out
 * is NULL and wt_plan_last_error(NULL) says why (likewise for the calls
 * below). */
wt_status wt_adamw_create(const wt_adamw_tensor *tensors, size_t n_tensors, const wt_adamw_options *opts,
                          wt_adamw **out);

/* Enqueues one step on `stream` (of the handle's device); returns without
 * waiting. When the norm is computed (max_norm > 0 or norm_out) and is not
 * finite, the step changes nothing but norm_out, so that one bad batch can be
 * left out. No allocation happens here, and a step may be captured: a replay
 * repeats it with the hyper values of the capture, apart from step_dev and
 * lr_dev (a step_dev below 1 counts as 1). With step_dev or lr_dev every
 * thread computes the step's factors for itself, about 1 us a step. The steps of one handle must be
 * ordered one behind the other, replays included: they update the same memory
 * and share the handle's workspace. WT_E_STATE if another thread is inside the
 * call with this handle; WT_E_INVAL for hyper values out of range; WT_E_HIP if
 * a launch fails. */
wt_status wt_adamw_step(wt_adamw *adamw, const wt_adamw_hyper *hyper, void *stream);

wt_status wt_adamw_get_info(const wt_adamw *adamw, wt_adamw_info *info);

/* Waits for the handle's device, then frees what the handle owns. A graph that
 * holds captured steps must not be launched after this. NULL is ignored. */
void wt_adamw_destroy(wt_adamw *adamw);

/* ---- Completion counters ----
 * Host-visible words that the GPU writes as parts of a replay finish, so a
 * host thread can start moving a part of the destination region (the one-sided
 * write to the inference side) as soon as it is final instead of waiting for
 * the whole replay ("RDMA point-to-point communication for LLM systems",
 * GPU-progress notification through memory words that kernels update and the
 * CPU polls; receiver-side counters per index). A replay finishes in units: the
 * launch over device-resident outputs (unit 0 when the plan has one), then
 * each pipeline chunk in order; wt_plan_info.n_units counts them and
 * wt_plan_task_unit maps a task to its unit. */

/* Attaches `words` (n_words >= n_units 8-byte words in pinned host memory,
 * 8-byte aligned; owned by the caller, who must keep it alive while the plan
 * replays) to the plan and resets the plan's replay counter. From then on the
 * r-th wt_prepare (r = 1, 2, ...) stores r into words[u] once every byte of
 * unit u is in the destination region: after the unit's prepare launch
 * (zero-copy) or after its destination copies (WT_DST_STAGED). The stores are
 * made by a one-thread kernel on the stream that ran the unit, with release
 * ordering at system scope, behind the unit's work. Passing words == NULL
 * detaches. Call only while no replay of this plan is in flight. The words are
 * never cleared by the library. WT_E_INVAL for a short, misaligned or
 * non-pinned array. */
wt_status wt_plan_set_progress(wt_plan *plan, uint64_t *words, size_t n_words);

/* *unit = the completion unit that covers task `task` (index into the table
 * given to wt_plan_create). WT_E_INVAL if task is out of range. */
wt_status wt_plan_task_unit(const wt_plan *plan, size_t task, int32_t *unit);

/* Host-side wait: polls *word (acquire loads) until it is >= target or
 * timeout_ns elapses. WT_OK when reached (the unit's bytes are then visible to
 * the host), WT_E_TIMEOUT otherwise, WT_E_INVAL for a NULL word. Makes no HIP
 * call. */
wt_status wt_progress_wait(const uint64_t *word, uint64_t target, uint64_t timeout_ns);

#ifdef __cplusplus
}
#endif

#endif /* WT_H */
