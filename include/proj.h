/*
 * proj.h - C ABI of the MI355X decode-projection library.
 *
 * The library computes one bias-free linear layer per call,
 *     out[i, n] = sum over k of x[i, k] * W[n, k]      (out = x @ W^T),
 * for five fixed weight matrices (guide ch. 1 "The problem, the judge and the
 * speed of light", §1.1, layer table):
 *
 *     layer      id  N x K         W      out
 *     qkv_gate    0  2304 x 8192   BF16   BF16
 *     o           1  8192 x 1024   BF16   BF16
 *     pooler      2  4096 x 8192   BF16   BF16
 *     unpooler    3  8192 x 4096   BF16   BF16  (m <= 8: only rows 0..1023)
 *     router      4   256 x 8192   FP32   FP32
 *
 * x is always BF16, m x K row-major. Accumulation is FP32 (notebook note
 * "Numerical formats and error": BF16 operands, FP32 accumulation, BF16
 * output). The call contract follows guide ch. 1 §1.6: weights are handed
 * over once to an untimed prepare step; the timed call is replayed inside a
 * graph, so it never synchronizes and branches on shapes only.
 *
 * Pointers named "device" are HIP device pointers of the device that was
 * current when the layer was prepared. Streams are hipStream_t passed as
 * void * (NULL = the null stream). Every function returns PROJ_OK (0) or a
 * negative proj_status; no function aborts the process.
 *
 * Threading: calls that touch one layer must not race each other. Launches
 * of one layer that overlap on the GPU must not share the layer's split-K
 * workspace: at most one proj_run per layer may be in flight at a time
 * (stream order of a single stream satisfies this).
 */
#ifndef PROJ_H
#define PROJ_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

enum proj_layer {
    PROJ_QKV_GATE = 0,
    PROJ_O = 1,
    PROJ_POOLER = 2,
    PROJ_UNPOOLER = 3,
    PROJ_ROUTER = 4,
    PROJ_NUM_LAYERS = 5
};

enum proj_status {
    PROJ_OK = 0,
    PROJ_ERR_LAYER = -1,        /* layer id not in 0..4 */
    PROJ_ERR_M = -2,            /* m < 1 or m > 2^30 */
    PROJ_ERR_NULL = -3,         /* a required pointer is NULL */
    PROJ_ERR_ALIGN = -4,        /* a pointer is not 16-byte aligned */
    PROJ_ERR_NOT_PREPARED = -5, /* proj_run before proj_prepare for that layer */
    PROJ_ERR_UNSUPPORTED = -6,  /* a requested kernel configuration is not built */
    PROJ_ERR_HIP = -7,          /* a HIP runtime call failed (see proj_last_hip_error) */
    PROJ_ERR_DEVICE = -8,       /* current device differs from the one the layer was prepared (or the tensors are) on */
    PROJ_ERR_SCRATCH = -9,      /* proj_run_noalloc: the plan needs more split-K scratch than it has */
    PROJ_ERR_ARG = -10,         /* block.h: a size, stride, type or index outside what the operator takes */
    PROJ_ERR_PAGES = -11        /* block.h: the page pool has too few free pages */
};

/*
 * proj_prepare - repack a layer's weights once (guide ch. 1 §1.6: prepare runs
 * once, untimed; the report's round-6 note and the notebook's packed-pooler
 * notes describe the same lossless reordering of W into the kernel's read
 * order).
 *
 * W: device pointer, N x K row-major contiguous, BF16 bit patterns (uint16)
 *    for layers 0..3 and FP32 for the router. Read only during the call; the
 *    caller keeps ownership and may free it on return.
 * Effect: allocates library-owned device memory for the packed copy (same
 *    byte count as W) and the layer's split-K workspaces (2 x 32 MB), runs the repack on
 *    the null stream and synchronizes the device. For the router (all 256
 *    rows) and the unpooler (its first 1024 rows) it also keeps a plain
 *    row-major copy of those rows for the row-dot kernel used at m <= 8
 *    (8 MB each). Then it warms up (guide ch. 10 "Measure, experiment, and
 *    try your own changes", Experiment D): every token count up to 16384 is
 *    planned and resolved (past that the plans reuse the same kernels), and
 *    each distinct kernel the plans name is launched once on zero
 *    activations, so no proj_run meets an unsupported configuration or pays
 *    a first launch. The device current at this call becomes the layer's
 *    device.
 *    Preparing a prepared layer replaces its weights: the new state is built
 *    and warmed up next to the old one, which is freed only on success (on
 *    an error the layer keeps its previous weights). Replacing or releasing a
 *    layer frees the buffers that graphs captured earlier point to: such
 *    graphs must not be replayed afterwards.
 * Errors: PROJ_ERR_LAYER, PROJ_ERR_NULL, PROJ_ERR_ALIGN, PROJ_ERR_HIP;
 *    PROJ_ERR_UNSUPPORTED if a plan names a kernel that is not built.
 */
int proj_prepare(int layer, const void *W);

/*
 * proj_run - out = x @ W^T for `m` tokens, launch only (guide ch. 1 §1.1 for
 * the operation, §1.6 for the graph-replay contract).
 *
 * x:   device, m x K row-major BF16 bits, 16-byte aligned.
 * out: device, m x proj_out_cols(layer, m) row-major, BF16 bits (router:
 *      FP32), 16-byte aligned. Fully overwritten.
 * stream: hipStream_t (NULL = null stream).
 * m:   any token count from 1 to 2^30 (offsets are computed in 64 bits;
 *      x and out must hold m rows; above 2^30 x alone would exceed 2 TB).
 * Effect: exactly one kernel launch on `stream`. No allocation, no
 *    synchronization, no host read of device memory, no memset; the choice
 *    of kernel depends on (layer, m) and on whether prepare built the
 *    layer's 12-bit form (proj_compressed(layer) >= 0, fixed per prepared
 *    weights), never on data. Safe to capture in a HIP graph and
 *    replay with new contents of x. Split-K state (arrival counters, or the
 *    empty marks of the polled partials) is restored on the GPU by the
 *    kernel itself.
 * Errors (checked on the host before launching): PROJ_ERR_LAYER, PROJ_ERR_M,
 *    PROJ_ERR_NULL, PROJ_ERR_ALIGN, PROJ_ERR_NOT_PREPARED, PROJ_ERR_DEVICE;
 *    PROJ_ERR_HIP if the launch is rejected.
 */
int proj_run(int layer, const void *x, int m, void *out, void *stream);

/*
 * proj_run_noalloc - proj_run for callers that cannot allocate device memory
 * (code under graph capture, tight serving loops, harnesses that forbid
 * hipMalloc). Same arguments, plan, kernels and results as proj_run; the
 * split-K partials and arrival counters live in one fixed device array of the
 * library (4 MiB of polled partials, 16 MiB of counted partials, 16384
 * counters; each GPU holds its own copy until the process ends), set up by the
 * first proj_prepare on that device. Allocates nothing and calls no
 * allocating routine. The kernels restore the array's empty marks and zeroed
 * counters themselves; every call on a GPU shares that GPU's array, so calls
 * that overlap on one GPU race (a single stream, or calls ordered between
 * streams, is safe); proj_run calls use the layer's own workspace and do not
 * interfere. A reducer give-up is counted for proj_split_giveups(layer), whose
 * reset also restores the array's marks.
 * Errors: those of proj_run, and PROJ_ERR_SCRATCH when (layer, m)'s plan needs
 * more partials or counters than the array holds (for instance the pooler at
 * 1000 tokens); nothing is launched then.
 */
int proj_run_noalloc(int layer, const void *x, int m, void *out, void *stream);

/*
 * proj_out_cols - columns of out: N, except 1024 for the unpooler at m <= 8
 * (guide ch. 1 §1.1: at <= 8 tokens only this GPU's slice, the first 1024
 * rows, is computed). Returns a negative proj_status for a bad layer or m.
 */
int proj_out_cols(int layer, int m);

/*
 * proj_layer_dims - the layer table: N, K and the element sizes of W and out
 * in bytes (2 for BF16, 4 for FP32). Any output pointer may be NULL.
 */
int proj_layer_dims(int layer, int *N, int *K, int *w_elem_bytes, int *out_elem_bytes);

/*
 * proj_compressed - whether prepare also stored the layer's weights in the
 * 12-bit lossless form (report "Muse Spark Open Kernel Challenge -
 * muse_bf16_proj", round 5: each BF16 weight keeps its low byte and gets a
 * sign plus a 3-bit code for one of eight exponent values chosen per
 * matrix; weights outside those eight are restored exactly from a per-row
 * correction list). Returns the correction slots per row (0..8) when it
 * did, -1 when the layer is FP32 (router) or some row would need more than 8
 * corrections (then only the BF16 form exists), PROJ_ERR_LAYER or
 * PROJ_ERR_NOT_PREPARED otherwise. Host-only; no GPU call.
 */
int proj_compressed(int layer);

/*
 * proj_split_giveups - how many times a polled split-K reducer of this layer
 * (kind 0 with ksplit > 1) stopped waiting for a partial since prepare or the
 * last reset. Each give-up wrote NaN where the missing partial belonged (the
 * bounded wait of the kind-0 configuration notes below). A partial published
 * after its reducer gave up would leave words that a later launch reads as
 * arrived, so reset != 0 also restores every empty mark of the layer's
 * workspace before zeroing the count. Synchronizes the device; not for use
 * inside a graph capture or while a proj_run of the layer is in flight on
 * another stream. Returns the count (>= 0) or PROJ_ERR_LAYER,
 * PROJ_ERR_NOT_PREPARED, PROJ_ERR_DEVICE, PROJ_ERR_HIP.
 */
int proj_split_giveups(int layer, int reset);

/* proj_release - free a layer's packed weights and workspace; idempotent. */
int proj_release(int layer);

/* proj_strerror - static text for a proj_status value. */
const char *proj_strerror(int status);

/* proj_last_hip_error - the hipError_t behind the last PROJ_ERR_HIP. */
int proj_last_hip_error(void);

/*
 * Kernel configurations (the m-keyed dispatch table and the tuner's view).
 *
 * A configuration names one compiled kernel variant plus its split:
 *   kind      0 = skinny MFMA kernel (16-row blocks, waves split K in the
 *               workgroup), 1 = tiled MFMA kernel (large m; weights streamed
 *               into registers, activation tiles staged in LDS), 2 = row-dot
 *               kernel (m <= 8, router and the unpooler's 1024-row slice
 *               only: whole rows per workgroup from a row-major weight copy,
 *               FP32 multiply-adds), 3 = wide-tile MFMA kernel (activations
 *               staged once per workgroup in LDS; 4 or 8 waves, tiles of 64-256
 *               rows x 16-128 tokens, K split unevenly over up to KS/2
 *               workgroups, KS/4 at prefetch depth 16)
 *   nt        token sub-tiles of 16 per workgroup (kinds 0, 1, 3); largest token
 *             count of the variant (kind 2)
 *   rb        16-row blocks per workgroup (kinds 0, 1, 3; a multiple of 4
 *             for kind 3); rows per workgroup (kind 2)
 *   waves     wavefronts per workgroup (4 for kind 2; 4 or 8 for kind 3, as
 *             compiled: 8 waves hold the same tile with half the rows per wave)
 *   spw       k-steps of 32 per wave (kind 0); weight prefetch distance in
 *             k-steps (kind 1: the k-steps of one workgroup must be a
 *             multiple of it; kind 3: 4, 8 or 16, any split);
 *             k chunks of 2048 per row (kind 2: K = 2048 * spw)
 *   ksplit    workgroups that split K for one tile (1 = no cross-workgroup
 *             reduction; >1 = one workgroup sums the partials in split order:
 *             kinds 1 and 3 the last to arrive, counted with an atomic;
 *             kind 0 the one the hardware dispatches last, which polls the
 *             others' partials (a bounded wait: after 2^18 polls missing
 *             words read as NaN, so a launch always ends, and the give-up
 *             is counted for proj_split_giveups))
 *   flags     bit 0 set: workgroup i keeps tile i. Clear (default): when the
 *             grid is a multiple of 8, consecutive tiles are grouped on one
 *             XCD (workgroups are dealt to the 8 XCDs round-robin).
 *             bit 2 set (kind 0 with nt 1 or 2 and waves 4 or 8): read the 12-bit
 *             weights (needs proj_compressed(layer) >= 0); the workgroup gets
 *             one more wave, which gathers the correction terms.
 *             bit 3 set (kind 3): stream mode. ksplit is then the number of
 *             workgroups (at most tiles x K/(32 S) super-steps, S = 2, or 4
 *             at depth 16); the super-steps of all tiles are dealt to them in
 *             equal contiguous shares, a share may finish one tile and start
 *             the next, and the workgroups sharing a tile sum their parts in
 *             workgroup order (the last to arrive stores the tile).
 *             bit 4 set (kind 0, tests only): the splits that do not reduce
 *             exit without publishing and the reducer polls once, so every
 *             reducer gives up (NaN outputs, counted by proj_split_giveups);
 *             a host-forced stand-in for a split that never arrives.
 *             bit 5 / bit 6 set (kind 0, nt 1, m <= 4 / m <= 8; not both):
 *             each wave loads its activation slice for 4 / 8 token rows into
 *             registers once, instead of one load per k-step (compiled for
 *             rb 1 with waves x spw 8 x 32 and 4 x 8). Same arithmetic and
 *             summation order as with the bit clear.
 *             bit 7 set (kind 3, BF16 weights): activations move from memory
 *             straight into the LDS ring by DMA instead of through registers;
 *             same arithmetic and summation order as with the bit clear.
 *             bit 8 set (kind 0, rb 1, ksplit 1, m <= 16 * nt): stream
 *             partition. The layer's (16-row block, k-step) pairs are dealt
 *             in equal contiguous shares of waves * spw to the workgroups
 *             (grid = row blocks * K/32 / (waves * spw), which must divide
 *             exactly, with waves * spw <= K/32); each row block's parts
 *             (at most 4) are summed by the share dispatched last (polled,
 *             bounded, counted like kind 0's split). Compiled for
 *             waves x spw = 144 (qkv_gate: 256 workgroups).
 *             Other bits, or a bit the kind does not use, are rejected.
 * proj_plan fills the configuration proj_run would use; proj_run_config runs
 * an explicit one and returns PROJ_ERR_UNSUPPORTED if it is not compiled or
 * does not tile the layer.
 */
typedef struct {
    int kind;
    int nt;
    int rb;
    int waves;
    int spw;
    int ksplit;
    int flags;     /* bit 0: keep hardware workgroup order (no XCD grouping); bit 2: 12-bit weights;
                      bit 3: stream mode (kind 3); bit 4: test-only lost split (kind 0);
                      bits 5 / 6: activations preloaded for <= 4 / <= 8 tokens (kind 0);
                      bit 7: activations by LDS DMA (kind 3); bit 8: stream partition (kind 0) */
    int grid;      /* filled by proj_plan: workgroups launched */
    int block;     /* filled by proj_plan: threads per workgroup */
} proj_config;

int proj_plan(int layer, int m, proj_config *cfg);
int proj_run_config(int layer, const void *x, int m, void *out, void *stream,
                    const proj_config *cfg);

/* Number of compiled variants and the i-th one (ksplit = 1). */
int proj_num_variants(void);
int proj_variant(int i, int *is_f32w, proj_config *cfg);

#ifdef __cplusplus
}
#endif

#endif /* PROJ_H */
