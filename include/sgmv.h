/*
 * sgmv.h -- C ABI of libsgmv.so, SGMV (segmented gather matrix-vector
 * multiplication) for multi-LoRA serving on AMD Instinct MI355X (gfx950).
 *
 * The operation.  A LoRA-adapted linear layer outputs the base product plus
 * a low-rank correction, y = xW + xAB, with A of shape [H1, r] and B of shape
 * [r, H2] (Punica walkthrough, omica.com.cn/news/959180, section 2.1).  A
 * batch mixes requests for many adapters; the correction for request i,
 * x_i A_i B_i, is computed in two steps: the shrink v_i = x_i A_i, a gather of
 * the request's A out of one back-to-back stack of all adapters' A matrices
 * followed by a vector-matrix product, and the expand v_i B_i over the
 * likewise stacked B matrices (same page, section 2.2; aivaro.ru answer 959,
 * section 3.2).  Requests for the same adapter form contiguous row segments
 * (segmented inputs and outputs: Punica review on nubint.ai, "Proposed
 * method").  This library adds the correction, times a scale s, to y:
 *
 *     for every segment t, every row i in [seg_indptr[t], seg_indptr[t+1]):
 *         a = adapter_ids[t]
 *         v[i, :] = x[i, :] @ A_stack[a]                  (shrink, H1 -> r)
 *         y[i, :] = y[i, :] + s * v[i, :] @ B_stack[a]    (expand, r -> H2)
 *
 * Layout (all row-major, dense, no padding):
 *     x        [num_rows, H1]              dtype
 *     y        [num_rows, H2]              dtype, updated in place
 *     A_stack  [num_adapters, H1, r]       dtype, adapter a at a*H1*r
 *     B_stack  [num_adapters, r, H2]       dtype, adapter a at a*r*H2
 *     v        [num_rows, r]               float32 (the shrink output)
 *     seg_indptr  int32 [num_segments + 1], non-decreasing, CSR row pointer
 *     adapter_ids int32 [num_segments]
 * x, A_stack, B_stack and y share one dtype; every sum is accumulated in
 * float32 and y is rounded once (nearest-even) to its dtype.
 *
 * Pointers.  Every array argument is a DEVICE pointer owned by the caller
 * (the host-side validator is the one exception and says so).  The library
 * keeps no state between calls, allocates no memory and never synchronises
 * the host with the device (sgmv_set_fused_wait() is the one process-wide
 * setting): each call only enqueues kernels on `stream`
 * (a hipStream_t; NULL means the default stream) and returns.
 *
 * Segment table.  Rows outside every segment are left untouched; empty
 * segments do nothing; an adapter may name several segments; segments must
 * not overlap.  The table is read on the device and is not validated on the
 * host (that would need a device-to-host copy).  For memory safety the
 * kernels clamp segment bounds to [0, num_rows) and skip a segment whose
 * adapter id lies outside [0, num_adapters); what a malformed table computes
 * is otherwise unspecified.  sgmv_validate_segments() checks a host copy.
 *
 * Workspace.  sgmv_shrink and lora_apply take caller-owned device scratch
 * (size from the *_workspace_bytes queries, a pure function of the shapes).
 * Its first 256 KiB hold synchronisation counters: they must be zero before
 * the buffer is first used (hipMemset once at allocation), and every call
 * leaves them zero again, so one buffer serves any sequence of calls of any
 * shapes, including calls captured in a HIP graph.  (The last 4 bytes of
 * that region are a sticky flag, set to 1 if a workgroup ever stopped
 * waiting and recomputed its input itself; results are the same either way.)
 * The rest holds float32 partial sums and may contain anything.  Two calls
 * that may run at the same time (e.g. on different streams) must not share
 * a workspace.
 *
 * Aliasing.  y must not overlap x, v, the stacks or the workspace.
 *
 * Errors.  Calls return SGMV_OK after enqueueing, or a status describing the
 * first problem found by the host-side checks (made before anything is
 * enqueued) or by the HIP launch.  Device faults surface at the caller's
 * next synchronisation, as usual for HIP.  num_rows == 0 or
 * num_segments == 0 is a valid no-op.
 *
 * Rank.  r is a runtime argument (any 1 <= r <= SGMV_MAX_RANK, no
 * recompilation: aivaro.ru answer 959, section 3.2).  Ranks 8, 16, 32, 64
 * and 128 (and 4 for float32) with 16-byte aligned arrays take the
 * vectorised kernels; anything else takes a slower general kernel that
 * computes the same thing.
 */
#ifndef SGMV_H
#define SGMV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SGMV_ABI_VERSION 1
#define SGMV_MAX_RANK 128

typedef enum {
    SGMV_F32 = 0,
    SGMV_F16 = 1,
    SGMV_BF16 = 2
} sgmv_dtype_t;

typedef enum {
    SGMV_OK = 0,
    SGMV_ERR_NULL_PTR = 1,     /* a required pointer is NULL                    */
    SGMV_ERR_BAD_SHAPE = 2,    /* negative size, r outside [1, SGMV_MAX_RANK]   */
    SGMV_ERR_BAD_DTYPE = 3,    /* dtype is not one of sgmv_dtype_t              */
    SGMV_ERR_UNSUPPORTED = 4,  /* sizes beyond what the kernels index (>2^31)   */
    SGMV_ERR_WORKSPACE = 5,    /* workspace NULL or smaller than required       */
    SGMV_ERR_HIP = 6,          /* a HIP launch reported an error                */
    SGMV_ERR_BAD_SEGMENTS = 7, /* (validator only) malformed segment table      */
    SGMV_ERR_SCRATCH = 8       /* lora_apply_noalloc: the call needs more than  */
                               /* SGMV_NOALLOC_SCRATCH_BYTES of scratch         */
} sgmv_status_t;

/* Version of this ABI (SGMV_ABI_VERSION of the library that was loaded). */
int sgmv_abi_version(void);

/* Human-readable name of a status code (static string, never NULL). */
const char* sgmv_status_string(int status);

/* Text of the last HIP error behind an SGMV_ERR_HIP returned to the calling
 * thread ("no error" if there was none; static string, never NULL). */
const char* sgmv_last_hip_error(void);

/*
 * Shrink: v[i, :] = x[i, :] @ A_stack[adapter_ids[t]] for every row i of
 * every segment t (overwrite; float32).  Rows of v outside every segment
 * keep their contents.  The reduction over H1 is split across workgroups and
 * combined in a fixed order, so repeated calls give identical bits.
 *
 * workspace: device scratch of at least sgmv_shrink_workspace_bytes(...)
 * bytes (see "Workspace" above).  May be NULL only when that size is 0.
 */
size_t sgmv_shrink_workspace_bytes(int32_t num_rows, int32_t num_segments,
                                   int32_t H1, int32_t r, int32_t dtype);
int sgmv_shrink(float* v, const void* x, const void* A_stack,
                const int32_t* seg_indptr, const int32_t* adapter_ids,
                int32_t num_segments, int32_t num_rows, int32_t num_adapters,
                int32_t H1, int32_t r, int32_t dtype,
                void* workspace, size_t workspace_bytes, void* stream);

/*
 * Expand: y[i, :] = round(y[i, :] + scale * (v[i, :] @ B_stack[adapter_ids[t]]))
 * for every row i of every segment t; v is float32 [num_rows, r], the sum
 * over r is taken in float32 and y is rounded once to its dtype.
 */
int sgmv_expand(void* y, const float* v, const void* B_stack,
                const int32_t* seg_indptr, const int32_t* adapter_ids,
                int32_t num_segments, int32_t num_rows, int32_t num_adapters,
                int32_t r, int32_t H2, float scale, int32_t dtype, void* stream);

/*
 * Fused add-on: y[i, :] = round(y[i, :] + scale * (x[i, :] @ A_a) @ B_a),
 * a = adapter_ids of row i's segment.  The intermediate v stays in float32
 * and never leaves the workspace.
 *
 * Decode- and prefill-shaped calls with a vectorised rank run as a single
 * kernel in which the expand workgroups wait, with bounded patience, for the
 * shrink workgroups of their rows; the result does not depend on how long
 * they wait.
 *
 * workspace: device scratch of at least lora_apply_workspace_bytes(...)
 * bytes (see "Workspace" above).
 */
size_t lora_apply_workspace_bytes(int32_t num_rows, int32_t num_segments,
                                  int32_t H1, int32_t H2, int32_t r, int32_t dtype);
int lora_apply(void* y, const void* x, const void* A_stack, const void* B_stack,
               const int32_t* seg_indptr, const int32_t* adapter_ids,
               int32_t num_segments, int32_t num_rows, int32_t num_adapters,
               int32_t H1, int32_t H2, int32_t r, float scale, int32_t dtype,
               void* workspace, size_t workspace_bytes, void* stream);

/*
 * lora_apply for callers that cannot allocate memory -- code being captured
 * into a HIP graph, tight serving loops, harnesses that forbid hipMalloc:
 * the same computation, kernels and results as lora_apply (bit for bit),
 * with no workspace argument.  Its scratch is a static device array inside
 * the library, SGMV_NOALLOC_SCRATCH_BYTES per GPU, held from the first call
 * on a GPU until the process ends.  The call allocates nothing: no hipMalloc,
 * no hipFree, no allocating library routine.
 *
 * Limit: a call whose lora_apply_workspace_bytes(...) exceeds
 * SGMV_NOALLOC_SCRATCH_BYTES returns SGMV_ERR_SCRATCH before enqueueing
 * anything (use lora_apply with a workspace of that size instead).
 *
 * The scratch is shared by every call on one GPU and keeps what the last
 * call left there: calls that may overlap on one GPU (different streams,
 * different host threads without ordering) race and must not be made.
 * Its synchronisation counters are zero when the library is loaded (static
 * storage) and every call leaves them zero; the first call on a GPU made
 * outside a graph capture also clears them with a small kernel on `stream`.
 * The current device must be the GPU that `stream` belongs to.  Arguments,
 * layout and the other errors are those of lora_apply.
 */
#define SGMV_NOALLOC_SCRATCH_BYTES (16u << 20)
int lora_apply_noalloc(void* y, const void* x, const void* A_stack, const void* B_stack,
                       const int32_t* seg_indptr, const int32_t* adapter_ids,
                       int32_t num_segments, int32_t num_rows, int32_t num_adapters,
                       int32_t H1, int32_t H2, int32_t r, float scale, int32_t dtype,
                       void* stream);

/*
 * Several LoRA add-ons over one batch -- e.g. the q, k, v and o projections
 * of a decoder layer -- in one call: for every problem p,
 *   problems[p].y[i, :] = round(y + scale_p * (x_p[i, :] @ A_p[a]) @ B_p[a])
 * with the shared segment table, num_rows, num_adapters, r and dtype, and
 * each problem's own arrays, H1, H2 and scale.  This amortises the launch
 * and the shrink-to-expand hand-off, which dominate a decode-sized call
 * (the pages stress kernel-launch overhead: Punica walkthrough,
 * omica.com.cn/news/959180, section 2.2).  Results equal those of one
 * lora_apply per problem.
 *
 * problems: HOST array of num_problems (1..SGMV_MAX_PROBLEMS) descriptors;
 * the pointers in them are device pointers, as for lora_apply, and the
 * problems must not overlap each other's y.  Decode-shaped calls (vector
 * ranks, aligned pointers, at most 1024 segments, segments of few rows) run
 * as one launch; any other call runs as one lora_apply per problem, in order.
 *
 * workspace: at least lora_apply_multi_workspace_bytes(...) bytes, with the
 * conventions of "Workspace" above.  Returns as lora_apply.
 */
#define SGMV_MAX_PROBLEMS 8
typedef struct {
    void* y;               /* [num_rows, H2], updated in place */
    const void* x;         /* [num_rows, H1] */
    const void* A_stack;   /* [num_adapters, H1, r] */
    const void* B_stack;   /* [num_adapters, r, H2] */
    int32_t H1;
    int32_t H2;
    float scale;
} sgmv_lora_problem;

size_t lora_apply_multi_workspace_bytes(const sgmv_lora_problem* problems,
                                        int32_t num_problems, int32_t num_rows,
                                        int32_t num_segments, int32_t r, int32_t dtype);
int lora_apply_multi(const sgmv_lora_problem* problems, int32_t num_problems,
                     const int32_t* seg_indptr, const int32_t* adapter_ids,
                     int32_t num_segments, int32_t num_rows, int32_t num_adapters,
                     int32_t r, int32_t dtype, void* workspace, size_t workspace_bytes,
                     void* stream);

/*
 * Adapted linear layer with the base product fused in:
 *   y[i, :] = round(x[i, :] @ W^T + bias + scale * (x[i, :] @ A_a) @ B_a)
 * for every row i, a = adapter_ids of row i's segment; rows outside every
 * segment (or in a segment whose adapter id is outside [0, num_adapters))
 * get round(x[i, :] @ W^T + bias).  This is the layer y = xW + xAB of Punica
 * walkthrough (omica.com.cn/news/959180, section 2.1) computed as one fused
 * kernel over the output, the correction added to each base tile before it
 * is stored (aivaro.ru answer 959, section 3.2: fusing the LoRA transform
 * into the base linear layer saves memory traffic), so y is written once
 * and never read.
 *
 * y: [num_rows, H2], overwritten.  x: [num_rows, H1].  W: [H2, H1], the row
 * of weights of each output feature (the usual layout of a linear layer's
 * weight; the page's W is its transpose).  bias: [H2] or NULL.  The stacks
 * and the segment table are those of lora_apply; with num_segments == 0
 * they may be NULL and the call computes the base layer alone.  All sums
 * are taken in float32 and y is rounded once.
 *
 * fp16/bf16 with H1 and H2 multiples of 8 and 16-byte aligned x, W, y,
 * bias and B_stack run on the matrix cores; any other call (float32
 * included) takes a slow element-wise kernel with the same definition.
 * Decode batches on the matrix cores (at most 64 rows, r in {16, 32, 64,
 * 128}, 16-byte aligned A_stack) take one launch: each workgroup of the
 * layer also computes a share of x @ A_a, publishes it, and waits for the
 * others' before adding its correction (the single-launch hand-off of
 * lora_apply, with the same patience, sgmv_set_fused_wait(); a workgroup
 * that stops waiting recomputes its share with the same arithmetic, so
 * the bits do not depend on it).  Other calls enqueue two launches: the
 * shrink of the add-on (skipped when num_segments == 0), then the layer.
 *
 * workspace: at least lora_linear_workspace_bytes(...) bytes, with the
 * conventions of "Workspace" above.  Returns as lora_apply; num_rows == 0
 * is a no-op.
 */
size_t lora_linear_workspace_bytes(int32_t num_rows, int32_t num_segments, int32_t H1,
                                   int32_t H2, int32_t r, int32_t dtype);
int lora_linear(void* y, const void* x, const void* W, const void* bias,
                const void* A_stack, const void* B_stack,
                const int32_t* seg_indptr, const int32_t* adapter_ids,
                int32_t num_segments, int32_t num_rows, int32_t num_adapters,
                int32_t H1, int32_t H2, int32_t r, float scale, int32_t dtype,
                void* workspace, size_t workspace_bytes, void* stream);

/*
 * On-demand adapter loading: copies `count` adapters from HOST memory into
 * slots [slot, slot + count) of the device stacks -- h_A [count, H1, r]
 * into A_stack[slot ..] and h_B [count, r, H2] into B_stack[slot ..], all
 * row-major in the stacks' dtype -- with two asynchronous copies on
 * `stream`, so that the next lora_apply on that stream sees them.  Adapters
 * not yet resident are brought in this way when a request needs them
 * (Punica review, nubint.ai, "Proposed method": the
 * system loads LoRA models on demand and keeps only the base model
 * resident).  For the copy to overlap other work the host buffers must be
 * pinned (hipHostMalloc); pageable buffers are staged by the runtime.  The
 * host buffers must stay valid until the copies have completed.  Returns
 * SGMV_OK, SGMV_ERR_NULL_PTR, SGMV_ERR_BAD_SHAPE (slots outside
 * [0, num_adapters), count < 1, bad sizes), SGMV_ERR_BAD_DTYPE or
 * SGMV_ERR_HIP.
 */
int sgmv_load_adapter(void* A_stack, void* B_stack, int32_t slot, int32_t count,
                      int32_t num_adapters, const void* h_A, const void* h_B, int32_t H1,
                      int32_t H2, int32_t r, int32_t dtype, void* stream);

/*
 * Process-wide patience, in seconds (0 <= seconds <= 10; default 0.02), of
 * the single-kernel lora_apply's expand workgroups waiting for their shrink
 * workgroups (and of the one-launch lora_linear's workgroups waiting for
 * each other's shares of x @ A_a).  A workgroup that stops waiting computes its input itself with
 * the same arithmetic in the same order, so results never depend on this
 * setting; 0 makes every expand workgroup do so without waiting (that is
 * how the path is tested).  This is the library's only state.  Returns SGMV_OK or
 * SGMV_ERR_BAD_SHAPE for a value out of range.
 */
int sgmv_set_fused_wait(double seconds);

/*
 * Host-side check of a segment table held in HOST memory: seg_indptr
 * non-decreasing from >= 0, seg_indptr[num_segments] <= num_rows, every
 * adapter id in [0, num_adapters).  Returns SGMV_OK or SGMV_ERR_BAD_SEGMENTS
 * (SGMV_ERR_NULL_PTR / SGMV_ERR_BAD_SHAPE for bad arguments).
 */
int sgmv_validate_segments(const int32_t* h_seg_indptr, const int32_t* h_adapter_ids,
                           int32_t num_segments, int32_t num_rows, int32_t num_adapters);

/*
 * Segment tables built on the device from per-row adapter ids (the
 * per-sample LoRA indices of Punica walkthrough, omica.com.cn/news/959180,
 * section 3.2; SGMV itself wants the batch "segmented" by adapter, Punica
 * review, nubint.ai, "Proposed method").
 *
 * row_ids [num_rows] int32: the adapter of each row; an id outside
 * [0, num_adapters) means "no adapter" (the row is left untouched by a
 * lora_apply over the resulting table).
 *
 * Outputs, all DEVICE arrays owned by the caller:
 *   seg_indptr [num_rows + 1], adapter_ids [num_rows]: a segment table of
 *     num_rows segments whose first *num_segments are the real ones; the
 *     rest are empty (seg_indptr = the end of the last real segment,
 *     adapter id -1).  So the table can be handed to lora_apply with
 *     num_segments = num_rows and no device-to-host read.
 *   num_segments [1]: the real segment count.
 *
 * sgmv_build_segments: one segment per maximal run of equal (normalised)
 * ids, in row order; no reordering of rows is needed.  Rows without an
 * adapter form segments with adapter id -1.
 *
 * sgmv_group_rows: also writes perm [num_rows], a stable grouping of the
 * rows: the rows of adapter 0 in increasing row order, then those of
 * adapter 1, ..., then the rows without an adapter.  Row j of the grouped
 * batch is row perm[j] of the original one.  The segment table describes
 * the grouped batch, with one segment per adapter present, in increasing
 * id order; the rows without an adapter come after the last segment.  Its
 * size is M = min(num_rows, num_adapters) segments instead of num_rows
 * (seg_indptr [M + 1], adapter_ids [M] are written), since there is at most
 * one segment per adapter; pass M to lora_apply.  num_adapters must be at
 * most 4096 (SGMV_ERR_UNSUPPORTED beyond).
 *
 * Both run as one workgroup on `stream` and return SGMV_OK after
 * enqueueing, SGMV_ERR_NULL_PTR / SGMV_ERR_BAD_SHAPE for bad arguments, or
 * SGMV_ERR_HIP.  num_rows == 0 writes seg_indptr[0] = 0 and a zero count.
 */
int sgmv_build_segments(const int32_t* row_ids, int32_t num_rows, int32_t num_adapters,
                        int32_t* seg_indptr, int32_t* adapter_ids, int32_t* num_segments,
                        void* stream);
int sgmv_group_rows(const int32_t* row_ids, int32_t num_rows, int32_t num_adapters,
                    int32_t* perm, int32_t* seg_indptr, int32_t* adapter_ids,
                    int32_t* num_segments, void* stream);

/*
 * The projections around the adapters: a base model with 4-bit weights, the
 * gated feed-forward block, rotary positions, and from the projections of q, k and v to attention over
 * a quantized cache.  These calls follow the
 * conventions above (device pointers, row-major arrays of one dtype, float32
 * sums, enqueue-only); a workspace is taken where one is named, and may hold anything.  Outputs must
 * not overlap inputs, except that h may be gate_add or up_add itself and rope and qk_norm_rope
 * work in place.
 */

/*
 * 4-bit weights.  W [out_features, in_features] is held as codes 0..15, one
 * scale per group of group_size consecutive input features of a row, and
 * optionally one zero point 0..15 per group (8 without):
 *     W[n, k] = scales[n, k / group_size] * (code[n, k] - zero[n, k / group_size]).
 * A user's arrays: codes [out_features, ceil(in_features / 2)] bytes, input
 * feature 2 j in the low and 2 j + 1 in the high half of byte j; scales
 * [out_features, groups] in the activations' dtype; zeros [out_features,
 * groups] bytes, or NULL; groups = ceil(in_features / group_size).
 * group_size is any multiple of 32 (the last group of a row may be shorter).
 *
 * q4_pack lays them out once for the matrix cores, into caller-owned,
 * 16-byte aligned device arrays: tiles (q4_tiles_bytes) and meta, the scales
 * and zero points (q4_meta_bytes).  The calls below read only these.
 */
typedef struct {
    const void* tiles;
    const void* meta;
} sgmv_q4_weight;

size_t q4_tiles_bytes(int32_t out_features, int32_t in_features);
size_t q4_meta_bytes(int32_t out_features, int32_t in_features, int32_t group_size, int32_t dtype);
int q4_pack(void* tiles, void* meta, const uint8_t* codes, const void* scales,
            const uint8_t* zeros, int32_t out_features, int32_t in_features, int32_t group_size,
            int32_t dtype, void* stream);

/*
 * y = round(x W^T + bias): x [num_rows, in_features], y [num_rows,
 * out_features] (overwritten), bias [out_features] or NULL.  For any number of rows
 * the codes, less their zero points, enter the products exactly and the scales
 * multiply float32 sums per group; y's rounding is the only one to fewer bits, so a
 * row's result depends on the rows beside it by the order of float32 sums alone.
 * An infinity in x gives a non-finite row (NaN where the products alone would give
 * an infinity).
 */
int q4_linear(void* y, const void* x, const sgmv_q4_weight* w, const void* bias, int32_t num_rows,
              int32_t out_features, int32_t in_features, int32_t group_size, int32_t dtype,
              void* stream);

/*
 * Gated feed-forward block: h = round(act(g) * u) with g = x Wg^T + gate_add
 * and u = x Wu^T + up_add, both products, the activation and the product in
 * one kernel.  gate_add, up_add [num_rows, out_features] or NULL: what the
 * rows' adapters add before the activation (lora_apply_multi on zeros).
 * q4_gated_ffn takes 4-bit weights of one group size, gated_ffn plain ones
 * [out_features, in_features].
 *
 * gated_ffn also stores g and u, rounded to dtype (finite values past its
 * largest as that), into g_saved and u_saved [num_rows, out_features] when these
 * are not NULL; gated_ffn_backward takes
 * them with dh = dL/dh and computes
 *     dg = dh * u * act'(g),  du = dh * act(g)   (also the addends' gradients)
 *     dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x
 * with dg and du rounded to dtype between the steps.  dx, or dWg and dWu,
 * may be NULL and are then not computed; dg and du are needed.  Options, OR-ed into
 * dtype (of the workspace query too):
 *   SGMV_FULL_GRADIENTS  g_saved, u_saved, g and u are float32, and dg and du go
 *                        through the products in two parts of dtype each (rounded
 *                        once where they are stored), so that no gradient is off by
 *                        more than float32 sums and its own rounding; the backward
 *                        products take twice as long.  Without it gradients carry
 *                        the roundings of g, u, dg and du.
 *   SGMV_ONE_WEIGHT      one of dWg and dWu alone may be NULL.
 * With
 * num_rows == 0 the weights' gradients are zero.  act' of relu at 0 is 0.  At
 * infinities the activations and act' are their limits: a g of minus infinity gives
 * h = 0 and no gradient.
 * Features beyond 2^20 return SGMV_ERR_UNSUPPORTED.
 * workspace: for dx, and with SGMV_FULL_GRADIENTS always, at least
 * gated_ffn_backward_workspace_bytes(...) bytes (0 for many sizes: it may then be
 * NULL), 16-byte aligned: dx of few rows is summed in ranges of out_features, whose
 * float32 sums stand there, and second parts of dg and du.  It may hold anything
 * before the call and does after it, from its first byte on: a buffer of the calls
 * above, whose counters have to be zero, must not be given here.
 */
typedef enum {
    SGMV_ACT_SILU = 0,
    SGMV_ACT_GELU = 1,      /* by the error function */
    SGMV_ACT_GELU_TANH = 2,
    SGMV_ACT_RELU = 3,
    SGMV_ACT_SIGMOID = 4
} sgmv_act_t;

#define SGMV_FULL_GRADIENTS 0x100
#define SGMV_ONE_WEIGHT 0x200

int q4_gated_ffn(void* h, const void* x, const sgmv_q4_weight* gate, const sgmv_q4_weight* up,
                 const void* gate_add, const void* up_add, int32_t num_rows, int32_t out_features,
                 int32_t in_features, int32_t group_size, int32_t act, int32_t dtype, void* stream);
int gated_ffn(void* h, void* g_saved, void* u_saved, const void* x, const void* Wg, const void* Wu,
              const void* gate_add, const void* up_add, int32_t num_rows, int32_t in_features,
              int32_t out_features, int32_t act, int32_t dtype, void* stream);
size_t gated_ffn_backward_workspace_bytes(int32_t num_rows, int32_t in_features,
                                          int32_t out_features, int32_t dtype);
int gated_ffn_backward(void* dx, void* dWg, void* dWu, void* dg, void* du, const void* dh,
                       const void* x, const void* Wg, const void* Wu, const void* g, const void* u,
                       int32_t num_rows, int32_t in_features, int32_t out_features, int32_t act,
                       int32_t dtype, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Rotary positions on q [num_rows, q_heads, head_dim] and k [num_rows,
 * k_heads, head_dim] (either may have no heads): pair j of the first
 * rotary_dim elements of every head, elements (j, j + rotary_dim / 2) or,
 * interleaved, (2 j, 2 j + 1), is turned by positions[row] * inv_freq[j]
 * radians and scaled by magnitude; the other elements are copied.  With
 * `inverse` it turns back (the gradients' form).
 *
 * positions: int32 or int64 (position_bytes 4 or 8); inv_freq: rotary_dim / 2
 * doubles.  Angles are formed in float64.  strides: HOST array of eight
 * element strides, for q {in row, in head, out row, out head} and then for
 * k; the last dimension is dense.  The outputs may be the inputs themselves
 * (equal pointers and strides) and must not overlap them otherwise.
 * rotary_dim is even and at most head_dim, head_dim at most 1024.
 */
int rope(void* q_out, void* k_out, const void* q, const void* k, const void* positions,
         int32_t position_bytes, const double* inv_freq, float magnitude, int32_t num_rows,
         int32_t q_heads, int32_t k_heads, int32_t head_dim, int32_t rotary_dim,
         const int64_t* strides, int32_t interleaved, int32_t inverse, int32_t dtype, void* stream);

/*
 * Norms of queries and keys for each head, with the rotation in the same
 * pass: a head x [head_dim] becomes Rot(x / sqrt(mean(x^2) + eps) * weight),
 * Rot as in rope (times magnitude, elements from rotary_dim on not turned),
 * rounded once.  weights [head_dim] of dtype, or NULL for ones.  strides as for
 * rope; the outputs may be the inputs themselves.  eps is not negative.
 *
 * qk_norm_rope_backward takes the outputs' gradients dq_out, dk_out and writes
 * dq, dk [num_rows, heads, head_dim] and the weights' gradients [head_dim]
 * (any of the four may be NULL and is then not computed; heads of zero leave a
 * side out, and its weight's gradient is zero).  strides: HOST array of
 * twelve, for q {in row, in head, gradient row, gradient head, dq row, dq
 * head} and then for k.  Sums are float32 in an order that depends on the sizes
 * alone.  workspace: qk_norm_rope_backward_workspace_bytes(...), 16-byte aligned, needed
 * where a weight's gradient is; it may hold anything.  With num_rows == 0
 * the weights' gradients are zero.
 */
int qk_norm_rope(void* q_out, void* k_out, const void* q, const void* k, const void* q_weight,
                 const void* k_weight, const void* positions, int32_t position_bytes,
                 const double* inv_freq, float magnitude, float eps, int32_t num_rows,
                 int32_t q_heads, int32_t k_heads, int32_t head_dim, int32_t rotary_dim,
                 const int64_t* strides, int32_t interleaved, int32_t dtype, void* stream);
size_t qk_norm_rope_backward_workspace_bytes(int32_t num_rows, int32_t head_dim, int32_t rotary_dim);
int qk_norm_rope_backward(void* dq, void* dk, void* dq_weight, void* dk_weight, const void* dq_out,
                          const void* dk_out, const void* q, const void* k, const void* q_weight,
                          const void* k_weight, const void* positions, int32_t position_bytes,
                          const double* inv_freq, float magnitude, float eps, int32_t num_rows,
                          int32_t q_heads, int32_t k_heads, int32_t head_dim, int32_t rotary_dim,
                          const int64_t* strides, int32_t interleaved, int32_t dtype,
                          void* workspace, size_t workspace_bytes, void* stream);

/*
 * A paged cache of K and V in 8 or 4 bits.  Token slots are numbered page by
 * page: slot = page * page_size + place in it.  Values are code * 2^e:
 *   SGMV_KV_FP8  e4m3 codes, one exponent per token and head (of K, of V);
 *   SGMV_KV_FP4  e2m1 codes, one exponent per 32 elements of a token's head.
 * e is the least exponent with |x| <= M 2^e over its group (M = 448 or 6), held to
 * what the type of the written rows represents exactly (float16: values of
 * 2^-24 to 57344 or 49152; else about 1e-38 to 3e38 or 2.5e38; larger ones saturate);
 * code is x 2^-e rounded to nearest even.  A token's head that holds a NaN or an
 * infinity reads as NaN, all of it.
 *
 * The caller owns the four device arrays (16-byte aligned; kv_codes_bytes for k and for v,
 * kv_scales_bytes for each scales array) and zeroes them once before use; their
 * layout is the library's own.  page_size is a multiple of 16, head_dim at most 256.
 *
 * kv_write quantizes row i of k and v [num_rows, kv_heads, head_dim] into
 * slots[i] (int32 or int64: slot_bytes 4 or 8); rows whose slot lies outside the
 * cache (-1 for padding) are skipped.  Slots of one call must differ: one named twice
 * holds parts of either row.  kv_read is the reverse, exact in the dtype that was written
 * (and in any wider one); rows without a slot read as zeros.  strides: HOST array of four element
 * strides, k {row, head}, v {row, head}; the last dimension is dense.
 */
typedef enum { SGMV_KV_FP8 = 0, SGMV_KV_FP4 = 1 } sgmv_kv_kind;

typedef struct {
    void* k;
    void* v;
    void* k_scales;
    void* v_scales;
    int32_t num_pages, page_size, kv_heads, head_dim;
    int32_t kind; /* sgmv_kv_kind */
} sgmv_kv_cache;

size_t kv_codes_bytes(int32_t num_pages, int32_t page_size, int32_t kv_heads, int32_t head_dim,
                      int32_t kind);
size_t kv_scales_bytes(int32_t num_pages, int32_t page_size, int32_t kv_heads, int32_t head_dim,
                       int32_t kind);
int kv_write(const sgmv_kv_cache* cache, const void* k, const void* v, const void* slots,
             int32_t slot_bytes, int32_t num_rows, const int64_t* strides, int32_t dtype,
             void* stream);
int kv_read(void* k, void* v, const sgmv_kv_cache* cache, const void* slots, int32_t slot_bytes,
            int32_t num_rows, const int64_t* strides, int32_t dtype, void* stream);

/*
 * Attention of a batch over such a cache.  num_seqs sequences have tokens of
 * their own in the cache; runs of consecutive sequences may share a prefix, which is
 * read for all of their rows together.  Rows of sequence s, row_indptr[s] up to
 * row_indptr[s + 1], are the last of its own tokens: row i of n sees the whole of its
 * run's prefix and the first lengths[s] - n + i + 1 of its own tokens,
 *     o = softmax(scale q K^T) V,   lse = log(sum of exp(scale q k)),
 * with float32 sums and maxima, rounded once.  q_heads / kv_heads consecutive heads of q share a
 * K / V head.  A row that sees no key gets zeros and an lse of minus infinity.  Rows of no
 * sequence are left as they are.  A visible NaN gives a row of NaN, whatever its weight; but for
 * that a score of minus infinity counts as a key that is not seen.  Weights
 * meet V with 11 bits or more where o is bfloat16, with 16 or more where it is float16 and with 22
 * or more where it is float32.  With many rows V is held in steps of 2^-31 of the largest scale that the
 * rows' tile meets, also of keys that a row does not see: exact over scales of 2^22, zero from 2^32 below it
 * on (caches of bfloat16 or float32 alone reach so far).  Sums of weights up to 2^4 times V have to
 * stay within float32, so V within about 1e37 over the keys.
 *
 * Tables, int32 device arrays: lengths [num_seqs], tokens in the cache (a step's new
 * ones among them, written before); row_indptr [num_seqs + 1], or NULL for one row each (row s
 * of sequence s); pages [num_seqs, pages_per_seq], the pages of a sequence's own tokens;
 * prefix_lengths [num_prefixes], prefix_pages [num_prefixes, pages_per_prefix]; prefix_indptr
 * [num_prefixes + 1], the first sequence of every run and the end (NULL with one prefix:
 * all sequences; sequences outside every run have no prefix).  They are
 * read on the device and not validated on the host: lengths are held to what the page tables have
 * room for, row and run bounds to the arrays, and tokens on a page outside the cache
 * are not seen; what a malformed table (one whose bounds decrease) computes is otherwise unspecified.
 *
 * prefix_plan cuts the work (prefix_plan_bytes, 16-byte aligned) from the lengths and
 * row tables: once per step, for all layers' prefix_attention calls with caches of the
 * same sizes; the page tables are read by these calls themselves.  The cache's
 * arrays are not read by prefix_plan.  prefix_attention needs a workspace
 * (prefix_attention_workspace_bytes, 16-byte aligned, any contents; calls that may run
 * at the same time must not share one).  It holds float32 results that are joined: without prefixes
 * at most 36 MB, whatever the batch; with them about as much and, since lengths are not known on the
 * host, room for two results of every row and head, 4 bytes an element of the padded head and 8 (578 MB
 * for 16384 rows of 32 heads of 128).  scale is positive and at most 2e38.  strides: HOST array of
 * element strides q {row, head}, o {row, head}; lse [num_rows, q_heads] or NULL.  o must not
 * overlap q.  Where lse is NULL nothing else changes.
 */
size_t prefix_plan_bytes(const sgmv_kv_cache* cache, int32_t num_rows, int32_t num_seqs,
                         int32_t num_prefixes, int32_t q_heads, int32_t dtype);
int prefix_plan(void* plan, size_t plan_bytes, const sgmv_kv_cache* cache, const int32_t* lengths,
                const int32_t* row_indptr, int32_t pages_per_seq, const int32_t* prefix_lengths,
                const int32_t* prefix_indptr, int32_t pages_per_prefix, int32_t num_rows,
                int32_t num_seqs, int32_t num_prefixes, int32_t q_heads, int32_t dtype,
                void* stream);
size_t prefix_attention_workspace_bytes(const sgmv_kv_cache* cache, int32_t num_rows,
                                        int32_t num_seqs, int32_t num_prefixes, int32_t q_heads,
                                        int32_t dtype);
int prefix_attention(void* o, float* lse, const void* q, const sgmv_kv_cache* cache,
                     const void* plan, const int32_t* pages, int32_t pages_per_seq,
                     const int32_t* prefix_pages, int32_t pages_per_prefix, int32_t num_rows,
                     int32_t num_seqs, int32_t num_prefixes, int32_t q_heads, float scale,
                     const int64_t* strides, int32_t dtype, void* workspace,
                     size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SGMV_H */
