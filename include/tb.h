/*
 * tb.h -- C ABI of the theta-bundle projection library (libtb.so), gfx950.
 *
 * The theta bundle ("The theta bundle", weightless docs, component table)
 * replaces a projection's dense weight [out_dim, in_dim] by
 *     W0 [out_dim, in_dim]   shared by every layer of a band, per family,
 *     s  [out_dim]           per layer, a scale of each output row of W0,
 *     U  [out_dim, rank]     per layer, left factor of the low-rank delta,
 *     V  [in_dim,  rank]     per layer, right factor of the low-rank delta,
 * with the weight rebuilt as diag(s) . W0 + U . V^T.  The band whose W0 a
 * layer uses comes from the contiguous band map ("Banded sharing", section
 * "How layers map to bands").
 *
 * Conventions shared by every entry point
 *   - Matrices are dense, row-major, with the leading dimension equal to the
 *     row length.  All pointers except band_out are DEVICE pointers on the
 *     current HIP device.  The caller owns all memory and the library keeps
 *     no caller pointer after a call returns.  The forward, reconstruct and
 *     error calls allocate and free nothing.  Two exceptions, both held until
 *     the process ends: tb_linear_forward_no_alloc's static device scratch
 *     (one per GPU, set up on its first call there), and the decomposition
 *     calls that multiply through rocBLAS (tb_lowrank_factors,
 *     tb_lowrank_factors_batch, tb_refine_shared_block), which create one
 *     rocBLAS handle per (device, stream) on first use; rocBLAS allocates
 *     that handle's own device workspace then.  Those three calls are
 *     therefore not for HIP graph capture or allocation-free callers.
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream).
 *     Device work is enqueued on it asynchronously; outputs are valid once
 *     the caller synchronises that stream.  No entry point synchronises.
 *   - Arguments are checked on the host before anything is enqueued.  On any
 *     status other than TB_OK nothing was enqueued and no output was written.
 *     tb_last_error() then describes the problem (per calling thread).
 *   - Matrix base pointers (x, w0, u, v, original, reconstructed, w_out) must
 *     be 16-byte aligned and in_dim / cols must be a multiple of 8; otherwise
 *     the call returns TB_ERR_UNSUPPORTED.  Every Gemma-shaped projection
 *     satisfies this.  s and y need only element alignment.
 *   - Sizes are 64-bit; an element count must fit in int64.
 */
#ifndef TB_H
#define TB_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum tb_status {
  TB_OK = 0,
  TB_ERR_INVALID_ARGUMENT = 1, /* a NULL pointer, a size out of range, ...  */
  TB_ERR_UNSUPPORTED = 2,      /* alignment / divisibility / dtype combination */
  TB_ERR_HIP = 3               /* the HIP runtime refused a query or launch  */
} tb_status;

typedef enum tb_dtype {
  TB_F32 = 0,  /* IEEE binary32 */
  TB_BF16 = 1, /* bfloat16, round-to-nearest-even on every store */
  TB_E4M3 = 2, /* 8-bit: 4 exponent bits, 3 mantissa bits, largest 448, no infinities; only where a call says so */
  TB_INT8 = 3  /* 8-bit whole numbers -127 .. 127; only where a call says so */
} tb_dtype;

/* How the scales of 8-bit blocks are stored (see tb_quantize_activations). */
typedef enum tb_scale {
  TB_SCALE_F32 = 0,  /* fp32: largest value of the block / 448 */
  TB_SCALE_E8M0 = 1  /* one byte, a power of two: exponent + 127 (255: NaN) */
} tb_scale;

/* Columns of an activation block; rows and columns of a weight block. */
#define TB_FP8_BLOCK 128

/* Largest in_dim and token count of the 8-bit calls. */
#define TB_FP8_MAX_IN_DIM (1 << 22)
#define TB_FP8_MAX_TOKENS (1 << 24)

/* Largest head of tb_head_norm_rotate, most heads of one token over all parts, most tokens. */
#define TB_MAX_HEAD_DIM 1024
#define TB_MAX_HEADS 65535
#define TB_MAX_HEAD_TOKENS (1 << 25)

/* Largest in_dim of the 8-bit integer calls, longest row of tb_residual_norm, most axes of a rotation. */
#define TB_INT8_MAX_IN_DIM 65536
#define TB_MAX_NORM_DIM 32768
#define TB_MAX_AXES 4

/* Most projections one tb_linear_forward_group call takes. */
#define TB_MAX_GROUP 8

/* Leading bytes of a forward workspace that hold control words: one block of
 * 64 KiB for each member a grouped call may have (a single call uses block 0). */
#define TB_WORKSPACE_CONTROL_BYTES (TB_MAX_GROUP * 65536)

/* Fixed workspace size of tb_rel_frobenius_error. */
#define TB_FROBENIUS_WORKSPACE_BYTES 65536

/* Most layers one band may hold in tb_shared_block. */
#define TB_MAX_BAND_LAYERS 128

/* Widest random probe (k = rank + oversampling) of tb_lowrank_factors. */
#define TB_MAX_PROBE 512

/*
 * tb_band_index -- band of one layer ("Banded sharing", "How layers map to
 * bands").  The num_layers layers are split into num_bands contiguous bands
 * whose sizes differ by at most one, the earlier bands taking the remainder:
 * with q = num_layers / num_bands and m = num_layers % num_bands, bands
 * 0..m-1 hold q+1 layers and the others q.  num_bands = 1 shares one W0 by
 * all layers; num_bands = num_layers is passthrough (band == layer).
 *
 *   num_layers >= 1, 1 <= num_bands <= num_layers, 0 <= layer < num_layers,
 *   band_out is a HOST pointer.  Host-only and pure; it touches no device.
 *   Errors: TB_ERR_INVALID_ARGUMENT (band_out untouched).
 */
tb_status tb_band_index(int32_t num_layers, int32_t num_bands, int32_t layer, int32_t *band_out);

/*
 * tb_linear_forward_workspace_size -- bytes of workspace tb_linear_forward
 * needs for these sizes on the current device (host-only query; it reads the
 * device's compute-unit count once).  *bytes_out >= TB_WORKSPACE_CONTROL_BYTES.
 */
tb_status tb_linear_forward_workspace_size(int64_t m, int64_t out_dim, int64_t in_dim, int64_t rank,
                                           tb_dtype dtype, size_t *bytes_out);

/*
 * tb_linear_forward -- one theta-bundle projection.
 *
 *     y[t, o] = s[o] * sum_i x[t, i] W0[o, i]  +  sum_j (sum_i x[t, i] V[i, j]) U[o, j]
 *
 * i.e. y = s (.) (x . W0^T) + (x . V) . U^T, the transpose of the
 * reconstruction formula weight = diag(s) W0 + U V^T ("The theta bundle"),
 * applied without forming the weight.  W0 is the block of the layer's band
 * (the caller selects it with tb_band_index).
 *
 *   x  [m, in_dim]        activations              (dtype)
 *   s  [out_dim]          row scale                (dtype; NULL: every row's scale is 1)
 *   w0 [out_dim, in_dim]  shared block             (dtype)
 *   u  [out_dim, rank]    left factor              (dtype; NULL allowed iff rank == 0)
 *   v  [in_dim, rank]     right factor             (dtype; NULL allowed iff rank == 0)
 *   y  [m, out_dim]       output                   (dtype), written, must not alias inputs
 *   m >= 1 tokens, out_dim >= 1, in_dim >= 8 and % 8 == 0, rank >= 0.
 *   Arithmetic: products and sums in fp32 (bf16 inputs are exact in fp32);
 *   the scale multiplies fp32 sums of x . W0^T before the delta is added
 *   (where a reduction over in_dim is split across workgroups, each part's
 *   sum is scaled and the parts are then added in a fixed order); for
 *   bf16 the intermediate x . V is rounded to bf16 before it meets U.  y is
 *   rounded once at the end.  Results are deterministic run to run.  For
 *   m <= 64, in_dim * element size * 96 must stay below 2^32 (else
 *   TB_ERR_UNSUPPORTED).
 *   workspace: device buffer of at least tb_linear_forward_workspace_size()
 *   bytes, 256-byte aligned.  Its first TB_WORKSPACE_CONTROL_BYTES bytes are
 *   control words: they must be zero before the first call that uses the
 *   buffer and must not be changed by the caller afterwards (each completed
 *   call, single or grouped, leaves all of them ready for the next; some
 *   carry state from call to call).  Word 2
 *   (uint32) is a sticky error flag: it becomes nonzero only when a bounded
 *   internal wait times out (the rows of y behind that wait are NaN), and a
 *   timed-out call may leave other control words stale.  While word 2 is set,
 *   every forward call on the workspace (tb_linear_forward, tb_dense_forward,
 *   tb_linear_forward_group) writes NaN to all of its y and reads or writes no
 *   other control word; zeroing the first TB_WORKSPACE_CONTROL_BYTES bytes
 *   again makes the workspace usable.  Calls that may run at the same time
 *   (different streams) must not share a workspace.
 *   Errors: TB_ERR_INVALID_ARGUMENT, TB_ERR_UNSUPPORTED, TB_ERR_HIP.
 */
tb_status tb_linear_forward(const void *x, const void *s, const void *w0, const void *u, const void *v,
                            void *y, int64_t m, int64_t out_dim, int64_t in_dim, int64_t rank,
                            tb_dtype dtype, void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of the device scratch that tb_linear_forward_no_alloc uses (96 MiB on
 * every GPU the library runs on, held until the process ends). */
#define TB_NO_ALLOC_SCRATCH_BYTES (96u << 20)

/*
 * tb_linear_forward_no_alloc -- tb_linear_forward for callers that cannot
 * allocate device memory: code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc.  The same computation, kernels, results
 * (bit for bit) and argument rules as tb_linear_forward, but the workspace is
 * the library's own static device array of TB_NO_ALLOC_SCRATCH_BYTES on the
 * current device; the call allocates and frees nothing.
 *   Every call on one GPU shares that GPU's array: calls that may overlap on
 *   one GPU (several streams, several host threads) race and must be
 *   serialised by the caller.  Each call first clears the array's control
 *   words (a small kernel on `stream`), so a call whose internal wait timed
 *   out (word 2 set, its y NaN) does not affect the next.  The array keeps
 *   the last call's contents.
 *   Errors: as tb_linear_forward; TB_ERR_UNSUPPORTED when the call would need
 *   more than TB_NO_ALLOC_SCRATCH_BYTES of workspace
 *   (tb_linear_forward_workspace_size tells), with nothing enqueued.
 */
tb_status tb_linear_forward_no_alloc(const void *x, const void *s, const void *w0, const void *u, const void *v,
                                     void *y, int64_t m, int64_t out_dim, int64_t in_dim, int64_t rank,
                                     tb_dtype dtype, void *stream);

/*
 * tb_dense_forward -- y = x . W^T for a weight held whole: the
 * materialise-once serving mode, where W = tb_reconstruct_weight(s, W0, U, V)
 * is formed once in the operand type ("Banded sharing", "Set G for serving":
 * the serve command that precomputes the weight outside the model graph;
 * "Quality": that path costs nothing measurable) and each call then streams
 * W alone.  It is tb_linear_forward with s = NULL (unit scale), rank 0:
 * the same kernels, workspace (tb_linear_forward_workspace_size with rank
 * 0), arithmetic, determinism, limits and errors.
 *
 *   x [m, in_dim], w [out_dim, in_dim], y [m, out_dim], all dtype, device.
 */
tb_status tb_dense_forward(const void *x, const void *w, void *y, int64_t m, int64_t out_dim, int64_t in_dim,
                           tb_dtype dtype, void *workspace, size_t workspace_bytes, void *stream);

/*
 * One projection of a group: the arguments of tb_linear_forward that may
 * differ between its members (same meaning, layout and alignment rules).
 */
typedef struct tb_projection {
  const void *x;
  const void *s;
  const void *w0;
  const void *u;
  const void *v;
  void *y;
  int64_t out_dim, in_dim, rank;
} tb_projection;

/*
 * tb_linear_forward_group_workspace_size -- bytes of workspace
 * tb_linear_forward_group needs for these projections (only their out_dim,
 * in_dim and rank are read) at m tokens: the control bytes plus each
 * member's buffers.
 */
tb_status tb_linear_forward_group_workspace_size(int32_t n, const tb_projection *projs, int64_t m, tb_dtype dtype,
                                                 size_t *bytes_out);

/*
 * tb_linear_forward_group -- n independent theta-bundle projections (the
 * computation of tb_linear_forward for each member) over the same token
 * count m and dtype.  Layers apply several projections to one input (q/k/v,
 * gate/up); each member still names its own x, which may be shared.  For
 * m <= 64 the members run in one launch when their plans can share one tile
 * shape, so the fixed cost of a launch and the wait for x . V are paid once.
 * For bf16 and m > 64, members that share in_dim and rank run as one x . V
 * launch and one GEMM launch over all their output tiles.  In one launch the
 * chip is shared out between the members, which may split a member's
 * reductions over in_dim differently from its own call, so its result may
 * differ from tb_linear_forward's in the last bits (same error bound; a given
 * group is deterministic run to run).  Other cases run the members one after
 * another, each exactly as its own call.
 *   n: 1 .. TB_MAX_GROUP.  projs: host array of n members (no y may alias
 *   any member's input or another member's y).
 *   workspace: as for tb_linear_forward, at least
 *   tb_linear_forward_group_workspace_size() bytes; member j uses control
 *   block j and its own buffers after the control bytes (a fused prefill
 *   launch uses block 0 and the buffers from the start).  A timed-out wait in
 *   any member sets word 2 of the workspace.
 *   Errors: TB_ERR_INVALID_ARGUMENT, TB_ERR_UNSUPPORTED, TB_ERR_HIP; a
 *   member that fails validation fails the call before anything is launched.
 */
tb_status tb_linear_forward_group(int32_t n, const tb_projection *projs, int64_t m, tb_dtype dtype, void *workspace,
                                  size_t workspace_bytes, void *stream);

/*
 * tb_reconstruct_weight -- w_out = diag(s) . W0 + U . V^T ("The theta bundle",
 * reconstruct_weight(s, W0, U, V)).
 *
 *   s [out_dim], w0 [out_dim, in_dim], u [out_dim, rank], v [in_dim, rank]
 *   in in_dtype; w_out [out_dim, in_dim] in out_dtype.  rank >= 0 (u, v may
 *   be NULL iff rank == 0), in_dim % 8 == 0.  fp32 accumulation; with
 *   rank == 0 and fp32 output the result is exact (s * W0 of bf16 inputs is
 *   representable in fp32).  Errors as above.
 */
tb_status tb_reconstruct_weight(const void *s, const void *w0, const void *u, const void *v, void *w_out,
                                int64_t out_dim, int64_t in_dim, int64_t rank,
                                tb_dtype in_dtype, tb_dtype out_dtype, void *stream);

/*
 * tb_rel_frobenius_error -- ||original - reconstructed||_F / ||original||_F
 * ("Quality", section "Reconstruction error"; the argument order of
 * relative_frobenius_error(original, reconstructed) in "The theta bundle").
 *
 *   original, reconstructed: [rows, cols] in dtype, cols % 8 == 0.
 *   result_device: DEVICE pointer to one double, written.  Differences,
 *   squares and sums are taken in fp64 in a fixed order (deterministic).
 *   When the difference is zero the result is 0; when only the original is
 *   zero it is +inf.  workspace: >= TB_FROBENIUS_WORKSPACE_BYTES device bytes,
 *   16-byte aligned.  Bytes [TB_FROBENIUS_WORKSPACE_BYTES - 8192,
 *   TB_FROBENIUS_WORKSPACE_BYTES) hold arrival counters: zero them before
 *   the first use; every call leaves them zero (the rest needs no
 *   initialisation).  Calls that share a workspace must not overlap (keep
 *   them on one stream).  Errors as above.
 */
tb_status tb_rel_frobenius_error(const void *original, const void *reconstructed, int64_t rows, int64_t cols,
                                 tb_dtype dtype, double *result_device, void *workspace,
                                 size_t workspace_bytes, void *stream);

/*
 * tb_reconstruction_error -- relative_frobenius_error(original,
 * reconstruct_weight(s, W0, U, V)) without writing the rebuilt weight ("The
 * theta bundle", reconstruction formula; "Quality", section "Reconstruction
 * error").  The rebuilt entries are formed in fp32 as tb_reconstruct_weight
 * forms them for fp32 output; differences, squares and sums are taken in
 * fp64 in a fixed order (deterministic).
 *
 *   s [out_dim], w0 [out_dim, in_dim], u [out_dim, rank], v [in_dim, rank]
 *   in bundle_dtype (u, v may be NULL iff rank == 0); original
 *   [out_dim, in_dim] in original_dtype; in_dim % 8 == 0.  result_device:
 *   DEVICE pointer to one double, written (0 when the two agree, +inf when
 *   only the original is zero).  workspace: as for tb_rel_frobenius_error
 *   (same size; the same arrival counters, zero before the first use and left
 *   zero by every call).  Errors as above.
 */
tb_status tb_reconstruction_error(const void *s, const void *w0, const void *u, const void *v, const void *original,
                                  int64_t out_dim, int64_t in_dim, int64_t rank, tb_dtype bundle_dtype,
                                  tb_dtype original_dtype, double *result_device, void *workspace,
                                  size_t workspace_bytes, void *stream);

/*
 * Analytic decomposition of one projection family ("The theta bundle",
 * section "Analytic decomposition"), in three steps per band and layer.
 * Outputs are fp32; the caller casts them for the forward path.
 *
 * tb_shared_block -- W0 = the mean of the band's weight matrices (Shared
 * block): summed in layer order in fp64, divided by n, rounded once to fp32.
 *   weights: HOST array of n DEVICE pointers, each [out_dim, in_dim] of
 *   weight_dtype; 1 <= n <= TB_MAX_BAND_LAYERS.  w0_out: device fp32
 *   [out_dim, in_dim].  Errors: TB_ERR_INVALID_ARGUMENT, TB_ERR_HIP.
 */
tb_status tb_shared_block(const void *const *weights, int32_t n, int64_t out_dim, int64_t in_dim,
                          tb_dtype weight_dtype, float *w0_out, void *stream);

/*
 * tb_row_scale -- s[o] = <weight[o], W0[o]> / <W0[o], W0[o]>, the per-row
 * least-squares fit of the weight against its band's block (Per-row scale);
 * 0 for a zero row of W0 (the minimum-norm solution).  fp64 sums in a fixed
 * order, one rounding to fp32.
 *   weight [out_dim, in_dim] (weight_dtype), w0 fp32 [out_dim, in_dim],
 *   s_out fp32 [out_dim], all device.  Errors: TB_ERR_INVALID_ARGUMENT, TB_ERR_HIP.
 */
tb_status tb_row_scale(const void *weight, const float *w0, int64_t out_dim, int64_t in_dim, tb_dtype weight_dtype,
                       float *s_out, void *stream);

/*
 * tb_lowrank_factors_workspace_size -- bytes of workspace tb_lowrank_factors
 * needs (host-only query; it reads the device's compute-unit count once).
 */
tb_status tb_lowrank_factors_workspace_size(int64_t out_dim, int64_t in_dim, int64_t rank, int64_t k,
                                            size_t *bytes_out);

/*
 * tb_lowrank_factors -- U [out_dim, rank], V [in_dim, rank] with U V^T the
 * rank-r cut of the residual E = weight - diag(s) W0 by the randomized SVD
 * the section names for large matrices (Low-rank residual; Halko,
 * Martinsson and Tropp, 2009).  U absorbs the singular values (columns by
 * decreasing singular value); a singular value at or below 1e-7 of the
 * largest counts as zero and gives zero columns in U and V.
 *   omega [in_dim, k] fp32: the random probe, drawn by the caller
 *   (k = rank + oversampling); power_iters re-orthonormalised power
 *   iterations (0..16).  The probe's range is found as in the method: Y = E
 *   omega, orthonormalised; each power iteration maps through E^T and E,
 *   orthonormalising each time; then the SVD of the k x in_dim projection.
 *   With k = min(out_dim, in_dim) the result is the exact truncated SVD up to
 *   rounding.  E is formed in fp32 (one rounding per entry), products in fp32,
 *   Gram matrices, Cholesky factors and the eigen-decomposition in fp64.
 *   weight (weight_dtype), w0, s, omega, u_out, v_out: device, 4-byte aligned.
 *   0 <= rank <= k <= min(out_dim, in_dim, TB_MAX_PROBE); out_dim * in_dim <
 *   2^31.  rank 0 writes nothing.  workspace: at least
 *   tb_lowrank_factors_workspace_size() bytes, 256-byte aligned, no initial
 *   contents.  Calls that may run at the same time must not share it.
 *   Errors: TB_ERR_INVALID_ARGUMENT, TB_ERR_UNSUPPORTED, TB_ERR_HIP (also for
 *   a failing rocBLAS call).
 */
tb_status tb_lowrank_factors(const void *weight, const float *w0, const float *s, int64_t out_dim, int64_t in_dim,
                             int64_t rank, tb_dtype weight_dtype, const float *omega, int64_t k, int32_t power_iters,
                             float *u_out, float *v_out, void *workspace, size_t workspace_bytes, void *stream);

/*
 * tb_lowrank_factors_batch -- tb_lowrank_factors for n matrices of one shape
 * (the layers of a projection family, each with its band's W0), in one pass:
 * every step runs on all of them together, so the single-workgroup solvers
 * of the n matrices share the chip.  Each matrix's result equals what
 * tb_lowrank_factors computes for it up to the rounding of the batched
 * products.
 *   weights, w0s: HOST arrays of n DEVICE pointers ([out_dim, in_dim]; weights
 *   of weight_dtype, w0s fp32), 1 <= n <= TB_MAX_BAND_LAYERS; s [n][out_dim],
 *   omega [n][in_dim][k],
 *   u_out [n][out_dim][rank], v_out [n][in_dim][rank], all fp32 device and
 *   contiguous.  workspace: n times tb_lowrank_factors_workspace_size()
 *   bytes, 256-byte aligned.  Other rules and errors as tb_lowrank_factors.
 */
tb_status tb_lowrank_factors_batch(const void *const *weights, int32_t n, const float *const *w0s, const float *s,
                                   int64_t out_dim, int64_t in_dim, int64_t rank, tb_dtype weight_dtype,
                                   const float *omega, int64_t k, int32_t power_iters, float *u_out, float *v_out,
                                   void *workspace, size_t workspace_bytes, void *stream);

/*
 * tb_refine_shared_block -- one least-squares refit of a band's shared block
 * with each layer's scale and factors held fixed, the alternating least
 * squares the "Quality" page reports on (Research: why shared configurations
 * need training): row by row
 *     W0[o] = sum_l s_l[o] (W_l - U_l V_l^T)[o] / sum_l s_l[o]^2,
 * and a row whose scales are all zero keeps its w0_prev value (a reading).
 * num = sum_l diag(s_l) W_l in fp64 sums (layer order, rounded to fp32),
 * minus the n layers' deltas as one fp32 GEMM of inner dimension n * rank
 * (rocBLAS), then the division in fp64.
 *   weights: HOST array of n DEVICE pointers ([out_dim, in_dim], weight_dtype);
 *   s, u, v: HOST arrays of n DEVICE fp32 pointers ([out_dim], [out_dim,
 *   rank], [in_dim, rank]; u, v may be NULL when rank is 0); w0_prev, w0_out:
 *   device fp32 [out_dim, in_dim] (they may be the same buffer).
 *   1 <= n <= TB_MAX_BAND_LAYERS, 0 <= rank <= TB_MAX_PROBE, out_dim *
 *   in_dim < 2^31.  workspace: tb_refine_shared_block_workspace_size()
 *   bytes, 256-byte aligned.  Errors: TB_ERR_INVALID_ARGUMENT,
 *   TB_ERR_UNSUPPORTED, TB_ERR_HIP.
 */
tb_status tb_refine_shared_block_workspace_size(int64_t out_dim, int64_t in_dim, int32_t n, int64_t rank,
                                                size_t *bytes_out);
tb_status tb_refine_shared_block(const void *const *weights, const float *const *s, const float *const *u,
                                 const float *const *v, int32_t n, int64_t out_dim, int64_t in_dim, int64_t rank,
                                 tb_dtype weight_dtype, const float *w0_prev, float *w0_out, void *workspace,
                                 size_t workspace_bytes, void *stream);

/*
 * 8-bit blocks: e4m3 numbers with one scale for each block, for serving a
 * materialised weight at one byte per entry on the matrix cores' 8-bit rate.
 *
 * tb_quantize_activations -- x [m, in_dim] (dtype, device) to
 *   q     [m, in_dim]                 e4m3
 *   scale [m, ceil(in_dim / 128)]     scale_type
 * one scale per row and 128 columns (the last block may be shorter).  With a
 * the block's largest magnitude:
 *   TB_SCALE_E8M0: scale = 2^max(ceil(log2(a / 448)), -127), q = e4m3(x / scale);
 *   TB_SCALE_F32:  scale = a' * (1 / 448), q = e4m3(x * (448 * (1 / a'))) with
 *                  a' = max(a, 2^-100), each operation rounded to fp32.
 * e4m3 rounds to nearest, ties to even.  A block that holds an infinity or NaN
 * gets a NaN scale and NaN entries.
 *   0 <= m <= TB_FP8_MAX_TOKENS (0: nothing is enqueued), in_dim >= 8, % 8 == 0
 *   and <= TB_FP8_MAX_IN_DIM.  x and q 16-byte aligned, scale element aligned; q
 *   and scale must not alias x.
 *   Errors: TB_ERR_INVALID_ARGUMENT, TB_ERR_UNSUPPORTED, TB_ERR_HIP.
 */
tb_status tb_quantize_activations(const void *x, void *q, void *scale, int64_t m, int64_t in_dim, tb_dtype dtype,
                                  tb_scale scale_type, void *stream);

/*
 * tb_reconstruct_weight_fp8 -- tb_reconstruct_weight into 8-bit blocks:
 * W = diag(s) W0 + U V^T is formed in fp32 as there and rounded once, to
 *   q     [out_dim, in_dim]                               e4m3
 *   scale [ceil(out_dim / 128), ceil(in_dim / 128)]       scale_type
 * one scale per 128 x 128 block, by the rules of tb_quantize_activations.
 * A dense weight is quantised with s = NULL (unit scale) and rank = 0.
 *   s, w0, u, v in dtype; in_dim % 8 == 0; w0, u, v and q 16-byte aligned; q and
 *   scale must not alias inputs.
 *   Errors as above.
 */
tb_status tb_reconstruct_weight_fp8(const void *s, const void *w0, const void *u, const void *v, void *q, void *scale,
                                    int64_t out_dim, int64_t in_dim, int64_t rank, tb_dtype dtype, tb_scale scale_type,
                                    void *stream);

/*
 * tb_dense_forward_fp8 -- tb_dense_forward for a weight in 8-bit blocks:
 *
 *     y[t, o] = sum_b xs[t, b] ws[o / 128, b] sum_{i in block b} xq[t, i] wq[o, i]
 *
 * over the blocks b of 128 columns.  The blocks' scaled sum is taken in fp32
 * and y is rounded once.  For y in TB_F32 the inner sums are fp32 as well.  For
 * TB_BF16 they run on the 8-bit matrix instructions, which cut the products of
 * each eight columns (8j .. 8j + 7) towards zero at 2^-13 of the largest
 * 2^(a + b) among them, a and b the exponents of a product's factors, before
 * the fp32 sum: y is off by at most 7 * 2^-13 of the sum of its terms'
 * magnitudes.  For normally distributed values that comes to about 2^-16 of the
 * result, below the rounding of y.  Where a few large terms cancel (channels of
 * outliers) it is no bound on the result: take y in TB_F32 there, which cuts
 * nothing.  Results are deterministic run to run.
 *   x  [m, in_dim]  in x_dtype.  TB_BF16 or TB_F32: x_scale is NULL and x is
 *      quantised within the call as tb_quantize_activations does (scales of
 *      scale_type).  TB_E4M3: x_scale [m, ceil(in_dim / 128)] are its scales;
 *      projections that share an input quantise it once this way.
 *   wq [out_dim, in_dim] e4m3, w_scale [ceil(out_dim / 128), ceil(in_dim / 128)]
 *   y  [m, out_dim] in y_dtype (TB_BF16 or TB_F32), must not alias inputs.
 *   Weights that share an input can be stacked along out_dim into one call
 *   where every one but the last has a multiple of 128 rows.
 *   0 <= m <= TB_FP8_MAX_TOKENS (0: nothing is enqueued), out_dim >= 1 and
 *   within one launch (8.0e8 up to 16 tokens, 5.3e8 up to 32, 4.0e8 up to 64),
 *   in_dim % 16 == 0 and <= TB_FP8_MAX_IN_DIM; x, wq 16-byte aligned.  The
 *   product xs * ws of two scales must be finite in fp32.
 *   workspace: at least tb_dense_forward_fp8_workspace_size() bytes, 256-byte
 *   aligned, no initial contents (NULL when 0).  Calls that may run at the same
 *   time must not share it.  The size does not grow with m everywhere: query each m.
 *   Errors: TB_ERR_INVALID_ARGUMENT, TB_ERR_UNSUPPORTED, TB_ERR_HIP.
 */
tb_status tb_dense_forward_fp8_workspace_size(int64_t m, int64_t out_dim, int64_t in_dim, tb_dtype x_dtype,
                                              tb_dtype y_dtype, tb_scale scale_type, size_t *bytes_out);
tb_status tb_dense_forward_fp8(const void *x, const void *x_scale, const void *wq, const void *w_scale, void *y,
                               int64_t m, int64_t out_dim, int64_t in_dim, tb_dtype x_dtype, tb_dtype y_dtype,
                               tb_scale scale_type, void *workspace, size_t workspace_bytes, void *stream);

/*
 * 8-bit integers with one scale per row, for activations (a scale per token) and
 * weights (a scale per output channel).
 *
 * tb_quantize_rows_int8 -- x [m, in_dim] (dtype, device) to
 *   q     [m, in_dim]  whole numbers, TB_INT8
 *   scale [m]          fp32
 * With a the row's largest magnitude and a' = max(a, 2^-100):
 *   scale = a' * (1 / 127),  q = round(x * (127 * (1 / a'))),
 * each operation rounded to fp32, ties to even.  A row that holds an infinity or
 * NaN gets a NaN scale and zeros.
 *   0 <= m <= TB_FP8_MAX_TOKENS (0: nothing is enqueued), in_dim >= 8, % 8 == 0
 *   and <= TB_INT8_MAX_IN_DIM.  x 16-byte, q 8-byte, scale element aligned; q and
 *   scale must not alias x.
 *   Errors: TB_ERR_INVALID_ARGUMENT, TB_ERR_UNSUPPORTED, TB_ERR_HIP.
 */
tb_status tb_quantize_rows_int8(const void *x, void *q, float *scale, int64_t m, int64_t in_dim, tb_dtype dtype,
                                void *stream);

/*
 * tb_dense_forward_int8 -- tb_dense_forward for a weight in 8-bit integers:
 *
 *     y[t, o] = (sum_i xq[t, i] wq[o, i]) * (xs[t] * ws[o])
 *
 * The sum is a whole number, held in 32 bits and exact, whatever y's type; it is
 * turned to fp32, scaled and rounded to y (fp32 operations, one rounding each).
 * So a result does not depend on how the call splits its work: a token's row is
 * the same bits in a batch and alone.
 *   x  [m, in_dim]  in x_dtype.  TB_BF16 or TB_F32: x_scale is NULL and x is
 *      quantised within the call as tb_quantize_rows_int8 does.  TB_INT8: x_scale
 *      [m] are its scales; projections that share an input quantise it once.
 *   wq [out_dim, in_dim] TB_INT8, w_scale [out_dim] fp32
 *   y  [m, out_dim] in y_dtype (TB_BF16 or TB_F32), must not alias inputs.
 *   Weights that share an input can be stacked along out_dim into one call.
 *   0 <= m <= TB_FP8_MAX_TOKENS (0: nothing is enqueued), out_dim >= 1, in_dim %
 *   16 == 0 and <= TB_INT8_MAX_IN_DIM; x, wq 16-byte aligned; the matrix must fit
 *   one launch as in tb_dense_forward_fp8.  q of -128 is allowed for.  The product
 *   xs * ws of two scales must be finite in fp32 (and loses digits below 2^-126).
 *   workspace: at least tb_dense_forward_int8_workspace_size() bytes, 256-byte
 *   aligned, no initial contents (NULL when 0).  Calls that may run at the same
 *   time must not share it.  The size does not grow with m everywhere: query each m.
 *   Errors: TB_ERR_INVALID_ARGUMENT, TB_ERR_UNSUPPORTED, TB_ERR_HIP.
 */
tb_status tb_dense_forward_int8_workspace_size(int64_t m, int64_t out_dim, int64_t in_dim, tb_dtype x_dtype,
                                               tb_dtype y_dtype, size_t *bytes_out);
tb_status tb_dense_forward_int8(const void *x, const float *x_scale, const void *wq, const float *w_scale, void *y,
                                int64_t m, int64_t out_dim, int64_t in_dim, tb_dtype x_dtype, tb_dtype y_dtype,
                                void *workspace, size_t workspace_bytes, void *stream);

/*
 * The tensors of tb_residual_norm: rows of n adjacent elements, row t of h at
 * h + t * h_stride (strides in elements).
 */
typedef struct tb_residual {
  const void *h;           /* [m, n] the residual stream (h_dtype) */
  const void *y;           /* [m, n] the block's output (dtype), or NULL: no block, h' = h */
  const void *post_weight; /* [n] (dtype) or NULL: none (and no offset) */
  const void *gate;        /* (dtype) row t takes row t / gate_rows; NULL: none */
  const void *weight;      /* [n] (dtype) or NULL: none (and no offset) */
  void *h_out;             /* [m, n] (h_dtype); NULL iff y is */
  void *z;                 /* [m, n] (z_dtype), or NULL: h' alone is wanted */
  void *z_scale;           /* the scales of an 8-bit z, else NULL */
  int64_t h_stride, y_stride, h_out_stride;
  int64_t z_stride;        /* of a z in dtype; an 8-bit z is dense */
  int64_t gate_rows;       /* consecutive rows that share a row of the gate, >= 1 */
  int64_t gate_stride;     /* between rows of the gate */
  int64_t gate_channels;   /* 1: a row of the gate holds n elements; 0: one, for the whole row */
} tb_residual;

/*
 * tb_residual_norm -- the norms before and after a block with its gate and
 * residual scale, in one pass: for each row
 *
 *     a  = y, or with post_norm y / sqrt(mean(y^2) + eps) * (post_weight + weight_offset)
 *     h' = residual_scale * h + gate * a
 *     z  = h' / sqrt(mean(h'^2) + eps) * (weight + weight_offset)
 *
 * h' is written to h_out, z to z in the type that the next projection takes.
 * Sums and products in fp32; h' and z are rounded once each, z from the h' that
 * is not yet rounded.  A row's results do not depend on the other rows or on how
 * many there are.
 *   z_dtype: dtype; TB_INT8 (z_scale [m] fp32, by the rules of
 *   tb_quantize_rows_int8); or TB_E4M3 (z_scale [m, ceil(n / 128)] scale_type, by
 *   the rules of tb_quantize_activations).
 *   0 <= m <= TB_FP8_MAX_TOKENS (0: nothing is enqueued), 1 <= n <=
 *   TB_MAX_NORM_DIM; an 8-bit z needs n % 8 == 0, rows (the gate's too where it has
 *   channels) and weights 16-byte aligned.  A wide z takes any n and element
 *   alignment: 16-byte pieces where n and the strides are multiples of eight and
 *   rows and weights 16-byte aligned; else the same pieces at element alignment
 *   (1.1 to 2.6 times as long, the most for the longest rows), and rows of fewer
 *   than eight elements one by one.  Strides of tensors with several rows are
 *   0 .. 2^35, those of outputs >= n.  h_out may be h, and a z in dtype may be y
 *   (same strides); other overlaps of an output with another tensor are refused,
 *   but for rows that interleave at one stride.  Without y there is no gate,
 *   post_norm or residual scale (1).  eps >= 0; rows must be small enough for their
 *   squares to sum up in fp32 (and, where eps is 0, large enough for the sum not to
 *   vanish).
 *   Errors: TB_ERR_INVALID_ARGUMENT, TB_ERR_UNSUPPORTED, TB_ERR_HIP.
 */
tb_status tb_residual_norm(const tb_residual *tensors, int64_t m, int64_t n, float residual_scale, float eps,
                           float weight_offset, int32_t post_norm, tb_dtype dtype, tb_dtype h_dtype, tb_dtype z_dtype,
                           tb_scale scale_type, void *stream);

/*
 * One tensor of heads in tb_head_norm_rotate: element (token t, head h, d) of
 * x is at x + t * x_token_stride + h * x_head_stride + d (strides in
 * elements), so queries and keys may be views of one packed projection output,
 * and y may be a view of a cache.
 */
typedef struct tb_head_part {
  const void *x;
  void *y;            /* x itself (same strides), or memory that overlaps no part's x and no other y */
  const void *weight; /* [head_dim], or NULL: no weight (and no offset) */
  int64_t heads;
  int64_t x_token_stride, x_head_stride;
  int64_t y_token_stride, y_head_stride;
} tb_head_part;

/*
 * tb_head_norm_rotate -- norms of queries and keys per head and their position
 * rotation, in one pass over all parts.  For each token and head
 *
 *     z = x / sqrt(mean(x^2) + eps) * (weight + weight_offset)
 *
 * over its head_dim elements; then, with r = rot_dim / 2 and the angles
 * a_p = positions[t] * freqs[p], each pair (i, j) of z's first rot_dim
 * elements is turned: y_i = z_i cos a_p - z_j sin a_p, y_j = z_j cos a_p +
 * z_i sin a_p.  Pair p is (p, p + r), or (2p, 2p + 1) when interleaved.  The
 * other elements are y = z.  Sums and products in fp32, angles in fp64 (right
 * to fp32 for positions up to 2^30), one rounding to y.
 *   n: 1 .. TB_MAX_GROUP parts (host array) of one dtype (x, y and weight);
 *   0 <= tokens <= TB_MAX_HEAD_TOKENS (0: nothing is enqueued); 1 <= head_dim <= TB_MAX_HEAD_DIM;
 *   0 <= rot_dim <= head_dim, even; positions [tokens] int64 and freqs [r]
 *   double, device (may be NULL where rot_dim is 0); eps >= 0.  Heads add up
 *   to TB_MAX_HEADS at most; a part may have none.  Strides are >= 0 and the
 *   rows of a y must not overlap one another.  Overlaps between a y and other
 *   tensors are refused where the two step alike over tokens and heads, or
 *   start at the same row; elsewhere keeping them apart is up to the caller.  16-byte aligned parts with
 *   strides, head_dim and (unless interleaved) r in multiples of 16 bytes are
 *   read and written in 16-byte pieces; everything else works, more slowly.
 *   x must be small enough for its squares to sum up in fp32 (and, where eps is
 *   0, large enough for the sum not to vanish).
 *   Errors: TB_ERR_INVALID_ARGUMENT, TB_ERR_UNSUPPORTED, TB_ERR_HIP.
 */
tb_status tb_head_norm_rotate(int32_t n, const tb_head_part *parts, int64_t tokens, int64_t head_dim, int64_t rot_dim,
                              int32_t interleaved, const int64_t *positions, const double *freqs, float eps,
                              float weight_offset, tb_dtype dtype, void *stream);

/* Where pair p of a rotation of r = rot_dim / 2 pairs lies. */
typedef enum tb_pairs {
  TB_PAIRS_HALF = 0,        /* (p, p + r) */
  TB_PAIRS_INTERLEAVED = 1, /* (2p, 2p + 1) */
  TB_PAIRS_AXIS = 2         /* in its axis's own span: with s pairs of the axes before and c of its own, (s + p, s + p + c) */
} tb_pairs;

/*
 * tb_head_norm_rotate_axes -- tb_head_norm_rotate for tokens with a position on
 * each of several axes (time, height, width): the angle of pair p is
 * positions[pair_axis[p]][t] * freqs[p].  With one axis and norm it is
 * tb_head_norm_rotate, bit for bit.
 *   positions [axes][tokens] int64, device; 1 <= axes <= TB_MAX_AXES.
 *   pair_axis: HOST array of rot_dim / 2 axes, each below `axes`; with
 *   TB_PAIRS_AXIS each axis's pairs are consecutive.  rot_dim >= 2.
 *   norm: 0: z = x, and no part has a weight (eps and weight_offset are not used).
 *   TB_PAIRS_AXIS takes 16-byte pieces where every axis's pairs come in multiples of them.
 *   Everything else, errors too, as tb_head_norm_rotate.
 */
tb_status tb_head_norm_rotate_axes(int32_t n, const tb_head_part *parts, int64_t tokens, int64_t head_dim,
                                   int64_t rot_dim, tb_pairs pairs, int32_t axes, const int64_t *positions,
                                   const uint8_t *pair_axis, const double *freqs, int32_t norm, float eps,
                                   float weight_offset, tb_dtype dtype, void *stream);

/*
 * tb_debug_set_wait_polls -- bound, in polls about 0.1 us apart, of the
 * forward kernels' internal waits (a decode streamer waiting for the x . V
 * products of its launch; a k-slice of a split prefill tile waiting for the
 * tile's other slices); default 1 << 20 (about 0.1 s).  It applies to
 * launches enqueued after the call, process-wide.  For tests of the timeout
 * path: 0 makes every such wait give up at once, so word 2 of the workspace
 * is set and y is NaN, with every kernel exiting normally.
 *   polls >= 0.  Errors: TB_ERR_INVALID_ARGUMENT.  Host-only.
 */
tb_status tb_debug_set_wait_polls(int32_t polls);

/* Static description of a status code. */
const char *tb_status_string(tb_status status);

/* Description of the last failure on the calling thread ("" if none). */
const char *tb_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* TB_H */
