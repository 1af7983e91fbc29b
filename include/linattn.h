/*
 * linattn.h -- C ABI of the GB300 (sm_103a) kernelised linear-attention
 * library (liblinattn.so).
 *
 * The operation ("Linear Attention", generalised-kernel equations and the
 * causal running statistics; "Story of Attention - Part 5: Linear Attention:
 * Kernels, Decay, and Gating", section 1a):
 *
 *   phi(x)  = elu(x) + 1   (alpha = 1), applied elementwise to q and k only
 *   non-causal   y_i = phi(q_i)^T [sum_j phi(k_j) v_j^T] / phi(q_i)^T [sum_j phi(k_j)]
 *   causal       S_t = g S_{t-1} + phi(k_t) v_t^T,  z_t = g z_{t-1} + phi(k_t),
 *                y_t = phi(q_t)^T S_t / phi(q_t)^T z_t      (update, then read)
 *
 * with an optional per-head scalar decay g ("Linear Attention: Removing the
 * Softmax Buys Associativity", the forget-gate passage; Part 5, section 4
 * recurrent form), g = 1 when no decay is given.  There is no 1/sqrt(d)
 * scaling and no epsilon in the denominator (phi > 0 makes it positive).
 *
 * Conventions shared by every entry point
 *   - All tensor pointers are DEVICE pointers owned by the caller (except
 *     la_forward_host's, which are host pointers); the library never frees
 *     or retains them after the call is enqueued.
 *   - Sequences are row-major contiguous [B][H][N][d] (d fastest); decode
 *     inputs are [B][H][d]; states S are [B][H][d][d] with S[a][c],
 *     a = key-feature index, c = value index; normalisers z are [B][H][d].
 *   - q, k, v and out share one dtype (`dtype`); outputs are rounded to it
 *     with round-to-nearest-even.  Accumulation is always fp32.
 *   - Every call is asynchronous on `stream` (a cudaStream_t; NULL = the
 *     legacy default stream) and performs no implicit synchronisation.
 *     Arguments are validated on the host before anything is enqueued; a
 *     rejected call enqueues nothing.
 *   - Calls are thread-safe.  The library's only global mutable state is a
 *     per-device status word written by kernels that detect a device-side
 *     problem (a bounded wait that ran out); read it with
 *     la_check_device_status().
 */
#ifndef LINATTN_H
#define LINATTN_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same underlying type as cudaStream_t, so that a cudaStream_t (or
 * torch.cuda.Stream.cuda_stream) can be passed directly. */
typedef struct CUstream_st *la_stream_t;

typedef enum {
    LA_OK = 0,
    LA_ERR_INVALID_ARG = 1,  /* null pointer, bad size, bad decay, ...      */
    LA_ERR_UNSUPPORTED = 2,  /* valid request this build cannot run          */
    LA_ERR_CUDA = 3,         /* a CUDA runtime call or launch failed         */
    LA_ERR_NO_MEMORY = 4,    /* workspace allocation failed                  */
    LA_ERR_TIMEOUT = 5,      /* a device-side bounded wait gave up           */
    LA_ERR_INTERNAL = 6      /* a debug build's device-side index check failed */
} la_status;

typedef enum { LA_F32 = 0, LA_BF16 = 1 } la_dtype;

/* Method variant for la_forward_variant / la_decode_step_variant. */
typedef enum { LA_PHI_ELU1 = 0, LA_PHI_IDENTITY = 1 } la_feature_map;
typedef struct {
    int feature_map; /* LA_PHI_ELU1: phi(x) = elu(x) + 1 (the default);
                        LA_PHI_IDENTITY: phi(x) = x                         */
    int normalise;   /* 1: divide by phi(q)^T z (the default); 0: no
                        denominator                                         */
} la_variant;

/* Largest head dimension accepted by any entry point. */
#define LA_MAX_D 256
/* Largest number of heads for which a per-head decay can be given. */
#define LA_MAX_DECAY_HEADS 1024

/*
 * la_forward -- full-sequence linear attention.
 *
 * Defined by the non-causal form phi(Q)[phi(K)^T V] / phi(Q)[phi(K)^T 1]
 * ("Story of Attention - Part 5", section 1a, matrix form) when causal == 0,
 * and by the causal running-state recurrence (same section, causal form;
 * "Linear Attention", cumulative running statistics) when causal == 1.
 *
 *   q, k, v  [B][H][N][d] device, dtype `dtype`, read only.
 *   out      [B][H][N][d] device, dtype `dtype`, written; may not alias
 *            q, k or v.
 *   B, H, N  >= 0 (B*H*N == 0 is a no-op returning LA_OK, and then q, k,
 *            v, out may be NULL); d in 1..LA_MAX_D.
 *   causal   0 or 1.
 *   decay    HOST array of H floats g_h in [0, 1] (read during the call, not
 *            retained), or NULL for g = 1.  Only valid with causal == 1:
 *            the pages define decay for the recurrence only, so a decay with
 *            causal == 0 is LA_ERR_INVALID_ARG.
 *   dtype    LA_F32 or LA_BF16.  fp32 inputs run on the fp32 CUDA-core path
 *            (no TF32); bf16 inputs with d in {64, 128} run on the tcgen05
 *            tensor-core kernels, other d on the CUDA-core path.
 *
 * Workspace: the tensor-core kernels, and the CUDA-core kernels when they
 * cut a sequence into segments (or reduce a non-causal state), need a small
 * stream-ordered scratch (per-segment states and flags), allocated with
 * cudaMallocAsync on `stream` and freed with cudaFreeAsync on the same
 * stream; LA_ERR_NO_MEMORY if that fails.
 */
la_status la_forward(const void *q, const void *k, const void *v, void *out,
                     int B, int H, int N, int d, int causal,
                     const float *decay, la_dtype dtype, la_stream_t stream);

/*
 * la_forward_ex -- la_forward with explicit kernel selection, for tests and
 * measurement.  `path`: 0 = automatic (what la_forward does), 1 = force the
 * fp32 CUDA-core kernels (any dtype), 2 = force the tensor-core kernels
 * (LA_ERR_UNSUPPORTED where they do not apply).  `segment_chunks`: 0 =
 * automatic, else the number of chunks per sequence segment that one CTA
 * takes (sequence parallelism inside a head; chunks of 128 tokens on the
 * tensor cores, of 32 on the CUDA cores).
 */
la_status la_forward_ex(const void *q, const void *k, const void *v,
                        void *out, int B, int H, int N, int d, int causal,
                        const float *decay, la_dtype dtype, int path,
                        int segment_chunks, la_stream_t stream);

/*
 * la_forward_host -- la_forward on HOST buffers (the one entry point whose
 * tensors are host pointers).  The pages define only the operation (as for
 * la_forward); moving the data to and from the GPU has no counterpart there.
 * The call copies q, k, v to a caller-provided device workspace, runs the
 * forward there and copies out back, split into at most 4 groups of heads so
 * that the host-to-device copy of one group, the kernels of the one before
 * and the device-to-host copy of the one before that overlap (two copy
 * streams owned by the library, one per direction, created on first use).
 *
 *   q, k, v   [B][H][N][d] host, dtype `dtype`, read only.  Page-locked
 *             memory (cudaHostAlloc, cudaHostRegister, torch pin_memory)
 *             gives asynchronous full-speed copies; pageable memory works,
 *             but the CUDA driver stages its copies and the call then blocks.
 *   out       [B][H][N][d] host, written; may not alias q, k or v.
 *   B, H, N, d, causal, decay, dtype   as la_forward (decay is a host
 *             array of H floats, read during the call).
 *   workspace device buffer, 256-byte aligned, of at least
 *             la_forward_host_workspace_bytes(B, H, N, d, dtype) bytes,
 *             owned by the caller; it holds the device copies of q, k, v and
 *             out and must not be used by anything else until `stream` has
 *             passed the call.
 *   stream    the copies start after the work already enqueued on `stream`;
 *             `stream` continues only after the last output copy, so out is
 *             complete once `stream` reaches work enqueued after the call
 *             (e.g. cudaStreamSynchronize(stream)).
 *
 * Errors: validation as la_forward (LA_ERR_INVALID_ARG also for a missing,
 * unaligned or too small workspace); a failure part-way through returns its
 * status with `stream` still ordered after the copies already enqueued, and
 * out unspecified.  Calls on one device are serialised on the host while
 * they enqueue (the copy streams and their events are shared).
 */
la_status la_forward_host(const void *q, const void *k, const void *v,
                          void *out, int B, int H, int N, int d, int causal,
                          const float *decay, la_dtype dtype, void *workspace,
                          size_t workspace_bytes, la_stream_t stream);

/* Device workspace bytes la_forward_host needs for this problem (0 for an
 * invalid shape or dtype). */
size_t la_forward_host_workspace_bytes(int B, int H, int N, int d,
                                       la_dtype dtype);

/*
 * la_decode_step -- one recurrent decode step per head: with
 * phi_k = phi(k), S <- S + phi_k v^T, z <- z + phi_k, then
 * out = phi(q)^T S / phi(q)^T z  (update, then read; "Linear Attention",
 * running statistics and per-token inference cost O(d^2) arithmetic and
 * O(d^2) memory, independent of history).
 *
 *   S        [B][H][d][d] fp32 device, read and written in place.
 *   z        [B][H][d]    fp32 device, read and written in place.
 *   q, k, v  [B][H][d] device, dtype `dtype`, read only.
 *   out      [B][H][d] device, dtype `dtype`, written.
 *   B, H >= 0 (B*H == 0 is a no-op), d in 1..LA_MAX_D.
 * The caller owns the recurrent state; saving and restoring S and z is how
 * a decode is checkpointed and resumed.
 */
la_status la_decode_step(float *S, float *z, const void *q, const void *k,
                         const void *v, void *out, int B, int H, int d,
                         la_dtype dtype, la_stream_t stream);

/*
 * la_decode_step_ex -- la_decode_step with a per-head decay g:
 * S <- g S + phi_k v^T, z <- g z + phi_k, then out = phi(q)^T S / phi(q)^T z
 * (the recurrence with the forget-gate passage's scalar g; "Story of
 * Attention - Part 5", section 4, recurrent form S_t = g S_{t-1} + k_t v_t^T).
 *   decay    HOST array of H floats in [0, 1] (read during the call), or NULL
 *            for g = 1 (then identical to la_decode_step).
 * Other arguments, layouts and errors as la_decode_step; LA_ERR_UNSUPPORTED
 * for a decay over more than LA_MAX_DECAY_HEADS heads.
 */
la_status la_decode_step_ex(float *S, float *z, const void *q, const void *k,
                            const void *v, void *out, int B, int H, int d,
                            const float *decay, la_dtype dtype,
                            la_stream_t stream);

/*
 * la_forward_causal_state -- the causal form of la_forward that also returns
 * the final state: S_N = sum_t g^(N-1-t) phi(k_t) v_t^T and z_N likewise,
 * i.e. the running statistics after the last token ("Linear Attention",
 * running statistics; the state an RNN-style decode continues from).  It is
 * the prefill half of a prefill -> decode hand-off: la_decode_step(_ex) on S
 * and z then continues the same sequences.
 *   q, k, v, out, B, H, N, d, decay, dtype   as la_forward with causal = 1.
 *   S        [B][H][d][d] fp32 device, written (S[a][c]: a key feature, c
 *            value column; the layout la_decode_step reads); 16-byte aligned.
 *   z        [B][H][d] fp32 device, written.
 * N == 0 writes the zero state.  Errors as la_forward, plus
 * LA_ERR_INVALID_ARG for a NULL or unaligned S or a NULL z.
 */
la_status la_forward_causal_state(const void *q, const void *k, const void *v,
                                  void *out, float *S, float *z, int B, int H,
                                  int N, int d, const float *decay,
                                  la_dtype dtype, la_stream_t stream);

/*
 * la_forward_variant / la_decode_step_variant -- la_forward_ex (automatic
 * kernel and segment choice) and la_decode_step_ex with the feature map and
 * the normaliser selectable.  With {LA_PHI_IDENTITY, 0} and a decay this is
 * retention ("Story of Attention - Part 5", section 4: recurrent form
 * S_t = g S_{t-1} + k_t v_t^T, o_t = q_t S_t; parallel form (Q K^T (.) D) V
 * with D_ij = g^(i-j) for i >= j); with {LA_PHI_ELU1, 0} linear attention
 * without the denominator.
 *   variant  NULL for {LA_PHI_ELU1, 1} (then identical to la_forward_ex /
 *            la_decode_step_ex); LA_ERR_INVALID_ARG for a feature_map other
 *            than the two above or a normalise other than 0 or 1.
 * Without the normaliser z is still carried (and, for the decode step,
 * updated) but not used.  Other arguments and errors as la_forward and
 * la_decode_step_ex.
 */
la_status la_forward_variant(const void *q, const void *k, const void *v,
                             void *out, int B, int H, int N, int d, int causal,
                             const float *decay, la_dtype dtype,
                             const la_variant *variant, la_stream_t stream);
la_status la_decode_step_variant(float *S, float *z, const void *q,
                                 const void *k, const void *v, void *out, int B,
                                 int H, int d, const float *decay,
                                 la_dtype dtype, const la_variant *variant,
                                 la_stream_t stream);

/*
 * la_forward_gated / la_decode_step_gated -- the causal recurrence with a
 * data-dependent scalar gate per token and head instead of a fixed decay:
 * S_t = alpha_t S_{t-1} + phi(k_t) v_t^T, z_t = alpha_t z_{t-1} + phi(k_t),
 * y_t = phi(q_t)^T S_t / phi(q_t)^T z_t ("Linear Attention", GLA's
 * S_t = G_t (.) S_{t-1} + k_t v_t^T with G_t = alpha_t, the scalar forget
 * gate alpha_t of "Story of Attention - Part 5", section 7).
 *   gates    DEVICE fp32, [B][H][N] for la_forward_gated (alpha of every
 *            token) or [B][H] for la_decode_step_gated (alpha of this step's
 *            token), values in [0, 1].  The values are not checked (they live
 *            on the device); outside [0, 1] the results are unspecified.
 *   variant  as la_forward_variant (NULL: elu(x) + 1 with the normaliser).
 * Other arguments as la_forward (causal) and la_decode_step.  The forward
 * runs where la_forward would (bf16 with d in {64, 128}: the tcgen05
 * kernels; otherwise the fp32 CUDA-core kernels); the decode step is the
 * same kernel as la_decode_step.
 */
la_status la_forward_gated(const void *q, const void *k, const void *v,
                           void *out, const float *gates, int B, int H, int N,
                           int d, la_dtype dtype, const la_variant *variant,
                           la_stream_t stream);
la_status la_decode_step_gated(float *S, float *z, const void *q, const void *k,
                               const void *v, void *out, const float *gates,
                               int B, int H, int d, la_dtype dtype,
                               const la_variant *variant, la_stream_t stream);

/*
 * la_decode_step_delta -- one delta-rule decode step per head ("Story of
 * Attention - Part 5", section 7, Gated DeltaNet / Delta Attention: one step
 * of online gradient descent on 1/2 ||S_{t-1} k_t - v_t||^2, with the scalar
 * forget gate alpha_t):
 *   S_t = alpha S_{t-1} + beta (v_t - alpha S_{t-1} k_t) k_t^T,  o_t = S_t q_t
 * in the page's orientation, where S k is the value stored for key k.  No
 * feature map and no normaliser (the page's form; a model normalises k).
 *   S        [B][H][d][d] fp32 device, read and written in place, stored as
 *            in la_decode_step: S[a][c] with a the key feature and c the
 *            value column (the transpose of the page's S).
 *   q, k, v  [B][H][d] device, dtype `dtype`, read only.
 *   out      [B][H][d] device, dtype `dtype`, written.
 *   beta     DEVICE fp32 [B][H]: this step's update strength per head.
 *   alpha    DEVICE fp32 [B][H]: this step's forget gate per head, or NULL
 *            for alpha = 1 (plain DeltaNet).  beta and alpha are not checked
 *            (the page's ranges are beta in [0, 1], alpha in (0, 1)).
 *   B, H >= 0 (B*H == 0 is a no-op), d in 1..LA_MAX_D.
 */
la_status la_decode_step_delta(float *S, const void *q, const void *k,
                               const void *v, void *out, const float *beta,
                               const float *alpha, int B, int H, int d,
                               la_dtype dtype, la_stream_t stream);

/*
 * la_forward_delta -- the delta rule of la_decode_step_delta over whole
 * sequences ("Story of Attention - Part 5", section 7): for t = 1..N,
 *   S_t = alpha_t S_{t-1} + beta_t (v_t - alpha_t S_{t-1} k_t) k_t^T,
 *   o_t = S_t q_t,
 * with one beta and one alpha per token and head.  The pages name a
 * chunkwise form of this rule but do not give it; this is the recurrent form
 * on CUDA cores in fp32 (value columns of a head in parallel, tokens in order).
 *   q, k, v  [B][H][N][d] device, dtype `dtype`, read only.
 *   out      [B][H][N][d] device, dtype `dtype`, written (o_t).
 *   beta     DEVICE fp32 [B][H][N]: each token's update strength.
 *   alpha    DEVICE fp32 [B][H][N]: each token's forget gate, or NULL for
 *            alpha = 1 (plain DeltaNet).  beta and alpha are not checked.
 *   S        DEVICE fp32 [B][H][d][d] (S[a][c], a key feature, as in
 *            la_decode_step_delta) holding the state before the first token;
 *            it receives the state after the last one, so that
 *            la_decode_step_delta continues the sequences.  NULL: start from
 *            zero and return no state.
 *   B, H, N >= 0 (B*H*N == 0 is a no-op), d in 1..LA_MAX_D.
 */
la_status la_forward_delta(const void *q, const void *k, const void *v, void *out,
                           const float *beta, const float *alpha, float *S, int B,
                           int H, int N, int d, la_dtype dtype, la_stream_t stream);

/*
 * Strides in elements of a [B][H][N][d] tensor whose last dimension is
 * contiguous.  Every row starts at data + i_b*b + i_h*h + i_n*n.  A
 * dimension of an input may have stride 0 (a broadcast input); the rows of a
 * written tensor may not overlap.
 */
typedef struct {
    long long b, h, n;
} la_strides;

/*
 * The position rotation of la_qk_norm_rope.  Pair i < rotary_dim / 2 of a
 * row at position p is turned by the angle p * frequencies[i] (radians).
 */
typedef struct {
    const double *frequencies; /* HOST array of rotary_dim / 2 values in
                                  [-1e9, 1e9], read during the call         */
    int rotary_dim;            /* even, 0..d; 0: no rotation                 */
    int interleaved;           /* 0: pair i is (x[i], x[i + rotary_dim / 2]);
                                  1: pair i is (x[2i], x[2i + 1])            */
    const void *positions;     /* DEVICE integers, one per batch entry and
                                  token, or NULL: token n is at position n   */
    int position_bytes;        /* 4 or 8 (signed); ignored without positions */
    long long position_stride_b, position_stride_n; /* in elements, >= 0     */
    long long offset;          /* added to every position                    */
} la_rope;

/*
 * la_qk_norm_rope -- queries and keys as the forward and decode entry points
 * take them, out of a projection's output, in one pass: each row (one token
 * of one head, d values) is divided by its root mean square, scaled by a
 * weight per feature and rotated by its position,
 *   n = x / sqrt(mean(x^2) + eps),  u = w (.) n,
 *   (y1, y2) = (u1 cos t - u2 sin t, u2 cos t + u1 sin t)  for each pair,
 * features from rotary_dim on pass without rotation (u as it is, whatever is in
 * the others).  The pages normalise k
 * for the delta rule and rotate q and k in retention models without giving
 * the formulas; these are the usual ones.  With the identity feature map and
 * no normaliser, <y_q, y_k> then depends on positions by their difference.
 *
 *   q, k       [B][Hq][N][d] and [B][Hk][N][d] device, dtype `dtype`, read only.
 *   q_out, k_out   like q and k, written; may be q and k themselves with the
 *              same strides, otherwise may not alias an input or each other.
 *   strides    4 strides, of q, k, q_out, k_out, or NULL: all contiguous
 *              [B][H][N][d].  A token-major projection [B][N][H*d] is
 *              {N*H*d, d, H*d}: the call then turns the layout as well.
 *   q_weight, k_weight   [d] device, dtype `weight_dtype`, or NULL for ones.
 *   norm       1, or 0: no normalisation (u = x; the weights must be NULL).
 *   eps        > 0 and finite (ignored without norm).
 *   rope       the rotation, or NULL for none.
 *   B, N, Hq, Hk >= 0 (Hq == 0 or Hk == 0 leaves that side out; its pointers
 *              may be NULL), d in 1..LA_MAX_D.
 * A decode step is N == 1 with one position per sequence.  Sums of squares
 * are fp32; the angle is exact in the position (64-bit fixed-point turns), so
 * far positions lose nothing.  A row's result does not depend on strides or
 * alignment.  Rows may be read in whole 16-byte units of memory: neighbouring
 * bytes of a unit that holds part of a row may be read and are not used.  One
 * kernel, no workspace.
 */
la_status la_qk_norm_rope(const void *q, const void *k, void *q_out, void *k_out,
                          const la_strides *strides, const void *q_weight,
                          const void *k_weight, int norm, float eps,
                          const la_rope *rope, int B, int Hq, int Hk, int N, int d,
                          la_dtype dtype, la_dtype weight_dtype, la_stream_t stream);

/*
 * la_backward_qk_norm_rope -- gradients of la_qk_norm_rope: with g the
 * gradient of a row's output turned back by its angle,
 *   dw = sum over rows of g (.) n,
 *   dx = (w (.) g - n mean(n (.) w (.) g)) / sqrt(mean(x^2) + eps).
 *   dq_out, dk_out   gradients of the outputs, like q and k, read only.
 *   q, k       the forward's inputs (may be NULL with norm == 0, whose
 *              gradient does not need them).
 *   dq, dk     gradients of the inputs, written; may be dq_out and dk_out
 *              themselves with the same strides, otherwise no aliasing.
 *   dq_weight, dk_weight   [d] fp32 device, written, or NULL: not computed.
 *              Summed in a fixed order (repeated calls are bit-identical) with
 *              compensation: off by at most 19 * 2^-24 sum |g (.) n| over the
 *              rows, however many, and the error of the terms themselves.
 *   strides    6 strides, of dq_out, dk_out, q, k, dq, dk, or NULL: contiguous.
 * Other arguments as la_qk_norm_rope (the same values as in the forward).
 *   workspace  device buffer for the weight gradients' partial sums, 16-byte
 *              aligned, of la_backward_qk_norm_rope_workspace_bytes(d) bytes, not
 *              used by anything else until `stream` has passed the call; or
 *              NULL: allocated stream-ordered (LA_ERR_NO_MEMORY if that fails).
 *              Without weight gradients none is needed.
 * B*N == 0 writes zero weight gradients.
 */
la_status la_backward_qk_norm_rope(const void *dq_out, const void *dk_out, const void *q,
                                   const void *k, void *dq, void *dk, float *dq_weight,
                                   float *dk_weight, const la_strides *strides,
                                   const void *q_weight, const void *k_weight, int norm,
                                   float eps, const la_rope *rope, int B, int Hq, int Hk,
                                   int N, int d, la_dtype dtype, la_dtype weight_dtype,
                                   void *workspace, size_t workspace_bytes,
                                   la_stream_t stream);

/* Workspace bytes that la_backward_qk_norm_rope needs at most on the current
 * device for head dimension d (0 for an invalid d). */
size_t la_backward_qk_norm_rope_workspace_bytes(int d);

/* What a gate tensor of the per-channel recurrence holds: the gate a itself,
 * its logarithm (a = exp(g)) or its logit (a = 1 / (1 + exp(-g))). */
typedef enum { LA_GATE_VALUE = 0, LA_GATE_LOG = 1, LA_GATE_LOGIT = 2 } la_gate;

/* Strides in elements of a [B][N][C] tensor whose last dimension is
 * contiguous; a dimension of an input may have stride 0. */
typedef struct {
    long long b, n;
} la_seq_strides;

/*
 * la_forward_recurrence -- the gated linear recurrence with a gate per
 * channel ("Linear Attention", GLA's S_t = G_t (.) S_{t-1} + ..., on a vector
 * state; the z_t of the running statistics under vector gates):
 *   h_t = a_t (.) h_{t-1} + x_t                 (complement == 0)
 *   h_t = a_t (.) h_{t-1} + (1 - a_t) (.) x_t   (complement == 1)
 * for t = 1..N, with out_t = h_t.
 *   x          [B][N][C] device, dtype `dtype`, read only.
 *   gates      [B][N][C] device, dtype `gate_dtype` (LA_F32, or `dtype`),
 *              holding a_t as `gate` says.  Not checked; values outside
 *              [0, 1] (positive logarithms) follow the formula while the
 *              products of gates stay finite.  A gate of 0 (logarithm or
 *              logit -inf) starts a new sequence; a gate of 1 (0, +inf) with
 *              x = 0, or with complement any finite x, keeps the state.
 *   h0         [B][C] fp32 device, the state before the first token, or NULL
 *              for zero.
 *   out        [B][N][C] device, dtype `dtype`, written; may be x itself with
 *              the same strides, otherwise no aliasing.
 *   h_last     [B][C] fp32 device, written with the state after the last
 *              token (unrounded), or NULL; may be h0 itself, otherwise no
 *              aliasing.
 *   strides    3 strides, of x, gates, out, or NULL: contiguous.
 *   B, N, C >= 0 (B*C == 0 is a no-op; N == 0 copies h0 to h_last); B * C / 32,
 *              C / 32 rounded up, below 2^24, else LA_ERR_UNSUPPORTED.
 *   workspace  device buffer, 16-byte aligned, of
 *              la_recurrence_workspace_bytes(B, C, dtype) bytes, not used by
 *              anything else until `stream` has passed the call; or NULL: a
 *              call that needs one (few channels, a long sequence) allocates it
 *              stream-ordered (LA_ERR_NO_MEMORY if that fails).
 * States and gate products are fp32.  Sequences are cut along N (the pieces
 * are joined in a fixed order: repeated calls are bit-identical).
 * A non-finite value stays within its sequence and channel.  Rows are read in
 * whole 16-byte units of memory: neighbouring bytes of a unit that holds part
 * of a row may be read and are not used.
 */
la_status la_forward_recurrence(const void *x, const void *gates, const float *h0,
                                void *out, float *h_last, const la_seq_strides *strides,
                                int B, int N, int C, la_gate gate, int complement,
                                la_dtype dtype, la_dtype gate_dtype, void *workspace,
                                size_t workspace_bytes, la_stream_t stream);

/* Workspace bytes that la_forward_recurrence and la_backward_recurrence need
 * at most for B sequences of C channels (0: none, or invalid arguments). */
size_t la_recurrence_workspace_bytes(int B, int C, la_dtype dtype);

/*
 * la_backward_recurrence -- gradients of la_forward_recurrence.  With c_t the
 * factor of x_t (1, or 1 - a_t) and, from the last token backwards,
 *   g_t = dout_t + a_{t+1} (.) g_{t+1}   (g_N = dout_N + dh_last),
 *   dx_t = c_t (.) g_t,   dh0 = a_1 (.) g_1,
 *   dgates_t = s_t (.) g_t (.) (h_{t-1} - x_t [complement]),
 * s_t = 1, a_t or a_t (1 - a_t) for a gate given as value, logarithm, logit.
 *   dout       [B][N][C] device, dtype `dtype`: the gradient of out.
 *   gates, h0  as in the forward.
 *   out        [B][N][C] device, dtype `dtype`: what the forward wrote (the
 *              states h_t, rounded to dtype, that dgates reads).
 *   x          the forward's input; needed with complement only, else NULL.
 *   dh_last    [B][C] fp32 device: gradient of h_last, or NULL for zero.
 *   dx         [B][N][C] device, dtype `dtype`, written; may be dout itself
 *              with the same strides.
 *   dgates     [B][N][C] device, dtype `gate_dtype`, written: the gradient of
 *              the gate tensor as given (value, logarithm or logit).
 *   dh0        [B][C] fp32 device, written, or NULL; may be dh_last itself,
 *              otherwise no aliasing.
 *   strides    6 strides, of dout, gates, out, x, dx, dgates, or NULL:
 *              contiguous.
 * Other arguments as la_forward_recurrence.  N == 0 copies dh_last to dh0.
 */
la_status la_backward_recurrence(const void *dout, const void *gates, const void *out,
                                 const void *x, const float *h0, const float *dh_last,
                                 void *dx, void *dgates, float *dh0,
                                 const la_seq_strides *strides, int B, int N, int C,
                                 la_gate gate, int complement, la_dtype dtype,
                                 la_dtype gate_dtype, void *workspace,
                                 size_t workspace_bytes, la_stream_t stream);

/*
 * la_decode_step_recurrence -- one token of la_forward_recurrence.
 *   h          [B][C] fp32 device, the state, read.
 *   h_out      [B][C] fp32 device, the new state, written; h itself for an
 *              update in place (or an fp32 x or gates laid out as h is).
 *   x, gates   [B][C] device; out [B][C] device, dtype `dtype`, written (h_out
 *              rounded); may be x itself with the same stride.
 *   strides    3 strides between batch entries, of x, gates, out, or NULL: C.
 * Other arguments as la_forward_recurrence.
 */
la_status la_decode_step_recurrence(const float *h, float *h_out, const void *x,
                                    const void *gates, void *out, const long long *strides,
                                    int B, int C, la_gate gate, int complement,
                                    la_dtype dtype, la_dtype gate_dtype,
                                    la_stream_t stream);

/*
 * A paged cache of keys and values: pages of page_size tokens each, in any
 * order, and a table that names the pages of each sequence.  Position p of
 * sequence b is in page table[b][p / page_size], slot p % page_size.
 */
typedef struct {
    void *k, *v;         /* DEVICE [pages][Hk][page_size][d], dtype `dtype`  */
    la_strides k_strides, v_strides; /* b: from page to page, h: from head to
                            head, n: from slot to slot; d is contiguous      */
    const int *table;    /* DEVICE [B][max_pages] page numbers; an entry that
                            is not in 0..pages-1 is no page                  */
    long long table_stride; /* elements from sequence to sequence           */
    const int *lengths;  /* DEVICE [B]: tokens of each sequence before this
                            call's; negative: a place of the batch that is
                            not in use                                       */
    int pages, page_size, max_pages; /* max_pages * page_size <= 2^30       */
} la_cache;

/*
 * la_append_cache -- T new tokens per sequence into a paged cache, keys and
 * queries rotated by their position on the way (the rotation of
 * la_qk_norm_rope).  Token t of sequence b is at position p = lengths[b] + t;
 * its key and value go to the cache's place for p, in all heads.
 *   q          [B][Hq][T][d] device, dtype `dtype`, read only; q_out likewise,
 *              written (every row): the queries as la_decode_step_paged takes
 *              them.  q_out may be q itself with the same strides.
 *   k, v       [B][Hk][T][d] device, dtype `dtype`, read only.
 *   cache      k and v are written at the new tokens' places, nowhere else.
 *   counts     DEVICE [B]: how many of the T tokens sequence b really has
 *              (a padded batch of prompts), or NULL: all T.
 *   strides    4 strides, of q, k, v, q_out, or NULL: contiguous.
 *   rope       the rotation, by p + offset (rope->positions must be NULL), or
 *              NULL for none.  Values, and features from rotary_dim on, pass
 *              bit for bit.
 *   B, Hq, Hk, T >= 0 (Hq == 0 leaves the queries out), Hq + 2 Hk < 2^31 - 4097,
 *              d in 1..LA_MAX_D.
 * A token whose place has no page (past the table, a table entry that is no
 * page) or whose sequence is not in use is not stored.  Two sequences that
 * append to one page at one slot leave either's token there.  Angles are exact
 * in the position.  One kernel, no workspace.
 */
la_status la_append_cache(const void *q, const void *k, const void *v, void *q_out,
                          const la_cache *cache, const int *counts,
                          const la_strides *strides, const la_rope *rope, int B, int Hq,
                          int Hk, int T, int d, la_dtype dtype, la_stream_t stream);

/*
 * la_decode_step_paged -- softmax attention of a sequence's newest T tokens
 * over its paged cache, the softmax layer of a stack that has a few of them
 * between its linear ones:
 *   o_t = sum_j exp(scale q_t . k_j) v_j / sum_j exp(scale q_t . k_j)
 * over the keys j <= p_t = lengths[b] + t, with window > 0 only those with
 * j > p_t - window.  The call's own keys are in the cache already
 * (la_append_cache with the same lengths): a step appends, attends, and adds T
 * to lengths once all layers are done.
 *   q          [B][Hq][T][d] device, dtype `dtype`, read only.
 *   out        [B][Hq][T][d] device, dtype `dtype`, written; may alias neither q
 *              nor the cache.
 *   cache      read only.  A key whose place has no page is left out.  Pages
 *              that lie wholly before all windows are not read and need no
 *              table entry.
 *   strides    2 strides, of q and out, or NULL: contiguous.
 *   scale      finite; usually 1 / sqrt(d).
 *   window     0: all keys.
 *   B, Hq, Hk, T >= 0, T <= 2^20, Hq a multiple of Hk (query head h reads
 *              head h / (Hq / Hk) of the cache), d in 1..LA_MAX_D.
 *   workspace  device buffer, 16-byte aligned, of
 *              la_decode_step_paged_workspace_bytes(...) bytes, not used by
 *              anything else until `stream` has passed the call; or NULL:
 *              allocated stream-ordered (LA_ERR_NO_MEMORY if that fails).
 * A query without keys (a sequence not in use) gives zeros.  What lies in the
 * cache outside the keys that a query looks at does not reach its output,
 * whatever it is.  Scores, the softmax's maximum and sum and the outputs are
 * fp32; with bf16 the weights are rounded to bf16 for their product with the
 * values (the sum is of the rounded ones).  The work is cut into equal pieces
 * along all sequences' lengths and joined in a fixed order: repeated calls are
 * bit-identical.  Two kernels.
 */
la_status la_decode_step_paged(const void *q, void *out, const la_cache *cache,
                               const la_strides *strides, float scale, int window,
                               int B, int Hq, int Hk, int T, int d, la_dtype dtype,
                               void *workspace, size_t workspace_bytes,
                               la_stream_t stream);

/* Workspace bytes that la_decode_step_paged needs at most on the current
 * device, whatever B and the lengths are (0 for invalid arguments). */
size_t la_decode_step_paged_workspace_bytes(int Hq, int Hk, int T, int d,
                                            la_dtype dtype);

/*
 * la_forward_cross -- linear attention of N queries per head to M keys and
 * values of another sequence, an encoder's (the non-causal form of la_forward
 * with two lengths, shared heads and padding):
 *   S = sum_j phi(k_j) v_j^T,  z = sum_j phi(k_j)   over j < lengths[b],
 *   y_i = phi(q_i)^T S / phi(q_i)^T z.
 *   q          [B][Hq][N][d] device, dtype `dtype`, read only.
 *   k, v       [B][Hk][M][d] device, dtype `dtype`, read only; what lies behind
 *              a sequence's length is not used, whatever it is.
 *   out        [B][Hq][N][d] device, dtype `dtype`, written.
 *   S, z       [B][Hk][d][d] and [B][Hk][d] fp32 device, written: the states,
 *              as la_decode_step has them (S[a][c], a the key feature).  They
 *              are all that la_decode_step_cross and la_backward_cross need of
 *              the encoder's side and of the forward.
 *   lengths    DEVICE [B]: tokens of each sequence's keys (taken as 0 below 0
 *              and M above M), or NULL: M.
 *   strides    4 strides, of q, k, v, out, or NULL: contiguous.
 *   B, Hq, Hk, N, M >= 0, Hq a multiple of Hk (query head h reads the state of
 *              head h / (Hq / Hk)), d in 1..LA_MAX_D; N, M <= 2^31 - 256.
 *   variant    as la_forward_variant.
 *   workspace  device buffer, 16-byte aligned, of la_cross_workspace_bytes(...,
 *              0) bytes, not used by anything else until `stream` has passed
 *              the call; or NULL: allocated stream-ordered (LA_ERR_NO_MEMORY if
 *              that fails).
 * A denominator of exactly 0 (a sequence without keys) gives zeros.  Values that
 * are not finite act as in the formulas, but with bf16 a result may be NaN
 * where the formula has an infinity.  No output may alias another tensor.  The
 * parts of a sum are joined in a fixed order: repeated calls are bit-identical.
 */
la_status la_forward_cross(const void *q, const void *k, const void *v, void *out,
                           float *S, float *z, const int *lengths,
                           const la_strides *strides, int B, int Hq, int Hk, int N,
                           int M, int d, const la_variant *variant, la_dtype dtype,
                           void *workspace, size_t workspace_bytes, la_stream_t stream);

/*
 * la_backward_cross -- gradients of la_forward_cross's `out` (S and z as
 * results of their own have none).  With f = phi(q_i), r = 1 / (f . z):
 *   t = r f . (S dy_i),  dphi(q_i) = r (S dy_i - t z),
 *   dS = sum r f dy_i^T,  dz = -sum r t f   over the queries of all heads that
 *   share the state,  dphi(k_j) = dS v_j + dz,  dv_j = dS^T phi(k_j).
 *   dout, dq   [B][Hq][N][d], dtype `dtype`: gradient of out, read; of q, written.
 *   dk, dv     [B][Hk][M][d], dtype `dtype`, written; 0 behind a sequence's
 *              length.
 *   S, z       what the forward wrote, read only.
 *   strides    7 strides, of dout, q, k, v, dq, dk, dv, or NULL: contiguous.
 *   workspace  as la_forward_cross, of la_cross_workspace_bytes(..., 1) bytes.
 * Other arguments as la_forward_cross (the same values as in the forward).
 * Where the denominator is 0 the gradients are 0.
 */
la_status la_backward_cross(const void *dout, const void *q, const void *k, const void *v,
                            const float *S, const float *z, const int *lengths, void *dq,
                            void *dk, void *dv, const la_strides *strides, int B, int Hq,
                            int Hk, int N, int M, int d, const la_variant *variant,
                            la_dtype dtype, void *workspace, size_t workspace_bytes,
                            la_stream_t stream);

/* Workspace bytes that la_forward_cross (backward == 0) or la_backward_cross
 * (1) needs at most on the current device (0: none, or invalid arguments). */
size_t la_cross_workspace_bytes(int B, int Hq, int Hk, int N, int M, int d,
                                la_dtype dtype, int backward);

/*
 * la_decode_step_cross -- a decoder's next token, or N of them, against the
 * states that la_forward_cross wrote once for the encoder's tokens: y =
 * phi(q)^T S / phi(q)^T z.  The states are read, not updated.
 *   q, out     [B][Hq][N][d] device, dtype `dtype`.
 *   strides    2 strides, of q and out, or NULL: contiguous.
 * Other arguments as la_forward_cross.  One kernel, no workspace.  fp32
 * throughout, but with bf16 and five or more tokens phi(q) and S may be rounded
 * to bf16 for their product, as in la_forward_cross.
 */
la_status la_decode_step_cross(const float *S, const float *z, const void *q, void *out,
                               const la_strides *strides, int B, int Hq, int Hk, int N,
                               int d, const la_variant *variant, la_dtype dtype,
                               la_stream_t stream);

/* Size of the fixed device scratch used by la_forward_causal_noalloc. */
#define LA_NOALLOC_SCRATCH_BYTES (16u << 20)

/*
 * la_forward_causal_noalloc -- the causal form of la_forward (bf16 only),
 * for callers that cannot allocate device memory: work recorded into a CUDA
 * graph whose capture forbids allocation, hosts that reserve all device
 * memory up front, and plug-in layers that are handed their buffers and may
 * not own allocations.  The pages have no counterpart of this entry point;
 * it exists only for such callers.
 *
 * Same arguments and meaning as la_forward with causal == 1 and
 * dtype == LA_BF16: q, k, v, out are caller-owned device tensors
 * [B][H][N][d] (16-byte aligned), d must be 64 or 128, `decay` is a host
 * array of H values in [0, 1] or NULL.  It runs the same tensor-core kernel,
 * but its workspace lives in a static device array of
 * LA_NOALLOC_SCRATCH_BYTES (16 MiB) that every GPU which loads the library's
 * causal kernels keeps until the process exits.  The call makes no
 * cudaMalloc/cudaFree or other allocating call.  It enqueues two kernels on
 * `stream`: a small zeroing kernel that clears the part of the scratch that
 * must start at zero (ticket counter and segment flags), then the forward,
 * launched with programmatic stream serialisation: it may run its set-up
 * while the zeroing kernel finishes and waits for it (griddepcontrol.wait)
 * before touching memory; stream capture records a programmatic edge
 * between the two kernel nodes.
 *   - Sequence segments are lengthened until the workspace fits the
 *     scratch; if it cannot fit even with one segment per head the call
 *     returns LA_ERR_UNSUPPORTED ("needs more workspace than ...") and
 *     enqueues nothing.  Other shapes or dtypes: LA_ERR_UNSUPPORTED.
 *   - The first call on each device looks up the scratch array's device
 *     address (cudaGetSymbolAddress) with that device current; make that
 *     first call before any stream capture.
 *   - All calls on a device share the one scratch array, which keeps the
 *     last call's contents.  Calls whose kernels can overlap on the GPU
 *     (different streams without ordering between them, or several host
 *     threads) race on it and give wrong results: order them.
 */
la_status la_forward_causal_noalloc(const void *q, const void *k,
                                    const void *v, void *out, int B, int H,
                                    int N, int d, const float *decay,
                                    la_stream_t stream);

/*
 * la_check_device_status -- synchronises `stream`, then reads and clears the
 * current device's status word.  Returns LA_ERR_TIMEOUT if a kernel gave up
 * on a bounded wait since the last check (its outputs are then not valid),
 * LA_ERR_INTERNAL if, in a library built with LA_DEBUG, a device-side index
 * check failed (la_last_error names the source line), LA_ERR_CUDA if the
 * synchronisation itself failed, else LA_OK.
 */
la_status la_check_device_status(la_stream_t stream);

/* Static, human-readable name of a status code. */
const char *la_status_string(la_status s);

/* Detail of the last failed call on the calling thread ("" if none). */
const char *la_last_error(void);

/* ABI version of this header: 1. */
int la_abi_version(void);

/* Number of kernels this library has enqueued in this process (all devices,
 * all streams) since it was loaded; for measurement and launch accounting. */
unsigned long long la_kernel_launch_count(void);

/*
 * Testing hooks.  The pages have no counterpart: these exist so that the
 * library's own tests can drive its failure paths without faulting a GPU.
 * Each applies to the calling thread only and is consumed by the next call
 * it affects.
 *
 * la_debug_inject_timeout -- the next d = 128 causal tensor-core launch
 * (la_forward and friends with bf16, d = 128, no gates) bounds every wait by
 * `wait_cycles` clock cycles (>= 4096) instead of about two seconds, and
 * segment `hold_segment` of every head never publishes the state it holds
 * (-1: all publish).  Segment s >= 1 holds the local state of segment s - 1
 * and publishes it when a segment after s needs it (s = 1 .. nseg - 2;
 * segment 0 and the last segment publish nothing).  The segments after
 * `hold_segment` then wait in vain and their waits run out: the launch records
 * LA_ERR_TIMEOUT in the device status word, every later wait of the launch
 * passes through, it finishes (outputs invalid) and la_check_device_status
 * reports LA_ERR_TIMEOUT.  LA_ERR_INVALID_ARG for wait_cycles < 4096.
 * A launch of la_forward_recurrence or la_backward_recurrence takes the hook
 * as well, whichever comes first: there, the first block of every thread-block
 * cluster never fetches its rows of round `hold_segment` (0 or 1, of the
 * first rounds; -1: fetches all).
 * So do la_decode_step_paged over pages of whole 16-key tiles (each warp never
 * fetches tile `hold_segment` of its own), and, where they run on the tensor
 * cores' tiles, la_forward_cross (its states), la_decode_step_cross and
 * la_backward_cross (both kernels): each block fetches nothing from its tile
 * `hold_segment` on.
 *
 * la_debug_fail_next_allocs -- the next `n` stream-ordered workspace
 * allocations of the forward kernels (tensor-core launches given no
 * workspace, and CUDA-core launches over more than one segment per head, or
 * non-causal), of the recurrence and of la_backward_qk_norm_rope (given no
 * workspace) fail: those calls return LA_ERR_NO_MEMORY and enqueue nothing,
 * la_backward_qk_norm_rope at most the zeros of a side without rows.
 * n = 0 clears the hook; LA_ERR_INVALID_ARG for n < 0.
 */
la_status la_debug_inject_timeout(long long wait_cycles, int hold_segment);
la_status la_debug_fail_next_allocs(int n);

#ifdef __cplusplus
}
#endif
#endif /* LINATTN_H */
