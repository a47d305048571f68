/*
 * gdn2.h -- C ABI of the MI355X (gfx950) Gated DeltaNet-2 chunked prefill
 * forward.
 *
 * The operation (FlashInfer chunk_gated_delta_rule2 documentation, recurrence
 * display equation): for every packed sequence and every value head, with a
 * K x V float32 state S,
 *
 *     S_t    = diag(exp(g_t)) S_{t-1}
 *     vnew_t = w_t * v_t - (beta_t * k_t)^T S_t
 *     S_t   += k_t vnew_t^T
 *     o_t    = scale * q_t^T S_t
 *
 * evaluated in 64-token chunks through the WY form (the chunked evaluation
 * the burn-gdn2 README "Fused CUDA kernels" section and the FlashRT card's
 * 64-token WY chain describe), returning the output and the final state.
 *
 * All entry points are plain C: no exceptions cross the boundary, no C++ or
 * framework types appear in the signatures.
 */
#ifndef GDN2_H
#define GDN2_H

#include <stdint.h>

#include <hip/hip_runtime_api.h> /* hipStream_t */

#ifdef __cplusplus
extern "C" {
#endif

#define GDN2_ABI_VERSION 7

/* Element types a tensor descriptor may carry. */
typedef enum gdn2_dtype {
    GDN2_DTYPE_BF16 = 1, /* bfloat16 */
    GDN2_DTYPE_F32 = 2,  /* IEEE float32 */
    GDN2_DTYPE_I32 = 3,  /* int32 */
    GDN2_DTYPE_F16 = 4,  /* IEEE float16 */
    GDN2_DTYPE_I64 = 5   /* int64 */
} gdn2_dtype;

/*
 * A view of caller-owned memory: `ndim` dimensions of `shape`, element
 * strides in `stride` (row-major contiguous tensors have
 * stride[d] = prod(shape[d+1..ndim-1])). `data` is a DEVICE pointer; it may
 * be NULL only when the tensor has zero elements.
 */
typedef struct gdn2_tensor {
    void *data;
    int32_t dtype; /* gdn2_dtype */
    int32_t ndim;
    int64_t shape[4];
    int64_t stride[4];
} gdn2_tensor;

/* Status codes. 0 is success; every failure is negative. */
enum {
    GDN2_OK = 0,
    GDN2_ERR_NULL_ARG = -1,    /* a required descriptor or pointer is NULL */
    GDN2_ERR_DTYPE = -2,       /* a tensor has the wrong element type */
    GDN2_ERR_SHAPE = -3,       /* ranks or extents disagree */
    GDN2_ERR_HEADS = -4,       /* HV is not a positive multiple of H */
    GDN2_ERR_UNSUPPORTED = -5, /* K or V not 64 or 128 (the backward: K != V), or an option out of range */
    GDN2_ERR_LAYOUT = -6,      /* a tensor's strides or alignment are not accepted */
    GDN2_ERR_ALIAS = -7,       /* an output overlaps an input */
    GDN2_ERR_HIP = -8,         /* the HIP runtime reported an error */
    GDN2_ERR_WORKSPACE = -9    /* a caller's workspace is missing, too small or not aligned */
};

/*
 * gdn2_chunk_fwd -- enqueue the GDN-2 chunked prefill forward on `stream`.
 *
 * Tensors (T = total packed tokens, N = number of sequences, H = q/k heads,
 * HV = value heads, K = key dim, V = value dim):
 *   q, k           [T, H, K]       bf16 or float16 (the io type: q's type,
 *                                  which k, v, beta, w and out must share)
 *   v, w           [T, HV, V]      io type
 *   g              [T, HV, K]      float32, bf16 or float16, natural-log
 *                                  decay, each value <= 0 and finite
 *                                  (precondition, not checked)
 *   beta           [T, HV, K]      io type (erase gate, taken as given, e.g.
 *                                  in [0, 1] or [0, 2]; not clamped)
 *   initial_state  [N, HV, K, V]   float32 or bf16, K-major (V innermost);
 *                                  V-major [N, HV, V, K] with the
 *                                  state_layout option
 *   cu_seqlens     [N + 1]         int32 or int64, device memory; cu[0] = 0,
 *                                  non-decreasing, cu[N] = T (precondition,
 *                                  not checked on the device)
 *   out            [T, HV, V]      io type, written for every token
 *   final_state    [N, HV, K, V]   float32 or bf16 (rounded to nearest
 *                                  even), layout as initial_state
 *
 * The FlashInfer parameter list names these element types (q, k, v at
 * float16 or bfloat16, beta and w read at q's type, g at float32, bfloat16
 * or float16, states at float32 or bfloat16, int32 or int64 cu_seqlens).
 * Arithmetic is float32 throughout (a bf16 state is widened on load and
 * carried in float32); the MFMA operands are bf16 for either io type.
 *
 * Value head hv reads q/k head hv / (HV / H) (contiguous groups of value
 * heads share one q/k head).
 *
 * Conditioning: each token's transition I - k (beta * k)^T (after the
 * decay; * elementwise) has the eigenvalue 1 - sum_c beta_c k_c^2, and all
 * its other eigenvalues are 1. With unit-norm keys (or qk_l2norm) and beta
 * in [0, 2] that eigenvalue stays within [-1, 1]; beyond that the
 * recurrence itself amplifies every rounding, and no two evaluations of it
 * (this library's or a float64 one) need agree. The accuracy figures of
 * this library hold in the contracting range.
 *
 * Optional arguments (the FlashInfer parameter-list defaults): g NULL means
 * g = 0, beta NULL means beta = 1, w NULL means w = 1, initial_state NULL
 * means a zero state, final_state NULL means the final state is not written,
 * cu_seqlens NULL means one sequence of T tokens (N = 1). scale == 0 means
 * 1/sqrt(K). A descriptor whose `data` is NULL but which has elements is an
 * error (NULL_ARG) for every tensor; an optional tensor is omitted by passing
 * a NULL descriptor pointer.
 *
 * Supported: K and V each 64 or 128, equal or not (the Flash-GDN-2 README,
 * training paragraph: both head dimensions in {64, 128}); any T >= 0,
 * N >= 1, H >= 1, HV a multiple of H. Empty sequences are allowed (their
 * final state equals their initial state).
 *
 * Ownership: the caller owns every buffer. Inputs and initial_state are only
 * read; out and final_state must be preallocated and are fully written. The
 * library keeps no pointer after the call returns. When it splits sequences
 * (see gdn2_chunk_fwd_opts) it takes a stream-ordered workspace of
 * N * HV * nseg * (2 K V + K K) * 4 bytes on `stream` and returns it with
 * hipFreeAsync on the same stream (nseg = segments per sequence, at most
 * ceil(ceil(T / 64) / segment chunks)); if that allocation fails it runs the
 * sequences whole instead. Otherwise it allocates no device memory.
 * Workspaces come from a memory pool the library creates on each device it
 * runs on (hipMemPoolCreate) with an unlimited release threshold: freed
 * workspace stays in that pool for later calls, so the pool holds up to the
 * largest workspace any call has used until the process ends.
 *
 * Layout (GDN2_ERR_LAYOUT otherwise; strides are in elements, as the
 * FlashInfer parameter list has it, only the innermost dimension needs to be
 * contiguous):
 *   q, k, v, g, beta, w, out: the K or V elements of each (token, head) row
 *     contiguous; the token and head strides free, non-negative and
 *     multiples of 16 bytes, with the token stride at least one row (K or V
 *     elements) and under 2^31 / 64 bytes; e.g. q, k, v as views of one
 *     fused [T, 3, H, D] projection. The rows of out must not overlap.
 *   initial_state, final_state, cu_seqlens: row-major contiguous.
 *   Every data pointer is 16-byte aligned.
 *
 * Aliasing: neither output (out, final_state) may overlap any input or the
 * other output; in particular final_state may not alias initial_state
 * (FlashInfer docs, output_state: the incoming state is read while outgoing
 * states are written): GDN2_ERR_ALIAS.
 *
 * Errors: every argument is validated on the host before anything is
 * enqueued; on failure nothing is enqueued, the return value says why and
 * gdn2_last_error() holds a message. Faults inside the kernel (e.g. a
 * cu_seqlens that breaks its precondition) surface at the caller's next
 * synchronisation with the stream.
 *
 * Semantics: asynchronous (returns after enqueueing, does not synchronise);
 * deterministic (no atomics; the same inputs give the same bits); reentrant.
 */
int gdn2_chunk_fwd(const gdn2_tensor *q, const gdn2_tensor *k,
                   const gdn2_tensor *v, const gdn2_tensor *g,
                   const gdn2_tensor *beta, const gdn2_tensor *w, float scale,
                   const gdn2_tensor *initial_state,
                   const gdn2_tensor *cu_seqlens, const gdn2_tensor *out,
                   const gdn2_tensor *final_state, hipStream_t stream);

/* State layouts (gdn2_fwd_options.state_layout). */
enum {
    GDN2_STATE_KV = 0, /* [N, HV, K, V]: V innermost (default) */
    GDN2_STATE_VK = 1  /* [N, HV, V, K]: K innermost, the FlashInfer layout */
};

/*
 * Options of gdn2_chunk_fwd_opts and gdn2_recurrent_fwd_opts. Set
 * `struct_size` to sizeof(gdn2_fwd_options); fields that lie past a smaller
 * struct_size (a caller built against an earlier version; at least the
 * first two fields) take their defaults (0).
 *
 * seq_split_chunks selects how a sequence is walked:
 *    0  automatic: gdn2_split_plan() for this shape and the current
 *       device's compute-unit count decides (what gdn2_chunk_fwd does);
 *   -1  never split: one workgroup walks each (sequence, value head);
 *  > 0  split every sequence into segments of this many 64-token chunks.
 *
 * A split run is the same computation in another order (the chunked WY form
 * is affine in the entering state): a transition pass gives every segment's
 * end state from a zero start and its K x K state transition, a combine
 * chains them into each segment's entering state, and an output pass runs
 * all segments at once. It pays when there are few (sequence, value head)
 * chains for the compute units and they are long (the parallel scan over
 * the sequence that the FlashInfer docs' output_state note alludes to when
 * it speaks of one sequence split across CTAs).
 */
typedef struct gdn2_fwd_options {
    int32_t struct_size;
    int32_t seq_split_chunks; /* chunked entry only; ignored by the recurrent one */
    /* GDN2_STATE_KV or GDN2_STATE_VK: the layout of initial_state and
     * final_state (FlashInfer parameter list: its states are V-major) */
    int32_t state_layout;
    /* 1: normalise every (token, head) row of q and of k to unit L2 norm
     * inside the kernel, x / max(||x||_2, 1e-12) in float32 from the stored
     * values (the FlashInfer use_qk_l2norm_in_kernel flag; the normalisation
     * is that of the Flash-GDN-2 quick start's torch normalize call); 0: q
     * and k are used as given */
    int32_t qk_l2norm;
} gdn2_fwd_options;

/*
 * gdn2_chunk_fwd_opts -- gdn2_chunk_fwd with options (NULL opts = defaults).
 * Same arguments, contract and errors as gdn2_chunk_fwd, plus
 * GDN2_ERR_SHAPE for a bad options struct (struct_size under 8,
 * seq_split_chunks < -1, state_layout or qk_l2norm out of range).
 */
int gdn2_chunk_fwd_opts(const gdn2_tensor *q, const gdn2_tensor *k,
                        const gdn2_tensor *v, const gdn2_tensor *g,
                        const gdn2_tensor *beta, const gdn2_tensor *w,
                        float scale, const gdn2_tensor *initial_state,
                        const gdn2_tensor *cu_seqlens, const gdn2_tensor *out,
                        const gdn2_tensor *final_state,
                        const gdn2_fwd_options *opts, hipStream_t stream);

/* Bytes of the fixed device array that gdn2_chunk_fwd_noalloc uses (64 MiB). */
#define GDN2_NOALLOC_SCRATCH_BYTES (64u << 20)

/*
 * gdn2_chunk_fwd_noalloc -- gdn2_chunk_fwd_opts for callers that cannot
 * allocate device memory: code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc. Same arguments, results and errors as
 * gdn2_chunk_fwd_opts; it calls no hipMalloc, hipMallocAsync, hipFree or
 * other allocating routine.
 *
 * Where the split run needs a workspace (N * HV * nseg * (2 K V + K K) * 4
 * bytes, see gdn2_chunk_fwd_opts), it is taken from a static device array of
 * GDN2_NOALLOC_SCRATCH_BYTES that each GPU the library runs on holds until
 * the process ends. Nothing in it needs clearing: every byte a call reads
 * was written earlier in the same call. With seq_split_chunks = 0 the
 * automatic plan lengthens its segments until the workspace fits (whole
 * sequences if none does); an explicit seq_split_chunks whose workspace
 * exceeds the array is rejected with GDN2_ERR_UNSUPPORTED and a message
 * naming both sizes. Device ordinals 0..63.
 *
 * All calls on one GPU share that GPU's array: calls that overlap in time on
 * one GPU (e.g. on two streams without ordering between them) race on it
 * and give undefined results. Calls ordered on one stream are safe.
 */
int gdn2_chunk_fwd_noalloc(const gdn2_tensor *q, const gdn2_tensor *k,
                           const gdn2_tensor *v, const gdn2_tensor *g,
                           const gdn2_tensor *beta, const gdn2_tensor *w,
                           float scale, const gdn2_tensor *initial_state,
                           const gdn2_tensor *cu_seqlens,
                           const gdn2_tensor *out,
                           const gdn2_tensor *final_state,
                           const gdn2_fwd_options *opts, hipStream_t stream);

/*
 * gdn2_recurrent_fwd -- the same operation evaluated token by token: for
 * decode (one new token per sequence) and short spans (a few tokens per
 * sequence, e.g. speculative or chunk-remainder steps), where the WY chunk
 * machinery would waste most of a 64-token chunk. Same tensors, dtypes,
 * defaults, varlen packing and errors as gdn2_chunk_fwd, with one
 * difference: final_state may be the very buffer of initial_state (same
 * data pointer and element type) to update the state in place; any other
 * overlap is GDN2_ERR_ALIAS. The arithmetic is the recurrence step by step
 * in float32 (state, gates, products); only the output (and a bf16 final
 * state) is rounded.
 *
 * Cost: every (sequence, value head) state is read and written once per
 * call (2 * K * V * 4 bytes), plus the tokens' vectors; one workgroup per
 * (sequence, value head, 32 value columns) walks the span in order, so long
 * sequences belong on gdn2_chunk_fwd. Allocates nothing.
 */
int gdn2_recurrent_fwd(const gdn2_tensor *q, const gdn2_tensor *k,
                       const gdn2_tensor *v, const gdn2_tensor *g,
                       const gdn2_tensor *beta, const gdn2_tensor *w,
                       float scale, const gdn2_tensor *initial_state,
                       const gdn2_tensor *cu_seqlens, const gdn2_tensor *out,
                       const gdn2_tensor *final_state, hipStream_t stream);

/*
 * gdn2_recurrent_fwd_opts -- gdn2_recurrent_fwd with options (NULL opts =
 * defaults): state_layout and qk_l2norm as for gdn2_chunk_fwd_opts;
 * seq_split_chunks is ignored. Errors as gdn2_chunk_fwd_opts.
 */
int gdn2_recurrent_fwd_opts(const gdn2_tensor *q, const gdn2_tensor *k,
                            const gdn2_tensor *v, const gdn2_tensor *g,
                            const gdn2_tensor *beta, const gdn2_tensor *w,
                            float scale, const gdn2_tensor *initial_state,
                            const gdn2_tensor *cu_seqlens,
                            const gdn2_tensor *out,
                            const gdn2_tensor *final_state,
                            const gdn2_fwd_options *opts, hipStream_t stream);

/* The host-side validation of gdn2_recurrent_fwd alone (no device work). */
int gdn2_recurrent_fwd_check(const gdn2_tensor *q, const gdn2_tensor *k,
                             const gdn2_tensor *v, const gdn2_tensor *g,
                             const gdn2_tensor *beta, const gdn2_tensor *w,
                             float scale, const gdn2_tensor *initial_state,
                             const gdn2_tensor *cu_seqlens,
                             const gdn2_tensor *out,
                             const gdn2_tensor *final_state);

/*
 * gdn2_split_plan -- the automatic choice of seq_split_chunks for T packed
 * tokens in N sequences with HV value heads on a device with num_cu compute
 * units: 0 (run whole sequences) or the segment length in chunks. Pure host
 * arithmetic (assumes equal sequence lengths); needs no GPU.
 */
int gdn2_split_plan(int64_t T, int32_t N, int32_t HV, int32_t num_cu);

/*
 * gdn2_chunk_fwd_check -- the host-side argument validation of
 * gdn2_chunk_fwd alone: same arguments (no stream), same return codes, same
 * gdn2_last_error() message. Touches no device memory and makes no HIP call,
 * so it can run on a machine without a GPU.
 */
int gdn2_chunk_fwd_check(const gdn2_tensor *q, const gdn2_tensor *k,
                         const gdn2_tensor *v, const gdn2_tensor *g,
                         const gdn2_tensor *beta, const gdn2_tensor *w,
                         float scale, const gdn2_tensor *initial_state,
                         const gdn2_tensor *cu_seqlens, const gdn2_tensor *out,
                         const gdn2_tensor *final_state);

/*
 * gdn2_chunk_bwd -- enqueue the backward of gdn2_chunk_fwd on `stream`: the
 * gradients of a scalar loss with respect to q, k, v, g, beta, w and the
 * initial state, given its gradients d_out with respect to the output and
 * d_final_state with respect to the final state. It differentiates the same
 * recurrence (FlashInfer chunk_gated_delta_rule2 docs, recurrence display
 * equation) through the same 64-token chunked WY form, so a training step
 * can pair the two calls.
 *
 * Tensors (every one dense, row-major; shapes and roles as in
 * gdn2_chunk_fwd):
 *   q, k [T, H, K], v, w [T, HV, V], beta [T, HV, K]      bf16 or float16, one type (required)
 *   g [T, HV, K]                                           float32, bf16 or float16 (required)
 *   initial_state [N, HV, K, V]                            float32, K-major, or NULL (zero)
 *   cu_seqlens [N + 1]                                     int32 or int64, or NULL (one sequence)
 *   d_out [T, HV, V]                                       q's type (required)
 *   d_final_state [N, HV, K, V]                            float32, or NULL (zero)
 * Outputs (caller-allocated, fully written):
 *   dq, dk [T, H, K]                                       q's type: sums over the value heads that
 *                                                          read each q/k head
 *   dv, dw [T, HV, V], dbeta [T, HV, K]                    q's type
 *   dg [T, HV, K]                                          g's type (gradient of the natural-log g)
 *   d_initial_state [N, HV, K, V]                          float32, or NULL (not written)
 * scale == 0 means 1/sqrt(K). Supported sizes: (K, V) = (64, 64) or
 * (128, 128) (GDN2_ERR_UNSUPPORTED otherwise; the forward also takes K != V).
 *
 * Strong decay: any g <= 0 is supported. A key channel whose running
 * in-chunk sum of g leaves about -83 (120 ln 2) within a chunk cannot use
 * the chunk-start factors e^G and e^-G (the second overflows); such a
 * channel's share of the intra-chunk products is differentiated exactly,
 * per pair of rows with e^(G_r - G_s) <= 1 (burn-gdn2 README, numerical
 * stability), at some extra cost for the chunks that have one.
 *
 * Evaluation: the forward runs again and keeps the state entering every
 * chunk (rounded to bf16) and each chunk's WY quantities (its record); one workgroup
 * per (sequence, value head) carries the state gradient over the chunks in
 * reverse; a chunk-parallel pass forms every gradient; a last pass sums dq
 * and dk over grouped value heads (HV > H). Arithmetic is float32 with bf16
 * MFMA operands, as in the forward.
 *
 * Streams: when every (sequence, value head) chain of the call can be
 * resident at once (more than half of the device's compute units and at
 * most all of them, whole sequences), the longer half of the sequences
 * (by chunk count, ranked on the device) runs its passes on `stream` and
 * the shorter half on a second stream. The library creates that stream
 * per device on first use, at the default priority, and keeps it until
 * the process ends. The work is forked from `stream` and joined back to it
 * with events, so the call is ordered on `stream` like any other. The
 * second stream is never created while `stream` is being captured into a
 * graph (such a call runs on `stream` alone); graph capture of the
 * backward is otherwise untested. Results are bit-identical either way.
 *
 * Ownership and memory: the caller owns every buffer; inputs are only read.
 * A stream-ordered workspace (from the library's pool, see gdn2_chunk_fwd;
 * released with hipFreeAsync on `stream`) of
 *   (T / 64 + N) * HV * (2 * K * V * 2 + 516 * K + 16384) bytes,
 *   plus 2 * T * HV * K * 4 bytes when HV > H (per-value-head dq and dk),
 *   plus N * 4 bytes when the call runs as two groups (each sequence's group)
 * (rounded up per part) holds the checkpoints, the records and partial
 * gradients; if it cannot be allocated the call fails with GDN2_ERR_HIP and
 * enqueues nothing.
 *
 * Errors as gdn2_chunk_fwd: NULL_ARG for a missing required tensor, DTYPE,
 * SHAPE, HEADS, UNSUPPORTED, LAYOUT for a non-dense tensor, ALIAS when an
 * output overlaps an input or another output. Asynchronous, deterministic
 * (no atomics), reentrant.
 */
int gdn2_chunk_bwd(const gdn2_tensor *q, const gdn2_tensor *k,
                   const gdn2_tensor *v, const gdn2_tensor *g,
                   const gdn2_tensor *beta, const gdn2_tensor *w, float scale,
                   const gdn2_tensor *initial_state,
                   const gdn2_tensor *cu_seqlens, const gdn2_tensor *d_out,
                   const gdn2_tensor *d_final_state, const gdn2_tensor *dq,
                   const gdn2_tensor *dk, const gdn2_tensor *dv,
                   const gdn2_tensor *dg, const gdn2_tensor *dbeta,
                   const gdn2_tensor *dw, const gdn2_tensor *d_initial_state,
                   hipStream_t stream);

/* The host-side validation of gdn2_chunk_bwd alone (no device work). */
int gdn2_chunk_bwd_check(const gdn2_tensor *q, const gdn2_tensor *k,
                         const gdn2_tensor *v, const gdn2_tensor *g,
                         const gdn2_tensor *beta, const gdn2_tensor *w,
                         float scale, const gdn2_tensor *initial_state,
                         const gdn2_tensor *cu_seqlens,
                         const gdn2_tensor *d_out,
                         const gdn2_tensor *d_final_state,
                         const gdn2_tensor *dq, const gdn2_tensor *dk,
                         const gdn2_tensor *dv, const gdn2_tensor *dg,
                         const gdn2_tensor *dbeta, const gdn2_tensor *dw,
                         const gdn2_tensor *d_initial_state);

/* ------------------------------------------------ scalar-gated delta rule --
 *
 * The gated delta rule with one decay and one gate per token and head, the
 * case g constant over the channels and w = beta = one scalar of the rule
 * above (FlashInfer chunk_gated_delta_rule2 docs: the reduction to the
 * scalar rule): per sequence and value head, with a K x V float32 state S,
 *
 *     S_t  = exp(g_t) S_{t-1}
 *     u_t  = beta_t (v_t - S_t^T k_t)
 *     S_t += k_t u_t^T
 *     o_t  = scale * q_t^T S_t
 *
 * gdn2_delta_chunk_fwd evaluates it in 64-token chunks (prefill, training),
 * gdn2_delta_recurrent_fwd token by token (decode and short spans), and
 * gdn2_delta_chunk_bwd computes the gradients. Tensors as in gdn2_chunk_fwd
 * but for the gates:
 *   q, k  [T, H, K], v, out [T, HV, V]   bf16 or float16, one io type
 *   g     [T, HV]   float32, bf16 or float16; natural log of the decay, <= 0
 *                   and finite (precondition, not checked), the type's lowest
 *                   value too: it forgets the state; NULL: 0
 *   beta  [T, HV]   io type, taken as given; NULL: 1
 *   initial_state, final_state [N, HV, K, V] float32 or bf16 (or V-major by
 *                   option), cu_seqlens [N + 1] int32 or int64
 * with the same defaults for NULL arguments and scale, the same sizes (K and
 * V each 64 or 128, HV a multiple of H), the same preconditions on cu_seqlens
 * and conditioning, and the same layouts; g and beta may have any
 * non-negative strides (elements) and need only their element's alignment.
 * opts: state_layout and qk_l2norm as for gdn2_chunk_fwd_opts (NULL:
 * defaults); of seq_split_chunks the chunked entry takes 0 (few long
 * sequences run as parallel segments, joined by their transitions; chosen
 * from T, N, HV, K and V alone) and -1 (never split), and refuses > 0
 * (GDN2_ERR_UNSUPPORTED); the recurrent one ignores it.
 * N * HV and (T / 64 + N) * HV may reach 5592405 (GDN2_ERR_SHAPE beyond).
 * Tokens behind the last sequence (cu_seqlens[N] < T, a padded batch) are not
 * read, and no output or gradient of theirs is written. An infinity or NaN in
 * a token reaches no other sequence; in the chunked entries it may reach the
 * earlier tokens of its 64-token chunk too.
 *
 * Accuracy: products run on fp16 MFMA with float32 accumulation; float32
 * operands are taken in two fp16 parts next to a power of two of their
 * column's largest value (22 significant bits), bf16 rows next to one of
 * their own; the state and all sums are float32. Float32 results
 * (final_state, dg, d_initial_state) are within about 1e-6 of a float64
 * evaluation, relative in the 2-norm, on unit-norm keys (within 1e-5 where a
 * chunk repeats one key, not decayed, at beta near 2); 16-bit results are
 * rounded once (a forward output of bf16 takes the state and the chunk's
 * factors in one such part, rounded to nearest: 11 bits next to its 8).
 *
 * Workspace: these entries allocate nothing and keep nothing between calls.
 * The caller passes device memory of at least the number of bytes that the
 * entry's _workspace function gives (0: NULL is accepted; it also gives 0 for
 * sizes that the entry refuses), 256-byte aligned and apart from every tensor
 * (GDN2_ERR_WORKSPACE, GDN2_ERR_ALIAS). Its contents before the call do not matter and are undefined after it; it may
 * be reused once the call's work on the stream is done. Calls that can
 * overlap in time need workspaces of their own. Every entry may be captured
 * into a graph; a graph's workspace belongs to that graph's replays.
 *
 * Asynchronous, deterministic (no atomics), reentrant. Errors as
 * gdn2_chunk_fwd. Each _check function is the host-side validation alone,
 * without the workspace: no HIP call, no device memory.
 */

/* Bytes of workspace of gdn2_delta_chunk_fwd: (T / 64 + N) * HV * 26880, and
 * at most 8 MiB for the segments where few long sequences are split. */
int64_t gdn2_delta_chunk_fwd_workspace(int64_t T, int32_t N, int32_t HV);

/* The chunked forward. final_state may not alias initial_state. */
int gdn2_delta_chunk_fwd(const gdn2_tensor *q, const gdn2_tensor *k,
                         const gdn2_tensor *v, const gdn2_tensor *g,
                         const gdn2_tensor *beta, float scale,
                         const gdn2_tensor *initial_state,
                         const gdn2_tensor *cu_seqlens, const gdn2_tensor *out,
                         const gdn2_tensor *final_state,
                         const gdn2_fwd_options *opts, void *workspace,
                         int64_t workspace_bytes, hipStream_t stream);
int gdn2_delta_chunk_fwd_check(const gdn2_tensor *q, const gdn2_tensor *k,
                               const gdn2_tensor *v, const gdn2_tensor *g,
                               const gdn2_tensor *beta, float scale,
                               const gdn2_tensor *initial_state,
                               const gdn2_tensor *cu_seqlens,
                               const gdn2_tensor *out,
                               const gdn2_tensor *final_state,
                               const gdn2_fwd_options *opts);

/* Token by token, without a workspace: every state is read and written once
 * per call. final_state may be initial_state's own buffer (same pointer and
 * type) to update the state in place. */
int gdn2_delta_recurrent_fwd(const gdn2_tensor *q, const gdn2_tensor *k,
                             const gdn2_tensor *v, const gdn2_tensor *g,
                             const gdn2_tensor *beta, float scale,
                             const gdn2_tensor *initial_state,
                             const gdn2_tensor *cu_seqlens,
                             const gdn2_tensor *out,
                             const gdn2_tensor *final_state,
                             const gdn2_fwd_options *opts, hipStream_t stream);
int gdn2_delta_recurrent_fwd_check(const gdn2_tensor *q, const gdn2_tensor *k,
                                   const gdn2_tensor *v, const gdn2_tensor *g,
                                   const gdn2_tensor *beta, float scale,
                                   const gdn2_tensor *initial_state,
                                   const gdn2_tensor *cu_seqlens,
                                   const gdn2_tensor *out,
                                   const gdn2_tensor *final_state,
                                   const gdn2_fwd_options *opts);

/*
 * The backward of gdn2_delta_chunk_fwd (without qk_l2norm; see
 * gdn2_qk_norm_rope_bwd for the norm's gradient). Every tensor dense and
 * 16-byte aligned; q, k, v, g, beta, d_out required; (K, V) = (64, 64) or
 * (128, 128); states K-major float32 (initial_state and d_final_state NULL:
 * zero; d_initial_state NULL: not written). dq, dk (summed over the value
 * heads that read each q/k head), dv and dbeta have q's type, dg g's.
 * Workspace: per (chunk, value head) 26880 + 8 K V + 514 V bytes, plus
 * 8 T HV K with grouped heads (HV > H), each part rounded up to 256 bytes,
 * and at most 12 MiB for the segments where few long sequences are split.
 */
int64_t gdn2_delta_chunk_bwd_workspace(int64_t T, int32_t N, int32_t H,
                                       int32_t HV, int32_t K, int32_t V);
int gdn2_delta_chunk_bwd(const gdn2_tensor *q, const gdn2_tensor *k,
                         const gdn2_tensor *v, const gdn2_tensor *g,
                         const gdn2_tensor *beta, float scale,
                         const gdn2_tensor *initial_state,
                         const gdn2_tensor *cu_seqlens,
                         const gdn2_tensor *d_out,
                         const gdn2_tensor *d_final_state,
                         const gdn2_tensor *dq, const gdn2_tensor *dk,
                         const gdn2_tensor *dv, const gdn2_tensor *dg,
                         const gdn2_tensor *dbeta,
                         const gdn2_tensor *d_initial_state, void *workspace,
                         int64_t workspace_bytes, hipStream_t stream);
int gdn2_delta_chunk_bwd_check(const gdn2_tensor *q, const gdn2_tensor *k,
                               const gdn2_tensor *v, const gdn2_tensor *g,
                               const gdn2_tensor *beta, float scale,
                               const gdn2_tensor *initial_state,
                               const gdn2_tensor *cu_seqlens,
                               const gdn2_tensor *d_out,
                               const gdn2_tensor *d_final_state,
                               const gdn2_tensor *dq, const gdn2_tensor *dk,
                               const gdn2_tensor *dv, const gdn2_tensor *dg,
                               const gdn2_tensor *dbeta,
                               const gdn2_tensor *d_initial_state);

/* ---------------------------------------- norms and rotation of q and k --
 *
 * What a model does to q and k before the rule, both in one launch: every
 * (token, head) row x of K elements becomes
 *
 *     z = x * r * weight,   r = 1 / max(|x|, eps)           (L2, the default)
 *                           r = 1 / sqrt(mean(x^2) + eps)   (RMS)
 *                           r = 1                           (NONE)
 *     y = z with its first rot elements turned by the token's position: each
 *         pair (a, b) becomes (a cos - b sin, a sin + b cos)
 *
 * in float32, rounded once. L2 with eps 1e-12 and no weight is what
 * qk_l2norm does in the forward entries; here it has a backward. A rotation
 * keeps a row's norm, so the rule's conditioning is that of the norm alone.
 *
 *   q [T, H, K], k [T, HK, K]   bf16 or float16 (one io type), K 64 or 128
 *   q_weight, k_weight [K]      float32 or the io type; NULL: 1
 *   rope [P, rot]               float32: rot / 2 cosines, then rot / 2 sines
 *                               of each position's angles (any frequencies and
 *                               scaling); NULL: no rotation. rot a multiple of
 *                               16, or of 2 with interleaved, at most K
 *   positions [T]               int32 or int64, in [0, P) (precondition, not
 *                               checked on the device: others read the
 *                               table's first or last row); with rope only
 *   q_out, k_out                q's and k's shapes and type
 * Pairs are (i, i + rot / 2), or (2 i, 2 i + 1) with interleaved. Rows as in
 * gdn2_chunk_fwd (token and head strides free, 16-byte multiples); weights,
 * table and positions dense and 16-byte aligned. Outputs may not overlap an
 * input or each other (their spans, also of interleaved views).
 */
enum {
    GDN2_QK_NORM_NONE = 0,
    GDN2_QK_NORM_L2 = 1,
    GDN2_QK_NORM_RMS = 2
};

/* struct_size: sizeof(gdn2_qk_options). NULL options: L2, 1e-12, halves. */
typedef struct gdn2_qk_options {
    int32_t struct_size;
    int32_t norm;        /* GDN2_QK_NORM_* */
    int32_t interleaved; /* 0 or 1 */
    float eps;           /* 0: 1e-12 (L2) or 1e-6 (RMS) */
} gdn2_qk_options;

int gdn2_qk_norm_rope_fwd(const gdn2_tensor *q, const gdn2_tensor *k,
                          const gdn2_tensor *q_weight,
                          const gdn2_tensor *k_weight, const gdn2_tensor *rope,
                          const gdn2_tensor *positions,
                          const gdn2_tensor *q_out, const gdn2_tensor *k_out,
                          const gdn2_qk_options *opts, hipStream_t stream);
int gdn2_qk_norm_rope_fwd_check(const gdn2_tensor *q, const gdn2_tensor *k,
                                const gdn2_tensor *q_weight,
                                const gdn2_tensor *k_weight,
                                const gdn2_tensor *rope,
                                const gdn2_tensor *positions,
                                const gdn2_tensor *q_out,
                                const gdn2_tensor *k_out,
                                const gdn2_qk_options *opts);

/*
 * Its backward: dq, dk from the inputs q, k and the gradients dq_out, dk_out
 * of the outputs (all of q's and k's shapes and type, rows as above), and,
 * where given, dq_weight and dk_weight [K] in the weight's type, summed over
 * all tokens and heads in float32 in a fixed order. The sums need a workspace
 * (as above; 0 bytes when neither is given).
 */
int64_t gdn2_qk_norm_rope_bwd_workspace(int64_t T, int32_t H, int32_t HK,
                                        int32_t K);
int gdn2_qk_norm_rope_bwd(const gdn2_tensor *q, const gdn2_tensor *k,
                          const gdn2_tensor *dq_out, const gdn2_tensor *dk_out,
                          const gdn2_tensor *q_weight,
                          const gdn2_tensor *k_weight, const gdn2_tensor *rope,
                          const gdn2_tensor *positions, const gdn2_tensor *dq,
                          const gdn2_tensor *dk, const gdn2_tensor *dq_weight,
                          const gdn2_tensor *dk_weight,
                          const gdn2_qk_options *opts, void *workspace,
                          int64_t workspace_bytes, hipStream_t stream);
int gdn2_qk_norm_rope_bwd_check(const gdn2_tensor *q, const gdn2_tensor *k,
                                const gdn2_tensor *dq_out,
                                const gdn2_tensor *dk_out,
                                const gdn2_tensor *q_weight,
                                const gdn2_tensor *k_weight,
                                const gdn2_tensor *rope,
                                const gdn2_tensor *positions,
                                const gdn2_tensor *dq, const gdn2_tensor *dk,
                                const gdn2_tensor *dq_weight,
                                const gdn2_tensor *dk_weight,
                                const gdn2_qk_options *opts);

/* --------------------------------------------- around the rule: a mixer's
 * other per-channel operators --
 *
 * What stands before and after a rule in a token mixer: the short causal
 * convolution of its inputs, the gated linear recurrence (a rule with a
 * vector for a state), and the norm of rows with a gate. Shared by all three:
 *   types   x and its like ("io type"): bf16, float16 or float32, one type
 *           per call; arithmetic, sums and statistics in float32, rounded
 *           once
 *   layout  the last dimension contiguous, the other strides free and
 *           non-negative (0 too, for inputs); pointers aligned to their
 *           element; the rows of an output may not overlap. Weights, states
 *           and cu_seqlens dense and 16-byte aligned.
 *   sizes   T and N any number to 2^31 - 65537, D to 2^24 (the norm: 16384),
 *           within the 2^32 - 1 threads that one launch can hold
 *           (GDN2_ERR_SHAPE beyond)
 *   cu_seqlens, workspaces, errors, streams, graphs: as for the
 *           scalar-gated rule above. Tokens behind the last sequence are not
 *           read, and nothing of theirs is written. An infinity or NaN in a
 *           token reaches no other sequence and no other channel (norm: no
 *           other row; the weights' gradients are sums over all). A state
 *           that is an infinity may be NaN in the tokens after it.
 * Outputs may not overlap inputs or each other (their spans, also of
 * interleaved views: GDN2_ERR_ALIAS).
 */

/*
 * The gated linear recurrence: per sequence and channel
 *
 *     h_t = e^(g_t) h_{t-1} + m_t w_t x_t,   out_t = h_t
 *     m   = 1,  1 - e^g  or  sqrt(1 - e^(2 g))
 *
 *   x, w, out [T, D]  io type; w NULL: 1
 *   g [T, D]          float32 or the io type: natural log of the decay, <= 0
 *                     (precondition, not checked), minus infinity or the
 *                     type's lowest value too: they forget the state
 *   initial_state, final_state [N, D]  float32 or bf16 (NULL: zero / not
 *                     written)
 *
 * gdn2_linear_scan_fwd runs over long sequences: whole ones side by side, or
 * few long ones in two passes over chunks of tokens, joined by the products of
 * their decays (chosen from T, N and D alone; only the second needs the
 * workspace). gdn2_linear_scan_recurrent_fwd walks token by token
 * (decode, short spans), where final_state may be initial_state's own buffer
 * (same pointer and type) to update the state in place.
 *
 * Slow decays are held in two parts, so that g near 0 keeps its precision.
 * Every step rounds the state: float32 results of a state that remembers M
 * steps (1 / |g|, or the sequence where that is shorter) are up to about 1e-6
 * + sqrt(2 M) 2^-24 off a float64 evaluation, relative in the 2-norm (M = 50:
 * 2e-6, and 1e-7 as measured; 6000: 8e-6), the gradient of g, a sum that may
 * cancel, 2.5 times that.
 */
enum {
    GDN2_SCAN_INPUT_NONE = 0,   /* m = 1 */
    GDN2_SCAN_INPUT_CONVEX = 1, /* m = 1 - e^g */
    GDN2_SCAN_INPUT_UNIT = 2    /* m = sqrt(1 - e^(2 g)) */
};

/* struct_size: sizeof(gdn2_scan_options). NULL options: m = 1. */
typedef struct gdn2_scan_options {
    int32_t struct_size;
    int32_t input_scale; /* GDN2_SCAN_INPUT_* */
} gdn2_scan_options;

int64_t gdn2_linear_scan_fwd_workspace(int64_t T, int32_t N, int32_t D);
int gdn2_linear_scan_fwd(const gdn2_tensor *x, const gdn2_tensor *g,
                         const gdn2_tensor *w, const gdn2_tensor *initial_state,
                         const gdn2_tensor *cu_seqlens, const gdn2_tensor *out,
                         const gdn2_tensor *final_state,
                         const gdn2_scan_options *opts, void *workspace,
                         int64_t workspace_bytes, hipStream_t stream);
int gdn2_linear_scan_fwd_check(const gdn2_tensor *x, const gdn2_tensor *g,
                               const gdn2_tensor *w,
                               const gdn2_tensor *initial_state,
                               const gdn2_tensor *cu_seqlens,
                               const gdn2_tensor *out,
                               const gdn2_tensor *final_state,
                               const gdn2_scan_options *opts);
int gdn2_linear_scan_recurrent_fwd(const gdn2_tensor *x, const gdn2_tensor *g,
                                   const gdn2_tensor *w,
                                   const gdn2_tensor *initial_state,
                                   const gdn2_tensor *cu_seqlens,
                                   const gdn2_tensor *out,
                                   const gdn2_tensor *final_state,
                                   const gdn2_scan_options *opts,
                                   hipStream_t stream);
int gdn2_linear_scan_recurrent_fwd_check(const gdn2_tensor *x,
                                         const gdn2_tensor *g,
                                         const gdn2_tensor *w,
                                         const gdn2_tensor *initial_state,
                                         const gdn2_tensor *cu_seqlens,
                                         const gdn2_tensor *out,
                                         const gdn2_tensor *final_state,
                                         const gdn2_scan_options *opts);

/*
 * Its backward: dx, dw (io type; dw with w, NULL: not written), dg (g's type),
 * d_initial_state [N, D] float32 (NULL: not written) from the inputs, d_out
 * (io type) and d_final_state [N, D] float32 (NULL: zero). The derivative of
 * sqrt(1 - e^(2 g)) at g = 0, where it is infinite, is taken as 0.
 */
int64_t gdn2_linear_scan_bwd_workspace(int64_t T, int32_t N, int32_t D);
int gdn2_linear_scan_bwd(const gdn2_tensor *x, const gdn2_tensor *g,
                         const gdn2_tensor *w, const gdn2_tensor *initial_state,
                         const gdn2_tensor *cu_seqlens,
                         const gdn2_tensor *d_out,
                         const gdn2_tensor *d_final_state,
                         const gdn2_tensor *dx, const gdn2_tensor *dg,
                         const gdn2_tensor *dw,
                         const gdn2_tensor *d_initial_state,
                         const gdn2_scan_options *opts, void *workspace,
                         int64_t workspace_bytes, hipStream_t stream);
int gdn2_linear_scan_bwd_check(const gdn2_tensor *x, const gdn2_tensor *g,
                               const gdn2_tensor *w,
                               const gdn2_tensor *initial_state,
                               const gdn2_tensor *cu_seqlens,
                               const gdn2_tensor *d_out,
                               const gdn2_tensor *d_final_state,
                               const gdn2_tensor *dx, const gdn2_tensor *dg,
                               const gdn2_tensor *dw,
                               const gdn2_tensor *d_initial_state,
                               const gdn2_scan_options *opts);

/*
 * The short causal convolution: per sequence and channel, with K = 2, 3 or 4
 * taps,
 *
 *     p_t = bias + sum_j weight[j] x_{t-(K-1)+j},   out_t = p_t or p_t sigmoid(p_t)
 *
 *   x, out [T, D], initial_state, final_state [N, K - 1, D]  io type: the K - 1
 *                    inputs before a sequence's first token and its last
 *                    K - 1, the oldest first (NULL: zeros / not written). A
 *                    sequence of under K - 1 tokens keeps rows of its initial
 *                    state in its final one.
 *   weight [D, K], bias [D]  float32 or the io type, both one type; bias NULL: 0
 *
 * gdn2_short_conv_recurrent_fwd walks token by token (decode, short spans);
 * there final_state may be initial_state's own buffer. No workspace.
 */
enum { GDN2_CONV_NONE = 0, GDN2_CONV_SILU = 1 };

/* struct_size: sizeof(gdn2_conv_options). NULL options: SiLU. */
typedef struct gdn2_conv_options {
    int32_t struct_size;
    int32_t activation; /* GDN2_CONV_* */
} gdn2_conv_options;

int gdn2_short_conv_fwd(const gdn2_tensor *x, const gdn2_tensor *weight,
                        const gdn2_tensor *bias,
                        const gdn2_tensor *initial_state,
                        const gdn2_tensor *cu_seqlens, const gdn2_tensor *out,
                        const gdn2_tensor *final_state,
                        const gdn2_conv_options *opts, hipStream_t stream);
int gdn2_short_conv_fwd_check(const gdn2_tensor *x, const gdn2_tensor *weight,
                              const gdn2_tensor *bias,
                              const gdn2_tensor *initial_state,
                              const gdn2_tensor *cu_seqlens,
                              const gdn2_tensor *out,
                              const gdn2_tensor *final_state,
                              const gdn2_conv_options *opts);
int gdn2_short_conv_recurrent_fwd(const gdn2_tensor *x,
                                  const gdn2_tensor *weight,
                                  const gdn2_tensor *bias,
                                  const gdn2_tensor *initial_state,
                                  const gdn2_tensor *cu_seqlens,
                                  const gdn2_tensor *out,
                                  const gdn2_tensor *final_state,
                                  const gdn2_conv_options *opts,
                                  hipStream_t stream);
int gdn2_short_conv_recurrent_fwd_check(const gdn2_tensor *x,
                                        const gdn2_tensor *weight,
                                        const gdn2_tensor *bias,
                                        const gdn2_tensor *initial_state,
                                        const gdn2_tensor *cu_seqlens,
                                        const gdn2_tensor *out,
                                        const gdn2_tensor *final_state,
                                        const gdn2_conv_options *opts);

/*
 * Its backward: dx, d_initial_state [N, K - 1, D] (io type; NULL: not
 * written), dweight and dbias (the weight's type; NULL: not written; dbias
 * with bias), summed over all tokens in float32 in a fixed order, from the
 * inputs, d_out and d_final_state (io type; NULL: zero). The sums need the
 * workspace (0 bytes when neither is given).
 */
int64_t gdn2_short_conv_bwd_workspace(int64_t T, int32_t D, int32_t K);
int gdn2_short_conv_bwd(const gdn2_tensor *x, const gdn2_tensor *weight,
                        const gdn2_tensor *bias,
                        const gdn2_tensor *initial_state,
                        const gdn2_tensor *cu_seqlens,
                        const gdn2_tensor *d_out,
                        const gdn2_tensor *d_final_state,
                        const gdn2_tensor *dx, const gdn2_tensor *dweight,
                        const gdn2_tensor *dbias,
                        const gdn2_tensor *d_initial_state,
                        const gdn2_conv_options *opts, void *workspace,
                        int64_t workspace_bytes, hipStream_t stream);
int gdn2_short_conv_bwd_check(const gdn2_tensor *x, const gdn2_tensor *weight,
                              const gdn2_tensor *bias,
                              const gdn2_tensor *initial_state,
                              const gdn2_tensor *cu_seqlens,
                              const gdn2_tensor *d_out,
                              const gdn2_tensor *d_final_state,
                              const gdn2_tensor *dx,
                              const gdn2_tensor *dweight,
                              const gdn2_tensor *dbias,
                              const gdn2_tensor *d_initial_state,
                              const gdn2_conv_options *opts);

/*
 * The norm of rows: every (token, head) row x of D elements, 1 <= D <= 16384,
 * becomes
 *
 *     n = (x - mean) / sqrt(var + eps)  (LAYER)  or  x / sqrt(mean x^2 + eps)  (RMS)
 *     y = n weight + bias,   times gate sigmoid(gate) where a gate is given
 *
 *   x, gate, out [T, H, D]  io type; gate NULL: none
 *   weight, bias [D]        float32 or the io type, each; NULL: 1, 0
 * T * H to 2^31 - 1. The output of a rule with its gate is [T, HV, V]; a
 * residual stream [T, D] is T rows of one head.
 */
enum { GDN2_NORM_LAYER = 0, GDN2_NORM_RMS = 1 };

/* struct_size: sizeof(gdn2_norm_options). NULL options: LAYER, 1e-5. */
typedef struct gdn2_norm_options {
    int32_t struct_size;
    int32_t norm; /* GDN2_NORM_* */
    float eps;    /* 0: 1e-5 (LAYER) or 1e-6 (RMS) */
} gdn2_norm_options;

int gdn2_layer_norm_fwd(const gdn2_tensor *x, const gdn2_tensor *gate,
                        const gdn2_tensor *weight, const gdn2_tensor *bias,
                        const gdn2_tensor *out, const gdn2_norm_options *opts,
                        hipStream_t stream);
int gdn2_layer_norm_fwd_check(const gdn2_tensor *x, const gdn2_tensor *gate,
                              const gdn2_tensor *weight,
                              const gdn2_tensor *bias, const gdn2_tensor *out,
                              const gdn2_norm_options *opts);

/*
 * Its backward: dx and (with gate) dgate, of x's shape and type, and, where
 * given, dweight and dbias [D] in their tensors' types, summed over all rows
 * in float32 in a fixed order, which need the workspace (0 bytes when neither
 * is given). Nothing is kept from the forward.
 */
int64_t gdn2_layer_norm_bwd_workspace(int64_t T, int32_t H, int32_t D);
int gdn2_layer_norm_bwd(const gdn2_tensor *x, const gdn2_tensor *gate,
                        const gdn2_tensor *weight, const gdn2_tensor *bias,
                        const gdn2_tensor *d_out, const gdn2_tensor *dx,
                        const gdn2_tensor *dgate, const gdn2_tensor *dweight,
                        const gdn2_tensor *dbias,
                        const gdn2_norm_options *opts, void *workspace,
                        int64_t workspace_bytes, hipStream_t stream);
int gdn2_layer_norm_bwd_check(const gdn2_tensor *x, const gdn2_tensor *gate,
                              const gdn2_tensor *weight,
                              const gdn2_tensor *bias, const gdn2_tensor *d_out,
                              const gdn2_tensor *dx, const gdn2_tensor *dgate,
                              const gdn2_tensor *dweight,
                              const gdn2_tensor *dbias,
                              const gdn2_norm_options *opts);

/* Message describing the last failure on the calling thread ("" if none).
 * The string stays valid until the next call on the same thread. */
const char *gdn2_last_error(void);

/* GDN2_ABI_VERSION of the built library. */
int gdn2_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN2_H */
