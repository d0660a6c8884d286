/*
 * gdn.h -- C ABI of the MI355X (gfx950) gated delta-rule library, libgdn.so.
 *
 * The library computes one gated delta-rule linear-attention layer core: the
 * per-token, per-value-head recurrence on an fp32 state S[dv][dk]
 *
 *     S <- exp(g) * S;   p = S k;   d = beta * (v - p);   S <- S + d k^T;   o = (S q) / sqrt(dk)
 *
 * (module doc of docs.rs ferrox-core 0.24.0 src/gdn.rs, `delta_step`; CPU reference
 * `cpu_segment` of docs.rs ferrum-kernels 0.8.0
 * src/backend/metal/vnext_ops/gated_delta_attention_tests.rs), plus the ops that
 * surround it in that reference: depthwise causal conv + SiLU with carried raw
 * inputs, L2 norm of q and k, the softplus/sigmoid gates, the grouped or tiled
 * k-head map, and the gated RMS norm of the output.
 *
 * Beside it: linear attention with a decay per head (the same state without the
 * delta rule), and what feeds a layer in 8 bits -- the RMS norm with the residual's
 * addition and an 8-bit output, and the product of 8-bit integers that projects
 * it to the mixed q, k, v row. And the softmax attention layers that stand between such
 * layers: rotary positions, attention over packed prompts and in decode steps over a
 * paged cache with a shared prefix, and the operations on that cache's pages.
 *
 * Conventions shared by every entry point
 *  - Every array pointer is a DEVICE pointer unless its comment says "host".
 *    The caller owns all memory; the library allocates nothing and keeps no
 *    state between calls.
 *  - Calls are asynchronous on `stream` (a hipStream_t; NULL = the default
 *    stream). Results are visible after the stream is synchronised. Calls are
 *    reentrant; calls that share output or state buffers must be ordered by the
 *    caller (same stream or events).
 *  - All arguments are validated on the host before any HIP call. A call that
 *    returns an error status has launched nothing and changed no buffer.
 *    GDN_ERR_LAUNCH is the only status reported after a launch was attempted.
 *  - Nothing aborts, prints or throws across this interface.
 *  - dtypes: activations may be f32, f16 or bf16 (gdn_dtype); states, gates given
 *    as g/beta, decay parameters, dt_bias and norm weights are f32.
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum gdn_status {
    GDN_OK = 0,
    GDN_ERR_NULL = 1,        /* a pointer the configuration needs is NULL */
    GDN_ERR_SHAPE = 2,       /* inconsistent sizes: counts < 0, Hv % Hk != 0, bad cu_seqlens */
    GDN_ERR_UNSUPPORTED = 3, /* valid but not built: head dims, conv width, dtype, flags */
    GDN_ERR_OVERFLOW = 4,    /* an element count or offset exceeds what the kernels index */
    GDN_ERR_ALIGN = 5,       /* a pointer or stride breaks the alignment a kernel needs */
    GDN_ERR_WORKSPACE = 6,   /* workspace NULL or smaller than the size query returned */
    GDN_ERR_LAUNCH = 7,      /* the HIP runtime reported an error for a launch */
    GDN_ERR_SCRATCH = 8      /* gdn_prefill_chunked_noalloc: the call needs more workspace
                                than its static scratch (GDN_NOALLOC_SCRATCH_BYTES) */
} gdn_status;

typedef enum gdn_dtype { GDN_F32 = 0, GDN_F16 = 1, GDN_BF16 = 2 } gdn_dtype;

/* Which k-head v-head h reads (docs.rs ferrox-core src/gdn.rs `HeadMap`;
 * ferrum-kernels tests page `GatedDeltaValueHeadMapping`):
 *   GROUPED: h / (Hv / Hk)   (Qwen3-Next order)
 *   TILED:   h % Hk          (Qwen3.5 order; "interleaved by key head")          */
typedef enum gdn_head_map { GDN_MAP_GROUPED = 0, GDN_MAP_TILED = 1 } gdn_head_map;

/* How the per-head decay parameter becomes the rate that multiplies softplus
 * (ferrum-kernels tests page, `cpu_segment` gate section):
 *   LOG_RATE:      rate = -exp(decay_param[h])   (decay_param is A_log)
 *   NEGATIVE_RATE: rate = decay_param[h]         (decay_param is -exp(A_log))   */
typedef enum gdn_decay { GDN_DECAY_LOG_RATE = 0, GDN_DECAY_NEGATIVE_RATE = 1 } gdn_decay;

/* gdn_dims.flags */
enum {
    /* q, k rows are normalised in-op: x * (sum x^2 + l2_eps)^(-1/2) per (token,
     * k-head) (ferrum-kernels tests page, `normalize_rows` and `cpu_segment`). */
    GDN_L2NORM_QK = 1u,
    /* gates from raw a, b: g = rate * softplus(a + dt_bias), beta = sigmoid(b)
     * (softplus with the +-20 cut-overs of that page's `softplus`). Without this
     * flag the caller passes g and beta directly. */
    GDN_RAW_GATES = 2u,
    /* output y = o * (mean_j o_j^2 + norm_eps)^(-1/2) * norm_weight * silu(z)
     * over the dv values of each (token, v-head) (that page's `cpu_segment`
     * output section). Without it the output is the core o itself. */
    GDN_GATED_NORM = 4u,
    /* Decode entry points only (the prefill returns UNSUPPORTED): a cache hint
     * for callers whose states do not stay in the GPU's last-level cache from
     * one call to the next (many layers or sequences, more state than the
     * cache holds). The state is loaded and stored with non-temporal hints;
     * results are bit for bit those of a call without the flag. On states the
     * cache does keep, the flag makes the step slower. */
    GDN_STREAM_STATE = 8u,
    /* gdn_linattn_* only (the gated delta entry points return UNSUPPORTED): every
     * token of v-head h decays by the one rate that decay_param[h] gives
     * (gdn_dims.decay). Without it the log decay is g, per token and head. */
    GDN_HEAD_DECAY = 16u
};

typedef struct gdn_dims {
    int32_t num_k_heads; /* Hk >= 1 */
    int32_t num_v_heads; /* Hv >= 1, Hv % Hk == 0 */
    int32_t head_dim_k;  /* dk */
    int32_t head_dim_v;  /* dv. Built (dk, dv), for every entry point: (32,32), (64,64),
                            (96,96), (128,128), (64,128), (128,64), (128,256),
                            (256,128), (256,256). Others: UNSUPPORTED. */
    int32_t head_map;    /* gdn_head_map */
    int32_t decay;       /* gdn_decay, used with GDN_RAW_GATES (and GDN_HEAD_DECAY) */
    uint32_t flags;      /* GDN_L2NORM_QK | GDN_RAW_GATES | GDN_GATED_NORM |
                            GDN_STREAM_STATE; gdn_linattn_*: GDN_HEAD_DECAY | GDN_STREAM_STATE */
    float scale;         /* read-out scale; 0 selects 1/sqrt(dk) */
    float l2_eps;        /* 0 selects 1e-6 */
    float norm_eps;      /* 0 selects 1e-6 */
} gdn_dims;

/* Per-token activations. A "token row" r indexes tokens: r = b * T + t for the
 * decode step (sequence b, token t of T) and the packed token index for the
 * prefill. Element (row r, head, i) of q is at q[r * q_stride + head * dk + i]
 * (same for k with k_stride, v with v_stride and dv), so q, k, v may be strided
 * views into one mixed [tokens][2*Hk*dk + Hv*dv] row. Strides are in elements.
 * The kernels read q, k and v in groups of 4 elements: each base pointer must be
 * aligned to 4 elements and each stride a multiple of 4 (else GDN_ERR_ALIGN). */
typedef struct gdn_inputs {
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    int32_t qkv_dtype;      /* gdn_dtype of q, k, v */
    /* GDN_RAW_GATES: a, b [tokens][Hv] contiguous in ab_dtype, aligned to their
     * element size; decay_param and dt_bias [Hv] f32. Every read stays within
     * the tokens*Hv elements. */
    const void *a, *b;
    int32_t ab_dtype;
    const float *decay_param, *dt_bias;
    /* no GDN_RAW_GATES: g (log decay, <= 0 in a real layer) and beta [tokens][Hv] f32,
     * 4-byte aligned */
    const float *g, *beta;
    /* GDN_GATED_NORM: z [tokens][Hv][dv] contiguous in z_dtype, 4-byte aligned
     * (read as 32-bit words; dv is even in every built shape, so no word reaches
     * past the last element); norm_weight [dv] f32 */
    const void *z;
    int32_t z_dtype;
    const float *norm_weight;
} gdn_inputs;

/* ---------------------------------------------------------------------------
 * gdn_conv_update -- depthwise causal conv1d + SiLU with carried raw inputs.
 * (ferrum-kernels tests page, `cpu_segment` conv section; docs.rs libmir-metal
 * 0.1.0 src/engine/gated_delta_layer/decode/mod.rs, `convolve`.)
 *
 * For sequence i with tokens [cu[i], cu[i+1]) and each channel c:
 *   y[r][c] = silu( sum_{m<K} weight[c][m] * xhat(t + m - (K-1)) ),  t = r - cu[i]
 * where xhat(j) = x[cu[i] + j][c] for j >= 0 and conv_state[i][c][(K-1) + j]
 * otherwise; afterwards conv_state[i][c][:] holds the last K-1 entries of
 * [old state || this call's inputs], oldest first. No bias. A zero-length
 * sequence leaves its state untouched.
 *
 *   channels      C >= 1
 *   kernel_size   K, 2 <= K <= 8
 *   num_seqs      N >= 0
 *   cu_seqlens    device int32 [N+1], cu[0] = 0, non-decreasing, cu[N] = total_tokens;
 *                 NULL means every sequence has total_tokens / N tokens (N must divide it)
 *   x             [total_tokens] rows of x_stride elements (>= C), x_dtype
 *   weight        [C][K] in x_dtype
 *   conv_state    [N][C][K-1] in x_dtype, updated in place
 *   y             [total_tokens] rows of y_stride elements (>= C), y_dtype; may not alias x
 * Errors: NULL, SHAPE (counts, strides), UNSUPPORTED (K, dtype), OVERFLOW.
 * ------------------------------------------------------------------------- */
gdn_status gdn_conv_update(int32_t channels, int32_t kernel_size, int32_t num_seqs,
                           const int32_t *cu_seqlens, int32_t total_tokens, int32_t x_dtype,
                           const void *x, int64_t x_stride, const void *weight, void *conv_state,
                           int32_t y_dtype, void *y, int64_t y_stride, void *stream);

/* ---------------------------------------------------------------------------
 * gdn_decode_step -- the recurrence for `batch` independent sequences of
 * `tokens_per_seq` tokens each, token order preserved, each sequence's state
 * read from HBM once and written once per call (ferrox-core src/gdn.rs
 * `delta_step` for one token; ferrum-kernels tests page `cpu_segment` for the
 * token loop, the gates and the gated norm).
 *
 *   dims            see gdn_dims; flags select L2 norm, raw gates, gated norm
 *   batch           B >= 0 sequences
 *   tokens_per_seq  T >= 1; token row of (b, t) is b*T + t
 *   in              activations; see gdn_inputs
 *   state           [num_slots][Hv][dv][dk] f32, key index innermost, 16-byte
 *                   aligned; updated in place
 *   state_slots     device int32 [B]: slot of sequence b; NULL means slot b.
 *                   A slot outside [0, num_slots) leaves that sequence's state
 *                   and output rows untouched.
 *   num_slots       number of state slots (>= B when state_slots is NULL)
 *   out_dtype, out  [B*T][Hv][dv]; may not alias any input or the state
 * Errors: NULL, SHAPE, UNSUPPORTED (dims, dtype), OVERFLOW, ALIGN (q/k/v groups of 4
 * elements; a, b to their element size; g, beta, z and norm_weight to 4 bytes; the
 * state to 16 bytes), LAUNCH.
 * ------------------------------------------------------------------------- */
gdn_status gdn_decode_step(const gdn_dims *dims, int32_t batch, int32_t tokens_per_seq,
                           const gdn_inputs *in, float *state, const int32_t *state_slots,
                           int32_t num_slots, int32_t out_dtype, void *out, void *stream);

/* The causal conv that gdn_decode_layer applies to q, k and v before the
 * recurrence: the same operation as gdn_conv_update over the channel order
 * [q (Hk*dk) | k (Hk*dk) | v (Hv*dv)] of the mixed projection row. */
typedef struct gdn_conv_args {
    int32_t kernel_size;  /* K; the built layer kernel supports K = 4 */
    const void *weight;   /* [channels][K] in the activations' dtype (qkv_dtype) */
    const void *state_in; /* [num_slots][channels][K-1], oldest first, qkv_dtype */
    void *state_out;      /* same shape; must not overlap state_in */
} gdn_conv_args;

/* ---------------------------------------------------------------------------
 * gdn_decode_layer -- one launch for the whole decode layer: causal conv + SiLU
 * of q, k, v with carried raw inputs (ferrum-kernels tests page, `cpu_segment`
 * conv section; libmir-metal decode/mod.rs `convolve`), then everything
 * gdn_decode_step does (L2 norm, gates, recurrence, gated norm).
 *
 * Arguments are those of gdn_decode_step, except:
 *   in->q, in->k, in->v  the PRE-conv projections (e.g. views into the mixed
 *                        [tokens][2*Hk*dk + Hv*dv] row)
 *   conv                 weights and conv state; the state is indexed by the
 *                        same slot as the delta state. The call reads state_in
 *                        and writes the window after its tokens to state_out
 *                        (a caller alternates two buffers); both must be aligned
 *                        to 4 elements. A slot outside [0, num_slots) leaves both
 *                        states and the output rows untouched.
 * Every v-head workgroup computes the conv of the q/k channels it reads; the
 * new q/k window is written by one workgroup per k-head, which is why the
 * state is not updated in place.
 * Slot pools: a call writes new windows only for the slots it names (and a
 * live slot's window only to state_out); for every other slot state_out keeps
 * what it held. A caller that alternates the two buffers while some calls do
 * not name every slot must therefore carry the windows of the slots a call left
 * out: e.g. copy those slots' windows from state_in to state_out after the
 * call, or keep per slot which buffer holds its latest window and gather the
 * windows of the next call's slots into the buffer passed as state_in. The
 * delta state is updated in place and needs no such care.
 * Errors: those of gdn_decode_step; NULL (conv pointers), UNSUPPORTED (K),
 * ALIGN (conv buffers), SHAPE (state_out overlapping state_in).
 * ------------------------------------------------------------------------- */
gdn_status gdn_decode_layer(const gdn_dims *dims, int32_t batch, int32_t tokens_per_seq,
                            const gdn_conv_args *conv, const gdn_inputs *in, float *state,
                            const int32_t *state_slots, int32_t num_slots, int32_t out_dtype,
                            void *out, void *stream);

/* ---------------------------------------------------------------------------
 * gdn_prefill_workspace_bytes -- device workspace gdn_prefill_chunked needs for
 * at most num_seqs sequences and total_tokens packed tokens (an upper bound
 * over every split of total_tokens into num_seqs lengths). Returns 0 when the
 * arguments are invalid.
 * ------------------------------------------------------------------------- */
size_t gdn_prefill_workspace_bytes(const gdn_dims *dims, int32_t num_seqs, int32_t total_tokens);

/* ---------------------------------------------------------------------------
 * gdn_prefill_chunked -- the same recurrence over packed variable-length
 * sequences, computed chunk-parallel (64-token chunks -- 32 when dk = 256 --
 * that start at each sequence's first token and never straddle two
 * sequences). Each path runs a kernel parallel over (chunk, k-head) that forms
 * the chunk's own quantities, then a carry per (sequence, v-head, slice of dv
 * rows) that runs the state-dependent products chunk after chunk. dk = dv = 128
 * takes f16 MFMA operands; the other head shapes keep f32 accuracy (f32 MFMA,
 * and bf16 hi/lo operand pairs on bf16 MFMA in the carry). The result equals
 * the token-by-token recurrence up to rounding order (ferrox-core src/gdn.rs
 * module doc: the chunked form is the same recurrence summed in another order;
 * ferrum-kernels tests page, `chunked_c64_matches_recurrent_oracle_and_
 * non_aligned_state_continuity`).
 *
 *   num_seqs         N >= 0
 *   cu_seqlens_host  host int32 [N+1] (validated: cu[0] = 0, non-decreasing,
 *                    cu[N] = total_tokens)
 *   cu_seqlens_dev   device int32 [N+1], the same values
 *   in               activations indexed by packed token row
 *   state            [N][Hv][dv][dk] f32: initial state in, final state out
 *   out_dtype, out   [total_tokens][Hv][dv]
 *   workspace        device, >= gdn_prefill_workspace_bytes(dims, N, total_tokens),
 *                    256-byte aligned; contents are scratch
 * Errors: NULL, SHAPE, UNSUPPORTED, OVERFLOW, ALIGN, WORKSPACE, LAUNCH.
 * ------------------------------------------------------------------------- */
gdn_status gdn_prefill_chunked(const gdn_dims *dims, int32_t num_seqs,
                               const int32_t *cu_seqlens_host, const int32_t *cu_seqlens_dev,
                               int32_t total_tokens, const gdn_inputs *in, float *state,
                               int32_t out_dtype, void *out, void *workspace,
                               size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * gdn_prefill_chunked_noalloc -- gdn_prefill_chunked for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation): the same kernels and results, with the
 * workspace in a static device array of the library instead of a caller buffer.
 *
 * Arguments and errors are those of gdn_prefill_chunked without the workspace.
 * The call allocates nothing. The array holds GDN_NOALLOC_SCRATCH_BYTES per GPU
 * (64 MiB: about 1,700 tokens of one sequence at Hk=16, Hv=32, dk=dv=128 without
 * the gated norm); a call whose gdn_prefill_workspace_bytes exceeds it returns
 * GDN_ERR_SCRATCH and launches nothing. Each GPU the library runs on holds its
 * own copy of the array until the process ends (its device address is looked
 * up on the first call on that device). Every call on one GPU shares that GPU's
 * copy and leaves its contents behind; nothing in it needs to start at zero.
 * Calls that overlap in time on one GPU (different streams, or different host
 * threads without ordering) race on the array: order them.
 * ------------------------------------------------------------------------- */
#define GDN_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
gdn_status gdn_prefill_chunked_noalloc(const gdn_dims *dims, int32_t num_seqs,
                                       const int32_t *cu_seqlens_host,
                                       const int32_t *cu_seqlens_dev, int32_t total_tokens,
                                       const gdn_inputs *in, float *state, int32_t out_dtype,
                                       void *out, void *stream);

/* ---------------------------------------------------------------------------
 * Linear attention with a decay: per v-head and token,
 *
 *     S <- exp(g) S + v k^T,   o = scale (S q)
 *
 * on the state layout, head maps, activations (gdn_inputs: q, k, v with their
 * strides and dtype) and head shapes of the gated delta entry points.
 *
 *   dims   flags: GDN_HEAD_DECAY, and GDN_STREAM_STATE for the decode step; others
 *          UNSUPPORTED. l2_eps and norm_eps are ignored.
 *   in     with GDN_HEAD_DECAY the log decay of head h is -exp(decay_param[h])
 *          (GDN_DECAY_LOG_RATE) or decay_param[h] (GDN_DECAY_NEGATIVE_RATE), [Hv]
 *          f32; without it in->g [tokens][Hv] f32. Both 4-byte aligned. The other
 *          gate fields, z and norm_weight are ignored.
 *
 * -inf stands for exp(g) = 0: the state is forgotten. Log decays above 0 let the state
 * grow; in the prefill exp of their sum over any run of a sequence's tokens must stay
 * finite, also where the state is 0.
 * A NaN or infinity in q, k, v or the state makes what the formula makes of it not
 * finite, and nothing else (where the formula has an infinity, the prefill may have a
 * NaN; a later exp(g) = 0 does not clear either).
 * Sums are f32 or more exact, whatever the output's type (of values below 2^-109 the
 * prefill may leave out what lies below 2^-133). A call without tokens does nothing,
 * whatever its per-token pointers.
 * ------------------------------------------------------------------------- */

/* gdn_linattn_decode_step -- B sequences of T tokens each; arguments, slots and
 * errors as gdn_decode_step's. Each state is read and written once per call. The
 * slots that a call names must differ from one another: a slot named twice holds
 * either sequence's rows afterwards. */
gdn_status gdn_linattn_decode_step(const gdn_dims *dims, int32_t batch, int32_t tokens_per_seq,
                                   const gdn_inputs *in, float *state, const int32_t *state_slots,
                                   int32_t num_slots, int32_t out_dtype, void *out, void *stream);

/* gdn_linattn_prefill_workspace_bytes -- device workspace that
 * gdn_linattn_prefill_chunked needs for at most num_seqs sequences and total_tokens
 * packed tokens. Returns 0 when the arguments are invalid. */
size_t gdn_linattn_prefill_workspace_bytes(const gdn_dims *dims, int32_t num_seqs,
                                           int32_t total_tokens);

/* gdn_linattn_prefill_chunked -- the same over packed variable-length sequences;
 * arguments and errors as gdn_prefill_chunked's, and: OVERFLOW for a row stride (of q, k
 * or v, or Hv*dv) of 2^24 elements or more, ALIGN for an out not aligned to 16 bytes. An
 * empty sequence keeps its state.
 * The workspace is scratch: calls that may overlap in time (other streams, two
 * captured graphs) need one each. */
gdn_status gdn_linattn_prefill_chunked(const gdn_dims *dims, int32_t num_seqs,
                                       const int32_t *cu_seqlens_host,
                                       const int32_t *cu_seqlens_dev, int32_t total_tokens,
                                       const gdn_inputs *in, float *state, int32_t out_dtype,
                                       void *out, void *workspace, size_t workspace_bytes,
                                       void *stream);

/* ---------------------------------------------------------------------------
 * gdn_add_rms_norm -- RMS norm of rows, with the residual's addition before it and
 * an 8-bit output after it, each as the caller asks:
 *
 *     h = x + residual;   y = h (mean_i h_i^2 + eps)^(-1/2) weight
 *     residual_out = h;   out = y;   out_scale = max_i |y_i| / 127
 *     out_q = y 127 / max_i |y_i|, rounded to nearest, ties to even
 *
 * computed in f32 from the unrounded h, each output rounded once.
 * A row whose squares' sum leaves f32's range has y = 0.
 * A row whose largest |y| is below 2^-100 has out_q = 0 and out_scale = 0. A row
 * with an infinite or NaN y has out_q = 0 and out_scale = NaN.
 *
 *   rows, hidden   >= 0 rows of 1 to 2^24 elements (more: OVERFLOW)
 *   dtype          of x, residual and residual_out
 *   x, residual    rows of x_stride / residual_stride elements (>= hidden), aligned to
 *                  their element size; residual may be NULL (h = x)
 *   residual_out   NULL, or rows of residual_out_stride elements; may be x's or
 *                  residual's own buffer (same pointer and stride), else may not
 *                  overlap an input
 *   weight         [hidden] f32, 4-byte aligned
 *   eps            0 selects 1e-6
 *   out            NULL, or rows of out_stride elements of out_dtype; may be x's own
 *                  buffer (same pointer, stride and dtype), else may not overlap an input
 *   out_q          NULL, or int8 rows of out_q_stride; out_scale [rows] f32 goes with it
 *                  (both or neither)
 * At least one of out and out_q. Outputs may not overlap one another.
 * Errors: NULL, SHAPE (counts, strides, eps), UNSUPPORTED (dtype), OVERFLOW, ALIGN, LAUNCH.
 * ------------------------------------------------------------------------- */
typedef struct gdn_norm_args {
    int32_t rows, hidden;
    int32_t dtype;
    const void *x;
    int64_t x_stride;
    const void *residual;
    int64_t residual_stride;
    void *residual_out;
    int64_t residual_out_stride;
    const float *weight;
    float eps;
    int32_t out_dtype;
    void *out;
    int64_t out_stride;
    int8_t *out_q;
    int64_t out_q_stride;
    float *out_scale;
} gdn_norm_args;
gdn_status gdn_add_rms_norm(const gdn_norm_args *args, void *stream);

/* ---------------------------------------------------------------------------
 * gdn_quant_matmul -- product of 8-bit integers with a scale for each token (row of
 * a) and each channel (row of w):
 *
 *     out[m][n] = (sum_k a[m][k] w[n][k]) a_scale[m] w_scale[n]
 *
 * The integer sums are exact (32 bits); the scales are applied in f32, a_scale first, and
 * the result is rounded once. A NaN scale makes its row or column NaN.
 *
 *   M, N, K      M, N >= 0, at most 2^31 - 256 and ceil(M / 256) ceil(N / 256) below 2^23
 *                (else OVERFLOW); K >= 1 a multiple of 16 (else UNSUPPORTED), at most
 *                131056 (else OVERFLOW: the sum could leave 32 bits)
 *   a            [M] int8 rows of a_stride bytes (>= K)
 *   w            [N] int8 rows of w_stride bytes (>= K): a torch Linear's weight layout
 *                a, w and both strides are multiples of 16 bytes, strides below 2^23
 *                (else OVERFLOW)
 *   a_scale      [M] f32; w_scale [N] f32; 4-byte aligned
 *   out          [M] rows of out_stride elements (>= N) of out_dtype, aligned to the element
 * Errors: NULL, SHAPE, UNSUPPORTED, OVERFLOW, ALIGN, LAUNCH.
 * ------------------------------------------------------------------------- */
gdn_status gdn_quant_matmul(int32_t M, int32_t N, int32_t K, const int8_t *a, int64_t a_stride,
                            const float *a_scale, const int8_t *w, int64_t w_stride,
                            const float *w_scale, int32_t out_dtype, void *out,
                            int64_t out_stride, void *stream);

/* ---------------------------------------------------------------------------
 * gdn_rope -- rotary positions: a pair (a, b) of a head's first rotary_dim elements, at
 * position p and with frequency w of the pair, becomes
 *
 *     (a c - b s, b c + a s),   c = magnitude cos(p w),   s = magnitude sin(p w)
 *
 * and the head's other elements stay. The angle is formed and reduced in 64 bits, the
 * pair is turned in f32, each output is rounded once. q, k, or both; with page pools
 * the turned k and v go to the cache's pages instead of rows.
 *
 *   tokens         >= 0 rows
 *   q_heads, kv_heads, head_dim   head_dim 2 to 1024; rotary_dim even, 2 to head_dim
 *   layout         GDN_ROPE_HALF pairs (i, i + rotary_dim / 2), GDN_ROPE_INTERLEAVED
 *                  (2 i, 2 i + 1)
 *   dtype          of every row and page
 *   positions      [tokens] int32, from 0 on (any other value turns as the formula has it)
 *   inv_freq       [rotary_dim / 2] f64, radians a token, finite
 *   magnitude      0 selects 1
 *   q, q_out       rows of q_heads * head_dim elements with strides q_stride, q_out_stride;
 *                  q_out may be q itself (same pointer and stride), else may not overlap
 *                  an input. Both NULL: no q.
 *   k, k_out       the same for k (kv_heads); k_out only without pages. k NULL: no k.
 *   k_pages, v_pages  NULL, or page pools (gdn_attention_args): row t of the turned k and
 *                  of v (rows of v_stride) goes to slot slots[t] = page * page_size + token
 *                  in page. A slot outside [0, num_pages * page_size) is not stored. Slots
 *                  of a call differ; of two tokens with one slot either may be stored.
 *   page_size      a power of two from 16 to 1024; num_pages * page_size below 2^31
 *   page_stride    elements from page to page, >= kv_heads * page_size * head_dim
 * Pointers are aligned to their element (positions, slots 4, inv_freq 8 bytes).
 * Errors: NULL, SHAPE, UNSUPPORTED (dtype, layout, head or rotary dims, page size),
 * OVERFLOW, ALIGN, LAUNCH.
 * ------------------------------------------------------------------------- */
typedef enum gdn_rope_layout { GDN_ROPE_HALF = 0, GDN_ROPE_INTERLEAVED = 1 } gdn_rope_layout;
typedef struct gdn_rope_args {
    int32_t tokens, q_heads, kv_heads, head_dim, rotary_dim;
    int32_t layout, dtype;
    float magnitude;
    const int32_t *positions;
    const double *inv_freq;
    const void *q;
    int64_t q_stride;
    void *q_out;
    int64_t q_out_stride;
    const void *k;
    int64_t k_stride;
    void *k_out;
    int64_t k_out_stride;
    const void *v;
    int64_t v_stride;
    void *k_pages, *v_pages;
    int64_t page_stride;
    int32_t num_pages, page_size;
    const int32_t *slots;
} gdn_rope_args;
gdn_status gdn_rope(const gdn_rope_args *args, void *stream);

/* gdn_rope_frequencies -- fills inv_freq (HOST, [rotary_dim / 2] f64) and magnitude (HOST)
 * for gdn_rope: theta^(-2 i / rotary_dim), stretched for contexts `factor` (>= 1) times as long:
 *   GDN_ROPE_PLAIN    as it is
 *   GDN_ROPE_LINEAR   divided by factor
 *   GDN_ROPE_BASE     theta times factor^(r / (r - 2)) (r = rotary_dim >= 4): the slowest pair
 *                     is divided by factor, the fastest stays
 *   GDN_ROPE_BANDS    pairs that turn beta_fast times or more in original_length tokens stay,
 *                     those that turn beta_slow times or less are divided by factor, between
 *                     them the two are mixed in proportion to the pair's index; magnitude
 *                     0.1 ln(factor) + 1 (1 with the other kinds)
 * The index at which a pair turns n times is r ln(original_length / (2 pi n)) / (2 ln theta),
 * rounded down for beta_fast and up for beta_slow and kept within [0, r - 1].
 * Makes no HIP call. Errors: NULL, SHAPE (theta <= 1, factor < 1, original_length < 1,
 * 0 < beta_slow <= beta_fast not held), UNSUPPORTED (kind, rotary_dim). */
typedef enum gdn_rope_scaling {
    GDN_ROPE_PLAIN = 0,
    GDN_ROPE_LINEAR = 1,
    GDN_ROPE_BASE = 2,
    GDN_ROPE_BANDS = 3
} gdn_rope_scaling;
gdn_status gdn_rope_frequencies(int32_t rotary_dim, double theta, int32_t scaling, double factor,
                                double original_length, double beta_fast, double beta_slow,
                                double *inv_freq, float *magnitude);

/* ---------------------------------------------------------------------------
 * Softmax attention of grouped heads: query head h reads key head h / (q_heads / kv_heads),
 *
 *     o_i = sum_j p_ij v_j,   p_ij = exp(scale q_i k_j) / sum_j exp(scale q_i k_j)
 *
 * over the keys j that query i sees. Scores, their maximum and sum and the outputs are
 * f32 sums; p enters the product with v rounded to the 16 bits of v, by up to half a step
 * (f16, below 2^-21 of the row's largest: by up to 2^-32 of that), and o is rounded once.
 * A query that sees no key, or whose scores are all -inf, has o = 0 and lse = -inf.
 * Infinities and NaN in keys, values or queries that a query does not see do not reach
 * it; in those it sees they make what the formula makes of them not finite (where that
 * is an infinity, a NaN may stand; the value of a key of score -inf may be left out instead).
 * Finite f16 values and scores have finite outputs. Outputs are summed before they are divided
 * by the sum of weights, of at most 2^8 each (f16 2^15): bf16 values of 2^90 and more may leave
 * f32 on the way, as may scores times scale.
 *
 *   q_heads, kv_heads   q_heads a multiple of kv_heads, both >= 1
 *   head_dim       64, 96, 128 or 256
 *   dtype          of q, k, v and out: f16 or bf16
 *   scale          0 selects head_dim^(-1/2)
 *   q, out         rows of q_heads * head_dim elements with strides q_stride, out_stride
 *   lse            NULL, or [rows][q_heads] f32: ln sum_j exp(scale q_i k_j)
 *   k, v           page_size 0: packed rows of kv_heads * head_dim elements, k_stride and
 *                  v_stride elements apart. Else pools of pages [kv_heads][page_size]
 *                  [head_dim], k_stride and v_stride elements from page to page
 *   page_size      0, or a power of two from 16 to 1024
 *   num_pages      pages of the pools
 *   table          [sequences][table_stride] int32: page of token n of a sequence is entry
 *                  n / page_size. Keys of an entry outside [0, num_pages) are not seen.
 * q, k, v, out and their strides are multiples of 16 bytes, lse, table 4 bytes.
 * out may not overlap an input.
 * ------------------------------------------------------------------------- */
typedef struct gdn_attention_args {
    int32_t q_heads, kv_heads, head_dim, dtype;
    float scale;
    const void *q;
    int64_t q_stride;
    void *out;
    int64_t out_stride;
    float *lse;
    const void *k, *v;
    int64_t k_stride, v_stride;
    int32_t page_size, num_pages;
    const int32_t *table;
    int64_t table_stride;
} gdn_attention_args;

/* gdn_attention_prefill -- prompts packed one after another, causal: sequence s has the
 * queries [cu_q[s], cu_q[s + 1]) and cu_k[s + 1] - cu_k[s] keys, of which its last query
 * sees all, the one before all but one, and so on. Packed keys are the rows
 * [cu_k[s], cu_k[s + 1]); on pages they are the first tokens of table row s. More queries
 * than keys: the first ones see none.
 *   cu_q, cu_k     [num_seqs + 1] int32, ascending from 0, on the host and on the device
 *                  with the same values; both cu_k NULL: cu_q
 *   workspace      of the bytes that the query gives for these counts, aligned to 256; NULL
 *                  where it gives 0. Scratch: calls that may overlap in time (other streams,
 *                  two captured graphs) need one each.
 * Rows behind cu_q[num_seqs] are not touched.
 * Errors: NULL, SHAPE (counts, strides, offsets; table rows shorter than a sequence),
 * UNSUPPORTED, OVERFLOW (a row stride of 2^24 elements or more, more than 2^31 - 1 rows times
 * heads, more than 2^21 keys of a sequence, which f32 sums no longer resolve, or a grid of 2^32
 * threads), ALIGN, WORKSPACE, LAUNCH. */
size_t gdn_attention_prefill_workspace_bytes(int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                             int32_t num_seqs, int32_t total_tokens);
gdn_status gdn_attention_prefill(const gdn_attention_args *args, int32_t num_seqs,
                                 const int32_t *cu_q_host, const int32_t *cu_q_dev,
                                 const int32_t *cu_k_host, const int32_t *cu_k_dev,
                                 void *workspace, size_t workspace_bytes, void *stream);

/* gdn_attention_decode -- tokens_per_seq (T) new tokens of each of `batch` sequences, whose
 * keys are on pages (page_size 0 UNSUPPORTED): first prefix_len keys that the whole batch
 * shares, read and multiplied once for all, then the sequence's own, lens[b] tokens (the T
 * new ones among them) of table row b. Query t sees the prefix and the first
 * lens[b] - T + 1 + t own keys.
 *   q, out, lse    row b * T + t
 *   lens           [batch] int32 on the device; of more than max_len tokens the first
 *                  max_len are there, below 0 counts as 0
 *   max_len        an upper bound of lens that sizes the grid and the workspace
 *   prefix_table   [ceil(prefix_len / page_size)] int32 pages of the prefix; NULL where
 *                  prefix_len is 0
 *   workspace      as above
 * Errors: as gdn_attention_prefill's (OVERFLOW: max_len above 2^30, prefix_len above 2^21). */
size_t gdn_attention_decode_workspace_bytes(int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                            int32_t batch, int32_t tokens_per_seq, int32_t max_len,
                                            int32_t prefix_len);
gdn_status gdn_attention_decode(const gdn_attention_args *args, int32_t batch,
                                int32_t tokens_per_seq, const int32_t *lens, int32_t max_len,
                                const int32_t *prefix_table, int32_t prefix_len, void *workspace,
                                size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * The pages of a cache. A table row lists the pages of one sequence in order, -1 where
 * there is none; refs counts the rows' references to each page, and a page with none is
 * free. Free pages are handed out lowest first, in the order of the requests and of a row's
 * entries. Pages of a row are its first entries.
 *
 *   table          [rows][table_stride] int32, width entries of each row in use
 *   refs           [num_pages] int32
 *   page_size      tokens a page holds, >= 1
 *   data           the pages of every layer's keys and values: num_planes planes of
 *                  num_pages pages of page_bytes, page and plane strides in bytes; all
 *                  multiples of 16, data too (page_bytes at most 2^30)
 * A request for a row outside [0, rows), to change a row that an earlier request of the
 * call names too, or on rows that do not hold what it needs is refused: its status is 2 and
 * nothing of it is done. Entries outside [0, num_pages) count as none.
 * Calls on one table and refs are ordered by the caller; n is at most 1024, num_pages, width
 * and rows * width at most 2^30 (else OVERFLOW).
 * Errors: NULL, SHAPE, OVERFLOW, ALIGN, WORKSPACE, LAUNCH.
 * ------------------------------------------------------------------------- */
typedef struct gdn_page_args {
    int32_t *table;
    int64_t table_stride;
    int32_t rows, width;
    int32_t *refs;
    int32_t num_pages, page_size;
    void *data;
    int32_t num_planes;
    int64_t plane_stride, page_stride, page_bytes;
} gdn_page_args;

/* gdn_pages_free -- releases the entries keep[i] and later (all, keep NULL) of row rows[i]:
 * their pages' refs go down by one, the entries become -1. A row named twice is released
 * once, from the lower of its keep on. data is not used. */
gdn_status gdn_pages_free(const gdn_page_args *args, int32_t n, const int32_t *rows,
                          const int32_t *keep, void *stream);

/* gdn_pages_reserve -- gives row rows[i] a page for each of the first ceil(lens[i] /
 * page_size) entries that has none. status[i]: 0 done, 1 pages are needed, but too few were
 * left for it and the requests before it (nothing of it done), 2 refused (also lens[i] below
 * 0 or past the row). data is not used. */
gdn_status gdn_pages_reserve(const gdn_page_args *args, int32_t n, const int32_t *rows,
                             const int32_t *lens, int32_t *status, void *stream);

/* gdn_pages_fork -- row dst[i], which holds no page, becomes the first lens[i] tokens of
 * row src[i]: full pages are shared (refs up by one), a last page filled in part is copied
 * to a free one, on every plane. status as gdn_pages_reserve's; refused also where the
 * source lacks a page of them or is a dst of the call. One source may be forked many times.
 * workspace: gdn_pages_workspace_bytes(num_pages), aligned to 256. */
size_t gdn_pages_workspace_bytes(int32_t num_pages);
gdn_status gdn_pages_fork(const gdn_page_args *args, int32_t n, const int32_t *src,
                          const int32_t *dst, const int32_t *lens, int32_t *status,
                          void *workspace, size_t workspace_bytes, void *stream);

/* gdn_pages_compact -- moves the pages in use together: with U of them, the i-th page in use
 * at U or later goes to the i-th free page below U, on every plane; table and refs follow
 * (the whole width of every row). page_map [num_pages]: where each page went, itself where
 * it did not move. used [1]: U. page_size is not used. workspace as gdn_pages_fork's. */
gdn_status gdn_pages_compact(const gdn_page_args *args, int32_t *page_map, int32_t *used,
                             void *workspace, size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * Kernel selection, for inspection and host-side tests. Which kernel a call runs
 * follows from its shape and from the device, as the ferrum-kernels tests page
 * checks for its own kernels (`chunk_k_gram_specialization_requires_repeated_
 * k128_heads`, `simd_delta_specialization_is_shape_and_device_capability_driven`).
 * These calls report the choice the corresponding entry point makes, from the
 * same code; they make no HIP call and launch nothing.
 * ------------------------------------------------------------------------- */
typedef struct gdn_launch_info {
    int32_t waves;             /* decode: waves per workgroup */
    int32_t lanes_per_row;     /* decode: lanes holding one dk-wide state row */
    int32_t token_mode;        /* decode: 0 any token count, 1 token groups (fused layer,
                                  T > 1), 2 one token per sequence */
    int32_t nontemporal;       /* decode: 1 when GDN_STREAM_STATE selects the hinted kernel */
    int32_t carry_kind;        /* prefill: 0 split carry (compute + output wave per dv
                                  slice), 1 carry (one wave per slice); 2 the f32 carry
                                  of the head shapes other than 128 x 128 */
    int32_t slices_per_workgroup; /* prefill: 16-row dv slices per carry workgroup */
    int32_t workgroups;        /* grid of the decode kernel, of the prefill carry, or of the
                                  int8 product (which has this and threads alone) */
    int32_t threads;           /* threads per workgroup of that kernel */
    int32_t prep_workgroups;   /* prefill: grid of the per-chunk preparation kernel */
} gdn_launch_info;

/* The decode kernel gdn_decode_step (fused_conv = 0) or gdn_decode_layer
 * (fused_conv = 1) runs for these dims (flags included), batch and tokens_per_seq.
 * Errors: NULL, SHAPE, UNSUPPORTED, as the entry points report them. */
gdn_status gdn_decode_launch_info(const gdn_dims *dims, int32_t batch, int32_t tokens_per_seq,
                                  int32_t fused_conv, gdn_launch_info *info);

/* The kernels gdn_prefill_chunked runs for these dims and sequences on a device
 * with `compute_units` CUs (the entry point queries the current device's count).
 * cu_seqlens_host: host int32 [N+1]. Errors: NULL, SHAPE, UNSUPPORTED. */
gdn_status gdn_prefill_launch_info(const gdn_dims *dims, int32_t num_seqs,
                                   const int32_t *cu_seqlens_host, int32_t total_tokens,
                                   int32_t compute_units, gdn_launch_info *info);

/* The kernel gdn_quant_matmul runs for these counts (none: workgroups 0). Errors: NULL, and
 * SHAPE, UNSUPPORTED, OVERFLOW as the entry point reports them for M, N, K. */
gdn_status gdn_quant_matmul_launch_info(int32_t M, int32_t N, int32_t K, gdn_launch_info *info);

/* Static, NUL-terminated description of a status code. */
const char *gdn_status_string(gdn_status status);

/* Library version as MAJOR * 10000 + MINOR * 100 + PATCH. */
int32_t gdn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H */
