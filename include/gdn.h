/*
 * gdn.h -- C ABI of the MI355X (gfx950) chunkwise-parallel gated delta rule.
 *
 * The operation (all pages agree once the orientation is fixed; S is
 * d_v x d_k and o = S q):
 *
 *     S_t = alpha_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T
 *     o_t = S_t q_t                     (the output sees token t's write)
 *
 * Sources: "从零开始的 GDN 推导", the recurrent form under the notation
 * section (gate alpha_t multiplying the erased state) and the section on O
 * (o_t = q_t S_{t+1}, i.e. inclusive); "RNN的复兴03:现代RNN的并行计算",
 * section 1, equation (2) (S in R^{d_v x d_k}); the circuit-complexity page,
 * "类 RNN 模型训练" (o_t = S_t q_t).  The library evaluates it with the
 * chunkwise-parallel method of "从零开始的 GDN 推导" (UT transform, W and U,
 * per-chunk state and output, chunks chained), which reaches the same result
 * up to rounding order.
 *
 * Conventions for every entry point:
 *  - Tensor pointers are DEVICE pointers to row-major, contiguous memory on
 *    the current HIP device; the caller owns all of them.  The library never
 *    allocates, frees or keeps a pointer after the call returns.
 *  - Calls are stream-ordered and asynchronous: `stream` is a hipStream_t
 *    (NULL = the default stream).  The return value reports argument
 *    validation and launch errors; a fault inside a kernel surfaces at the
 *    caller's next synchronisation.
 *  - No global mutable state: the functions are thread-safe and re-entrant.
 *  - Values are not checked: NaN or Inf in the inputs propagate to the
 *    outputs of the affected (b, h) sequence only.
 *  - Nothing is written when validation fails.
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    GDN_OK = 0,
    GDN_ERR_NULL_ARG = 1,     /* a required pointer is NULL                   */
    GDN_ERR_BAD_SHAPE = 2,    /* B, H, T < 1, or a dimension out of range     */
    GDN_ERR_BAD_DTYPE = 3,    /* dtype code not one of gdn_dtype              */
    GDN_ERR_UNSUPPORTED = 4,  /* valid but not built: e.g. chunk/d_k/dtype mix */
    GDN_ERR_WORKSPACE = 5,    /* workspace smaller than the query returned    */
    GDN_ERR_HIP = 6           /* the HIP runtime reported an error            */
} gdn_status;

typedef enum { GDN_BF16 = 0, GDN_F32 = 1 } gdn_dtype;

typedef struct {
    int32_t B, H, T;          /* batch, heads, sequence length (T >= 1)        */
    int32_t d_k, d_v;         /* key/query and value head dimensions           */
    int32_t chunk_size;       /* C: tokens per chunk                           */
    int32_t qkv_dtype;        /* gdn_dtype of q, k and v (one dtype for all)   */
    int32_t o_dtype;          /* gdn_dtype of O (GDN_F32 recommended)          */
} gdn_shape;

/*
 * Supported combinations (anything else that is well-formed returns
 * GDN_ERR_UNSUPPORTED):
 *   chunk_size in {16, 32, 64};
 *   qkv_dtype GDN_BF16: d_k in {16, 32, 64, 96, 128, 256} (d_k 16 runs on
 *                       the d_k 32 kernel with the keys and queries padded
 *                       with zeros as they are staged: the MFMAs take 32
 *                       elements per k-step; no sequence-parallel segments);
 *   qkv_dtype GDN_F32:  d_k in {16, 32, 64, 128, 256};
 *   at d_k 256 a chunk of 64 tokens is computed as two chunks of 32 (its
 *   64-token tiles would need more than the 160 KB of LDS of one compute
 *   unit): the same recurrence grouped differently, so the same result up
 *   to rounding (gdn_chunk_fwd_stages, whose T is laid out per chunk, and
 *   gdn_chunk_prep reject that case);
 *   d_v a multiple of 16 in [16, 1024]; one head's largest tensor (T x
 *   max(d_k, d_v) x 4 bytes) below 2 GiB.
 * T may be any value >= 1; a last chunk shorter than chunk_size is handled
 * exactly (padding tokens are identity transitions).
 *
 * Arithmetic.  bf16 inputs run one fused kernel whose matrix products take
 * fp16 operands (11 significant bits; bf16 inputs convert exactly) with fp32
 * accumulation and an fp32 state: against the exact result the normwise
 * error is near 6e-4 on gated workloads.  Operands must stay inside the fp16
 * range (|x| < 65504; the state and the values are the ones that grow).
 * Without decay and with beta near 2 (reflections) the state keeps every
 * rounding, so the error grows with the number of chunks; gdn_chunk_fwd_precise
 * then keeps it near 1e-5.  f32 inputs use fp32 matrix products throughout.
 */

/*
 * Bytes of device workspace gdn_chunk_fwd (and gdn_chunk_fwd_eta) needs for
 * this shape on the current device: 0 unless the call takes the
 * sequence-parallel form (see gdn_chunk_fwd_seq), which it does for bf16
 * inputs when the heads and value tiles would leave compute units idle (few
 * heads, long sequences).  Returns (size_t)-1 if the shape is invalid or
 * unsupported.
 */
size_t gdn_chunk_fwd_workspace_bytes(const gdn_shape* s);

/*
 * Chunkwise-parallel forward pass.  Layouts:
 *   q, k     [B, H, T, d_k]   qkv_dtype   (k rows are usually L2-normalised
 *                                          by the caller; not required)
 *   v        [B, H, T, d_v]   qkv_dtype
 *   alpha    [B, H, T] float, gate in (0, 1]; NULL means alpha = 1 (no gate).
 *            alpha <= 0 is outside the method (its logarithm is used).
 *   beta     [B, H, T] float, any finite value (the pages use (0, 2)).
 *   S0       [B, H, d_v, d_k] float initial state; NULL means zero.
 *   O        [B, H, T, d_v]   o_dtype, written.
 *   S_final  [B, H, d_v, d_k] float, written; may be the same pointer as S0
 *            (the state is updated in place).
 * workspace / workspace_bytes: at least gdn_chunk_fwd_workspace_bytes(s)
 * bytes of device memory (may be NULL when that is 0).
 */
gdn_status gdn_chunk_fwd(const gdn_shape* s,
                         const void* q, const void* k, const void* v,
                         const float* alpha, const float* beta, const float* S0,
                         void* O, float* S_final,
                         void* workspace, size_t workspace_bytes,
                         void* stream);

/*
 * The same pass with a separate write strength eta ("RNN的复兴03", section 1:
 * erase strength beta, write strength eta):
 *     S_t = alpha_t S_{t-1} (I - beta_t k_t k_t^T) + eta_t v_t k_t^T.
 * eta [B, H, T] float, any finite value; NULL means eta = beta, which is
 * exactly gdn_chunk_fwd.  beta = 0, eta = 1 gives gated linear attention
 * ("从电路复杂性理论的角度分析大模型的可并行性和表达能力", GLA).
 * Everything else as gdn_chunk_fwd.
 */
gdn_status gdn_chunk_fwd_eta(const gdn_shape* s,
                             const void* q, const void* k, const void* v,
                             const float* alpha, const float* beta, const float* eta,
                             const float* S0, void* O, float* S_final,
                             void* workspace, size_t workspace_bytes,
                             void* stream);

/*
 * gdn_chunk_fwd_eta with the sequence-parallel form chosen by the caller.
 * The state recurrence is linear in the state, so it is associative and can
 * be evaluated by a parallel scan ("Параллельность RNN?", section
 * "Уровень 2"); the chunk form already passes each chunk's end state to the
 * next ("从零开始的 GDN 推导", 总结).  Each sequence is cut into segments of
 * seg_chunks chunks (the last one shorter).  All segments run at once: the
 * first from S0; every later one from a zero state, together with the d_k
 * rows of its transition M = A_first ... A_last (A_t = alpha_t (I - beta_t
 * k_t k_t^T)) started from the identity, whose outputs are the queries
 * carried through the segment, qm_t = A_first ... A_t q_t.  A combine over
 * segments (X_{j+1} = X_j M_j + E_j, E_j the end state from zero) and a
 * correction o_t += X_j qm_t finish the pass.  Results equal those of the
 * plain form up to rounding (the combine and the correction multiply
 * split-bf16 operands, about 16 significant bits, with fp32 accumulation).
 *   seg_chunks  0: the form and segment length gdn_chunk_fwd would choose;
 *               >= 1: segments of that many chunks (one segment, i.e.
 *               seg_chunks >= ceil(T / chunk_size), is the plain form);
 *               < 0: GDN_ERR_BAD_SHAPE.  More than one segment needs bf16
 *               inputs (else GDN_ERR_UNSUPPORTED).
 * workspace: at least gdn_chunk_fwd_seq_workspace_bytes(s, seg_chunks)
 * bytes of device memory, 256-byte aligned (GDN_ERR_WORKSPACE if smaller or
 * NULL when needed).  After the call it holds, from offset 0,
 *   [B*H][n_seg][d_v + d_k][d_k] float: rows 0..d_v-1 of segment j: its end
 *     state from a zero state (segment 0: from S0); rows d_v.. : M_j
 *     transposed, row c holding M_j[0..d_k-1][c] (segments >= 1);
 *   then, at the next multiple of 256 bytes, [B*H*T][d_k] float: qm_t for
 *     the tokens of segments >= 1;
 *   then (bf16 O only) [B*H*T][d_v] float: outputs from a zero state.
 * Everything else as gdn_chunk_fwd_eta.
 */
size_t gdn_chunk_fwd_seq_workspace_bytes(const gdn_shape* s, int seg_chunks);
gdn_status gdn_chunk_fwd_seq(const gdn_shape* s, int seg_chunks,
                             const void* q, const void* k, const void* v,
                             const float* alpha, const float* beta, const float* eta,
                             const float* S0, void* O, float* S_final,
                             void* workspace, size_t workspace_bytes,
                             void* stream);

/*
 * gdn_chunk_fwd_seq without a workspace argument, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving
 * loops, harnesses that forbid allocation): the workspace is a 64 MiB
 * (67108864-byte) device array inside the library, one copy per GPU,
 * looked up on the first call on each device and held until the process
 * ends.  The call allocates nothing.  Plans whose workspace
 * (gdn_chunk_fwd_seq_workspace_bytes) exceeds 64 MiB return
 * GDN_ERR_WORKSPACE and write nothing.  Nothing in the array needs to start
 * at zero (every byte a call reads was written earlier in the same call),
 * and it keeps the last call's contents.  Calls that overlap on one GPU
 * (two streams, two threads) share that array and race: serialize them.
 * Runs on the current device.  Everything else as gdn_chunk_fwd_seq.
 */
gdn_status gdn_chunk_fwd_seq_noalloc(const gdn_shape* s, int seg_chunks,
                                     const void* q, const void* k, const void* v,
                                     const float* alpha, const float* beta, const float* eta,
                                     const float* S0, void* O, float* S_final,
                                     void* stream);

/*
 * The same pass with bf16 inputs through the split-bf16 kernels: every
 * derived matrix-product operand is a pair of bf16 numbers (hi + lo, about
 * 16 significant bits), which keeps the normwise error near 1e-5 whatever
 * the gates, at roughly twice the run time of gdn_chunk_fwd.  Shapes: bf16
 * with chunk_size in {32, 64} and d_k in {64, 128} take the pipelined
 * split kernel, bf16 d_k 32 and all f32 shapes the generic one (the other
 * bf16 shapes, chunk_size 16 or d_k 16 / 96 / 256, return GDN_ERR_UNSUPPORTED).
 * eta may
 * be NULL (eta = beta).  Arguments and conventions as gdn_chunk_fwd_eta,
 * without a workspace.
 */
gdn_status gdn_chunk_fwd_precise(const gdn_shape* s,
                                 const void* q, const void* k, const void* v,
                                 const float* alpha, const float* beta, const float* eta,
                                 const float* S0, void* O, float* S_final,
                                 void* stream);

/*
 * gdn_chunk_fwd_eta (bf16 inputs only) with two intermediates of the kernel
 * written out, for stage-by-stage checks of the pass itself:
 *   T_out  [B, H, NT, C, C] float: T = (I - A)^{-1} of every chunk as the
 *          kernel holds it (fp16 values, NT = ceil(T / C); zero above the
 *          diagonal and, in a ragged last chunk, identity past its end);
 *          A strictly lower with A_ri = -beta_r exp(g_r - g_i) k_r.k_i
 *          ("从零开始的 GDN 推导", UT transform, with L = -A);
 *   Vp_out [B, H, T, d_v] float: the pseudo-values V' = U - W S^T of every
 *          chunk ("从零开始的 GDN 推导", S update), before their rounding to
 *          the fp16 operands of the output and state products.
 * Either may be NULL.  O and S_final are written as by gdn_chunk_fwd_eta.
 * Shapes: bf16 as for gdn_chunk_fwd; f32 inputs return GDN_ERR_UNSUPPORTED.
 */
gdn_status gdn_chunk_fwd_stages(const gdn_shape* s,
                                const void* q, const void* k, const void* v,
                                const float* alpha, const float* beta, const float* eta,
                                const float* S0, void* O, float* S_final,
                                float* T_out, float* Vp_out,
                                void* stream);

/*
 * Chunk-local quantities of the same method, for inspection and testing of
 * the intermediate stages.  For every chunk c (NT = ceil(T / C) chunks, the
 * last one zero-padded to C tokens):
 *   T_out  [B, H, NT, C, C] float: T = (I - A)^{-1}, A strictly lower with
 *          A_ri = -beta_r exp(g_r - g_i) k_r.k_i (i < r), g the chunk-local
 *          inclusive cumulative sum of log alpha ("从零开始的 GDN 推导",
 *          UT transform, with L = -A);
 *   W_out  [B, H, T, d_k] float: W = T diag(beta) diag(exp(g)) K;
 *   U_out  [B, H, T, d_v] float: U = T diag(beta) V ("S 的推导").
 * Any of the three output pointers may be NULL (that output is skipped).
 * Computed by the generic stage kernel (fp32 solve, split-bf16 products):
 * bf16 with chunk_size in {32, 64} and d_k in {32, 64, 128}, f32 as for
 * gdn_chunk_fwd; other shapes return GDN_ERR_UNSUPPORTED.
 */
gdn_status gdn_chunk_prep(const gdn_shape* s,
                          const void* k, const void* v,
                          const float* alpha, const float* beta,
                          float* T_out, float* W_out, float* U_out,
                          void* workspace, size_t workspace_bytes,
                          void* stream);

/*
 * Recurrent (token-by-token) forward pass: the same recurrence applied one
 * token at a time ("从零开始的 GDN 推导", recurrent form; "RNN的复兴03",
 * section 1), for short sequences such as a decode step appended to a
 * chunked prefill.  The state is read once, kept on chip for all T tokens
 * and written once, so for T = 1 the cost is one pass of the state through
 * HBM.  Same tensors, layouts and conventions as gdn_chunk_fwd:
 *   q, k [B, H, T, d_k], v [B, H, T, d_v] (qkv_dtype), alpha (NULL = 1) and
 *   beta [B, H, T] float, S0 [B, H, d_v, d_k] float (NULL = zero),
 *   O [B, H, T, d_v] (o_dtype), S_final [B, H, d_v, d_k] float; S_final may
 *   be the same pointer as S0 (in-place update), other overlaps are not
 *   allowed.  chunk_size is ignored.
 * Supported: qkv_dtype GDN_BF16 or GDN_F32; d_k in {16, 32, 64, 96, 128,
 * 192, 256}; 1 <= d_v <= 65536; any T >= 1 (the work is serial in T, so long
 * sequences belong to gdn_chunk_fwd).  Pointers 16-byte aligned.  Errors are
 * returned before any launch, as for gdn_chunk_fwd.
 */
gdn_status gdn_recurrent_fwd(const gdn_shape* s,
                             const void* q, const void* k, const void* v,
                             const float* alpha, const float* beta, const float* S0,
                             void* O, float* S_final,
                             void* stream);

/* gdn_recurrent_fwd with a separate write strength eta (NULL means
 * eta = beta), as for gdn_chunk_fwd_eta. */
gdn_status gdn_recurrent_fwd_eta(const gdn_shape* s,
                                 const void* q, const void* k, const void* v,
                                 const float* alpha, const float* beta, const float* eta,
                                 const float* S0, void* O, float* S_final,
                                 void* stream);

/* ------------------------------------------------------------------------
 * The operators around the recurrence of a mixing layer: the short causal
 * convolution before it, the diagonal (selective state space) recurrence
 * that takes the delta rule's place in some layers, and the normalisation
 * and gate of the heads after it.  The conventions above hold, except that
 * inputs whose strides are in a shape struct need only a contiguous last
 * dimension (strides count elements, are >= 0, and may be 0: a broadcast
 * input), that pointers need only the alignment of their type (16-byte
 * aligned rows run the wide kernels), and that rows may be padded:
 *   lens  [B] int32 or NULL (every sequence has T tokens): the number of
 *         tokens of each sequence, clamped to [0, T].  Rows at and after it
 *         are not read as tokens: their contents, NaN included, reach no
 *         output; the output and gradient rows there are written as zero;
 *         the final state is the one after the last token (the initial one
 *         for a length of 0).
 * Outputs may not overlap inputs or each other, except where stated (checked
 * by the entries for one token, whose state is updated in place).
 * Gradients of parameters and of broadcast rows are sums in fp32 in a fixed
 * order: the same call gives the same bits.
 */

/* Short causal convolution of each channel over W tokens. */
typedef struct {
    int32_t B, T, D;          /* sequences, tokens, channels                   */
                              /* (T up to 2^31 - 128, D up to 2^25)            */
    int32_t W;                /* taps: 2, 3 or 4                               */
    int32_t H;                /* heads of y and dy (D a multiple of H)         */
    int32_t dtype;            /* gdn_dtype of x, y, the states, their gradients */
    int32_t silu;             /* 1: y = SiLU(p), 0: y = p                      */
    int64_t x_stride_b, x_stride_t;   /* x [B, T, D]                           */
} gdn_conv_shape;

/*
 *     p_t = bias + sum_{j < W} weight_j x_{t-W+1+j},   y_t = p_t SiLU-ed
 * per channel, with x_{-W+1} .. x_{-1} the rows of state0 (oldest first).
 *   x          [B, T, D]        dtype, strided
 *   weight     [D, W] float;  bias [D] float or NULL
 *   state0     [B, W-1, D]      dtype, or NULL (zero)
 *   y          [B, H, T, D/H]   dtype, contiguous (H = 1: [B, T, D]; H heads:
 *                               q, k or v of gdn_chunk_fwd)
 *   state_out  [B, W-1, D]      dtype or NULL; may be state0 (in place)
 */
gdn_status gdn_conv_fwd(const gdn_conv_shape* s, const void* x, const float* weight,
                        const float* bias, const void* state0, const int32_t* lens,
                        void* y, void* state_out, void* stream);

/* One token of every sequence (T must be 1): gdn_conv_fwd with the state
 * updated in place.  x [B, D] (rows x_stride_b apart), y [B, D]. */
gdn_status gdn_conv_step(const gdn_conv_shape* s, const void* x, const float* weight,
                         const float* bias, void* state, void* y, void* stream);

/*
 * Gradient of gdn_conv_fwd.  dy [B, H, T, D/H]; dstate_out (the gradient of
 * state_out) [B, W-1, D] or NULL; dx [B, T, D] contiguous, all dtype;
 * dweight [D, W], dbias [D] float (dbias may be NULL); dstate0 [B, W-1, D]
 * dtype or NULL.  workspace: gdn_conv_bwd_workspace_bytes(s) bytes
 * ((size_t)-1 for an invalid shape).
 */
size_t gdn_conv_bwd_workspace_bytes(const gdn_conv_shape* s);
gdn_status gdn_conv_bwd(const gdn_conv_shape* s, const void* dy, const void* x,
                        const float* weight, const float* bias, const void* state0,
                        const void* dstate_out, const int32_t* lens,
                        void* dx, float* dweight, float* dbias, void* dstate0,
                        void* workspace, size_t workspace_bytes, void* stream);

/* Selective state space recurrence: a diagonal state of N numbers for every
 * channel. */
typedef struct {
    int32_t B, T, D;          /* sequences, tokens, channels                   */
    int32_t N;                /* states per channel: 1 .. 64                   */
    int32_t G;                /* groups of B and C (D a multiple of G)         */
                              /* (D and the strides of tokens: up to 2^24,     */
                              /* T up to 2^31 - 128)                           */
    int32_t dtype;            /* gdn_dtype of x, dt, Bm, C, z, y and their gradients */
    int32_t dt_softplus;      /* 1: dt passes through softplus, 0: as it is    */
    int64_t x_stride_b, x_stride_t;     /* x  [B, T, D]                        */
    int64_t dt_stride_b, dt_stride_t;   /* dt [B, T, D]                        */
    int64_t z_stride_b, z_stride_t;     /* z  [B, T, D]                        */
    int64_t b_stride_b, b_stride_t;     /* Bm [B, T, G, N] ([G, N] contiguous) */
    int64_t c_stride_b, c_stride_t;     /* C  [B, T, G, N] ([G, N] contiguous) */
} gdn_ssm_shape;

/*
 *     s_t = softplus(dt_t + dt_bias)      (dt_t + dt_bias with dt_softplus 0)
 *     h_t = exp(s_t A) h_{t-1} + s_t x_t Bm_t
 *     y_t = (C_t . h_t + Dskip x_t) SiLU(z_t)
 * for every channel d, with A, h of N numbers and Bm_t, C_t those of the
 * channel's group (channels [g D/G, (g+1) D/G) belong to group g).
 *   A        [D, N] float (negative in a decaying state)
 *   Dskip    [D] float or NULL (0);  dt_bias [D] float or NULL (0)
 *   z        dtype or NULL (no gate)
 *   h0       [B, D, N] float or NULL (zero)
 *   y        [B, T, D] dtype, contiguous
 *   h_final  [B, D, N] float or NULL; may be h0 (in place)
 * The state is held in fp32.  Few channels on long sequences: the tokens are
 * cut into segments that run at once, from summaries of the segments before
 * them.  workspace: gdn_ssm_fwd_workspace_bytes(s) bytes (0 without segments;
 * with them their summaries, 13 MB at B 4, T 4096, D 2048, N 16 and four times
 * that at N 64; (size_t)-1 for an invalid shape).
 */
size_t gdn_ssm_fwd_workspace_bytes(const gdn_ssm_shape* s);
gdn_status gdn_ssm_fwd(const gdn_ssm_shape* s, const void* x, const void* dt, const float* A,
                       const void* Bm, const void* C, const float* Dskip, const void* z,
                       const float* dt_bias, const float* h0, const int32_t* lens,
                       void* y, float* h_final,
                       void* workspace, size_t workspace_bytes, void* stream);

/* One token of every sequence (T must be 1, B at most 65535): gdn_ssm_fwd with
 * the state h [B, D, N] updated in place.  x, dt, z [B, D], Bm, C [B, G, N], rows their
 * stride_b apart; y [B, D]. */
gdn_status gdn_ssm_step(const gdn_ssm_shape* s, const void* x, const void* dt, const float* A,
                        const void* Bm, const void* C, const float* Dskip, const void* z,
                        const float* dt_bias, float* h, void* y, void* stream);

/*
 * Gradient of gdn_ssm_fwd.  dy [B, T, D] dtype contiguous; dh_final
 * [B, D, N] float or NULL (zero).  Written, all contiguous: dx, ddt, dz
 * [B, T, D] and dBm, dC [B, T, G, N] in dtype (dz NULL without z); dA [D, N],
 * dDskip [D], ddt_bias [D] float (the last two may be NULL); dh0 [B, D, N]
 * float or NULL.  The states are computed again from the inputs.
 * workspace: gdn_ssm_bwd_workspace_bytes(s) bytes ((size_t)-1 for an
 * invalid shape).  It holds the state after every eight tokens and each tile's
 * part of dBm and dC: about 0.8 N' bytes for each token and channel, up to 1.2
 * N' in small calls (N' = N rounded up to 4, 8, 16, 32 or 64, and the channels of
 * a group rounded up to a multiple of 64), 212 MB at B 2, T 4096, D 2048, N 16.
 */
size_t gdn_ssm_bwd_workspace_bytes(const gdn_ssm_shape* s);
gdn_status gdn_ssm_bwd(const gdn_ssm_shape* s, const void* dy, const void* x, const void* dt,
                       const float* A, const void* Bm, const void* C, const float* Dskip,
                       const void* z, const float* dt_bias, const float* h0,
                       const float* dh_final, const int32_t* lens,
                       void* dx, void* ddt, float* dA, void* dBm, void* dC, float* dDskip,
                       void* dz, float* ddt_bias, float* dh0,
                       void* workspace, size_t workspace_bytes, void* stream);

/* Normalisation of each head of each token, with an activation or a gate. */
typedef struct {
    int32_t B, T, G, d;       /* sequences, tokens, heads (groups), head size 1 .. 4096 */
                              /* (G below 2^24; weights [G, d]: G d up to 2^27,
                                 in the gradient below it) */
    int32_t x_dtype;          /* gdn_dtype of x and dx                         */
    int32_t o_dtype;          /* gdn_dtype of y, dy, z and dz                  */
    int32_t center;           /* 1: subtract the mean, 0: root mean square only */
    int32_t w_per_group;      /* weight and bias: 0 [d] for all heads, 1 [G, d] */
    int32_t silu;             /* 1: SiLU, 0: no activation                     */
    float eps;                /* > 0                                           */
    int64_t x_stride_b, x_stride_t, x_stride_g;   /* x [B, T, G, d]: the delta
                                 rule's O [B, H, T, d] is read as it lies      */
    int64_t z_stride_b, z_stride_t, z_stride_g;   /* z [B, T, G, d]            */
} gdn_norm_shape;

/*
 *     n = (x - mean) / sqrt(var + eps)    over the d numbers of a head of a
 *         token (mean = 0 and var = mean square where not centred)
 *     p = n weight + bias
 *     y = p act(z) with z, act(p) without  (act: SiLU or nothing)
 * weight, bias float or NULL (1, 0); z o_dtype or NULL; y [B, T, G, d]
 * o_dtype contiguous.  Statistics are taken in fp32 over the values in
 * registers, the variance from the differences to the mean.
 */
gdn_status gdn_norm_fwd(const gdn_norm_shape* s, const void* x, const float* weight,
                        const float* bias, const void* z, void* y, void* stream);

/*
 * Gradient of gdn_norm_fwd.  dy [B, T, G, d] o_dtype contiguous.  Written:
 * dx x_dtype, with memory laid out by dx_stride_b, _t, _g (elements; its
 * last dimension contiguous); dz [B, T, G, d] o_dtype contiguous (NULL
 * without z); dweight, dbias float, shaped as weight (either may be NULL).
 * workspace: gdn_norm_bwd_workspace_bytes(s) bytes ((size_t)-1 for an
 * invalid shape).
 */
size_t gdn_norm_bwd_workspace_bytes(const gdn_norm_shape* s);
gdn_status gdn_norm_bwd(const gdn_norm_shape* s, const void* dy, const void* x,
                        const float* weight, const float* bias, const void* z,
                        void* dx, int64_t dx_stride_b, int64_t dx_stride_t, int64_t dx_stride_g,
                        float* dweight, float* dbias, void* dz,
                        void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Linear attention with a decay for each head: the delta rule's state without
 * its erasing.  The conventions of the operators above hold (strides, lens,
 * padded rows, sums in a fixed order).
 *     S_t = a_t S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t,   a_t = exp(log_alpha_t)
 * log_alpha <= 0 decays; minus infinity starts anew at its token (documents
 * packed into one row); values above 0 grow.  A value below -256 ln 2 counts
 * as minus infinity.
 */
typedef struct {
    int32_t B, H, T;          /* sequences, heads of values, tokens            */
                              /* (T up to 2^31 - 128)                          */
    int32_t Hq, Hk;           /* heads of queries and of keys, each a divisor of H:
                                 head h reads heads h / (H / Hq), h / (H / Hk) */
    int32_t d_k, d_v;         /* 1 .. 256                                      */
    int32_t dtype;            /* gdn_dtype of q, k, v, dO and their gradients  */
    int32_t o_dtype;          /* gdn_dtype of O                                */
    int32_t per_head;         /* log_alpha: 0 [B, H, T], 1 [H]                 */
    float scale;
    int64_t q_stride_b, q_stride_h, q_stride_t;   /* q [B, Hq, T, d_k]         */
    int64_t k_stride_b, k_stride_h, k_stride_t;   /* k [B, Hk, T, d_k]         */
    int64_t v_stride_b, v_stride_h, v_stride_t;   /* v [B, H, T, d_v]          */
    int64_t a_stride_b, a_stride_h, a_stride_t;   /* log_alpha (not read for [H],
                                                     which is contiguous)      */
} gdn_lin_shape;

/*
 *   log_alpha  float, strided, or NULL (no decay)
 *   S0         [B, H, d_v, d_k] float or NULL (zero)
 *   O          [B, H, T, d_v] o_dtype, contiguous
 *   S_final    [B, H, d_v, d_k] float or NULL; may be S0 (in place)
 * Chunks of 64 tokens (32 for fp32, and above d_k 128) on the matrix units; bf16
 * products of what is computed take two or three bf16 numbers that add up to
 * it, so that results are those of fp32 arithmetic to about 1e-5 of a tensor's
 * largest number, rounded once where they are bf16.  Any finite numbers whose products and sums of them over a
 * chunk fit fp32, with 2^48 to spare on both sides in chunks that decay by as
 * much as 2^-96.
 * An infinite or NaN input reaches what the formulas make from it, as infinity
 * or NaN: outputs of its sequence and head (where heads share queries or keys, of
 * those heads) from its token on, an infinite q that token's alone.  A decay of 0
 * does not end it (0 times infinity is NaN).  Few heads on long sequences:
 * the tokens are cut into segments that run at once, from what each adds to the
 * state.  workspace: gdn_lin_fwd_workspace_bytes(s) bytes (0 without segments;
 * (size_t)-1 for an invalid shape).
 */
size_t gdn_lin_fwd_workspace_bytes(const gdn_lin_shape* s);
gdn_status gdn_lin_fwd(const gdn_lin_shape* s, const void* q, const void* k, const void* v,
                       const float* log_alpha, const float* S0, const int32_t* lens,
                       void* O, float* S_final,
                       void* workspace, size_t workspace_bytes, void* stream);

/* One token of every sequence (T must be 1): gdn_lin_fwd with the state S
 * [B, H, d_v, d_k] updated in place; O [B, H, d_v].  Token strides are not read. */
gdn_status gdn_lin_step(const gdn_lin_shape* s, const void* q, const void* k, const void* v,
                        const float* log_alpha, float* S, void* O, void* stream);

/*
 * Gradient of gdn_lin_fwd (o_dtype is not read).  dO [B, H, T, d_v] dtype
 * contiguous; dS_final [B, H, d_v, d_k] float or NULL (zero).  Written, all
 * contiguous: dq [B, Hq, T, d_k], dk [B, Hk, T, d_k] (sums over the heads that
 * share one), dv [B, H, T, d_v] in dtype; dlog_alpha float shaped as log_alpha
 * ([B, H, T] or [H]; NULL without log_alpha, or where it is not wanted; 0 where
 * the decay itself is 0); dS0 float or NULL.  The states are computed again.
 * Each number of dlog_alpha is a sum of its own terms alone: off by 2^-16 of the
 * sum of their absolute values at most (2e-7 of the tensor in the mean), however
 * large the gradients of other tokens are.
 * workspace: gdn_lin_bwd_workspace_bytes(s) bytes: with dlog_alpha mostly a state
 * in fp32 for each head and 64 tokens (32 for fp32 rows and above d_v 128; d_k
 * rounded up to 32), 268 MB at 4 x 16 heads x 4096 tokens of 128/128; without
 * dlog_alpha that part is not touched.
 */
size_t gdn_lin_bwd_workspace_bytes(const gdn_lin_shape* s);
gdn_status gdn_lin_bwd(const gdn_lin_shape* s, const void* dO, const void* q, const void* k, const void* v,
                       const float* log_alpha, const float* S0, const float* dS_final, const int32_t* lens,
                       void* dq, void* dk, void* dv, float* dlog_alpha, float* dS0,
                       void* workspace, size_t workspace_bytes, void* stream);

/* The norms after and before a block, with the block's gate, the scale of its
 * part and the residual stream between them. */
typedef struct {
    int32_t B, T, D;          /* sequences, tokens, channels (D up to 16384)   */
    int32_t dtype;            /* gdn_dtype of o, gate, y and their gradients   */
    int32_t x_dtype;          /* gdn_dtype of x, x_out and their gradients     */
    int32_t post;             /* 1: o is normalised, 0: taken as it is         */
    int32_t act;              /* of the gate: 0 none, 1 sigmoid, 2 SiLU        */
    float eps;                /* > 0                                           */
    int64_t o_stride_b, o_stride_t;   /* o    [B, T, D]                        */
    int64_t x_stride_b, x_stride_t;   /* x    [B, T, D]                        */
    int64_t g_stride_b, g_stride_t;   /* gate [B, T, D]                        */
} gdn_block_norm_shape;

/*
 *     n = o / sqrt(mean(o^2) + eps) w_post     (post 0: n = o)
 *     x_out = x + scale act(gate) n
 *     y = x_out / sqrt(mean(x_out^2) + eps) w_pre
 * over the D channels of a token: o is what a block computed, x the residual
 * stream, y what the next block reads (of x_out before it is rounded to x_dtype).
 * Statistics are fp32: for rows whose squares and their sums fit it.
 *   gate      dtype or NULL (act(gate) = 1);  w_post, scale, w_pre  [D] float or
 *             NULL (1)
 *   x_out     [B, T, D] x_dtype, contiguous; may be x where x is contiguous (in
 *             place)
 *   y         [B, T, D] dtype, contiguous, or NULL (not wanted)
 */
gdn_status gdn_block_norm_fwd(const gdn_block_norm_shape* s, const void* o, const void* x, const void* gate,
                              const float* w_post, const float* scale, const float* w_pre,
                              void* x_out, void* y, void* stream);

/*
 * Gradient of gdn_block_norm_fwd from what it was given and x_out (strided as x
 * in the shape; statistics are taken from it as it is stored).  dx_out [B, T, D]
 * x_dtype, dy [B, T, D] dtype, contiguous, either may be NULL (zero), not both.
 * Written, contiguous: dx x_dtype, dO (the gradient of o) and dgate (NULL
 * without a gate) dtype; dw_post, dscale, dw_pre [D] float, each with the input
 * that it belongs to or NULL.  workspace: gdn_block_norm_bwd_workspace_bytes(s)
 * bytes.
 */
size_t gdn_block_norm_bwd_workspace_bytes(const gdn_block_norm_shape* s);
gdn_status gdn_block_norm_bwd(const gdn_block_norm_shape* s, const void* dx_out, const void* dy,
                              const void* x_out, const void* o, const void* gate,
                              const float* w_post, const float* scale, const float* w_pre,
                              void* dx, void* dO, void* dgate, float* dw_post, float* dscale, float* dw_pre,
                              void* workspace, size_t workspace_bytes, void* stream);

/* Static text for a status code. */
const char* gdn_status_string(gdn_status st);

/* Text of the last error on the calling thread (HIP error string or the
 * reason a shape was rejected); "" if none.  Valid until the next call. */
const char* gdn_last_error(void);

/* Library version: major * 10000 + minor * 100 + patch. */
int32_t gdn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H */
