/*
 * selscan.h -- C ABI of libselscan, the Mamba-1 selective scan for B200
 * (sm_100a).
 *
 * The operation (pages: "Mamba & State Space Models — Guide Complet" §1
 * "Discrétisation" and §4 "Implémentation du SSM sélectif (S6)";
 * "Mamba и State Space Models: альтернатива Transformer", "SSM as RNN",
 * "Discretization" and "Mamba Block"). For every batch row b, channel d and
 * state index n, with h = 0 before the first token:
 *
 *     Δ_t      = softplus(delta[b,t,d] + delta_bias[d])   (or no softplus)
 *     Abar_t   = exp(Δ_t · A[d,n])
 *     h_t[n]   = Abar_t · h_{t-1}[n] + Δ_t · B[b,t,n] · x[b,t,d]
 *     y[b,t,d] = (Σ_n C[b,t,n] · h_t[n] + D[d] · x[b,t,d]) · silu(z[b,t,d])
 *
 * Δ, B and C vary per token (the "selection"); A is diagonal per channel and
 * fixed; the input term is Δ·B ("SSM as RNN" scales B by delta); y reads the
 * state after the token's update; D·x is added before the gate.
 *
 * Conventions shared by every entry point:
 *  - All tensor pointers are DEVICE pointers on the current CUDA device,
 *    row-major and contiguous, last index fastest. The caller owns every
 *    buffer; the library keeps no pointer after a call returns.
 *  - `dtype` is the element type of x, delta, z, B, C and y. A, D,
 *    delta_bias and all states are always float32. Arithmetic is float32.
 *    bf16 results are rounded to nearest even.
 *  - Pointers must be aligned to their element size; y must not overlap any
 *    input.
 *  - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *    default stream). The return value reports argument validation and
 *    launch errors (cudaGetLastError after the launches), not completion.
 *  - "required" pointers may be NULL only when their tensor has zero
 *    elements.
 *  - Return values: SELSCAN_OK (0) or one of the negative SELSCAN_ERR_*
 *    codes; nothing is launched when validation fails.
 */
#ifndef SELSCAN_H_
#define SELSCAN_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define SELSCAN_API __attribute__((visibility("default")))
#else
#define SELSCAN_API
#endif

/* Same type as cudaStream_t; spelled out so that this header needs no CUDA
 * header. */
typedef struct CUstream_st *selscan_stream_t;

typedef enum {
    SELSCAN_F32 = 0,  /* float32 x, delta, z, B, C, y */
    SELSCAN_BF16 = 1  /* bfloat16 x, delta, z, B, C, y */
} selscan_dtype_t;

enum {
    SELSCAN_OK = 0,
    SELSCAN_ERR_NULL_ARG = -1,           /* a required pointer is NULL */
    SELSCAN_ERR_BAD_DIM = -2,            /* a size is negative or too large */
    SELSCAN_ERR_BAD_DTYPE = -3,          /* dtype is not a selscan_dtype_t */
    SELSCAN_ERR_MISALIGNED = -4,         /* a pointer is not element-aligned */
    SELSCAN_ERR_DSTATE_UNSUPPORTED = -5, /* dstate outside 1..SELSCAN_MAX_DSTATE
                                            (1..SELSCAN_MAX_DSTATE_BWD for selscan_bwd) */
    SELSCAN_ERR_CUDA = -6,               /* a CUDA call failed */
    SELSCAN_ERR_ALIAS = -7,              /* y overlaps an input */
    SELSCAN_ERR_WORKSPACE = -8           /* the given or static workspace is too small
                                            (selscan_fwd_noalloc, selscan_bwd_workspace) */
};

/* Largest d_state of the forward and decode entry points. d_state ≤ 16 takes
 * the TMA-staged and register-resident kernels; 17..256 take a kernel that
 * splits each chain's states over 2-16 lanes (one pass, no chunking,
 * batch ≤ 65535). The gradient (selscan_bwd) takes d_state ≤ 256 as well. */
#define SELSCAN_MAX_DSTATE 256
#define SELSCAN_MAX_DSTATE_BWD 256

/*
 * selscan_fwd -- selective scan over whole sequences (the forward pass).
 *
 *   x, delta      [batch, seqlen, dim]      dtype        required
 *   A             [dim, dstate]             float32      required; a channel
 *                                                        whose A[d,n] are all
 *                                                        within 2^-21 of
 *                                                        (n+1)·A[d,0] (the
 *                                                        S4D/Mamba −(1..N),
 *                                                        also −exp(log(1..N))
 *                                                        in float32) is scanned
 *                                                        with (n+1)·A[d,0]:
 *                                                        powers of one decay
 *                                                        per token, a relative
 *                                                        change of Δ·|A|·2^-21
 *                                                        in exp(Δ·A)
 *   B, C          [batch, seqlen, dstate]   dtype        required; shared by
 *                                                        all channels
 *   D             [dim]                     float32      NULL -> no skip term
 *   z             [batch, seqlen, dim]      dtype        NULL -> no gate
 *   delta_bias    [dim]                     float32      NULL -> zero bias
 *   softplus_flag nonzero -> Δ = softplus(delta + bias), zero -> Δ = delta + bias
 *   y             [batch, seqlen, dim]      dtype        required output
 *   final_state   [batch, dim, dstate]      float32      NULL -> not written;
 *                                                        else h after the
 *                                                        last token (zeros if
 *                                                        seqlen == 0)
 *   batch, seqlen, dim >= 0 (any of them 0 -> nothing to compute);
 *   1 <= dstate <= SELSCAN_MAX_DSTATE.
 *
 * The sequence is processed in chunks whose final states are carried to the
 * next chunk (the pages' blockwise scan with its state carried across blocks,
 * "Hardware-Aware Scan", and the associative operator of Guide Complet §4
 * "Parallel Associative Scan"). Depending on the sizes, chunks run one after
 * another with the state handed over on the device, or in parallel followed
 * by a carry pass. Either takes a stream-ordered device workspace
 * (cudaMallocAsync / cudaFreeAsync on `stream`; its size is reported by
 * selscan_fwd_plan); no other memory is allocated.
 */
SELSCAN_API int selscan_fwd(const void *x, const void *delta, const float *A,
                const void *B, const void *C, const float *D, const void *z,
                const float *delta_bias, int softplus_flag, void *y,
                float *final_state, int64_t batch, int64_t seqlen, int64_t dim,
                int64_t dstate, selscan_dtype_t dtype, selscan_stream_t stream);

/*
 * selscan_fwd_from_state -- selscan_fwd starting from a given state instead
 * of h = 0 before the first token: the state carried across blocks of a
 * sequence ("Mamba и State Space Models: альтернатива Transformer",
 * "Hardware-Aware Scan") handed in from outside, e.g. the final state of a
 * previous call on the preceding tokens or a state advanced by
 * selscan_state_update. Arguments as selscan_fwd, plus
 *   initial_state [batch, dim, dstate]   float32   NULL -> zero (== selscan_fwd)
 * initial_state may be the same buffer as final_state (the state is then
 * advanced in place); any other overlap with an output is rejected. With
 * seqlen == 0 the final state is a copy of the initial state.
 */
SELSCAN_API int selscan_fwd_from_state(const void *x, const void *delta, const float *A,
                                       const void *B, const void *C, const float *D,
                                       const void *z, const float *delta_bias,
                                       int softplus_flag, const float *initial_state,
                                       void *y, float *final_state, int64_t batch,
                                       int64_t seqlen, int64_t dim, int64_t dstate,
                                       selscan_dtype_t dtype, selscan_stream_t stream);

/*
 * selscan_fwd_conv -- the Mamba block's causal depthwise convolution and SiLU
 * in front of the scan, fused into it ("Mamba и State Space Models:
 * альтернатива Transformer", "Mamba Block": Conv1d with one filter per
 * channel and d_conv − 1 leading zeros; "Mamba & State Space Models — Guide
 * Complet" §7: kernel width 4, the first L outputs, Conv1D → SiLU → SSM).
 * The scan's x is
 *   x[b,t,d] = silu( conv_bias[d] + Σ_{k<K} conv_weight[d,k] · x_in[b, t−(K−1)+k, d] )
 * (x_in = 0 before the first token of each sequence; a cross-correlation like
 * torch's Conv1d), used both in Δ·B·x and in D·x; x itself is not written.
 *   x_in          [batch, seqlen, dim]      dtype        required
 *   conv_weight   [dim, conv_width]         float32      required
 *   conv_bias     [dim]                     float32      NULL -> zero
 *   conv_width    1 .. 4
 *   conv_init     [batch, dim, 3]           float32      NULL -> zero: the x_in
 *                 values of the 3 tokens before token 0, oldest first (with
 *                 initial_state, continues a sequence exactly: pass the last 3
 *                 x_in tokens of the preceding call)
 * Other arguments as selscan_fwd_from_state (initial_state may be NULL).
 */
SELSCAN_API int selscan_fwd_conv(const void *x_in, const float *conv_weight,
                                 const float *conv_bias, int conv_width,
                                 const float *conv_init, const void *delta,
                                 const float *A, const void *B, const void *C, const float *D,
                                 const void *z, const float *delta_bias, int softplus_flag,
                                 const float *initial_state, void *y, float *final_state,
                                 int64_t batch, int64_t seqlen, int64_t dim, int64_t dstate,
                                 selscan_dtype_t dtype, selscan_stream_t stream);

/* Input term of the discretisation. */
enum {
    SELSCAN_BBAR_DELTA = 0, /* Bbar·x = Δ·B·x ("SSM as RNN"; the default everywhere) */
    SELSCAN_BBAR_ZOH = 1    /* Bbar·x = (exp(Δ·A) − 1)/A · B·x, zero-order hold ("Mamba &
                               State Space Models — Guide Complet" §1 "Discrétisation",
                               diagonal A; Δ·B·x where A = 0) */
};

/* Options of selscan_fwd_ex; a zero-initialised struct (or NULL) is
 * selscan_fwd. Fields as in selscan_fwd_from_state and selscan_fwd_conv
 * (conv_width 0: no conv). */
typedef struct {
    const float *initial_state; /* [batch, dim, dstate] or NULL */
    const float *conv_weight;   /* [dim, conv_width] (conv_width > 0) */
    const float *conv_bias;     /* [dim] or NULL */
    const float *conv_init;     /* [batch, dim, 3] or NULL */
    int conv_width;             /* 0 .. 4 */
    int bbar_mode;              /* SELSCAN_BBAR_DELTA or SELSCAN_BBAR_ZOH */
} selscan_fwd_options_t;

/*
 * selscan_fwd_ex -- selscan_fwd with every option: an initial state, the
 * causal conv in front, and the input term (Δ·B·x or the zero-order-hold
 * term, both on the TMA-staged kernel where the shape allows it, else on the
 * generic kernels). options NULL: selscan_fwd. Unknown bbar_mode:
 * SELSCAN_ERR_BAD_DIM.
 */
SELSCAN_API int selscan_fwd_ex(const void *x, const void *delta, const float *A,
                               const void *B, const void *C, const float *D, const void *z,
                               const float *delta_bias, int softplus_flag,
                               const selscan_fwd_options_t *options, void *y,
                               float *final_state, int64_t batch, int64_t seqlen,
                               int64_t dim, int64_t dstate, selscan_dtype_t dtype,
                               selscan_stream_t stream);

/*
 * selscan_fwd_noalloc -- selscan_fwd without any device allocation.
 *
 * The pages have no counterpart of this call; it exists for callers that
 * cannot allocate device memory while they run: code whose device memory is
 * all handed out by another allocator (a framework's caching allocator, an
 * arena reserved at start-up), latency-critical loops where an allocation may
 * block or fail, and processes without stream-ordered memory pools.
 *
 * Same arguments, results and launch plan as selscan_fwd. When the plan is
 * chunked, the chunk workspace is a fixed array inside the library of
 * SELSCAN_NOALLOC_WORKSPACE_BYTES bytes, held on every GPU that loads the
 * library until the process exits; sizes whose workspace (selscan_fwd_plan)
 * exceeds it are rejected with SELSCAN_ERR_WORKSPACE before anything runs.
 * This call never calls cudaMalloc, cudaMallocAsync or cudaFree.
 *  - Every call that needs the workspace looks up the array's device address
 *    on the current device (cudaGetSymbolAddress); nothing is cached, so a
 *    device reset or a re-created primary context, after which the array may
 *    sit at a new address, is picked up by the next call. The first such
 *    call on a device also loads the library's device code there; make it
 *    before any stream capture.
 *  - All calls on a device share the one array, and it keeps the contents
 *    of the last call. Calls that overlap on the GPU (e.g. on two streams
 *    without ordering between them) race on it and give wrong results; order
 *    them. The call itself clears, on `stream` and before its kernels, the
 *    counters that must start at zero (cudaMemsetAsync, no allocation); every
 *    other workspace element is written before it is read.
 */
#define SELSCAN_NOALLOC_WORKSPACE_BYTES (16u << 20)

SELSCAN_API int selscan_fwd_noalloc(const void *x, const void *delta, const float *A,
                                    const void *B, const void *C, const float *D,
                                    const void *z, const float *delta_bias,
                                    int softplus_flag, void *y, float *final_state,
                                    int64_t batch, int64_t seqlen, int64_t dim,
                                    int64_t dstate, selscan_dtype_t dtype,
                                    selscan_stream_t stream);

/*
 * selscan_fwd_plan -- the launch plan selscan_fwd would use for these sizes
 * with bf16 tensors on 16-byte boundaries (host only; no CUDA work). Writes,
 * through each non-NULL pointer, the number of sequence chunks (0 when there
 * is nothing to compute), the number of kernel launches (1 single pass; 3
 * chunked: chunk aggregates, carry, rescan) and the bytes of stream-ordered
 * workspace that call allocates. Returns SELSCAN_OK or the size errors of
 * selscan_fwd. The plan depends on the current device's SM count.
 */
SELSCAN_API int selscan_fwd_plan(int64_t batch, int64_t seqlen, int64_t dim,
                                 int64_t dstate, int64_t *chunks, int64_t *launches,
                                 int64_t *workspace_bytes);

/*
 * selscan_state_update -- one token of recurrent inference, in place
 * ("SSM as Convolution": recurrent mode for inference; Guide Complet §6: a
 * constant-size state instead of a growing cache).
 *
 *   state         [batch, dim, dstate]      float32      required, read and
 *                                                        overwritten with h_t
 *   x, delta      [batch, dim]              dtype        required
 *   A             [dim, dstate]             float32      required
 *   B, C          [batch, dstate]           dtype        required
 *   D             [dim]                     float32      NULL -> no skip term
 *   z             [batch, dim]              dtype        NULL -> no gate
 *   delta_bias    [dim]                     float32      NULL -> zero bias
 *   softplus_flag as for selscan_fwd
 *   y             [batch, dim]              dtype        required output
 *
 * A final_state from selscan_fwd is a valid `state`: steps continue the
 * sequence exactly where the scan stopped. No memory is allocated.
 */
SELSCAN_API int selscan_state_update(float *state, const void *x, const void *delta,
                         const float *A, const void *B, const void *C,
                         const float *D, const void *z,
                         const float *delta_bias, int softplus_flag, void *y,
                         int64_t batch, int64_t dim, int64_t dstate,
                         selscan_dtype_t dtype, selscan_stream_t stream);

/*
 * selscan_bwd -- gradient of selscan_fwd (the backward pass), with the
 * forward states recomputed instead of stored ("Mamba: co potrafią modele
 * przestrzeni stanów", "Cena selekcji": the backward pass recomputes the
 * intermediate states).
 *
 * For the loss Σ dy·y + Σ dfinal_state·final_state of the selscan_fwd call
 * with the same inputs, writes the loss's gradient with respect to each
 * input. With λ_t = ∂loss/∂h_t, λ after the last token = dfinal_state and
 * λ_t = ds_t·C_t + Abar_{t+1}·λ_{t+1}, ds_t = dy_t·silu(z_t):
 *
 *   x, delta, A, B, C, D, z, delta_bias, softplus_flag   as in selscan_fwd
 *   dy            [batch, seqlen, dim]      dtype        required
 *   dfinal_state  [batch, dim, dstate]      float32      NULL -> zero
 *   dx, ddelta    [batch, seqlen, dim]      dtype        required outputs
 *   dA            [dim, dstate]             float32      required output
 *                                                        (sum over batch and tokens)
 *   dB, dC        [batch, seqlen, dstate]   float32      required outputs
 *                                                        (sums over channels)
 *   dD            [dim]                     float32      NULL -> not written
 *   dz            [batch, seqlen, dim]      dtype        required iff z != NULL
 *   ddelta_bias   [dim]                     float32      NULL -> not written
 *   batch <= 65535, dstate 1..SELSCAN_MAX_DSTATE_BWD; other limits as in
 *   selscan_fwd.
 *
 * Every output is overwritten (not accumulated into); dB, dC, dA, dD and
 * ddelta_bias are float32 whatever `dtype` is. Results are deterministic
 * (fixed summation order, no atomics). Outputs must not overlap any input.
 * Takes a stream-ordered device workspace (cudaMallocAsync / cudaFreeAsync
 * on `stream`) of selscan_bwd_workspace_bytes() bytes: the state entering
 * every 8-token tile of every chain, and per-channel-tile partial sums of dB
 * and dC. Above 16 states the states go in groups of 16 computed side by
 * side; the workspace then holds every group's checkpoints and partials and
 * three float32 [batch, seqlen, dim] arrays per group, summed in group
 * order.
 */
SELSCAN_API int selscan_bwd(const void *x, const void *delta, const float *A,
                            const void *B, const void *C, const float *D, const void *z,
                            const float *delta_bias, int softplus_flag, const void *dy,
                            const float *dfinal_state, void *dx, void *ddelta, float *dA,
                            float *dB, float *dC, float *dD, void *dz, float *ddelta_bias,
                            int64_t batch, int64_t seqlen, int64_t dim, int64_t dstate,
                            selscan_dtype_t dtype, selscan_stream_t stream);

/* Host-only: device workspace bytes selscan_bwd takes for these sizes
 * (0 for empty or invalid sizes). */
SELSCAN_API int64_t selscan_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim,
                                                int64_t dstate);

/*
 * selscan_bwd_workspace -- selscan_bwd on a workspace the caller provides
 * (e.g. from its own caching allocator) instead of one allocated on the
 * stream: same arguments and results, plus
 *   workspace        device buffer, 256-byte aligned, must not overlap any
 *                    input or output; NULL only when no token is processed
 *   workspace_bytes  its size: at least selscan_bwd_workspace_bytes() for
 *                    these sizes, else SELSCAN_ERR_WORKSPACE
 * Nothing is allocated. The workspace is free for reuse once the call's work
 * on `stream` has completed; its contents are not meaningful afterwards.
 */
SELSCAN_API int selscan_bwd_workspace(const void *x, const void *delta, const float *A,
                                      const void *B, const void *C, const float *D,
                                      const void *z, const float *delta_bias,
                                      int softplus_flag, const void *dy,
                                      const float *dfinal_state, void *dx, void *ddelta,
                                      float *dA, float *dB, float *dC, float *dD, void *dz,
                                      float *ddelta_bias, int64_t batch, int64_t seqlen,
                                      int64_t dim, int64_t dstate, selscan_dtype_t dtype,
                                      void *workspace, int64_t workspace_bytes,
                                      selscan_stream_t stream);

/*
 * selscan_bwd_from_state -- the gradient of selscan_fwd_from_state: as
 * selscan_bwd_workspace, plus
 *   initial_state   [batch, dim, dstate]  float32  the forward's initial state
 *                                                  (NULL: zero)
 *   dinitial_state  [batch, dim, dstate]  float32  output: the loss's gradient
 *                                                  with respect to it (NULL: not
 *                                                  written); λ carried past the
 *                                                  first token, Abar_0·λ_0
 * workspace NULL: allocated on the stream as selscan_bwd does.
 */
SELSCAN_API int selscan_bwd_from_state(const void *x, const void *delta, const float *A,
                                       const void *B, const void *C, const float *D,
                                       const void *z, const float *delta_bias,
                                       int softplus_flag, const float *initial_state,
                                       const void *dy, const float *dfinal_state, void *dx,
                                       void *ddelta, float *dA, float *dB, float *dC,
                                       float *dD, void *dz, float *ddelta_bias,
                                       float *dinitial_state, int64_t batch, int64_t seqlen,
                                       int64_t dim, int64_t dstate, selscan_dtype_t dtype,
                                       void *workspace, int64_t workspace_bytes,
                                       selscan_stream_t stream);

/*
 * selscan_bwd_conv -- the gradient of selscan_fwd_conv (conv_init NULL: the
 * conv sees zeros before token 0): as selscan_bwd_from_state with x_in, the
 * conv arguments, and
 *   dx_in          [batch, seqlen, dim]  dtype    output: gradient w.r.t. x_in
 *                                                 (through the conv and SiLU)
 *   dconv_weight   [dim, conv_width]     float32  output
 *   dconv_bias     [dim]                 float32  output (NULL: not written)
 * The workspace (NULL: allocated on the stream) needs
 * selscan_bwd_conv_workspace_bytes() bytes: besides the scan gradient's it
 * holds the conv output's gradient (float32 [batch, seqlen, dim]) and conv
 * partial sums. The conv output is recomputed, never stored.
 */
SELSCAN_API int selscan_bwd_conv(const void *x_in, const float *conv_weight,
                                 const float *conv_bias, int conv_width, const void *delta,
                                 const float *A, const void *B, const void *C, const float *D,
                                 const void *z, const float *delta_bias, int softplus_flag,
                                 const float *initial_state, const void *dy,
                                 const float *dfinal_state, void *dx_in, void *ddelta,
                                 float *dA, float *dB, float *dC, float *dD, void *dz,
                                 float *ddelta_bias, float *dinitial_state,
                                 float *dconv_weight, float *dconv_bias, int64_t batch,
                                 int64_t seqlen, int64_t dim, int64_t dstate,
                                 selscan_dtype_t dtype, void *workspace,
                                 int64_t workspace_bytes, selscan_stream_t stream);

/* Options of selscan_bwd_ex; zero-initialised (or NULL) is selscan_bwd. */
typedef struct {
    const float *initial_state;  /* [batch, dim, dstate] or NULL (the forward's) */
    float *dinitial_state;       /* [batch, dim, dstate] or NULL: its gradient */
    const float *conv_weight;    /* [dim, conv_width] (conv_width > 0): x is then the
                                    conv's input and dx its gradient */
    const float *conv_bias;      /* [dim] or NULL */
    int conv_width;              /* 0 .. 4 */
    float *dconv_weight;         /* [dim, conv_width] (conv_width > 0) */
    float *dconv_bias;           /* [dim] or NULL */
    int bbar_mode;               /* SELSCAN_BBAR_DELTA or SELSCAN_BBAR_ZOH */
} selscan_bwd_options_t;

/*
 * selscan_bwd_ex -- the gradient of selscan_fwd_ex with every option of the
 * forward that has one: initial state, the conv front end, and the input
 * term. With SELSCAN_BBAR_ZOH the forward input is c·B·x with
 * c = (exp(Δ·A[d,n]) − 1)/A[d,n] ("Mamba & State Space Models — Guide
 * Complet" §1, zero-order hold); its gradient uses ∂c/∂Δ = exp(Δ·A) and
 * ∂c/∂A = Δ²·f'(Δ·A), f(z) = (e^z − 1)/z. Arguments as selscan_bwd plus
 * the options; workspace NULL -> allocated on the stream, else at least
 * selscan_bwd_conv_workspace_bytes() (conv) or selscan_bwd_workspace_bytes()
 * bytes. Unknown bbar_mode or a negative conv_width: SELSCAN_ERR_BAD_DIM.
 */
SELSCAN_API int selscan_bwd_ex(const void *x, const void *delta, const float *A, const void *B,
                               const void *C, const float *D, const void *z,
                               const float *delta_bias, int softplus_flag, const void *dy,
                               const float *dfinal_state, const selscan_bwd_options_t *options,
                               void *dx, void *ddelta, float *dA, float *dB, float *dC, float *dD,
                               void *dz, float *ddelta_bias, int64_t batch, int64_t seqlen,
                               int64_t dim, int64_t dstate, selscan_dtype_t dtype,
                               void *workspace, int64_t workspace_bytes, selscan_stream_t stream);

/* Host-only: workspace bytes selscan_bwd_conv takes (0 for empty or invalid sizes). */
SELSCAN_API int64_t selscan_bwd_conv_workspace_bytes(int64_t batch, int64_t seqlen,
                                                     int64_t dim, int64_t dstate);

/*
 * selscan_state_update_conv -- selscan_state_update with the causal conv +
 * SiLU of selscan_fwd_conv in front, for decoding after a selscan_fwd_conv
 * prefill: the token's x is silu(conv_bias + Σ_k conv_weight[d,k] · window),
 * the window being the 3 previous inputs kept in conv_state followed by
 * x_in; conv_state is then shifted to end with x_in.
 *   conv_state    [batch, dim, 3]           float32      in-out: the x_in values
 *                                                        of the 3 previous tokens,
 *                                                        oldest first
 *   x_in          [batch, dim]              dtype        required
 *   conv_weight   [dim, conv_width], conv_bias [dim] (NULL -> zero), conv_width 1..4
 * Other arguments as selscan_state_update. conv_state must not overlap any
 * other argument.
 */
SELSCAN_API int selscan_state_update_conv(float *state, float *conv_state, const void *x_in,
                                          const float *conv_weight, const float *conv_bias,
                                          int conv_width, const void *delta, const float *A,
                                          const void *B, const void *C, const float *D,
                                          const void *z, const float *delta_bias,
                                          int softplus_flag, void *y, int64_t batch,
                                          int64_t dim, int64_t dstate, selscan_dtype_t dtype,
                                          selscan_stream_t stream);

/* Options of selscan_state_update_ex; zero-initialised (or NULL) is
 * selscan_state_update. Fields as in selscan_state_update_conv. */
typedef struct {
    float *conv_state;          /* [batch, dim, 3], in-out (conv_width > 0) */
    const float *conv_weight;   /* [dim, conv_width] */
    const float *conv_bias;     /* [dim] or NULL */
    int conv_width;             /* 0 .. 4 */
    int bbar_mode;              /* SELSCAN_BBAR_DELTA or SELSCAN_BBAR_ZOH */
} selscan_step_options_t;

/* selscan_state_update with every option (conv window, input term). */
SELSCAN_API int selscan_state_update_ex(float *state, const void *x, const void *delta,
                                        const float *A, const void *B, const void *C,
                                        const float *D, const void *z, const float *delta_bias,
                                        int softplus_flag, const selscan_step_options_t *options,
                                        void *y, int64_t batch, int64_t dim, int64_t dstate,
                                        selscan_dtype_t dtype, selscan_stream_t stream);

/*
 * selscan_ssd_fwd -- the scan with one scalar A per head, computed in the
 * chunked matrix form of "Mamba & State Space Models — Guide Complet" §5
 * ("SSD — State Space Dual": y = (L ◦ S)·u, a causal mask times a structured
 * semiseparable matrix). Channel d = h·headdim + p of head h:
 *   Δ_t = softplus(dt[b,t,h] + dt_bias[h]) (or no softplus),
 *   h_t[n] = exp(Δ_t·A[h])·h_{t−1}[n] + Δ_t·B[b,t,n]·x[b,t,d],
 *   y[b,t,d] = (Σ_n C[b,t,n]·h_t[n] + D[h]·x[b,t,d])·silu(z[b,t,d]),
 * i.e. selscan_fwd_from_state with delta, delta_bias, A and D broadcast from
 * the heads to their channels.
 *   x, z          [batch, seqlen, nheads·headdim]   dtype   (z NULL -> no gate)
 *   dt            [batch, seqlen, nheads]           dtype
 *   A, D, dt_bias [nheads]                          float32 (D, dt_bias nullable)
 *   B, C          [batch, seqlen, dstate]           dtype   (one group)
 *   initial_state, final_state [batch, nheads·headdim, dstate] float32, nullable
 *   headdim 1..64, dstate 1..128, batch and nheads ≤ 65535.
 * float32 I/O: 64-token chunks, products in float32 on the CUDA cores.
 * bfloat16 I/O: 128-token chunks on the tensor cores (tcgen05, float32
 * accumulators); the operands that are not inputs (the masked decay matrix
 * M, w ◦ x for the chunk states, the carried state h_in) are split into
 * bfloat16 high/low pairs, so the products keep about 16 significant bits.
 * Workspace (NULL: allocated on the stream) of selscan_ssd_workspace_bytes()
 * bytes; the caller owns every buffer. No output may overlap an input
 * (SELSCAN_ERR_ALIAS). Asynchronous like selscan_fwd.
 */
SELSCAN_API int selscan_ssd_fwd(const void *x, const void *dt, const float *A, const void *B,
                                const void *C, const float *D, const void *z,
                                const float *dt_bias, int softplus_flag,
                                const float *initial_state, void *y, float *final_state,
                                int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim,
                                int64_t dstate, selscan_dtype_t dtype, void *workspace,
                                int64_t workspace_bytes, selscan_stream_t stream);

/* Host-only: workspace bytes selscan_ssd_fwd takes (0 for empty or invalid sizes). */
SELSCAN_API int64_t selscan_ssd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t nheads,
                                                int64_t headdim, int64_t dstate);

/* Options of selscan_linattn_fwd and selscan_linattn_bwd; zero-initialised (or
 * NULL): no decay, a zero first state, every token of every row, contiguous
 * operands. At most one of the two decays is given (else SELSCAN_ERR_BAD_DIM). */
typedef struct {
    const void *log_decay;       /* [batch, seqlen, heads] dtype: g of every token */
    const float *head_log_decay; /* [heads]: one g for all tokens of a head */
    const float *initial_state;  /* [batch, heads, dk, dv]: S before token 0 */
    const int32_t *seqlens;      /* [batch], on the device: tokens of each row (clamped to
                                    0..seqlen); NULL -> seqlen */
    int64_t q_stride, k_stride, v_stride; /* elements between tokens; 0 -> contiguous.
                                    A row's heads are contiguous, batch rows seqlen tokens
                                    apart: q, k and v may be slices of one projection */
} selscan_linattn_options_t;

/*
 * selscan_linattn_fwd -- linear attention with a decay for each head: the
 * matrix form of "Mamba & State Space Models — Guide Complet" §5 ("SSD — State
 * Space Dual") with a query and a key of their own for each head (or shared by
 * heads/qk_heads neighbouring heads) and free log decays. Per (batch row, head):
 *   S_t = exp(g_t)·S_{t−1} + k_t v_tᵀ,    y_t = scale·S_tᵀ q_t
 *   q, k          [batch, seqlen, qk_heads, dk]   dtype     required
 *   v, y          [batch, seqlen, heads, dv]      dtype     required (y: output)
 *   final_state   [batch, heads, dk, dv]          float32   NULL -> not written; may be
 *                                                 options->initial_state itself
 *   heads a multiple of qk_heads, 1 <= dk, dv <= 128, batch·heads <= 2^22.
 * A log decay of −∞ (any below −87.4, whose factor float32 flushes to zero)
 * resets: what came before that token does not count, whatever it holds. Tokens
 * at or behind a row's length are not used: their y is zero and final_state is
 * the state after the row's last token; their k and v may hold anything.
 * A value that is not finite reaches y of its token and of later ones up to the
 * next reset, and the state leaving, as long as float32 holds its weight; one of
 * v only its own column. What it reaches is infinite or NaN (the state takes an
 * infinite v as it stands), and nothing else changes.
 * Chunks of 64 tokens; float32 state, sums and decays. bfloat16 I/O whose rows
 * suit it (dk, dv multiples of 8, 16-byte rows) runs on the tensor cores
 * (tcgen05) with the products' weights and the entering state as bfloat16
 * operands, the state's own update keeping 24 bits; there a chunk's decay stands
 * between its factors on the way, so that y is finite where the sums of
 * |scale·(q·k)·v| stay below 2^96. Everything else runs in float32 on the CUDA
 * cores. Few (batch row, head) pairs: a sequence is cut into segments that run
 * side by side after a pass over their own states.
 * Workspace (256-byte aligned; NULL: allocated on the stream) of
 * selscan_linattn_workspace_bytes() bytes. Results do not depend on anything
 * but the inputs (fixed summation order). Asynchronous like selscan_fwd.
 */
SELSCAN_API int selscan_linattn_fwd(const void *q, const void *k, const void *v, float scale,
                                    const selscan_linattn_options_t *options, void *y,
                                    float *final_state, int64_t batch, int64_t seqlen,
                                    int64_t qk_heads, int64_t heads, int64_t dk, int64_t dv,
                                    selscan_dtype_t dtype, void *workspace,
                                    int64_t workspace_bytes, selscan_stream_t stream);

/* Host-only: workspace bytes selscan_linattn_fwd takes (0 for empty or invalid sizes). */
SELSCAN_API int64_t selscan_linattn_workspace_bytes(int64_t batch, int64_t seqlen,
                                                    int64_t qk_heads, int64_t heads, int64_t dk,
                                                    int64_t dv, selscan_dtype_t dtype);

/*
 * selscan_linattn_bwd -- the gradient of selscan_linattn_fwd for the loss
 * Σ dy·y + Σ dfinal_state·final_state. With N_t = ∂loss/∂S_t (N after the last
 * token = dfinal_state), N_t = scale·q_t dy_tᵀ + exp(g_{t+1})·N_{t+1}:
 *   dq_t = scale·S_t dy_t, dk_t = N_t v_t, dv_t = N_tᵀ k_t (sums over the heads
 *   that share a q and a k), dg_t = exp(g_t)·<S_{t−1}, N_t>
 *   dy             [batch, seqlen, heads, dv]     dtype     required
 *   dfinal_state   [batch, heads, dk, dv]         float32   NULL -> zero
 *   dq, dk         [batch, seqlen, qk_heads, dk]  dtype     required outputs
 *   dv             [batch, seqlen, heads, dv]     dtype     required output
 *   dlog_decay     [batch, seqlen, heads]         dtype     NULL -> not written;
 *                                                 needs options->log_decay (a decay
 *                                                 given by head is a constant)
 *   dinitial_state [batch, heads, dk, dv]         float32   NULL -> not written
 * States are recomputed. Every output is overwritten; those of tokens behind a
 * row's length are zero. dlog_decay is made as a running sum over the later
 * tokens, from the next reset back, of q·dq − k·dk: it carries the errors of
 * these products, which cancel (2^-20 of their size in float32, 2^-17 in
 * bfloat16), and a value that is not finite makes it so back to the last reset.
 * The other gradients take such values as the forward does: dq those of earlier
 * tokens, dk and dv those of later ones. Options, limits and workspace
 * (selscan_linattn_bwd_workspace_bytes()) as for the forward. Outputs are
 * contiguous and overlap no input.
 */
SELSCAN_API int selscan_linattn_bwd(const void *q, const void *k, const void *v, float scale,
                                    const selscan_linattn_options_t *options, const void *dy,
                                    const float *dfinal_state, void *dq, void *dk_out,
                                    void *dv_out, void *dlog_decay, float *dinitial_state,
                                    int64_t batch, int64_t seqlen, int64_t qk_heads,
                                    int64_t heads, int64_t dk, int64_t dv, selscan_dtype_t dtype,
                                    void *workspace, int64_t workspace_bytes,
                                    selscan_stream_t stream);

/* Host-only: workspace bytes selscan_linattn_bwd takes (0 for empty or invalid sizes). */
SELSCAN_API int64_t selscan_linattn_bwd_workspace_bytes(int64_t batch, int64_t seqlen,
                                                        int64_t qk_heads, int64_t heads,
                                                        int64_t dk, int64_t dv,
                                                        selscan_dtype_t dtype);

/*
 * selscan_linattn_step -- one token of selscan_linattn_fwd, the state updated
 * in place (recurrent inference after a prompt's final_state):
 *   state       [batch, heads, dk, dv]   float32   read and overwritten
 *   q, k        [batch, qk_heads, dk]    dtype     required
 *   v, y        [batch, heads, dv]       dtype     required (y: output)
 *   log_decay   [batch, heads] dtype, or head_log_decay [heads] float32, or
 *               neither (no decay); both: SELSCAN_ERR_BAD_DIM
 * A log decay of −∞ resets the state (its old content does not count). No
 * memory is allocated.
 */
SELSCAN_API int selscan_linattn_step(float *state, const void *q, const void *k, const void *v,
                                     const void *log_decay, const float *head_log_decay,
                                     float scale, void *y, int64_t batch, int64_t qk_heads,
                                     int64_t heads, int64_t dk, int64_t dv, selscan_dtype_t dtype,
                                     selscan_stream_t stream);

/* Where the gate silu(z) of selscan_block_norm_fwd stands. */
enum {
    SELSCAN_GATE_NONE = 0,
    SELSCAN_GATE_BEFORE = 1, /* the block's output is gated, then normed */
    SELSCAN_GATE_AFTER = 2   /* normed, then gated */
};

/* Options of selscan_block_norm_fwd and selscan_block_norm_bwd. */
typedef struct {
    const void *z;            /* [rows, dim] dtype (gate != SELSCAN_GATE_NONE) */
    int64_t x_stride, z_stride; /* elements between rows; 0 -> dim */
    const float *weight;      /* [dim]: the norm after the block; NULL -> no such norm */
    const void *residual;     /* [rows, dim]; NULL -> none */
    const float *res_scale;   /* [dim]: scale of the block's branch; NULL -> one */
    const float *next_weight; /* [dim]: the norm before the next block; NULL -> none */
    int64_t groups;           /* groups of the norm after the block (0 -> 1; needs weight when
                                 above 1; divides dim; up to 1024) */
    int gate;                 /* SELSCAN_GATE_* */
    int residual_f32;         /* residual, out, dout and dresidual are float32 whatever dtype is */
    float eps;                /* >= 0 */
} selscan_block_norm_options_t;

/*
 * selscan_block_norm_fwd -- what stands between two blocks, in one pass: the
 * norm of the block's output with its gate ("Mamba Block": y·silu(z)), the
 * scaled residual sum, and the norm before the next block. Per row:
 *   a   = x                (SELSCAN_GATE_BEFORE: x·silu(z))
 *   p   = a·rsqrt(mean_group(a²) + eps)·weight     (weight NULL: p = a)
 *   u   = p                (SELSCAN_GATE_AFTER: p·silu(z))
 *   out = residual + res_scale·u
 *   y   = out·rsqrt(mean(out²) + eps)·next_weight  (from the unrounded out)
 *   x, y   [rows, dim]   dtype            x required; y required iff next_weight is given
 *   out    [rows, dim]   residual's type  NULL -> not written (then y is); may be
 *                                         residual itself
 *   1 <= dim <= 16384, rows < 2^31. Arithmetic and sums are float32.
 */
SELSCAN_API int selscan_block_norm_fwd(const void *x, const selscan_block_norm_options_t *options,
                                       void *out, void *y, int64_t rows, int64_t dim,
                                       selscan_dtype_t dtype, selscan_stream_t stream);

/*
 * selscan_block_norm_bwd -- the gradient of selscan_block_norm_fwd for the loss
 * Σ dout·out + Σ dy·y, everything of the forward recomputed from its inputs:
 *   dout       [rows, dim]  residual's type  NULL -> zero (then dy is given)
 *   dy         [rows, dim]  dtype            required iff next_weight is given
 *   dx         [rows, dim]  dtype            required output
 *   dz         [rows, dim]  dtype            required output with a gate
 *   dresidual  [rows, dim]  residual's type  NULL -> not written
 *   dweight, dres_scale, dnext_weight [dim] float32, sums over the rows in a
 *              fixed order; NULL -> not written
 * Outputs are contiguous, overwritten, and overlap no input. Workspace
 * (256-byte aligned; NULL: allocated on the stream) of
 * selscan_block_norm_bwd_workspace_bytes() bytes.
 */
SELSCAN_API int selscan_block_norm_bwd(const void *x, const selscan_block_norm_options_t *options,
                                       const void *dout, const void *dy, void *dx, void *dz,
                                       void *dresidual, float *dweight, float *dres_scale,
                                       float *dnext_weight, int64_t rows, int64_t dim,
                                       selscan_dtype_t dtype, void *workspace,
                                       int64_t workspace_bytes, selscan_stream_t stream);

/* Host-only: workspace bytes selscan_block_norm_bwd takes (0 for empty or invalid sizes). */
SELSCAN_API int64_t selscan_block_norm_bwd_workspace_bytes(int64_t rows, int64_t dim);

/*
 * selscan_device_status -- the library's sticky device-side error word on
 * the current device (synchronous: waits for prior work). 0 means no device
 * wait has given up; otherwise the code of the first one that did (1: a
 * sequence chunk waited too long for its predecessor's state; 2, 3: a
 * pipeline stage waited too long; 4: a tensor-core MMA or its operand copy
 * of selscan_ssd_fwd did not complete in time; 5: the state copy of a
 * selscan_state_update step did not complete in time; 6: a step of the tensor-core pipeline of
 * selscan_linattn_fwd or _bwd; 7: a row copy of selscan_block_norm_fwd or _bwd).
 * Every device-side wait in the library is
 * bounded (2 s); a wait that gives up records its code here and the kernel
 * returns instead of hanging, leaving its outputs undefined. `clear` nonzero
 * resets the word to 0 after reading it.
 */
SELSCAN_API int selscan_device_status(int *status, int clear);

/* Static, NUL-terminated description of a status code (never NULL). */
SELSCAN_API const char *selscan_status_string(int status);

/* Text of the CUDA error behind the calling thread's last SELSCAN_ERR_CUDA
 * (static storage; "no error" if none). */
SELSCAN_API const char *selscan_last_cuda_error(void);

#ifdef __cplusplus
}
#endif

#endif /* SELSCAN_H_ */
