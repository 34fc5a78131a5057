// linattn_params.cuh -- launch parameters and entry points of linear attention
// with a decay for each head (linattn.cu, linattn_tc.cu, linattn_step.cu).
//
// Everything is built from one sweep over a sequence. For one (batch row,
// head), tokens 0 .. n − 1 and log decays g_t:
//   forward in time   S_t = exp(g_t)·S_{t−1} + c·k_t v_tᵀ,   y_t = r·S_tᵀ q_t
//   reverse in time   S_t = exp(g_{t+1})·S_{t+1} + c·k_t v_tᵀ, y_t = r·S_tᵀ q_t
// with scale factors c and r (c·r = the attention's scale). The forward pass
// is one sweep; its gradient is three:
//   dq = forward sweep of (q ← dy, k ← v, v ← k)
//   dk = reverse sweep of (q ← v, k ← dy, v ← q)
//   dv = reverse sweep of (q ← k, k ← q, v ← dy)
// and the log decays' gradient is a running sum of q·dq − k·dk.
#pragma once

#include "selscan_device.cuh"

namespace selscan {

constexpr int kLaChunk = 64;     // tokens per chunk
constexpr int kLaMaxDim = 128;   // largest head dimension of q/k and of v

struct SweepArgs {
    const void *q, *k, *v;        // token t of head h at row (b·seqlen + t)·*_row + (h / *_group)·dim
    const void *dot;              // NULL, or an operand with v's dims: dot_out = y · dot per token
    long long q_row, k_row, v_row, dot_row;    // elements between tokens
    int q_group, k_group, v_group, dot_group;  // heads that share one head of the operand
    int dk, dv;
    int reverse;
    float p_scale;                // on the products inside a chunk (c·r)
    float row_scale, col_scale;   // r on what a state gives, c on what a state takes
    void *y;                      // [batch][seqlen][heads][dv]
    int y_f32;                    // y in float32 whatever the I/O type
    float *dot_out;               // [ceil(dv / 64)][batch][heads][seqlen] partial sums
    const float *h_init;          // [batch][heads][dk][dv] (h_init_t: [dv][dk]) or NULL: the state entering
    float *h_final;               // likewise, the state leaving, or NULL
    int h_init_t, h_final_t;
    int fine_state;               // h_final is a result of the call: its sums keep 24 bits
    float *seg_state;             // [batch·heads][nseg][dk][dv]: segments' states
    float *seg_decay;             // [batch·heads][nseg]
    int map[4], map_y;            // tensor-core path: tensor maps of q, k, v, dot and y
};

struct LinattnParams {
    const void *g;                // [batch][seqlen][heads] log decays, or NULL
    const float *g_head;          // [heads] log decays, or NULL (both NULL: no decay)
    const int *seqlens;           // [batch] or NULL
    long long batch, seqlen;
    int heads;
    int nchunks, nseg, first_chunks, seg_chunks;
    int order0, orders;           // the segments of a launch, in the sweep's order (set by it)
    int nsweeps;
    int vec;                      // every operand row allows 4-element vector loads
    int *status;                  // the library's device error word
    SweepArgs sweep[3];
};

// Log decays (times log2 e) below this act as −∞: 2^−160 is zero in float32,
// and finite sums keep differences of resets well defined.
constexpr double kLaResetLog2 = -160.0;

// Plan: a sequence cut into segments. The first (in the sweep's order) runs whole
// while a second kernel on the SMs left over finds the own states of the others but
// the last; a carry turns these into the states entering, and the others run whole.
// The first segment is the shorter one: its full pass takes as long as a state pass
// over the others' seg_chunks. `ctas`: blocks of one segment; `slots`: blocks the
// device runs at a time.
struct LinattnPlan {
    int nchunks, nseg, first_chunks, seg_chunks;
};

// Chunks [*first, *last) of a sweep's segment.
__device__ __forceinline__ void linattn_segment(const LinattnParams &p, bool reverse, int order,
                                                int *first, int *last) {
    const int from = order ? p.first_chunks + (order - 1) * p.seg_chunks : 0;
    const int to = min(p.nchunks, from + (order ? p.seg_chunks : p.first_chunks));
    *first = reverse ? p.nchunks - to : from;
    *last = reverse ? p.nchunks - from : to;
}

// The first segment's kernel, called at its start: the state kernel may take the SMs
// that are left over.
__device__ __forceinline__ void linattn_let_states_start() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// The state kernel, at its end: what follows waits for both kernels.
__device__ __forceinline__ void linattn_wait_for_first() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// `head`: a block's start-up, `own`: the state pass's time, in chunk passes
// and as a share of the full pass.
LinattnPlan linattn_plan(long long seqlen, long long ctas, int slots, double head, double own);

// CUDA-core path: any sizes and alignment, both I/O types.
int linattn_tiles(int dv);  // 64-column tiles of a sweep (blocks per head and segment)
int linattn_slots(int dk, int dv);
cudaError_t launch_linattn_sweeps(const LinattnParams &p, bool bf16, cudaStream_t stream);
// Carry: seg_state[s] becomes the state entering segment s. A segment with decay
// zero (the first, whose state has its initial one in it) is not added to.
cudaError_t launch_linattn_carry(const LinattnParams &p, cudaStream_t stream);

// The launches of a sweep: `full` and `state` take the arguments behind p, on
// per_seg blocks a segment.
template <typename Kernel, typename... Args>
cudaError_t linattn_launch(Kernel full, Kernel state, int threads, int smem_full, int smem_state,
                           long long per_seg, LinattnParams p, cudaStream_t stream,
                           const Args &...args) {
    p.order0 = 0;
    p.orders = 1;
    full<<<(unsigned)per_seg, threads, smem_full, stream>>>(p, args...);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.nseg == 1) return e;
    p.order0 = 1;
    p.orders = p.nseg - 2;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t config{};
    config.gridDim = dim3((unsigned)(per_seg * p.orders));
    config.blockDim = dim3((unsigned)threads);
    config.dynamicSmemBytes = (size_t)smem_state;
    config.stream = stream;
    config.attrs = &attr;
    config.numAttrs = 1;
    e = cudaLaunchKernelEx(&config, state, p, args...);
    if (e == cudaSuccess) e = launch_linattn_carry(p, stream);
    if (e != cudaSuccess) return e;
    p.orders = p.nseg - 1;
    full<<<(unsigned)(per_seg * p.orders), threads, smem_full, stream>>>(p, args...);
    return cudaGetLastError();
}

// Tensor-core path (linattn_tc.cu): bfloat16 I/O, operands whose rows TMA can
// read (16-byte rows and bases, dims multiples of 8); one block an SM.
bool linattn_tc_rows(const void *ptr, long long row, int dim, long long seqlen);
cudaError_t launch_linattn_tc(const LinattnParams &p, cudaStream_t stream);

// Sums of the `group` heads that share one query/key head, of dq and of dk:
// src [tokens][qk_heads][group][dim] float32 -> dst [tokens][qk_heads][dim].
cudaError_t launch_linattn_group_sums(const float *const src[2], void *const dst[2],
                                      long long tokens, int qk_heads, int group, int dim, bool bf16,
                                      cudaStream_t stream);

// dlog_decay from the per-token dot products (rows = q·dq, cols = k·dk, each
// `tiles` partial sums of [batch][heads][seqlen]) and, when dfinal is given,
// the inner product of the last state with its gradient.
struct LinattnDecayGrad {
    const float *rows, *cols;
    int tiles;
    const float *last_state, *dfinal;  // [batch][heads][dk·dv]
    long long state_size;
    const int *seqlens;
    long long batch, seqlen;
    int heads;
    const void *g;                     // the log decays
    int has_init;                      // a first state was given
    void *dg;                          // [batch][seqlen][heads]
};
cudaError_t launch_linattn_decay_grad(const LinattnDecayGrad &p, bool bf16, cudaStream_t stream);

// One token.
struct LinattnStepParams {
    float *state;                 // [batch][heads][dk][dv]
    const void *q, *k, *v;        // [batch][qk_heads][dk], [batch][heads][dv]
    const void *g;                // [batch][heads] or NULL
    const float *g_head;          // [heads] or NULL
    void *y;                      // [batch][heads][dv]
    long long batch;
    int heads, group, dk, dv;
    float scale;
};
cudaError_t launch_linattn_step(const LinattnStepParams &p, bool bf16, cudaStream_t stream);

}  // namespace selscan
