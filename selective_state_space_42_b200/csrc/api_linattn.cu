// api_linattn.cu -- C entry points of linear attention with a decay for each
// head and of the block-norm junction: argument validation, workspace layout
// and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <stdint.h>

#include "api_util.cuh"
#include "block_norm.cuh"
#include "linattn_params.cuh"
#include "selscan.h"

using namespace selscan;

namespace {

constexpr int64_t kMaxPairs = (int64_t)1 << 22;  // batch·heads: rows of a one-dimensional grid

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// Bytes from the first to the last element of `rows` rows of `dim` elements,
// `stride` apart.
size_t strided_bytes(int64_t rows, int64_t stride, int64_t dim, size_t es) {
    return rows > 0 ? ((size_t)(rows - 1) * (size_t)stride + (size_t)dim) * es : 0;
}

struct LaDims {
    int64_t batch, seqlen, qk_heads, heads, dk, dv;
    size_t es;
    bool bf16;
    int64_t tokens() const { return batch * seqlen; }
    int64_t pairs() const { return batch * heads; }
    size_t state_bytes() const { return (size_t)(pairs() * dk * dv) * sizeof(float); }
};

int check_dims(const LaDims &d, int dtype) {
    if (dtype != SELSCAN_F32 && dtype != SELSCAN_BF16) return SELSCAN_ERR_BAD_DTYPE;
    if (d.batch < 0 || d.seqlen < 0 || d.heads < 0 || d.qk_heads < 0 || d.dk < 1 ||
        d.dk > kLaMaxDim || d.dv < 1 || d.dv > kLaMaxDim || d.heads > 65535 ||
        (d.heads > 0 && (d.qk_heads == 0 || d.heads % d.qk_heads != 0)))
        return SELSCAN_ERR_BAD_DIM;
    if (!mul_le(d.batch, std::max<int64_t>(d.heads, 1), kMaxPairs) ||
        d.seqlen > ((int64_t)1 << 36) ||
        !mul_le(std::max<int64_t>(d.batch, 1) * std::max<int64_t>(d.heads, 1) * kLaMaxDim,
                d.seqlen, kMaxElems))
        return SELSCAN_ERR_BAD_DIM;
    return SELSCAN_OK;
}

// tc: the tensor-core kernels.
LinattnPlan plan_for(const LaDims &d, int nsweeps, bool tc) {
    const int64_t ctas = d.pairs() * nsweeps;
    if (tc) return linattn_plan(d.seqlen, ctas, sm_count(), 3.0, 0.55);
    return linattn_plan(d.seqlen, ctas * linattn_tiles((int)std::max(d.dk, d.dv)),
                        sm_count() * linattn_slots((int)d.dk, (int)d.dv), 0.5, 0.5);
}

// Workspace of one call (offsets in bytes).
struct LaLayout {
    size_t seg_state[3], seg_decay[3];
    size_t rows, cols;     // q·dq and k·dk per token
    size_t dq, dk;         // float32 gradients of each head where heads share q and k
    size_t last_state;
    size_t total;
};

LaLayout layout_for(const LaDims &d, const LinattnPlan &pl, bool bwd) {
    LaLayout l{};
    size_t off = 0;
    auto take = [&off](size_t n) {
        const size_t at = off;
        off += align256(n);
        return at;
    };
    if (pl.nseg > 1)
        for (int s = 0; s < (bwd ? 3 : 1); ++s) {
            l.seg_state[s] = take(d.state_bytes() * pl.nseg);
            l.seg_decay[s] = take((size_t)(d.pairs() * pl.nseg) * sizeof(float));
        }
    if (bwd) {
        const size_t n = (size_t)(d.pairs() * d.seqlen) * sizeof(float) * linattn_tiles((int)d.dk);
        l.rows = take(n);
        l.cols = take(n);
        l.last_state = take(d.state_bytes());
        if (d.heads != d.qk_heads) {
            const size_t g = (size_t)(d.tokens() * d.heads * d.dk) * sizeof(float);
            l.dq = take(g);
            l.dk = take(g);
        }
    }
    l.total = off;
    return l;
}

int64_t workspace_for(const LaDims &d, int dtype, bool bwd) {
    if (check_dims(d, dtype) != SELSCAN_OK || d.pairs() * d.seqlen == 0) return 0;
    // the larger of the two paths' (which one runs depends on the operands' rows)
    const int n = bwd ? 3 : 1;
    size_t total = layout_for(d, plan_for(d, n, false), bwd).total;
    if (d.bf16) total = std::max(total, layout_for(d, plan_for(d, n, true), bwd).total);
    return (int64_t)total;
}

// Checks shared by the forward and the gradient, on the operands and options.
struct LaInputs {
    const void *q, *k, *v;
    selscan_linattn_options_t o;
    int64_t q_row, k_row, v_row;
};

int check_inputs(const LaDims &d, const void *q, const void *k, const void *v,
                 const selscan_linattn_options_t *options, LaInputs *in) {
    in->q = q;
    in->k = k;
    in->v = v;
    in->o = options ? *options : selscan_linattn_options_t{};
    const selscan_linattn_options_t &o = in->o;
    if (o.log_decay && o.head_log_decay) return SELSCAN_ERR_BAD_DIM;
    const int64_t qd = d.qk_heads * d.dk, vd = d.heads * d.dv;
    in->q_row = o.q_stride ? o.q_stride : qd;
    in->k_row = o.k_stride ? o.k_stride : qd;
    in->v_row = o.v_stride ? o.v_stride : vd;
    if (in->q_row < qd || in->k_row < qd || in->v_row < vd) return SELSCAN_ERR_BAD_DIM;
    const int64_t widest = std::max(in->q_row, std::max(in->k_row, in->v_row));
    if (!mul_le(d.tokens(), widest, kMaxElems)) return SELSCAN_ERR_BAD_DIM;
    if (d.pairs() * d.seqlen > 0 && (!q || !k || !v)) return SELSCAN_ERR_NULL_ARG;
    if (misaligned(q, d.es) || misaligned(k, d.es) || misaligned(v, d.es) ||
        misaligned(o.log_decay, d.es) || misaligned(o.head_log_decay, 4) ||
        misaligned(o.initial_state, 4) || misaligned(o.seqlens, 4))
        return SELSCAN_ERR_MISALIGNED;
    return SELSCAN_OK;
}

int input_spans(const LaDims &d, const LaInputs &in, Span *s) {
    const selscan_linattn_options_t &o = in.o;
    int n = 0;
    s[n++] = {in.q, strided_bytes(d.tokens(), in.q_row, d.qk_heads * d.dk, d.es)};
    s[n++] = {in.k, strided_bytes(d.tokens(), in.k_row, d.qk_heads * d.dk, d.es)};
    s[n++] = {in.v, strided_bytes(d.tokens(), in.v_row, d.heads * d.dv, d.es)};
    s[n++] = {o.log_decay, (size_t)(d.tokens() * d.heads) * d.es};
    s[n++] = {o.head_log_decay, (size_t)d.heads * 4};
    s[n++] = {o.seqlens, (size_t)d.batch * 4};
    return n;  // the initial state is checked by the caller (it may be the final state)
}

LinattnParams base_params(const LaDims &d, const LaInputs &in, const LinattnPlan &pl) {
    LinattnParams p{};
    p.g = in.o.log_decay;
    p.g_head = in.o.head_log_decay;
    p.seqlens = in.o.seqlens;
    p.batch = d.batch;
    p.seqlen = d.seqlen;
    p.heads = (int)d.heads;
    p.nchunks = pl.nchunks;
    p.nseg = pl.nseg;
    p.first_chunks = pl.first_chunks;
    p.seg_chunks = pl.seg_chunks;
    return p;
}

bool rows_vec(const void *p, int64_t row, int64_t dim, size_t es) {
    return !misaligned(p, 4 * es) && row % 4 == 0 && dim % 4 == 0;
}

cudaError_t set_state(float *dst, const float *src, size_t n, cudaStream_t stream) {
    if (!dst || n == 0 || dst == src) return cudaSuccess;
    return src ? cudaMemcpyAsync(dst, src, n, cudaMemcpyDeviceToDevice, stream)
               : cudaMemsetAsync(dst, 0, n, stream);
}

// The workspace given, or one allocated on the stream.
int take_workspace(void **ws, void *given, int64_t given_bytes, size_t need, const Span *outs,
                   int no, const Span *ins, int ni, cudaStream_t stream) {
    *ws = given;
    if (need == 0) return SELSCAN_OK;
    if (given) {
        if (given_bytes < (int64_t)need) return SELSCAN_ERR_WORKSPACE;
        const Span w[] = {{given, need}};
        if (any_overlap(w, 1, outs, no) || any_overlap(w, 1, ins, ni)) return SELSCAN_ERR_ALIAS;
        return SELSCAN_OK;
    }
    const cudaError_t e = cudaMallocAsync(ws, need, stream);
    return e == cudaSuccess ? SELSCAN_OK : cuda_fail(e);
}

int finish(cudaError_t e, void *ws, bool own, cudaStream_t stream) {
    if (own && ws) {
        const cudaError_t ef = cudaFreeAsync(ws, stream);
        if (e == cudaSuccess) e = ef;
    }
    return e == cudaSuccess ? SELSCAN_OK : cuda_fail(e);
}

}  // namespace

extern "C" {

int64_t selscan_linattn_workspace_bytes(int64_t batch, int64_t seqlen, int64_t qk_heads,
                                        int64_t heads, int64_t dk, int64_t dv,
                                        selscan_dtype_t dtype) {
    const LaDims d{batch, seqlen, qk_heads, heads, dk, dv, dtype == SELSCAN_BF16 ? 2u : 4u,
                   dtype == SELSCAN_BF16};
    return workspace_for(d, dtype, false);
}

int64_t selscan_linattn_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t qk_heads,
                                            int64_t heads, int64_t dk, int64_t dv,
                                            selscan_dtype_t dtype) {
    const LaDims d{batch, seqlen, qk_heads, heads, dk, dv, dtype == SELSCAN_BF16 ? 2u : 4u,
                   dtype == SELSCAN_BF16};
    return workspace_for(d, dtype, true);
}

int selscan_linattn_fwd(const void *q, const void *k, const void *v, float scale,
                        const selscan_linattn_options_t *options, void *y, float *final_state,
                        int64_t batch, int64_t seqlen, int64_t qk_heads, int64_t heads, int64_t dk,
                        int64_t dv, selscan_dtype_t dtype, void *workspace,
                        int64_t workspace_bytes, selscan_stream_t stream_) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    const LaDims d{batch, seqlen, qk_heads, heads, dk, dv, dtype == SELSCAN_BF16 ? 2u : 4u,
                   dtype == SELSCAN_BF16};
    int rc = check_dims(d, dtype);
    if (rc != SELSCAN_OK) return rc;
    LaInputs in;
    rc = check_inputs(d, q, k, v, options, &in);
    if (rc != SELSCAN_OK) return rc;
    const bool has_tokens = d.pairs() * seqlen > 0;
    if (has_tokens && !y) return SELSCAN_ERR_NULL_ARG;
    if (misaligned(y, d.es) || misaligned(final_state, 4) || misaligned(workspace, 256))
        return SELSCAN_ERR_MISALIGNED;
    const float *h0 = in.o.initial_state;
    const Span outs[] = {{y, (size_t)(d.tokens() * heads * dv) * d.es},
                         {final_state, d.state_bytes()}};
    Span ins[8];
    int ni = input_spans(d, in, ins);
    if (h0 != final_state) ins[ni++] = {h0, d.state_bytes()};
    if (any_overlap(outs, 2, ins, ni)) return SELSCAN_ERR_ALIAS;
    if (!has_tokens) {
        const cudaError_t e = set_state(final_state, h0, d.state_bytes(), stream);
        return e == cudaSuccess ? SELSCAN_OK : cuda_fail(e);
    }
    const bool tc = d.bf16 && linattn_tc_rows(q, in.q_row, (int)dk, seqlen) &&
                    linattn_tc_rows(k, in.k_row, (int)dk, seqlen) &&
                    linattn_tc_rows(v, in.v_row, (int)dv, seqlen) &&
                    linattn_tc_rows(y, heads * dv, (int)dv, seqlen);
    const LinattnPlan pl = plan_for(d, 1, tc);
    const LaLayout l = layout_for(d, pl, false);
    void *ws = nullptr;
    rc = take_workspace(&ws, workspace, workspace_bytes, l.total, outs, 2, ins, ni, stream);
    if (rc != SELSCAN_OK) return rc;
    char *w = static_cast<char *>(ws);
    LinattnParams p = base_params(d, in, pl);
    p.nsweeps = 1;
    p.vec = rows_vec(q, in.q_row, dk, d.es) && rows_vec(k, in.k_row, dk, d.es) &&
            rows_vec(v, in.v_row, dv, d.es) && !misaligned(y, 4 * d.es);
    const int group = (int)(heads / qk_heads);
    SweepArgs &a = p.sweep[0];
    a.q = q; a.k = k; a.v = v;
    a.q_row = in.q_row; a.k_row = in.k_row; a.v_row = in.v_row;
    a.q_group = a.k_group = group; a.v_group = 1; a.dot_group = 1;
    a.dk = (int)dk; a.dv = (int)dv;
    a.p_scale = a.row_scale = scale;
    a.col_scale = 1.f;
    a.y = y;
    a.h_init = h0;
    a.h_final = final_state;
    if (pl.nseg > 1) {
        a.seg_state = reinterpret_cast<float *>(w + l.seg_state[0]);
        a.seg_decay = reinterpret_cast<float *>(w + l.seg_decay[0]);
    }
    cudaError_t e = device_status_address(&p.status);
    if (e == cudaSuccess)
        e = tc ? launch_linattn_tc(p, stream) : launch_linattn_sweeps(p, d.bf16, stream);
    return finish(e, ws, !workspace, stream);
}

int selscan_linattn_bwd(const void *q, const void *k, const void *v, float scale,
                        const selscan_linattn_options_t *options, const void *dy,
                        const float *dfinal_state, void *dq, void *dk_, void *dv_,
                        void *dlog_decay, float *dinitial_state, int64_t batch, int64_t seqlen,
                        int64_t qk_heads, int64_t heads, int64_t dk, int64_t dv,
                        selscan_dtype_t dtype, void *workspace, int64_t workspace_bytes,
                        selscan_stream_t stream_) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    const LaDims d{batch, seqlen, qk_heads, heads, dk, dv, dtype == SELSCAN_BF16 ? 2u : 4u,
                   dtype == SELSCAN_BF16};
    int rc = check_dims(d, dtype);
    if (rc != SELSCAN_OK) return rc;
    LaInputs in;
    rc = check_inputs(d, q, k, v, options, &in);
    if (rc != SELSCAN_OK) return rc;
    const bool has_tokens = d.pairs() * seqlen > 0;
    if (has_tokens && (!dy || !dq || !dk_ || !dv_ || (dlog_decay && !in.o.log_decay)))
        return SELSCAN_ERR_NULL_ARG;
    if (misaligned(dy, d.es) || misaligned(dq, d.es) || misaligned(dk_, d.es) ||
        misaligned(dv_, d.es) || misaligned(dlog_decay, d.es) || misaligned(dfinal_state, 4) ||
        misaligned(dinitial_state, 4) || misaligned(workspace, 256))
        return SELSCAN_ERR_MISALIGNED;
    const float *h0 = in.o.initial_state;
    const size_t nqk = (size_t)(d.tokens() * qk_heads * dk) * d.es;
    const size_t nv = (size_t)(d.tokens() * heads * dv) * d.es;
    const Span outs[] = {{dq, nqk}, {dk_, nqk}, {dv_, nv},
                         {dlog_decay, (size_t)(d.tokens() * heads) * d.es},
                         {dinitial_state, d.state_bytes()}};
    Span ins[10];
    int ni = input_spans(d, in, ins);
    ins[ni++] = {h0, d.state_bytes()};
    ins[ni++] = {dy, nv};
    ins[ni++] = {dfinal_state, d.state_bytes()};
    if (any_overlap(outs, 5, ins, ni)) return SELSCAN_ERR_ALIAS;
    if (!has_tokens) {
        const cudaError_t e = set_state(dinitial_state, dfinal_state, d.state_bytes(), stream);
        return e == cudaSuccess ? SELSCAN_OK : cuda_fail(e);
    }
    const bool shared = heads != qk_heads;
    const bool tc = d.bf16 && linattn_tc_rows(q, in.q_row, (int)dk, seqlen) &&
                    linattn_tc_rows(k, in.k_row, (int)dk, seqlen) &&
                    linattn_tc_rows(v, in.v_row, (int)dv, seqlen) &&
                    linattn_tc_rows(dy, heads * dv, (int)dv, seqlen) &&
                    (shared || (linattn_tc_rows(dq, heads * dk, (int)dk, seqlen) &&
                                linattn_tc_rows(dk_, heads * dk, (int)dk, seqlen))) &&
                    linattn_tc_rows(dv_, heads * dv, (int)dv, seqlen) &&
                    seqlen * heads * std::max(dk, dv) < (1ll << 37);
    const LinattnPlan pl = plan_for(d, 3, tc);
    const LaLayout l = layout_for(d, pl, true);
    void *ws = nullptr;
    rc = take_workspace(&ws, workspace, workspace_bytes, l.total, outs, 5, ins, ni, stream);
    if (rc != SELSCAN_OK) return rc;
    char *w = static_cast<char *>(ws);
    LinattnParams p = base_params(d, in, pl);
    p.nsweeps = 3;
    p.vec = rows_vec(q, in.q_row, dk, d.es) && rows_vec(k, in.k_row, dk, d.es) &&
            rows_vec(v, in.v_row, dv, d.es) && rows_vec(dy, heads * dv, dv, d.es) &&
            (shared || (!misaligned(dq, 4 * d.es) && !misaligned(dk_, 4 * d.es))) &&
            !misaligned(dv_, 4 * d.es);
    const int group = (int)(heads / qk_heads);
    const bool want_dg = dlog_decay != nullptr;
    for (int s = 0; s < 3; ++s) {
        SweepArgs &a = p.sweep[s];
        a.p_scale = scale;
        a.dot_group = group;
        if (pl.nseg > 1) {
            a.seg_state = reinterpret_cast<float *>(w + l.seg_state[s]);
            a.seg_decay = reinterpret_cast<float *>(w + l.seg_decay[s]);
        }
    }
    {   // dq: (q ← dy, k ← v, v ← k), forward in time; its state is Sᵀ
        SweepArgs &a = p.sweep[0];
        a.q = dy; a.q_row = heads * dv; a.q_group = 1;
        a.k = v; a.k_row = in.v_row; a.k_group = 1;
        a.v = k; a.v_row = in.k_row; a.v_group = group;
        a.dk = (int)dv; a.dv = (int)dk;
        a.row_scale = scale; a.col_scale = 1.f;
        a.y = shared ? static_cast<void *>(w + l.dq) : dq;
        a.y_f32 = shared;
        a.h_init = h0; a.h_init_t = 1;
        if (want_dg) {
            a.dot = q; a.dot_row = in.q_row;
            a.dot_out = reinterpret_cast<float *>(w + l.rows);
            if (dfinal_state) {
                a.h_final = reinterpret_cast<float *>(w + l.last_state);
                a.h_final_t = 1;
            }
        }
    }
    {   // dk: (q ← v, k ← dy, v ← q), backwards; its state is the transposed state gradient
        SweepArgs &a = p.sweep[1];
        a.q = v; a.q_row = in.v_row; a.q_group = 1;
        a.k = dy; a.k_row = heads * dv; a.k_group = 1;
        a.v = q; a.v_row = in.q_row; a.v_group = group;
        a.dk = (int)dv; a.dv = (int)dk;
        a.reverse = 1;
        a.row_scale = 1.f; a.col_scale = scale;
        a.y = shared ? static_cast<void *>(w + l.dk) : dk_;
        a.y_f32 = shared;
        a.h_init = dfinal_state; a.h_init_t = 1;
        if (want_dg) {
            a.dot = k; a.dot_row = in.k_row;
            a.dot_out = reinterpret_cast<float *>(w + l.cols);
        }
    }
    {   // dv: (q ← k, k ← q, v ← dy), backwards
        SweepArgs &a = p.sweep[2];
        a.q = k; a.q_row = in.k_row; a.q_group = group;
        a.k = q; a.k_row = in.q_row; a.k_group = group;
        a.v = dy; a.v_row = heads * dv; a.v_group = 1;
        a.dk = (int)dk; a.dv = (int)dv;
        a.reverse = 1;
        a.row_scale = 1.f; a.col_scale = scale;
        a.y = dv_;
        a.h_init = dfinal_state;
        a.h_final = dinitial_state;
        a.fine_state = dinitial_state != nullptr;
    }
    cudaError_t e = device_status_address(&p.status);
    if (e == cudaSuccess)
        e = tc ? launch_linattn_tc(p, stream) : launch_linattn_sweeps(p, d.bf16, stream);
    if (shared) {
        const float *src[2] = {reinterpret_cast<float *>(w + l.dq),
                               reinterpret_cast<float *>(w + l.dk)};
        void *dst[2] = {dq, dk_};
        if (e == cudaSuccess)
            e = launch_linattn_group_sums(src, dst, d.tokens(), (int)qk_heads, group, (int)dk,
                                          d.bf16, stream);
    }
    if (want_dg && e == cudaSuccess) {
        LinattnDecayGrad g{};
        g.rows = reinterpret_cast<const float *>(w + l.rows);
        g.cols = reinterpret_cast<const float *>(w + l.cols);
        g.tiles = tc ? 1 : linattn_tiles((int)dk);  // the tensor-core blocks hold all columns
        g.dfinal = dfinal_state;
        g.last_state = reinterpret_cast<const float *>(w + l.last_state);
        g.state_size = dk * dv;
        g.seqlens = in.o.seqlens;
        g.batch = batch;
        g.seqlen = seqlen;
        g.heads = (int)heads;
        g.g = in.o.log_decay;
        g.has_init = h0 != nullptr;
        g.dg = dlog_decay;
        e = launch_linattn_decay_grad(g, d.bf16, stream);
    }
    return finish(e, ws, !workspace, stream);
}

int selscan_linattn_step(float *state, const void *q, const void *k, const void *v,
                         const void *log_decay, const float *head_log_decay, float scale, void *y,
                         int64_t batch, int64_t qk_heads, int64_t heads, int64_t dk, int64_t dv,
                         selscan_dtype_t dtype, selscan_stream_t stream_) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    const LaDims d{batch, 1, qk_heads, heads, dk, dv, dtype == SELSCAN_BF16 ? 2u : 4u,
                   dtype == SELSCAN_BF16};
    const int rc = check_dims(d, dtype);
    if (rc != SELSCAN_OK) return rc;
    if (log_decay && head_log_decay) return SELSCAN_ERR_BAD_DIM;
    if (d.pairs() > 0 && (!state || !q || !k || !v || !y)) return SELSCAN_ERR_NULL_ARG;
    if (misaligned(q, d.es) || misaligned(k, d.es) || misaligned(v, d.es) ||
        misaligned(y, d.es) || misaligned(log_decay, d.es) || misaligned(state, 4) ||
        misaligned(head_log_decay, 4))
        return SELSCAN_ERR_MISALIGNED;
    const size_t nqk = (size_t)(batch * qk_heads * dk) * d.es, nv = (size_t)(d.pairs() * dv) * d.es;
    const Span outs[] = {{y, nv}, {state, d.state_bytes()}};
    const Span ins[] = {{q, nqk}, {k, nqk}, {v, nv}, {log_decay, (size_t)d.pairs() * d.es},
                        {head_log_decay, (size_t)heads * 4}};
    if (any_overlap(outs, 2, ins, 5)) return SELSCAN_ERR_ALIAS;
    if (d.pairs() == 0) return SELSCAN_OK;
    LinattnStepParams p{};
    p.state = state;
    p.q = q; p.k = k; p.v = v;
    p.g = log_decay; p.g_head = head_log_decay;
    p.y = y;
    p.batch = batch;
    p.heads = (int)heads;
    p.group = (int)(heads / qk_heads);
    p.dk = (int)dk; p.dv = (int)dv;
    p.scale = scale;
    const cudaError_t e = launch_linattn_step(p, d.bf16, stream);
    return e == cudaSuccess ? SELSCAN_OK : cuda_fail(e);
}

// ---- the block-norm junction ------------------------------------------------------

static int norm_params(const void *x, const selscan_block_norm_options_t *options, int64_t rows,
                       int64_t dim, int dtype, BlockNormParams *p, Span *ins, int *ni,
                       size_t *es_out, size_t *rs_out) {
    if (dtype != SELSCAN_F32 && dtype != SELSCAN_BF16) return SELSCAN_ERR_BAD_DTYPE;
    const selscan_block_norm_options_t o = options ? *options : selscan_block_norm_options_t{};
    const int64_t groups = o.groups ? o.groups : 1;
    if (rows < 0 || rows > 0x7FFFFFFF || dim < 1 || dim > kBnMaxDim || groups < 1 ||
        groups > kBnMaxGroups || dim % groups != 0 || (groups > 1 && !o.weight) ||
        o.gate < kGateNone || o.gate > kGateAfter || !(o.eps >= 0.f))
        return SELSCAN_ERR_BAD_DIM;
    const int64_t xr = o.x_stride ? o.x_stride : dim, zr = o.z_stride ? o.z_stride : dim;
    if (xr < dim || zr < dim || !mul_le(rows, std::max(xr, zr), kMaxElems))
        return SELSCAN_ERR_BAD_DIM;
    if ((rows > 0 && !x) || (rows > 0 && o.gate != kGateNone && !o.z)) return SELSCAN_ERR_NULL_ARG;
    const size_t es = dtype == SELSCAN_F32 ? 4 : 2;
    const size_t rs = dtype == SELSCAN_F32 || o.residual_f32 ? 4 : 2;
    if (misaligned(x, es) || misaligned(o.z, es) || misaligned(o.residual, rs) ||
        misaligned(o.weight, 4) || misaligned(o.res_scale, 4) || misaligned(o.next_weight, 4))
        return SELSCAN_ERR_MISALIGNED;
    p->x = x;
    p->z = o.gate != kGateNone ? o.z : nullptr;
    p->x_row = xr;
    p->z_row = zr;
    p->weight = o.weight;
    p->res_scale = o.res_scale;
    p->next_weight = o.next_weight;
    p->res = o.residual;
    p->rows = rows;
    p->dim = (int)dim;
    p->groups = (int)groups;
    p->gate = o.gate;
    p->res_f32 = rs == 4;
    p->eps = o.eps;
    const size_t nw = (size_t)dim * 4;
    int n = 0;
    ins[n++] = {x, strided_bytes(rows, xr, dim, es)};
    ins[n++] = {p->z, strided_bytes(rows, zr, dim, es)};
    ins[n++] = {o.weight, nw};
    ins[n++] = {o.res_scale, nw};
    ins[n++] = {o.next_weight, nw};
    *ni = n;  // the residual is checked by the caller (the forward may write over it)
    p->vec = dim % 8 == 0 && xr % 8 == 0 && zr % 8 == 0 && !misaligned(x, 16) &&
             !misaligned(p->z, 16) && !misaligned(o.residual, 16) && !misaligned(o.weight, 16) &&
             !misaligned(o.res_scale, 16) && !misaligned(o.next_weight, 16);
    *es_out = es;
    *rs_out = rs;
    return SELSCAN_OK;
}

int selscan_block_norm_fwd(const void *x, const selscan_block_norm_options_t *options, void *out,
                           void *y, int64_t rows, int64_t dim, selscan_dtype_t dtype,
                           selscan_stream_t stream_) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    BlockNormParams p{};
    Span ins[8];
    int ni = 0;
    size_t es = 0, rs = 0;
    const int rc = norm_params(x, options, rows, dim, dtype, &p, ins, &ni, &es, &rs);
    if (rc != SELSCAN_OK) return rc;
    if (rows > 0 && ((!out && !y) || (p.next_weight && !y) || (y && !p.next_weight)))
        return SELSCAN_ERR_NULL_ARG;
    if (misaligned(out, rs) || misaligned(y, es)) return SELSCAN_ERR_MISALIGNED;
    const size_t n = (size_t)(rows * dim);
    const Span outs[] = {{out, n * rs}, {y, n * es}};
    if (out != p.res) ins[ni++] = {p.res, n * rs};
    if (any_overlap(outs, 2, ins, ni)) return SELSCAN_ERR_ALIAS;
    const Span yo[] = {{y, n * es}}, ro[] = {{p.res, n * rs}};
    if (any_overlap(yo, 1, ro, 1)) return SELSCAN_ERR_ALIAS;
    if (rows == 0) return SELSCAN_OK;
    p.out = out;
    p.y = y;
    p.vec = p.vec && !misaligned(out, 16) && !misaligned(y, 16);
    cudaError_t e = device_status_address(&p.status);
    if (e == cudaSuccess) e = launch_block_norm_fwd(p, dtype == SELSCAN_BF16, stream);
    return e == cudaSuccess ? SELSCAN_OK : cuda_fail(e);
}

int64_t selscan_block_norm_bwd_workspace_bytes(int64_t rows, int64_t dim) {
    if (rows < 1 || rows > 0x7FFFFFFF || dim < 1 || dim > kBnMaxDim) return 0;
    return (int64_t)block_norm_bwd_blocks(rows, (int)dim) * 2 * dim * (int64_t)sizeof(float);
}

int selscan_block_norm_bwd(const void *x, const selscan_block_norm_options_t *options,
                           const void *dout, const void *dy, void *dx, void *dz, void *dresidual,
                           float *dweight, float *dres_scale, float *dnext_weight, int64_t rows,
                           int64_t dim, selscan_dtype_t dtype, void *workspace,
                           int64_t workspace_bytes, selscan_stream_t stream_) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    BlockNormParams p{};
    Span ins[8];
    int ni = 0;
    size_t es = 0, rs = 0;
    int rc = norm_params(x, options, rows, dim, dtype, &p, ins, &ni, &es, &rs);
    if (rc != SELSCAN_OK) return rc;
    if (rows > 0 &&
        (!dx || (p.gate != kGateNone && !dz) || (p.next_weight ? !dy : dy != nullptr) ||
         (!dout && !dy)))
        return SELSCAN_ERR_NULL_ARG;
    if (misaligned(dout, rs) || misaligned(dy, es) || misaligned(dx, es) || misaligned(dz, es) ||
        misaligned(dresidual, rs) || misaligned(dweight, 4) || misaligned(dres_scale, 4) ||
        misaligned(dnext_weight, 4) || misaligned(workspace, 256))
        return SELSCAN_ERR_MISALIGNED;
    const size_t n = (size_t)(rows * dim), nw = (size_t)dim * 4;
    if (p.gate == kGateNone) dz = nullptr;
    if (!p.res) dresidual = nullptr;
    if (!p.weight) dweight = nullptr;
    if (!p.res_scale) dres_scale = nullptr;
    if (!p.next_weight) dnext_weight = nullptr;
    const Span outs[] = {{dx, n * es}, {dz, n * es}, {dresidual, n * rs},
                         {dweight, nw}, {dres_scale, nw}, {dnext_weight, nw}};
    ins[ni++] = {p.res, n * rs};
    ins[ni++] = {dout, n * rs};
    ins[ni++] = {dy, n * es};
    if (any_overlap(outs, 6, ins, ni)) return SELSCAN_ERR_ALIAS;
    if (rows == 0) {
        cudaError_t e = cudaSuccess;
        for (float *w : {dweight, dres_scale, dnext_weight})
            if (w && e == cudaSuccess) e = cudaMemsetAsync(w, 0, nw, stream);
        return e == cudaSuccess ? SELSCAN_OK : cuda_fail(e);
    }
    const size_t need = (size_t)selscan_block_norm_bwd_workspace_bytes(rows, dim);
    void *ws = nullptr;
    rc = take_workspace(&ws, workspace, workspace_bytes, need, outs, 6, ins, ni, stream);
    if (rc != SELSCAN_OK) return rc;
    p.dout = dout;
    p.dy = dy;
    p.dx = dx;
    p.dz = dz;
    p.dres = dresidual;
    p.dweight = dweight;
    p.dres_scale = dres_scale;
    p.dnext_weight = dnext_weight;
    p.partial = static_cast<float *>(ws);
    p.vec = p.vec && !misaligned(dout, 16) && !misaligned(dy, 16) && !misaligned(dx, 16) &&
            !misaligned(dz, 16) && !misaligned(dresidual, 16);
    cudaError_t e = device_status_address(&p.status);
    if (e == cudaSuccess) e = launch_block_norm_bwd(p, dtype == SELSCAN_BF16, stream);
    return finish(e, ws, !workspace, stream);
}

}  // extern "C"
