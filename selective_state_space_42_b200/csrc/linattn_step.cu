// linattn_step.cu -- one token of linear attention with a decay for each head,
// the state updated in place (recurrent inference, "SSM as Convolution"):
//   S ← exp(g)·S + k vᵀ,   y = scale·Sᵀ q      per (batch row, head), S [dk][dv]
//
// Bound: HBM, the float32 state read and written once. One block per (batch
// row, head) and column slab; every thread loads all of its state rows
// (float4s of one column group) before it computes, so that a whole slab is
// in flight at once (64 KB a block at 128×128). Fewer (row, head) pairs than
// two an SM: the columns are split over up to four blocks, which shortens the
// latency of a small batch's call. 256 rows of 32 heads of 128 × 128: 162 µs, the
// copy rate of HBM; one row: 2.5 µs.
#include "api_util.cuh"
#include "linattn_params.cuh"

namespace selscan {
namespace {

constexpr int kThr = 256;
constexpr int kMaxRows = 16;  // state rows a thread holds: 128 / (256 / 32)

// kCols float4 columns per block; thread t: column t % kCols, rows t / kCols
// and on in steps of 256 / kCols.
template <typename T, int kCols>
__global__ void __launch_bounds__(kThr) linattn_step_vec_kernel(const LinattnStepParams p) {
    constexpr int kRowsPer = kThr / kCols;
    constexpr int kRows = kLaMaxDim / kRowsPer;
    static_assert(kRows <= kMaxRows, "");
    __shared__ float qs[kLaMaxDim], ks[kLaMaxDim];
    __shared__ float4 part[kThr / 32][kCols];
    const int t = threadIdx.x, c = t % kCols, r0 = t / kCols;
    const long long bh = blockIdx.x;
    const long long b = bh / p.heads;
    const int h = (int)(bh % p.heads);
    const int v = 4 * ((int)blockIdx.y * kCols + c);
    const bool in = v < p.dv;
    float *st = p.state + bh * p.dk * p.dv + v;
    float4 s[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int d = r0 + i * kRowsPer;
        if (in && d < p.dk) s[i] = *reinterpret_cast<const float4 *>(st + (long long)d * p.dv);
    }
    const long long qk = (b * (p.heads / p.group) + h / p.group) * p.dk;
    if (t < p.dk)
        qs[t] = ldg_f32(static_cast<const T *>(p.q) + qk + t);
    else if (t >= kLaMaxDim && t - kLaMaxDim < p.dk)
        ks[t - kLaMaxDim] = ldg_f32(static_cast<const T *>(p.k) + qk + t - kLaMaxDim);
    float a = 1.f;
    if (p.g)
        a = ex2_approx(ldg_f32(static_cast<const T *>(p.g) + bh) * kLog2e);
    else if (p.g_head)
        a = ex2_approx(__ldg(p.g_head + h) * kLog2e);
    float vv[4] = {0.f, 0.f, 0.f, 0.f};
    if (in) {
        const T *vp = static_cast<const T *>(p.v) + bh * p.dv + v;
#pragma unroll
        for (int e = 0; e < 4; ++e) vv[e] = ldg_f32(vp + e);
    }
    __syncthreads();
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int d = r0 + i * kRowsPer;
        if (!in || d >= p.dk) continue;
        const float kd = ks[d], qd = qs[d];
        // a decay of zero resets: the old state does not count
        float4 o = a == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : s[i];
        o.x = fmaf(a, o.x, kd * vv[0]);
        o.y = fmaf(a, o.y, kd * vv[1]);
        o.z = fmaf(a, o.z, kd * vv[2]);
        o.w = fmaf(a, o.w, kd * vv[3]);
        *reinterpret_cast<float4 *>(st + (long long)d * p.dv) = o;
        y.x = fmaf(qd, o.x, y.x);
        y.y = fmaf(qd, o.y, y.y);
        y.z = fmaf(qd, o.z, y.z);
        y.w = fmaf(qd, o.w, y.w);
    }
#pragma unroll
    for (int m = kCols; m < 32; m <<= 1) {
        y.x += __shfl_xor_sync(0xffffffffu, y.x, m);
        y.y += __shfl_xor_sync(0xffffffffu, y.y, m);
        y.z += __shfl_xor_sync(0xffffffffu, y.z, m);
        y.w += __shfl_xor_sync(0xffffffffu, y.w, m);
    }
    if ((t & 31) < kCols) part[t >> 5][t & 31] = y;
    __syncthreads();
    if (t < 4 * kCols) {
        const int col = 4 * (int)blockIdx.y * kCols + t;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kThr / 32; ++w) sum += reinterpret_cast<const float *>(&part[w][0])[t];
        if (col < p.dv) static_cast<T *>(p.y)[bh * p.dv + col] = from_f32<T>(sum * p.scale);
    }
}

// Any dv and alignment: one column per thread of a warp's 32, rows over warps.
template <typename T>
__global__ void __launch_bounds__(kThr) linattn_step_kernel(const LinattnStepParams p) {
    __shared__ float part[kThr / 32][32];
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    const long long bh = blockIdx.x;
    const long long b = bh / p.heads;
    const int h = (int)(bh % p.heads);
    const int v = 32 * (int)blockIdx.y + lane;
    const bool in = v < p.dv;
    const long long qk = (b * (p.heads / p.group) + h / p.group) * p.dk;
    const T *q = static_cast<const T *>(p.q) + qk, *k = static_cast<const T *>(p.k) + qk;
    float a = 1.f;
    if (p.g)
        a = ex2_approx(ldg_f32(static_cast<const T *>(p.g) + bh) * kLog2e);
    else if (p.g_head)
        a = ex2_approx(__ldg(p.g_head + h) * kLog2e);
    float y = 0.f;
    if (in) {
        const float vv = ldg_f32(static_cast<const T *>(p.v) + bh * p.dv + v);
        float *st = p.state + bh * p.dk * p.dv + v;
#pragma unroll 4
        for (int d = w; d < p.dk; d += kThr / 32) {
            const float old = a == 0.f ? 0.f : st[(long long)d * p.dv];
            const float o = fmaf(a, old, ldg_f32(k + d) * vv);
            st[(long long)d * p.dv] = o;
            y = fmaf(ldg_f32(q + d), o, y);
        }
    }
    part[w][lane] = y;
    __syncthreads();
    if (w == 0 && in) {
        float sum = 0.f;
#pragma unroll
        for (int k2 = 0; k2 < kThr / 32; ++k2) sum += part[k2][lane];
        static_cast<T *>(p.y)[bh * p.dv + v] = from_f32<T>(sum * p.scale);
    }
}

template <typename T>
cudaError_t launch_typed(const LinattnStepParams &p, cudaStream_t stream) {
    const long long pairs = p.batch * p.heads;
    const bool vec = p.dv % 4 == 0 && (reinterpret_cast<uintptr_t>(p.state) & 15) == 0;
    if (!vec) {
        linattn_step_kernel<T>
            <<<dim3((unsigned)pairs, (unsigned)((p.dv + 31) / 32)), kThr, 0, stream>>>(p);
    } else if (p.dv <= 32 || pairs < 2ll * sm_count()) {
        linattn_step_vec_kernel<T, 8>
            <<<dim3((unsigned)pairs, (unsigned)((p.dv + 31) / 32)), kThr, 0, stream>>>(p);
    } else if (p.dv <= 64) {
        linattn_step_vec_kernel<T, 16>
            <<<dim3((unsigned)pairs, 1), kThr, 0, stream>>>(p);
    } else {
        linattn_step_vec_kernel<T, 32>
            <<<dim3((unsigned)pairs, 1), kThr, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linattn_step(const LinattnStepParams &p, bool bf16, cudaStream_t stream) {
    return bf16 ? launch_typed<__nv_bfloat16>(p, stream) : launch_typed<float>(p, stream);
}

}  // namespace selscan
