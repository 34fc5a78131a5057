// block_norm.cu -- the junction around a block: the norm after it with its
// gate, the scaled residual sum, and the norm before the next block, in one
// pass over the rows; and its gradient.
//
//   a   = x            (gate before: x·silu(z))
//   p   = a·rsqrt(mean_group(a²) + eps)·weight          (no weight: p = a)
//   u   = p            (gate after: p·silu(z))
//   out = res + res_scale·u
//   y   = out·rsqrt(mean(out²) + eps)·next_weight
// ("Mamba Block": the gated output, y·silu(z), between norm and residual.)
//
// Bound: HBM; each row is read once and held in registers between its (at
// most two, in the gradient three) reductions. A block works on one row at a
// time, or on several where a row needs no more than a warp: thread t holds
// kNV vectors of kVec elements of its group's columns, so that sums over a
// group stay within its threads. All arithmetic and all sums are float32; the
// only roundings to bfloat16 are the stores.
#include "block_norm.cuh"

#include <algorithm>

namespace selscan {
namespace {

// kVec consecutive elements as floats (plain loads: `out` may be `res`).
template <typename T, int kVec> struct Io;
template <> struct Io<float, 8> {
    static __device__ __forceinline__ void ld(const void *p, long long i, float (&v)[8]) {
        const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        const float4 a = q[0], b = q[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
    static __device__ __forceinline__ void st(void *p, long long i, const float (&v)[8]) {
        float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
};
template <> struct Io<__nv_bfloat16, 8> {
    static __device__ __forceinline__ void ld(const void *p, long long i, float (&v)[8]) {
        const uint4 u =
            *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p) + i);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[2 * k] = __uint_as_float(w[k] << 16);
            v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ void st(void *p, long long i, const float (&v)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
            w[k] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p) + i) =
            make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <typename T> struct Io<T, 1> {
    static __device__ __forceinline__ void ld(const void *p, long long i, float (&v)[1]) {
        v[0] = to_f32(static_cast<const T *>(p)[i]);
    }
    static __device__ __forceinline__ void st(void *p, long long i, const float (&v)[1]) {
        static_cast<T *>(p)[i] = from_f32<T>(v[0]);
    }
};

// Where a thread's columns are. tg threads a group, groups·tg threads a row,
// rows_per rows a block.
struct Map {
    int tg, row_threads, rows_per;
};

// Sum over the tg threads of this thread's group (a power of two up to a
// warp, or whole warps); `red` has a float per warp. Every thread of the
// block calls it.
__device__ __forceinline__ float group_sum(float v, int tg, float *red) {
    const int w = threadIdx.x >> 5;
    if (tg <= 32) {
        for (int m = tg >> 1; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
        return v;
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    __syncthreads();  // readers of the previous sum are done
    if ((threadIdx.x & 31) == 0) red[w] = v;
    __syncthreads();
    const int per = tg >> 5, first = w / per * per;
    float s = 0.f;
    for (int k = 0; k < per; ++k) s += red[first + k];
    return s;
}

// Sums over a row's threads. Rows of more than a warp have the block to
// themselves; a row of fewer threads than a warp has a power of two.
__device__ __forceinline__ float row_sum(float v, int row_threads, float *red) {
    if (row_threads <= 32) {
        for (int m = row_threads >> 1; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
        return v;
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
    const int nw = ((int)blockDim.x + 31) >> 5;
    for (int k = 0; k < nw; ++k) s += red[k];
    return s;
}

template <typename T, typename TR, int kVec, int kNV>
__global__ void __launch_bounds__(1024) block_norm_fwd_kernel(const BlockNormParams p, const Map m) {
    __shared__ float red[32];
    const int t = threadIdx.x, local = t % m.row_threads;
    const long long row = (long long)blockIdx.x * m.rows_per + t / m.row_threads;
    const int gs = p.dim / p.groups, grp = local / m.tg, lane = local % m.tg;
    const bool live = row < p.rows && grp < p.groups;
    float v[kNV][kVec], gate[kNV][kVec], res[kNV][kVec];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
        const int e = (i * m.tg + lane) * kVec;
        if (!live || e >= gs) continue;
        const long long c = (long long)grp * gs + e;
        Io<T, kVec>::ld(p.x, row * p.x_row + c, v[i]);
        if (p.gate != kGateNone) Io<T, kVec>::ld(p.z, row * p.z_row + c, gate[i]);
        if (p.res) Io<TR, kVec>::ld(p.res, row * p.dim + c, res[i]);
    }
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
        const int e = (i * m.tg + lane) * kVec;
        if (!live || e >= gs) continue;
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
            if (p.gate != kGateNone) gate[i][k] = silu_f32(gate[i][k]);
            if (p.gate == kGateBefore) v[i][k] *= gate[i][k];
            sum = fmaf(v[i][k], v[i][k], sum);
        }
    }
    float rstd = 1.f;
    if (p.weight) rstd = rsqrtf(group_sum(sum, m.tg, red) / (float)gs + p.eps);
    float sum2 = 0.f;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
        const int e = (i * m.tg + lane) * kVec;
        if (!live || e >= gs) continue;
        const int c = grp * gs + e;
        float w[kVec], s[kVec];
        if (p.weight) Io<float, kVec>::ld(p.weight, c, w);
        if (p.res_scale) Io<float, kVec>::ld(p.res_scale, c, s);
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
            float u = v[i][k];
            if (p.weight) u = u * rstd * w[k];
            if (p.gate == kGateAfter) u *= gate[i][k];
            if (p.res_scale) u *= s[k];
            if (p.res) u += res[i][k];
            v[i][k] = u;
            sum2 = fmaf(u, u, sum2);
        }
        if (p.out) Io<TR, kVec>::st(p.out, row * p.dim + c, v[i]);
    }
    if (!p.next_weight) return;
    const float rstd2 = rsqrtf(row_sum(sum2, m.row_threads, red) / (float)p.dim + p.eps);
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
        const int e = (i * m.tg + lane) * kVec;
        if (!live || e >= gs) continue;
        const int c = grp * gs + e;
        float w[kVec];
        Io<float, kVec>::ld(p.next_weight, c, w);
#pragma unroll
        for (int k = 0; k < kVec; ++k) v[i][k] = v[i][k] * rstd2 * w[k];
        Io<T, kVec>::st(p.y, row * p.dim + c, v[i]);
    }
}

// The gradient. With n = a·rstd, mm = out·rstd2, dm = dy·next_weight:
//   dr = dout + rstd2·(dm − mm·mean(dm·mm))       (= dres)
//   dres_scale = Σ dr·u,  du = dr·res_scale
//   gate after:  dgate = du·p, dp = du·silu(z)
//   dweight = Σ dp·n,  dn = dp·weight,  da = rstd·(dn − n·mean_group(dn·n))
//   gate before: dgate = da·x, dx = da·silu(z)
//   dz = dgate·silu'(z),  silu' = σ·(1 + z·(1 − σ))
// Everything of the forward is recomputed from the inputs. Blocks stride over
// the rows and keep the three column sums of their rows in registers; a
// second kernel adds the blocks' sums in a fixed order.
template <typename T, typename TR, int kVec, int kNV, int kThreads>
__global__ void __launch_bounds__(kThreads) block_norm_bwd_kernel(const BlockNormParams p, const Map m) {
    __shared__ float red[32];
    const int t = threadIdx.x, local = t % m.row_threads;
    const int gs = p.dim / p.groups, grp = local / m.tg, lane = local % m.tg;
    const int sub = t / m.row_threads;
    float aw[kNV][kVec], as[kNV][kVec], an[kNV][kVec];
#pragma unroll
    for (int i = 0; i < kNV; ++i)
#pragma unroll
        for (int k = 0; k < kVec; ++k) aw[i][k] = as[i][k] = an[i][k] = 0.f;

    for (long long base = (long long)blockIdx.x * m.rows_per; base < p.rows;
         base += (long long)gridDim.x * m.rows_per) {
        const long long row = base + sub;
        const bool live = row < p.rows && grp < p.groups;
        float x[kNV][kVec], z[kNV][kVec], r[kNV][kVec], dr[kNV][kVec], dm[kNV][kVec];
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            const int e = (i * m.tg + lane) * kVec;
            if (!live || e >= gs) continue;
            const long long c = (long long)grp * gs + e;
            Io<T, kVec>::ld(p.x, row * p.x_row + c, x[i]);
            if (p.gate != kGateNone) Io<T, kVec>::ld(p.z, row * p.z_row + c, z[i]);
            if (p.res) Io<TR, kVec>::ld(p.res, row * p.dim + c, r[i]);
            if (p.dout) Io<TR, kVec>::ld(p.dout, row * p.dim + c, dr[i]);
            if (p.next_weight) Io<T, kVec>::ld(p.dy, row * p.dim + c, dm[i]);
        }
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            const int e = (i * m.tg + lane) * kVec;
            if (!live || e >= gs) continue;
#pragma unroll
            for (int k = 0; k < kVec; ++k) {
                float a = x[i][k];
                if (p.gate == kGateBefore) a *= silu_f32(z[i][k]);
                sum = fmaf(a, a, sum);
            }
        }
        float rstd = 1.f;
        if (p.weight) rstd = rsqrtf(group_sum(sum, m.tg, red) / (float)gs + p.eps);
        // out, its norm's statistics
        float s_rr = 0.f, s_dr = 0.f;
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            const int e = (i * m.tg + lane) * kVec;
            if (!live || e >= gs) continue;
            const int c = grp * gs + e;
            float w[kVec], s[kVec], w2[kVec];
            if (p.weight) Io<float, kVec>::ld(p.weight, c, w);
            if (p.res_scale) Io<float, kVec>::ld(p.res_scale, c, s);
            if (p.next_weight) Io<float, kVec>::ld(p.next_weight, c, w2);
#pragma unroll
            for (int k = 0; k < kVec; ++k) {
                if (!p.dout) dr[i][k] = 0.f;
                if (!p.next_weight) continue;
                float u = x[i][k];
                if (p.gate == kGateBefore) u *= silu_f32(z[i][k]);
                if (p.weight) u *= rstd * w[k];
                if (p.gate == kGateAfter) u *= silu_f32(z[i][k]);
                if (p.res_scale) u *= s[k];
                if (p.res) u += r[i][k];
                r[i][k] = u;
                s_rr = fmaf(u, u, s_rr);
                s_dr = fmaf(dm[i][k] * w2[k], u, s_dr);
            }
        }
        float rstd2 = 1.f, coef = 0.f;
        if (p.next_weight) {
            rstd2 = rsqrtf(row_sum(s_rr, m.row_threads, red) / (float)p.dim + p.eps);
            coef = row_sum(s_dr, m.row_threads, red) * rstd2 / (float)p.dim;
        }
        float s_dn = 0.f;
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            const int e = (i * m.tg + lane) * kVec;
            if (!live || e >= gs) continue;
            const int c = grp * gs + e;
            float w[kVec], s[kVec], w2[kVec];
            if (p.weight) Io<float, kVec>::ld(p.weight, c, w);
            if (p.res_scale) Io<float, kVec>::ld(p.res_scale, c, s);
            if (p.next_weight) Io<float, kVec>::ld(p.next_weight, c, w2);
#pragma unroll
            for (int k = 0; k < kVec; ++k) {
                if (p.next_weight) {
                    const float mm = r[i][k] * rstd2;
                    an[i][k] = fmaf(dm[i][k], mm, an[i][k]);
                    dr[i][k] += rstd2 * (dm[i][k] * w2[k] - mm * coef);
                }
            }
            if (p.dres) Io<TR, kVec>::st(p.dres, row * p.dim + c, dr[i]);
#pragma unroll
            for (int k = 0; k < kVec; ++k) {
                const float gate = p.gate != kGateNone ? silu_f32(z[i][k]) : 1.f;
                float a = x[i][k];
                if (p.gate == kGateBefore) a *= gate;
                const float n = a * rstd;
                const float pp = p.weight ? n * w[k] : a;
                float d = dr[i][k];
                if (p.res_scale) {
                    as[i][k] = fmaf(d, p.gate == kGateAfter ? pp * gate : pp, as[i][k]);
                    d *= s[k];
                }
                float dg = 0.f;
                if (p.gate == kGateAfter) {
                    dg = d * pp;
                    d *= gate;
                }
                if (p.weight) {
                    aw[i][k] = fmaf(d, n, aw[i][k]);
                    d *= w[k];
                    s_dn = fmaf(d, n, s_dn);
                }
                dr[i][k] = d;   // dn (or da where there is no norm)
                dm[i][k] = dg;  // dgate of a gate after
            }
        }
        float cg = 0.f;
        if (p.weight) cg = group_sum(s_dn, m.tg, red) / (float)gs;
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            const int e = (i * m.tg + lane) * kVec;
            if (!live || e >= gs) continue;
            const long long c = (long long)grp * gs + e;
#pragma unroll
            for (int k = 0; k < kVec; ++k) {
                float a = x[i][k], sig = 0.f, gate = 1.f;
                if (p.gate != kGateNone) {
                    sig = sigmoid_f32(z[i][k]);
                    gate = z[i][k] * sig;
                }
                if (p.gate == kGateBefore) a *= gate;
                float d = dr[i][k];
                if (p.weight) d = rstd * (d - a * rstd * cg);
                float dg = dm[i][k];
                if (p.gate == kGateBefore) {
                    dg = d * x[i][k];
                    d *= gate;
                }
                dr[i][k] = d;
                if (p.gate != kGateNone) dm[i][k] = dg * sig * (1.f + z[i][k] * (1.f - sig));
            }
            Io<T, kVec>::st(p.dx, row * p.dim + c, dr[i]);
            if (p.gate != kGateNone) Io<T, kVec>::st(p.dz, row * p.dim + c, dm[i]);
        }
    }
    // the block's column sums, of each of its row slots
    float *part = p.partial + ((long long)blockIdx.x * m.rows_per + sub) * 3 * p.dim;
    if (grp < p.groups) {
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            const int e = (i * m.tg + lane) * kVec;
            if (e >= gs) continue;
            const int c = grp * gs + e;
            if (p.weight) Io<float, kVec>::st(part, c, aw[i]);
            if (p.res_scale) Io<float, kVec>::st(part + p.dim, c, as[i]);
            if (p.next_weight) Io<float, kVec>::st(part + 2 * p.dim, c, an[i]);
        }
    }
}

// Column sums over the partials' `n` row slots: 32 columns a block, 8 slices
// of slots.
__global__ void __launch_bounds__(256)
block_norm_reduce_kernel(const float *__restrict__ partial, int n, int dim, float *dweight,
                         float *dres_scale, float *dnext_weight) {
    __shared__ float s[8][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, which = blockIdx.y;
    float *out = which == 0 ? dweight : which == 1 ? dres_scale : dnext_weight;
    if (!out) return;
    float v = 0.f;
    if (c < dim)
        for (int k = w; k < n; k += 8) v += partial[((long long)k * 3 + which) * dim + c];
    s[w][lane] = v;
    __syncthreads();
    if (w == 0 && c < dim) {
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += s[k][lane];
        out[c] = sum;
    }
}

int pow2_floor(int v) {
    int p = 1;
    while (2 * p <= v) p *= 2;
    return p;
}

// Threads of a group for `per` elements each (a power of two up to a warp, or
// whole warps, as far as `threads` a block allow), and rows a block.
Map make_map(int dim, int groups, int per, int threads) {
    const int want = (dim / groups + per - 1) / per;
    const int room = threads / groups;
    Map m;
    if (want <= 32 || room < 64) {
        m.tg = 1;
        while (m.tg < want && m.tg < 32) m.tg *= 2;
        m.tg = std::min(m.tg, pow2_floor(room));
    } else {
        m.tg = std::min((want + 31) / 32 * 32, room / 32 * 32);
    }
    // a row's threads are whole warps, or a power of two inside one
    m.row_threads = m.tg * groups;
    if (m.row_threads > 32)
        m.row_threads = (m.row_threads + 31) / 32 * 32;
    else if (m.row_threads > 1)
        m.row_threads = 2 * pow2_floor(m.row_threads - 1);
    m.rows_per = m.row_threads <= 32 ? 128 / m.row_threads : 1;
    return m;
}

// The map if it leaves every thread at most nv vectors of `vec` elements.
bool fits(const BlockNormParams &p, int vec, int nv, int threads, Map *m) {
    if (p.groups > threads) return false;
    *m = make_map(p.dim, p.groups, vec * nv, threads);
    return (p.dim / p.groups + m->tg * vec - 1) / (m->tg * vec) <= nv;
}

bool use_vec(const BlockNormParams &p) { return p.vec && (p.dim / p.groups) % 8 == 0; }

template <typename T, typename TR, int kVec, int kNV>
cudaError_t fwd(const BlockNormParams &p, const Map &m, cudaStream_t stream) {
    const long long blocks = (p.rows + m.rows_per - 1) / m.rows_per;
    block_norm_fwd_kernel<T, TR, kVec, kNV>
        <<<(unsigned)blocks, m.row_threads * m.rows_per, 0, stream>>>(p, m);
    return cudaGetLastError();
}

template <typename T, typename TR>
cudaError_t fwd_typed(const BlockNormParams &p, cudaStream_t stream) {
    Map m;
    if (use_vec(p)) {
        if (fits(p, 8, 1, 1024, &m)) return fwd<T, TR, 8, 1>(p, m, stream);
        if (fits(p, 8, 2, 1024, &m)) return fwd<T, TR, 8, 2>(p, m, stream);
        if (fits(p, 8, 4, 1024, &m)) return fwd<T, TR, 8, 4>(p, m, stream);
    }
    if (fits(p, 1, 8, 1024, &m)) return fwd<T, TR, 1, 8>(p, m, stream);
    if (fits(p, 1, 32, 1024, &m)) return fwd<T, TR, 1, 32>(p, m, stream);
    return cudaErrorInvalidValue;
}

template <typename T, typename TR, int kVec, int kNV, int kThreads>
cudaError_t bwd(const BlockNormParams &p, const Map &m, cudaStream_t stream) {
    const long long want = (p.rows + m.rows_per - 1) / m.rows_per;
    const int blocks =
        (int)std::min<long long>(want, block_norm_bwd_slots(p.rows, p.dim) / m.rows_per);
    block_norm_bwd_kernel<T, TR, kVec, kNV, kThreads>
        <<<blocks, m.row_threads * m.rows_per, 0, stream>>>(p, m);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !(p.weight || p.res_scale || p.next_weight)) return e;
    block_norm_reduce_kernel<<<dim3((unsigned)((p.dim + 31) / 32), 3), 256, 0, stream>>>(
        p.partial, blocks * m.rows_per, p.dim, p.weight ? p.dweight : nullptr,
        p.res_scale ? p.dres_scale : nullptr, p.next_weight ? p.dnext_weight : nullptr);
    return cudaGetLastError();
}

template <typename T, typename TR>
cudaError_t bwd_typed(const BlockNormParams &p, cudaStream_t stream) {
    Map m;
    if (use_vec(p)) {
        if (fits(p, 8, 1, 512, &m)) return bwd<T, TR, 8, 1, 512>(p, m, stream);
        if (fits(p, 8, 2, 512, &m)) return bwd<T, TR, 8, 2, 512>(p, m, stream);
        if (fits(p, 8, 4, 1024, &m)) return bwd<T, TR, 8, 4, 1024>(p, m, stream);
    }
    if (fits(p, 1, 4, 512, &m)) return bwd<T, TR, 1, 4, 512>(p, m, stream);
    if (fits(p, 1, 16, 512, &m)) return bwd<T, TR, 1, 16, 512>(p, m, stream);
    if (fits(p, 1, 32, 1024, &m)) return bwd<T, TR, 1, 32, 1024>(p, m, stream);
    return cudaErrorInvalidValue;
}

}  // namespace

// Row slots the gradient's blocks keep column sums for: about a thousand
// threads an SM at eight columns a thread, two blocks an SM at least.
int block_norm_bwd_slots(long long rows, int dim) {
    const long long most = std::max<long long>(2 * 148, 148ll * 8 * 1024 / dim);
    return (int)std::max<long long>(128, std::min(rows + 127, most));
}

cudaError_t launch_block_norm_fwd(const BlockNormParams &p, bool bf16, cudaStream_t stream) {
    if (!bf16) return fwd_typed<float, float>(p, stream);
    return p.res_f32 ? fwd_typed<__nv_bfloat16, float>(p, stream)
                     : fwd_typed<__nv_bfloat16, __nv_bfloat16>(p, stream);
}

cudaError_t launch_block_norm_bwd(const BlockNormParams &p, bool bf16, cudaStream_t stream) {
    if (!bf16) return bwd_typed<float, float>(p, stream);
    return p.res_f32 ? bwd_typed<__nv_bfloat16, float>(p, stream)
                     : bwd_typed<__nv_bfloat16, __nv_bfloat16>(p, stream);
}

}  // namespace selscan
