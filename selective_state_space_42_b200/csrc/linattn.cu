// linattn.cu -- linear attention with a decay for each head on the CUDA cores:
// the sweep of linattn_params.cuh in chunks of 64 tokens, for every size and
// alignment and both I/O types, with float32 products (the float32 I/O path;
// bfloat16 I/O comes here only when its rows do not suit the tensor-core
// kernels).
//
// With within-chunk prefix sums G_i of the log decays (G_end their total), a
// chunk's outputs and state are dense products ("Mamba & State Space Models —
// Guide Complet" §5 "SSD — State Space Dual", with a key and a query of their
// own for each head):
//   forward:  y_i  = Σ_{j ≤ i} p·exp(G_i − G_j)·(q_i·k_j)·v_j + r·exp(G_i)·S_inᵀ q_i
//             S_out = exp(G_end)·S_in + Σ_j c·exp(G_end − G_j)·k_j v_jᵀ
//   reverse:  y_j  = Σ_{i ≥ j} p·exp(G_i − G_j)·(q_j·k_i)·v_i + r·exp(G_end − G_j)·S_inᵀ q_j
//             S_out = exp(G_end)·S_in + Σ_i c·exp(G_i)·k_i v_iᵀ
// A block carries the state of one head and 64 of its value columns through
// the chunks of one segment, in registers (with a shared-memory copy for the
// product with q). Too few heads to fill the device: the sequence is cut into
// segments (LinattnPlan).
//
// Bound: the float32 FMAs, at 8 warps an SM, which register tiles (4×4, and (DKP/16)×4
// for the state) feed from shared memory. A chunk of a head needs 2·64·64·(dk + dv) +
// 2·2·64·dk·dv operations; a block executes 2·64·64·(2·dk + DKP + 64) for its 64 value
// columns, DKP the larger dimension of both rounded up to 64 or 128, and two blocks both
// make the scores. On 3 × 1111 tokens of 6 heads 48 → 80 in float32 (107 µs; 125 with
// equal segments after a pass over all their states) that is 4.7 MFLOP a chunk for 2.0,
// 19 µs, four chunks a block.
#include "linattn_params.cuh"

#include <algorithm>

namespace selscan {
namespace {

constexpr int kC = kLaChunk;
constexpr int kVt = 64;        // value columns per block
constexpr int kThr = 256;
constexpr int kLd = kC + 4;    // row stride of the token-minor tiles (keeps 16-byte rows, spreads banks)

template <int DKP> struct SweepSmem {
    float Q[DKP][kLd];   // [d][token]
    float K[DKP][kLd];
    float V[kC][kVt];    // [token][column]
    float P[kC][kLd];    // [col token][row token]
    float S[DKP][kVt];   // the state entering the chunk
    float gh[kC], gl[kC];        // prefix sums times log2(e), as high + low
    float rowf[kC], colw[kC];
    float decay;
    float decay_log2_h, decay_log2_l;
};

// Four consecutive elements from `c` of a row with `n` valid ones, zero past them.
template <typename T>
__device__ __forceinline__ float4 ld4(const T *row, int c, int n, bool vec);
template <>
__device__ __forceinline__ float4 ld4<float>(const float *row, int c, int n, bool vec) {
    if (vec && c + 4 <= n) return __ldg(reinterpret_cast<const float4 *>(row + c));
    float4 v;
    v.x = c < n ? __ldg(row + c) : 0.f;
    v.y = c + 1 < n ? __ldg(row + c + 1) : 0.f;
    v.z = c + 2 < n ? __ldg(row + c + 2) : 0.f;
    v.w = c + 3 < n ? __ldg(row + c + 3) : 0.f;
    return v;
}
template <>
__device__ __forceinline__ float4 ld4<__nv_bfloat16>(const __nv_bfloat16 *row, int c, int n,
                                                     bool vec) {
    if (vec && c + 4 <= n) {
        const uint2 u = __ldg(reinterpret_cast<const uint2 *>(row + c));
        return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u),
                           __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u));
    }
    float4 v;
    v.x = c < n ? ldg_f32(row + c) : 0.f;
    v.y = c + 1 < n ? ldg_f32(row + c + 1) : 0.f;
    v.z = c + 2 < n ? ldg_f32(row + c + 2) : 0.f;
    v.w = c + 3 < n ? ldg_f32(row + c + 3) : 0.f;
    return v;
}

__device__ __forceinline__ void st4(float *p, const float4 &v) {
    *reinterpret_cast<float4 *>(p) = v;
}
__device__ __forceinline__ void st4(__nv_bfloat16 *p, const float4 &v) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&lo),
                                               *reinterpret_cast<const uint32_t *>(&hi));
}

__device__ __forceinline__ bool all_finite(const float4 &v) {
    // products with zero: zero, or NaN
    return fmaf(0.f, v.x, 0.f * v.y) + fmaf(0.f, v.z, 0.f * v.w) == 0.f;
}

// A [nq tokens][n columns] tile into shared memory as [column][token], zero
// outside. Lanes run over tokens, so that the transposed stores hit distinct
// banks; the four elements a lane reads per step share a sector with its
// next step's. True if the thread met a value that is not finite.
template <typename T, int DKP>
__device__ __forceinline__ bool load_transposed(float (*dst)[kLd], const T *base, long long row,
                                                int nq, int n, bool vec) {
    const int tok = threadIdx.x & (kC - 1), grp = threadIdx.x / kC;
    const T *r = base + tok * row;
    bool odd = false;
#pragma unroll
    for (int it = 0; it < DKP / 16; ++it) {
        const int d = 4 * (grp + 4 * it);
        const float4 v = tok < nq ? ld4<T>(r, d, n, vec) : make_float4(0.f, 0.f, 0.f, 0.f);
        dst[d][tok] = v.x;
        dst[d + 1][tok] = v.y;
        dst[d + 2][tok] = v.z;
        dst[d + 3][tok] = v.w;
        odd = odd || !all_finite(v);
    }
    return odd;
}

__device__ __forceinline__ void fma4(float4 &a, float s, const float4 &b) {
    a.x = fmaf(s, b.x, a.x);
    a.y = fmaf(s, b.y, a.y);
    a.z = fmaf(s, b.z, a.z);
    a.w = fmaf(s, b.w, a.w);
}

// Prefix sums of the chunk's log decays (one warp, two tokens a lane, in
// double: 64 tokens of strong decay would otherwise leave float32 too few
// bits for the difference of two neighbours) and the factors made from them.
template <typename T>
__device__ __forceinline__ void chunk_decays(const LinattnParams &p, const SweepArgs &a,
                                             long long b, int h, long long t0, int nq, float *gh,
                                             float *gl, float *rowf, float *colw, float *decay,
                                             float *total_h, float *total_l) {
    const int lane = threadIdx.x;
    double s[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int t = 2 * lane + e;
        double g = 0.0;
        if (t < nq) {
            if (p.g)
                g = (double)ldg_f32(static_cast<const T *>(p.g) +
                                    (b * p.seqlen + t0 + t) * p.heads + h);
            else if (p.g_head)
                g = (double)__ldg(p.g_head + h);
            g *= 1.4426950408889634;
            g = g < kLaResetLog2 ? kLaResetLog2 : g;
        }
        s[e] = g;
    }
    double sum = s[0] + s[1];
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const double o = __shfl_up_sync(0xffffffffu, sum, m);
        if (lane >= m) sum += o;
    }
    const double end = __shfl_sync(0xffffffffu, sum, 31);
    const double G[2] = {sum - s[1], sum};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int t = 2 * lane + e;
        const float hi = (float)G[e];
        gh[t] = hi;
        gl[t] = (float)(G[e] - (double)hi);
        const float up = ex2_approx((float)G[e]), down = ex2_approx((float)(end - G[e]));
        rowf[t] = a.row_scale * (a.reverse ? down : up);
        colw[t] = a.col_scale * (a.reverse ? up : down);
    }
    if (lane == 0) {
        *decay = ex2_approx((float)end);
        *total_h = (float)end;
        *total_l = (float)(end - (double)(float)end);
    }
}

// One block: one (sweep, batch row, head, segment, 64 value columns).
// kFull false: only the segment's own state, from zero.
template <typename T, int DKP, bool kFull>
__global__ void __launch_bounds__(kThr) linattn_sweep_kernel(const __grid_constant__ LinattnParams p) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    SweepSmem<DKP> &S = *reinterpret_cast<SweepSmem<DKP> *>(smem_raw);
    constexpr int kTiles = DKP / kVt;
    long long id = blockIdx.x;
    const int tile = (int)(id % kTiles);
    id /= kTiles;
    const int order = p.order0 + (int)(id % p.orders);  // position in the sweep's direction
    id /= p.orders;
    const int sw = (int)(id % p.nsweeps);
    const long long bh = id / p.nsweeps;
    const SweepArgs &a = p.sweep[sw];
    const int v0 = tile * kVt;
    if (kFull && p.nseg > 1 && order == 0) linattn_let_states_start();
    if (v0 >= a.dv) {
        if (!kFull && blockIdx.x == gridDim.x - 1) linattn_wait_for_first();
        return;
    }
    const long long b = bh / p.heads;
    const int h = (int)(bh % p.heads);
    const int seg = a.reverse ? p.nseg - 1 - order : order;
    const int t = threadIdx.x, tx = t & 15, ty = t >> 4;
    const long long len = p.seqlens
                              ? min((long long)max(__ldg(p.seqlens + b), 0), p.seqlen)
                              : p.seqlen;
    const long long row0 = b * p.seqlen;
    const T *Q = static_cast<const T *>(a.q) + row0 * a.q_row + (long long)(h / a.q_group) * a.dk;
    const T *K = static_cast<const T *>(a.k) + row0 * a.k_row + (long long)(h / a.k_group) * a.dk;
    const T *V = static_cast<const T *>(a.v) + row0 * a.v_row + (long long)(h / a.v_group) * a.dv;
    const bool vec = p.vec != 0;
    const long long state_elems = (long long)a.dk * a.dv;

    // the state: rows d = ty + 16·r, columns v0 + 4·tx .. + 3
    constexpr int kR = DKP / 16;
    float4 st[kR];
#pragma unroll
    for (int r = 0; r < kR; ++r) {
        const int d = ty + 16 * r;
        float e[4] = {0.f, 0.f, 0.f, 0.f};
        if (kFull && d < a.dk) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int v = v0 + 4 * tx + c;
                if (v >= a.dv) continue;
                if (order > 0)
                    e[c] = a.seg_state[(bh * p.nseg + seg) * state_elems + (long long)d * a.dv + v];
                else if (a.h_init)
                    e[c] = a.h_init[bh * state_elems + (a.h_init_t ? (long long)v * a.dk + d
                                                                   : (long long)d * a.dv + v)];
            }
        }
        st[r] = make_float4(e[0], e[1], e[2], e[3]);
    }
    double seg_log2 = 0.0;  // of the segment's decay (thread 0)

    int c_first, c_last;
    linattn_segment(p, a.reverse != 0, order, &c_first, &c_last);
    for (int i = 0; i < c_last - c_first; ++i) {
        const int c = a.reverse ? c_last - 1 - i : c_first + i;
        const long long t0 = (long long)c * kC;
        const int nq = (int)max(0ll, min((long long)kC, len - t0));
        const int nl = (int)min((long long)kC, p.seqlen - t0);
        if (nq == 0 && !kFull) continue;
        __syncthreads();  // the tiles' readers of the previous chunk are done
        bool odd = false;  // k or v holds a value that is not finite
        if (nq > 0) {
            if (kFull) load_transposed<T, DKP>(S.Q, Q + t0 * a.q_row, a.q_row, nq, a.dk, vec);
            odd = load_transposed<T, DKP>(S.K, K + t0 * a.k_row, a.k_row, nq, a.dk, vec);
#pragma unroll
            for (int k = 0; k < kC * kVt / 4 / kThr; ++k) {
                const int it = t + k * kThr, tok = it / (kVt / 4), c4 = 4 * (it % (kVt / 4));
                const float4 v = tok < nq ? ld4<T>(V + (t0 + tok) * a.v_row, v0 + c4, a.dv, vec)
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
                *reinterpret_cast<float4 *>(&S.V[tok][c4]) = v;
                odd = odd || !all_finite(v);
            }
            if (kFull) {
#pragma unroll
                for (int r = 0; r < kR; ++r)
                    *reinterpret_cast<float4 *>(&S.S[ty + 16 * r][4 * tx]) = st[r];
            }
            if (t < 32)
                chunk_decays<T>(p, a, b, h, t0, nq, S.gh, S.gl, S.rowf, S.colw, &S.decay,
                                &S.decay_log2_h, &S.decay_log2_l);
        }
        // A pair without a weight (a later token, one before a reset) does not count, and
        // zero times a value that is not finite would: such a chunk skips those pairs.
        odd = __syncthreads_or(odd) != 0;
        auto exponent = [&](int i0, int j0) {  // log2 of the pair's weight
            const float d = (S.gh[i0] - S.gh[j0]) + (S.gl[i0] - S.gl[j0]);
            return a.reverse ? -d : d;
        };
        float4 acc[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (nq > 0) {
            if (kFull) {
                // P[row 4·ty + r][col 4·tx + c]
#pragma unroll 4
                for (int d = 0; d < a.dk; ++d) {
                    const float4 q4 = *reinterpret_cast<const float4 *>(&S.Q[d][4 * ty]);
                    const float4 k4 = *reinterpret_cast<const float4 *>(&S.K[d][4 * tx]);
                    fma4(acc[0], q4.x, k4);
                    fma4(acc[1], q4.y, k4);
                    fma4(acc[2], q4.z, k4);
                    fma4(acc[3], q4.w, k4);
                }
                float w[4][4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i0 = 4 * ty + r;
                    const float *av = reinterpret_cast<const float *>(&acc[r]);
#pragma unroll
                    for (int cc = 0; cc < 4; ++cc) {
                        const int j0 = 4 * tx + cc;
                        const bool in = (a.reverse ? j0 >= i0 : j0 <= i0) && i0 < nq && j0 < nq;
                        const float e = ex2_approx(exponent(i0, j0));
                        w[cc][r] = in && e != 0.f ? av[cc] * (a.p_scale * e) : 0.f;
                    }
                }
#pragma unroll
                for (int cc = 0; cc < 4; ++cc)
                    *reinterpret_cast<float4 *>(&S.P[4 * tx + cc][4 * ty]) =
                        make_float4(w[cc][0], w[cc][1], w[cc][2], w[cc][3]);
                // what the entering state gives
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                for (int d = 0; d < a.dk; ++d) {
                    const float4 q4 = *reinterpret_cast<const float4 *>(&S.Q[d][4 * ty]);
                    const float4 s4 = *reinterpret_cast<const float4 *>(&S.S[d][4 * tx]);
                    fma4(acc[0], q4.x, s4);
                    fma4(acc[1], q4.y, s4);
                    fma4(acc[2], q4.z, s4);
                    fma4(acc[3], q4.w, s4);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float f = S.rowf[4 * ty + r];
                    // a factor of zero is a reset: the state before it does not count
                    acc[r] = f == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                                      : make_float4(acc[r].x * f, acc[r].y * f, acc[r].z * f,
                                                    acc[r].w * f);
                }
            }
            // the state leaving
            const float dec = S.decay;
#pragma unroll
            for (int r = 0; r < kR; ++r)
                st[r] = dec == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                                   : make_float4(st[r].x * dec, st[r].y * dec, st[r].z * dec,
                                                 st[r].w * dec);
            if (odd) {
#pragma unroll 1
                for (int j = 0; j < kC; ++j) {
                    const float w = S.colw[j];
                    if (w == 0.f) continue;
                    float4 v4 = *reinterpret_cast<const float4 *>(&S.V[j][4 * tx]);
                    v4 = make_float4(v4.x * w, v4.y * w, v4.z * w, v4.w * w);
#pragma unroll
                    for (int r = 0; r < kR; ++r) fma4(st[r], S.K[ty + 16 * r][j], v4);
                }
            }
#pragma unroll 2
            for (int j = odd ? kC : 0; j < kC; j += 4) {
                const float4 w4 = *reinterpret_cast<const float4 *>(&S.colw[j]);
                float4 v4[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v4[e] = *reinterpret_cast<const float4 *>(&S.V[j + e][4 * tx]);
                    const float w = e == 0 ? w4.x : e == 1 ? w4.y : e == 2 ? w4.z : w4.w;
                    v4[e] = make_float4(v4[e].x * w, v4[e].y * w, v4[e].z * w, v4[e].w * w);
                }
#pragma unroll
                for (int r = 0; r < kR; ++r) {
                    const float4 k4 = *reinterpret_cast<const float4 *>(&S.K[ty + 16 * r][j]);
                    fma4(st[r], k4.x, v4[0]);
                    fma4(st[r], k4.y, v4[1]);
                    fma4(st[r], k4.z, v4[2]);
                    fma4(st[r], k4.w, v4[3]);
                }
            }
            if (!kFull && t == 0)
                seg_log2 += (double)S.decay_log2_h + (double)S.decay_log2_l;
        }
        if (!kFull) continue;
        __syncthreads();  // P is whole
        if (nq > 0) {
            if (odd) {
#pragma unroll 1
                for (int j = 0; j < kC; ++j) {
                    const float4 v4 = *reinterpret_cast<const float4 *>(&S.V[j][4 * tx]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int i0 = 4 * ty + r;
                        if ((a.reverse ? j >= i0 : j <= i0) && ex2_approx(exponent(i0, j)) != 0.f)
                            fma4(acc[r], S.P[j][i0], v4);
                    }
                }
            }
#pragma unroll 4
            for (int j = odd ? kC : 0; j < kC; ++j) {
                const float4 p4 = *reinterpret_cast<const float4 *>(&S.P[j][4 * ty]);
                const float4 v4 = *reinterpret_cast<const float4 *>(&S.V[j][4 * tx]);
                fma4(acc[0], p4.x, v4);
                fma4(acc[1], p4.y, v4);
                fma4(acc[2], p4.z, v4);
                fma4(acc[3], p4.w, v4);
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i0 = 4 * ty + r;
            const long long tok = row0 + t0 + i0;
            const float *av = reinterpret_cast<const float *>(&acc[r]);
            if (a.dot) {  // every lane takes part in the shuffles
                float d = 0.f;
                if (i0 < nq) {
                    const T *dr = static_cast<const T *>(a.dot) + tok * a.dot_row +
                                  (long long)(h / a.dot_group) * a.dv;
                    const float4 o = ld4<T>(dr, v0 + 4 * tx, a.dv, vec);
                    d = fmaf(av[0], o.x, fmaf(av[1], o.y, fmaf(av[2], o.z, av[3] * o.w)));
                }
#pragma unroll
                for (int m = 1; m < 16; m <<= 1) d += __shfl_xor_sync(0xffffffffu, d, m);
                if (tx == 0 && i0 < nq)
                    a.dot_out[((long long)tile * p.batch * p.heads + bh) * p.seqlen + t0 + i0] = d;
            }
            if (i0 < nl) {
                // rows behind the sequence's length are zero
                const long long off = (tok * p.heads + h) * a.dv + v0 + 4 * tx;
                if (vec && i0 < nq && v0 + 4 * tx + 4 <= a.dv) {
                    if (a.y_f32)
                        *reinterpret_cast<float4 *>(static_cast<float *>(a.y) + off) = acc[r];
                    else
                        st4(static_cast<T *>(a.y) + off, acc[r]);
                    continue;
                }
#pragma unroll
                for (int cc = 0; cc < 4; ++cc) {
                    if (v0 + 4 * tx + cc >= a.dv) break;
                    const float o = i0 < nq ? av[cc] : 0.f;
                    if (a.y_f32)
                        static_cast<float *>(a.y)[off + cc] = o;
                    else
                        static_cast<T *>(a.y)[off + cc] = from_f32<T>(o);
                }
            }
        }
    }

    float *out = nullptr;
    bool transposed = false;
    if (!kFull || (p.nseg > 1 && order == 0)) {
        out = a.seg_state + (bh * p.nseg + seg) * state_elems;
        if (t == 0 && tile == 0)
            a.seg_decay[bh * p.nseg + seg] = kFull ? 0.f : ex2_approx((float)seg_log2);
    } else if (a.h_final && order == p.nseg - 1) {
        out = a.h_final + bh * state_elems;
        transposed = a.h_final_t != 0;
    }
    if (out) {
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            const int d = ty + 16 * r;
            const float *e = reinterpret_cast<const float *>(&st[r]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int v = v0 + 4 * tx + c;
                if (d < a.dk && v < a.dv)
                    out[transposed ? (long long)v * a.dk + d : (long long)d * a.dv + v] = e[c];
            }
        }
    }
    if (!kFull && blockIdx.x == gridDim.x - 1) linattn_wait_for_first();
}

// seg_state[s]: the segment's own state -> the state entering it, in the
// sweep's order. A thread carries kV neighbouring elements; eight segments'
// loads are in flight before the first is used.
template <int kV>
__global__ void __launch_bounds__(kThr)
linattn_carry_kernel(const __grid_constant__ LinattnParams p, unsigned blocks_per) {
    constexpr int kAhead = 8;
    const unsigned id = blockIdx.x / blocks_per;
    const SweepArgs &a = p.sweep[id % (unsigned)p.nsweeps];
    const long long bh = id / (unsigned)p.nsweeps;
    const int n = a.dk * a.dv;
    const int e0 = ((int)(blockIdx.x % blocks_per) * kThr + (int)threadIdx.x) * kV;
    if (e0 >= n) return;
    float h[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        const int e = e0 + v;
        h[v] = a.h_init ? a.h_init[bh * n + (a.h_init_t ? (e % a.dv) * a.dk + e / a.dv : e)] : 0.f;
    }
    float *base = a.seg_state + bh * p.nseg * n + e0;
    const float *decay = a.seg_decay + bh * p.nseg;
    for (int o0 = 0; o0 < p.nseg; o0 += kAhead) {
        float own[kAhead][kV], dec[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int o = o0 + k, s = a.reverse ? p.nseg - 1 - o : o;
            if (o + 1 >= p.nseg) continue;  // the last segment's own state is not made
            dec[k] = __ldg(decay + s);
            if (kV == 4) {
                const float4 f = *reinterpret_cast<const float4 *>(base + (long long)s * n);
                own[k][0] = f.x;
                own[k][kV > 1 ? 1 : 0] = f.y;
                own[k][kV > 2 ? 2 : 0] = f.z;
                own[k][kV > 3 ? 3 : 0] = f.w;
            } else {
                own[k][0] = base[(long long)s * n];
            }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int o = o0 + k, s = a.reverse ? p.nseg - 1 - o : o;
            if (o >= p.nseg) break;
            float *x = base + (long long)s * n;
            if (kV == 4)
                *reinterpret_cast<float4 *>(x) = make_float4(h[0], h[kV > 1 ? 1 : 0],
                                                             h[kV > 2 ? 2 : 0], h[kV > 3 ? 3 : 0]);
            else
                *x = h[0];
            if (o + 1 >= p.nseg) break;
#pragma unroll
            for (int v = 0; v < kV; ++v)  // a decay of zero is a reset
                h[v] = dec[k] == 0.f ? own[k][v] : fmaf(dec[k], h[v], own[k][v]);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThr)
linattn_group_sum_kernel(const float *__restrict__ src0, T *__restrict__ dst0,
                         const float *__restrict__ src1, T *__restrict__ dst1, long long n,
                         int group, int dim) {
    const float *src = blockIdx.y ? src1 : src0;
    T *dst = blockIdx.y ? dst1 : dst0;
    for (long long e = (long long)blockIdx.x * kThr + threadIdx.x; e < n;
         e += (long long)gridDim.x * kThr) {
        const float *s = src + (e / dim) * group * dim + e % dim;
        float sum = 0.f;
        for (int k = 0; k < group; ++k) sum += s[(long long)k * dim];
        dst[e] = from_f32<T>(sum);
    }
}

// dlog_decay_t = X + Σ_{i ≥ t} (q_i·dq_i − k_i·dk_i), X = <S_last, dS_last>:
// with λ_t the loss's gradient with respect to S_t, <S_t, λ_t> equals both
// dg_t + k_t·dk_t and q_t·dq_t + dg_{t+1}. The running sum is kept in double:
// its terms cancel over the sequence, so dg carries the float32 errors of the
// dot products it sums. Where exp(g_t)·S_{t−1} is zero (a reset; the first
// token without a first state) dg is zero, and the sum starts from nothing
// again at a reset: neither the errors nor a NaN of what stands behind it
// reach the tokens before. A reset here is a factor that the sweeps' ex2.approx
// flushes to zero, below 2^−126. One block per (batch row, head), tokens from
// the last to the first in tiles of 4·1024; a partial sum goes with a flag that
// says whether it begins at a reset, and one with the flag takes nothing from
// before.
constexpr int kDgThr = 1024, kDgPer = 4;
constexpr double kDgResetLog2 = -126.0;
template <typename T>
__global__ void __launch_bounds__(kDgThr) linattn_decay_grad_kernel(const LinattnDecayGrad p) {
    __shared__ double wsum[32];
    __shared__ int wreset[32];
    const long long bh = blockIdx.x, b = bh / p.heads;
    const int h = (int)(bh % p.heads), t = threadIdx.x, lane = t & 31, w = t >> 5;
    const long long len = p.seqlens
                              ? min((long long)max(__ldg(p.seqlens + b), 0), p.seqlen)
                              : p.seqlen;
    double x = 0.0;
    if (p.dfinal)
        for (long long e = t; e < p.state_size; e += kDgThr)
            x += (double)p.last_state[bh * p.state_size + e] * p.dfinal[bh * p.state_size + e];
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    if (lane == 0) wsum[w] = x;
    __syncthreads();
    double carry = wsum[lane];
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) carry += __shfl_xor_sync(0xffffffffu, carry, m);
    const T *g = static_cast<const T *>(p.g) + b * p.seqlen * p.heads + h;
    T *out = static_cast<T *>(p.dg) + b * p.seqlen * p.heads + h;
    for (long long i = len + t; i < p.seqlen; i += kDgThr) out[i * p.heads] = from_f32<T>(0.f);
    const long long plane = p.batch * p.heads * p.seqlen;
    const float *rows = p.rows + bh * p.seqlen, *cols = p.cols + bh * p.seqlen;
    for (long long end = len; end > 0; end -= kDgThr * kDgPer) {
        // thread t takes tokens end − 1 − 4·t − e
        double v[kDgPer];
        float r[kDgPer], c[kDgPer], gt[kDgPer];  // every load before the first sum
#pragma unroll
        for (int e = 0; e < kDgPer; ++e) {
            const long long i = end - 1 - (long long)kDgPer * t - e;
            r[e] = i >= 0 ? rows[i] : 0.f;
            c[e] = i >= 0 ? cols[i] : 0.f;
            gt[e] = i >= 0 ? ldg_f32(g + i * p.heads) : 0.f;
        }
        double s = 0.0;
        bool reset = false;  // s begins at a reset among the thread's tokens
        bool own[kDgPer];    // and so does v[e]
#pragma unroll
        for (int e = 0; e < kDgPer; ++e) {
            const long long i = end - 1 - (long long)kDgPer * t - e;
            s += (double)r[e] - (double)c[e];
            if (p.tiles > 1 && i >= 0) s += (double)rows[plane + i] - (double)cols[plane + i];
            if ((double)gt[e] * 1.4426950408889634 < kDgResetLog2) {
                s = 0.0;
                reset = true;
            }
            v[e] = s;
            own[e] = reset;
        }
        double incl = s;
        int from = reset;
        auto scan = [&](double &sum, int &flag) {  // over the warp, later tokens first
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const double o = __shfl_up_sync(0xffffffffu, sum, m);
                const int f = __shfl_up_sync(0xffffffffu, flag, m);
                if (lane >= m) {
                    if (!flag) sum += o;
                    flag |= f;
                }
            }
        };
        scan(incl, from);
        __syncthreads();  // the readers of the previous tile's sums are done
        if (lane == 31) {
            wsum[w] = incl;
            wreset[w] = from;
        }
        __syncthreads();
        double sums = wsum[lane];  // of the warps up to warp `lane`
        int froms = wreset[lane];
        scan(sums, froms);
        // what stands before this thread's tokens: its warp's lanes, the warps, the tiles
        double base = __shfl_up_sync(0xffffffffu, incl, 1);
        int base_from = __shfl_up_sync(0xffffffffu, from, 1);
        if (lane == 0) {
            base = 0.0;
            base_from = 0;
        }
        const double before = __shfl_sync(0xffffffffu, sums, (w + 31) & 31);
        const int before_from = __shfl_sync(0xffffffffu, froms, (w + 31) & 31);
        if (!base_from) {
            if (w > 0) base += before;
            if (w == 0 || !before_from) base += carry;
        }
#pragma unroll
        for (int e = 0; e < kDgPer; ++e) {
            const long long i = end - 1 - (long long)kDgPer * t - e;
            if (i < 0) continue;
            const bool none = i == 0 && !p.has_init;
            out[i * p.heads] = from_f32<T>(none ? 0.f : (float)(own[e] ? v[e] : base + v[e]));
        }
        const double total = __shfl_sync(0xffffffffu, sums, 31);
        carry = __shfl_sync(0xffffffffu, froms, 31) ? total : carry + total;
    }
}

template <typename T, int DKP>
cudaError_t launch_sweeps(const LinattnParams &p, cudaStream_t stream) {
    const size_t smem = sizeof(SweepSmem<DKP>);
    auto full = linattn_sweep_kernel<T, DKP, true>;
    auto state = linattn_sweep_kernel<T, DKP, false>;
    cudaError_t e =
        cudaFuncSetAttribute(full, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(state, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return linattn_launch(full, state, kThr, (int)smem, (int)smem,
                          p.batch * p.heads * p.nsweeps * (DKP / kVt), p, stream);
}

}  // namespace

LinattnPlan linattn_plan(long long seqlen, long long ctas, int slots, double head, double own) {
    LinattnPlan pl;
    pl.nchunks = (int)((seqlen + kLaChunk - 1) / kLaChunk);
    pl.nseg = 1;
    pl.first_chunks = pl.seg_chunks = pl.nchunks;
    // estimated time in chunk passes: waves of blocks × (start-up + chunks a
    // segment); with several segments the first's and the states' kernels side by
    // side, the others' full pass, the carry and the two further launches
    auto waves = [&](long long blocks) { return (double)((blocks + slots - 1) / slots); };
    double best = waves(ctas) * (head + pl.nchunks);
    const int most = ctas >= 8ll * slots ? 1 : pl.nchunks < 64 ? pl.nchunks : 64;
    for (int n = 3; n <= most; ++n) {
        const int per = (int)(pl.nchunks / (n - 1 + own)) + 1;
        const int segs = 1 + (pl.nchunks - 1) / per;  // the first has what is left: 1 .. per
        if (segs < 3) continue;
        const int first = pl.nchunks - (segs - 1) * per;
        const double both = waves(ctas * (segs - 1));
        const double cost = both * (head + own * per) + std::max(0.0, first - own * per) +
                            both * (head + per) + 6.0 + 0.05 * segs;
        if (cost < best) {
            best = cost;
            pl.nseg = segs;
            pl.first_chunks = first;
            pl.seg_chunks = per;
        }
    }
    return pl;
}

int linattn_tiles(int dv) { return dv > kVt ? 2 : 1; }

// Blocks the device holds at a time: two on an SM where both head dimensions
// fit the 64-wide tiles (85 KB of shared memory each), else one (136 KB).
int linattn_slots(int dk, int dv) { return dk <= 64 && dv <= 64 ? 2 : 1; }

cudaError_t launch_linattn_sweeps(const LinattnParams &p, bool bf16, cudaStream_t stream) {
    int most = 0;
    for (int s = 0; s < p.nsweeps; ++s) most = std::max(most, std::max(p.sweep[s].dk, p.sweep[s].dv));
    if (bf16)
        return most <= 64 ? launch_sweeps<__nv_bfloat16, 64>(p, stream)
                          : launch_sweeps<__nv_bfloat16, 128>(p, stream);
    return most <= 64 ? launch_sweeps<float, 64>(p, stream) : launch_sweeps<float, 128>(p, stream);
}

cudaError_t launch_linattn_carry(const LinattnParams &p, cudaStream_t stream) {
    const int n = p.sweep[0].dk * p.sweep[0].dv;  // the same for every sweep
    const int v = n % 4 == 0 ? 4 : 1;
    const unsigned per = (unsigned)((n / v + kThr - 1) / kThr);
    const unsigned blocks = (unsigned)(p.batch * p.heads * p.nsweeps) * per;
    if (v == 4)
        linattn_carry_kernel<4><<<blocks, kThr, 0, stream>>>(p, per);
    else
        linattn_carry_kernel<1><<<blocks, kThr, 0, stream>>>(p, per);
    return cudaGetLastError();
}

cudaError_t launch_linattn_group_sums(const float *const src[2], void *const dst[2],
                                      long long tokens, int qk_heads, int group, int dim, bool bf16,
                                      cudaStream_t stream) {
    const long long n = tokens * qk_heads * dim;
    const dim3 grid((unsigned)std::min((n + kThr - 1) / kThr, 1ll << 20), 2);
    if (bf16)
        linattn_group_sum_kernel<<<grid, kThr, 0, stream>>>(
            src[0], static_cast<__nv_bfloat16 *>(dst[0]), src[1],
            static_cast<__nv_bfloat16 *>(dst[1]), n, group, dim);
    else
        linattn_group_sum_kernel<<<grid, kThr, 0, stream>>>(src[0], static_cast<float *>(dst[0]),
                                                            src[1], static_cast<float *>(dst[1]),
                                                            n, group, dim);
    return cudaGetLastError();
}

cudaError_t launch_linattn_decay_grad(const LinattnDecayGrad &p, bool bf16, cudaStream_t stream) {
    const unsigned blocks = (unsigned)(p.batch * p.heads);
    if (bf16)
        linattn_decay_grad_kernel<__nv_bfloat16><<<blocks, kDgThr, 0, stream>>>(p);
    else
        linattn_decay_grad_kernel<float><<<blocks, kDgThr, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace selscan
