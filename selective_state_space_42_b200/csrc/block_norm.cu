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
// only roundings to bfloat16 are the stores. 16384 rows of 5120 in bfloat16: 187 µs,
// 70% of the HBM copy rate (the instructions' issue is at 75%); the gradient of 16384
// rows of 2560, 286 µs, 50%: its column sums and operands take 96 registers a thread and
// 100 bytes of spills, which leaves 20 warps an SM to hide two barriers a row.
#include "block_norm.cuh"
#include "tma_util.cuh"

#include <algorithm>
#include <atomic>

#include "api_util.cuh"

namespace selscan {
namespace {

// kVec consecutive elements of a row, as they stand in memory until they are
// used (a bfloat16 vector takes half the registers of its floats).
template <typename T, int kVec> struct Raw;
template <> struct Raw<float, 8> {
    float4 a, b;
    __device__ __forceinline__ void ld(const void *p, long long i) {
        const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        a = q[0];
        b = q[1];
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
    static __device__ __forceinline__ void st(void *p, long long i, const float (&v)[8]) {
        float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
};
template <> struct Raw<__nv_bfloat16, 8> {
    uint4 u;
    __device__ __forceinline__ void ld(const void *p, long long i) {
        u = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p) + i);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
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
template <typename T> struct Raw<T, 1> {
    T u;
    __device__ __forceinline__ void ld(const void *p, long long i) {
        u = static_cast<const T *>(p)[i];
    }
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = to_f32(u); }
    static __device__ __forceinline__ void st(void *p, long long i, const float (&v)[1]) {
        static_cast<T *>(p)[i] = from_f32<T>(v[0]);
    }
};
template <int kVec>
__device__ __forceinline__ void ld_weight(const float *p, int c, float (&v)[kVec]) {
    Raw<float, kVec> r;
    r.ld(p, c);
    r.get(v);
}

// Where a thread's columns are: tg threads a group, row_threads a row, rows_per
// rows a block.
struct Map {
    int tg, row_threads, rows_per;
};

// Sums of kN floats over the threads of this thread's group or row: `threads` is
// a power of two up to a warp, or whole warps starting at a multiple of it (the
// whole block for a row); `first` is its first warp. Every thread of the block
// calls it; `red` has a float2 per warp, and is not another call's until two block
// barriers later. Behind the barrier every warp adds the warps' sums by shuffles again (one shared-memory read a
// lane; reading them one after another took 0.4 µs a sum at 20 warps).
template <int kN>
__device__ __forceinline__ void sum_over(float (&v)[kN], int threads, int first, float2 *red) {
    if (threads <= 32) {
        for (int m = threads >> 1; m > 0; m >>= 1)
#pragma unroll
            for (int k = 0; k < kN; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], m);
        return;
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1)
#pragma unroll
        for (int k = 0; k < kN; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], m);
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) red[w] = make_float2(v[0], v[kN - 1]);
    __syncthreads();
    const float2 r = lane < threads >> 5 ? red[first + lane] : make_float2(0.f, 0.f);
    v[0] = r.x;
    if (kN > 1) v[kN - 1] = r.y;
#pragma unroll
    for (int m = 16; m > 0; m >>= 1)
#pragma unroll
        for (int k = 0; k < kN; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], m);
}

// A sum over the row's threads and one over the group's behind one barrier.
__device__ __forceinline__ void sum_row_and_group(float &row, float &group, const Map &m,
                                                  int first_g, float2 *red) {
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) {
        row += __shfl_xor_sync(0xffffffffu, row, k);
        const float g = __shfl_xor_sync(0xffffffffu, group, k);
        if (k < m.tg) group += g;
    }
    if (lane == 0) red[w] = make_float2(row, group);
    __syncthreads();
    row = lane < m.row_threads >> 5 ? red[lane].x : 0.f;
    float g = lane < m.tg >> 5 ? red[first_g + lane].y : 0.f;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) {
        row += __shfl_xor_sync(0xffffffffu, row, k);
        g += __shfl_xor_sync(0xffffffffu, g, k);
    }
    if (m.tg > 32) group = g;
}

// ---- rows through shared memory -------------------------------------------------------
// With many rows a block, each row's operands come by bulk copies into a ring of
// stages, several rows ahead, so that the memory system stays busy through the
// sums' barriers. A row's last barrier also serves the next row's first sum, whose
// operands are read from the next stage a second time: a forward row has one
// barrier, a gradient's two. Behind it thread 0 refills the row's stage.
constexpr int kMaxStages = 8;
constexpr uint64_t kRowWaitNs = 2000000000ull;  // a copy that takes longer is given up
constexpr int kStatusRowCopy = 7;                // device error code
__device__ const int kNoAbortRow = 0;

__device__ __forceinline__ void bulk_row(void *dst, const void *src, uint32_t bytes,
                                         uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
        ::"r"(smem_addr(dst)), "l"(src), "r"(bytes), "r"(smem_addr(bar))
        : "memory");
}

// Thread 0: row `row` into a stage.
template <typename T, typename TR>
__device__ __forceinline__ void fetch_row(const BlockNormParams &p, unsigned char *stage,
                                          uint64_t *bar, long long row, bool bwd) {
    const uint32_t nt = (uint32_t)p.dim * sizeof(T), nr = (uint32_t)p.dim * sizeof(TR);
    const bool z = p.gate != kGateNone, res = p.res && (!bwd || p.next_weight),
               dy = bwd && p.next_weight, dout = bwd && p.dout;
    mbar_arrive_expect_tx(bar, nt * (1 + z + dy) + nr * (res + dout));
    bulk_row(stage, static_cast<const T *>(p.x) + row * p.x_row, nt, bar);
    if (z) bulk_row(stage + p.off_z, static_cast<const T *>(p.z) + row * p.z_row, nt, bar);
    if (res) bulk_row(stage + p.off_res, static_cast<const TR *>(p.res) + row * p.dim, nr, bar);
    if (dy) bulk_row(stage + p.off_dy, static_cast<const T *>(p.dy) + row * p.dim, nt, bar);
    if (dout) bulk_row(stage + p.off_dout, static_cast<const TR *>(p.dout) + row * p.dim, nr, bar);
}

// A thread's part of the first sum of the row in a stage.
template <typename T, int kVec, int kNV>
__device__ __forceinline__ float stage_sum(const BlockNormParams &p, const unsigned char *at,
                                           bool mine, int grp, int lane, int tg, int gs) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
        const int e = (i * tg + lane) * kVec;
        if (!mine || e >= gs) continue;
        Raw<T, kVec> x;
        float v[kVec];
        x.ld(at, grp * gs + e);
        x.get(v);
        if (p.gate == kGateBefore) {
            float g[kVec];
            x.ld(at + p.off_z, grp * gs + e);
            x.get(g);
#pragma unroll
            for (int k = 0; k < kVec; ++k) v[k] *= silu_f32(g[k]);
        }
#pragma unroll
        for (int k = 0; k < kVec; ++k) sum = fmaf(v[k], v[k], sum);
    }
    return sum;
}

// A copy did not come in time: it is recorded, and the block goes once the copies
// still on their way have landed (or been given up too).
__device__ __noinline__ void row_copy_failed(const BlockNormParams &p, uint64_t *full, int stage,
                                             uint32_t phase, long long base, int copies) {
    if (threadIdx.x == 0) {
        if (p.status) atomicCAS(p.status, 0, kStatusRowCopy);
        for (int k = 0; k < copies && base + (long long)k * gridDim.x < p.rows; ++k) {
            mbar_wait(&full[stage], phase, &kNoAbortRow, kRowWaitNs);
            if (++stage == p.stages) {
                stage = 0;
                phase ^= 1;
            }
        }
    }
    __syncthreads();
}

template <typename T, typename TR, int kVec, int kNV, int kThreads, int kBlocks, bool kRing>
__global__ void __launch_bounds__(kThreads, kBlocks)
block_norm_fwd_kernel(const __grid_constant__ BlockNormParams p, const Map m) {
    __shared__ float2 reds[2][2][32];  // of rows in turn: a row may have a single barrier
    __shared__ uint64_t full[kMaxStages];
    __shared__ int failed[2];  // of rows in turn as well
    extern __shared__ __align__(128) unsigned char dyn[];
    const int t = threadIdx.x, local = t % m.row_threads;
    const int gs = p.dim / p.groups, grp = local / m.tg, lane = local % m.tg;
    if (kRing) {
        if (t == 0) {
            failed[0] = failed[1] = 0;
            for (int k = 0; k < p.stages; ++k) mbar_init(&full[k], 1);
            fence_barrier_init();
            for (int k = 0; k < p.stages; ++k) {
                const long long r = blockIdx.x + (long long)k * gridDim.x;
                if (r < p.rows)
                    fetch_row<T, TR>(p, dyn + (size_t)k * p.stage_bytes, &full[k], r, false);
            }
        }
        __syncthreads();
    }
    const float inv_gs = 1.f / (float)gs, inv_dim = 1.f / (float)p.dim;
    const int first_g = m.tg > 32 ? t / m.tg * (m.tg >> 5) : 0,
              first_r = t / m.row_threads * (m.row_threads >> 5);
    int stage = 0;
    uint32_t phase = 0, odd = 0;
    float first[1] = {0.f};  // the row's first sum, where the ring brings it
    if (kRing) {
        if (!mbar_wait(&full[0], 0, &kNoAbortRow, kRowWaitNs)) failed[1] = 1;
        first[0] = stage_sum<T, kVec, kNV>(p, dyn, grp < p.groups, grp, lane, m.tg, gs);
        sum_over(first, m.tg, first_g, reds[0][1]);
        __syncthreads();
        if (failed[1]) {
            row_copy_failed(p, full, 0, 0, blockIdx.x, p.stages);
            return;
        }
    }
    for (long long base = (long long)blockIdx.x * m.rows_per; base < p.rows;
         base += (long long)gridDim.x * m.rows_per) {
        const long long row = base + t / m.row_threads;
        const bool live = row < p.rows && grp < p.groups;
        float2(*red)[32] = reds[odd];
        if (!kRing) odd ^= 1;
        unsigned char *at = dyn + (size_t)stage * p.stage_bytes;
        Raw<T, kVec> x[kNV], z[kNV];
        Raw<TR, kVec> res[kNV];
        float v[kNV][kVec];
        float sum[1] = {0.f};
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            const int e = (i * m.tg + lane) * kVec;
            if (!live || e >= gs) continue;
            const long long c = (long long)grp * gs + e;
            if (kRing) {
                x[i].ld(at, c);
                if (p.gate != kGateNone) z[i].ld(at + p.off_z, c);
                if (p.res) res[i].ld(at + p.off_res, c);
            } else {
                x[i].ld(p.x, row * p.x_row + c);
                if (p.gate != kGateNone) z[i].ld(p.z, row * p.z_row + c);
                if (p.res) res[i].ld(p.res, row * p.dim + c);
            }
        }
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            const int e = (i * m.tg + lane) * kVec;
            if (!live || e >= gs) continue;
            x[i].get(v[i]);
            if (p.gate == kGateBefore) {
                float g[kVec];
                z[i].get(g);
#pragma unroll
                for (int k = 0; k < kVec; ++k) v[i][k] *= silu_f32(g[k]);
            }
#pragma unroll
            for (int k = 0; k < kVec; ++k)
                if (!kRing) sum[0] = fmaf(v[i][k], v[i][k], sum[0]);
        }
        float rstd = 1.f;
        if (p.weight) {
            if (kRing) sum[0] = first[0];
            else sum_over(sum, m.tg, first_g, red[0]);
            rstd = rsqrtf(sum[0] * inv_gs + p.eps);
        }
        float sum2[1] = {0.f};
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            const int e = (i * m.tg + lane) * kVec;
            if (!live || e >= gs) continue;
            const int c = grp * gs + e;
            float f[kVec];
            if (p.weight) {
                ld_weight<kVec>(p.weight, c, f);
#pragma unroll
                for (int k = 0; k < kVec; ++k) v[i][k] *= rstd * f[k];
            }
            if (p.gate == kGateAfter) {
                z[i].get(f);
#pragma unroll
                for (int k = 0; k < kVec; ++k) v[i][k] *= silu_f32(f[k]);
            }
            if (p.res_scale) {
                ld_weight<kVec>(p.res_scale, c, f);
#pragma unroll
                for (int k = 0; k < kVec; ++k) v[i][k] *= f[k];
            }
            if (p.res) {
                res[i].get(f);
#pragma unroll
                for (int k = 0; k < kVec; ++k) v[i][k] += f[k];
            }
#pragma unroll
            for (int k = 0; k < kVec; ++k) sum2[0] = fmaf(v[i][k], v[i][k], sum2[0]);
            if (p.out) Raw<TR, kVec>::st(p.out, row * p.dim + c, v[i]);
        }
        if (kRing) {
            const long long next = base + gridDim.x, later = base + (long long)p.stages * gridDim.x;
            const int was = stage;
            if (++stage == p.stages) {
                stage = 0;
                phase ^= 1;
            }
            first[0] = 0.f;
            if (next < p.rows) {
                if (!mbar_wait(&full[stage], phase, &kNoAbortRow, kRowWaitNs)) failed[odd] = 1;
                if (p.weight)
                    first[0] = stage_sum<T, kVec, kNV>(p, dyn + (size_t)stage * p.stage_bytes,
                                                       grp < p.groups, grp, lane, m.tg, gs);
            }
            sum_row_and_group(sum2[0], first[0], m, first_g, red[0]);
            if (*(volatile int *)&failed[odd]) {
                row_copy_failed(p, full, stage, phase, next, p.stages - 1);
                return;
            }
            if (t == 0 && later < p.rows) fetch_row<T, TR>(p, at, &full[was], later, false);
            odd ^= 1;
        }
        if (!p.next_weight) continue;
        if (!kRing) sum_over(sum2, m.row_threads, first_r, red[1]);
        const float rstd2 = rsqrtf(sum2[0] * inv_dim + p.eps);
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            const int e = (i * m.tg + lane) * kVec;
            if (!live || e >= gs) continue;
            const int c = grp * gs + e;
            float w[kVec];
            ld_weight<kVec>(p.next_weight, c, w);
#pragma unroll
            for (int k = 0; k < kVec; ++k) v[i][k] *= rstd2 * w[k];
            Raw<T, kVec>::st(p.y, row * p.dim + c, v[i]);
        }
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
// the rows and keep the column sums of their rows in registers; a second kernel
// adds the blocks' sums in a fixed order. Two sums do for three gradients: with
// b = Σ dr·n (gate after: Σ dr·n·silu(z)), u = n·weight and dp = dr·res_scale (each
// times the gate) make dres_scale = weight·b and dweight = res_scale·b.
template <typename T, typename TR, int kVec, int kNV, int kThreads, int kBlocks, bool kRing>
__global__ void __launch_bounds__(kThreads, kBlocks)
block_norm_bwd_kernel(const __grid_constant__ BlockNormParams p, const Map m) {
    __shared__ float2 reds[2][3][32];  // of rows in turn: a row may have a single barrier
    __shared__ uint64_t full[kMaxStages];
    __shared__ int failed[2];
    extern __shared__ __align__(128) unsigned char dyn[];
    float *sums = reinterpret_cast<float *>(dyn);  // [2][dim] where a block has several rows
    const int t = threadIdx.x, local = t % m.row_threads;
    const int gs = p.dim / p.groups, grp = local / m.tg, lane = local % m.tg;
    const int sub = t / m.row_threads;
    const bool before = p.gate == kGateBefore, after = p.gate == kGateAfter;
    float ab[kNV][kVec], an[kNV][kVec];
#pragma unroll
    for (int i = 0; i < kNV; ++i)
#pragma unroll
        for (int k = 0; k < kVec; ++k) ab[i][k] = an[i][k] = 0.f;
    if (kRing) {
        if (t == 0) {
            failed[0] = failed[1] = 0;
            for (int k = 0; k < p.stages; ++k) mbar_init(&full[k], 1);
            fence_barrier_init();
            for (int k = 0; k < p.stages; ++k) {
                const long long r = blockIdx.x + (long long)k * gridDim.x;
                if (r < p.rows)
                    fetch_row<T, TR>(p, dyn + (size_t)k * p.stage_bytes, &full[k], r, true);
            }
        }
        __syncthreads();
    }
    const float inv_gs = 1.f / (float)gs, inv_dim = 1.f / (float)p.dim;
    const int first_g = m.tg > 32 ? t / m.tg * (m.tg >> 5) : 0,
              first_r = sub * (m.row_threads >> 5);
    int stage = 0;
    uint32_t phase = 0, odd = 0;
    float first[1] = {0.f};  // the row's first sum, where the ring brings it
    if (kRing) {
        if (!mbar_wait(&full[0], 0, &kNoAbortRow, kRowWaitNs)) failed[1] = 1;
        first[0] = stage_sum<T, kVec, kNV>(p, dyn, grp < p.groups, grp, lane, m.tg, gs);
        sum_over(first, m.tg, first_g, reds[0][0]);
        __syncthreads();
        if (failed[1]) {
            row_copy_failed(p, full, 0, 0, blockIdx.x, p.stages);
            return;
        }
    }
    for (long long base = (long long)blockIdx.x * m.rows_per; base < p.rows;
         base += (long long)gridDim.x * m.rows_per) {
        const long long row = base + sub;
        const bool live = row < p.rows && grp < p.groups;
        float2(*red)[32] = reds[odd];
        unsigned char *at = dyn + (size_t)stage * p.stage_bytes;
        Raw<T, kVec> xr[kNV], zr[kNV], yr[kNV];
        Raw<TR, kVec> rr[kNV], dr[kNV];
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            const int e = (i * m.tg + lane) * kVec;
            if (!live || e >= gs) continue;
            const long long c = (long long)grp * gs + e;
            if (kRing) {
                xr[i].ld(at, c);
                if (p.gate != kGateNone) zr[i].ld(at + p.off_z, c);
                if (p.res && p.next_weight) rr[i].ld(at + p.off_res, c);
                if (p.next_weight) yr[i].ld(at + p.off_dy, c);
            } else {
                xr[i].ld(p.x, row * p.x_row + c);
                if (p.gate != kGateNone) zr[i].ld(p.z, row * p.z_row + c);
                if (p.res && p.next_weight) rr[i].ld(p.res, row * p.dim + c);
                if (p.next_weight) yr[i].ld(p.dy, row * p.dim + c);
                if (p.dout) dr[i].ld(p.dout, row * p.dim + c);
            }
        }
        float sum[1] = {0.f};
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            const int e = (i * m.tg + lane) * kVec;
            if (kRing || !live || e >= gs || !p.weight) continue;
            float x[kVec], z[kVec];
            xr[i].get(x);
            if (before) {
                zr[i].get(z);
#pragma unroll
                for (int k = 0; k < kVec; ++k) x[k] *= silu_f32(z[k]);
            }
#pragma unroll
            for (int k = 0; k < kVec; ++k) sum[0] = fmaf(x[k], x[k], sum[0]);
        }
        float rstd = 1.f;
        if (p.weight) {
            if (kRing) sum[0] = first[0];
            else sum_over(sum, m.tg, first_g, red[0]);
            rstd = rsqrtf(sum[0] * inv_gs + p.eps);
        }
        // out, its norm's statistics
        float r[kNV][kVec];
        float s2[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            const int e = (i * m.tg + lane) * kVec;
            if (!live || e >= gs || !p.next_weight) continue;
            const int c = grp * gs + e;
            float f[kVec];
            xr[i].get(r[i]);
            if (p.gate != kGateNone) {
                zr[i].get(f);
#pragma unroll
                for (int k = 0; k < kVec; ++k) r[i][k] *= silu_f32(f[k]);
            }
            if (p.weight) {
                ld_weight<kVec>(p.weight, c, f);
#pragma unroll
                for (int k = 0; k < kVec; ++k) r[i][k] *= rstd * f[k];
            }
            if (p.res_scale) {
                ld_weight<kVec>(p.res_scale, c, f);
#pragma unroll
                for (int k = 0; k < kVec; ++k) r[i][k] *= f[k];
            }
            if (p.res) {
                rr[i].get(f);
#pragma unroll
                for (int k = 0; k < kVec; ++k) r[i][k] += f[k];
            }
            float dy[kVec];
            yr[i].get(dy);
            ld_weight<kVec>(p.next_weight, c, f);
#pragma unroll
            for (int k = 0; k < kVec; ++k) {
                s2[0] = fmaf(r[i][k], r[i][k], s2[0]);
                s2[1] = fmaf(dy[k] * f[k], r[i][k], s2[1]);
            }
        }
        float rstd2 = 1.f, coef = 0.f;
        if (p.next_weight) {
            sum_over(s2, m.row_threads, first_r, red[1]);
            rstd2 = rsqrtf(s2[0] * inv_dim + p.eps);
            coef = s2[1] * rstd2 * inv_dim;
        }
        float s_dn[1] = {0.f};
        float d[kNV][kVec];
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            const int e = (i * m.tg + lane) * kVec;
            if (!live || e >= gs) continue;
            const int c = grp * gs + e;
            float f[kVec];
            if (p.dout) {
                if (kRing) dr[i].ld(at + p.off_dout, c);
                dr[i].get(d[i]);
            } else {
#pragma unroll
                for (int k = 0; k < kVec; ++k) d[i][k] = 0.f;
            }
            if (p.next_weight) {
                float dy[kVec];
                if (kRing) yr[i].ld(at + p.off_dy, c);
                yr[i].get(dy);
                ld_weight<kVec>(p.next_weight, c, f);
#pragma unroll
                for (int k = 0; k < kVec; ++k) {
                    const float mm = r[i][k] * rstd2;
                    an[i][k] = fmaf(dy[k], mm, an[i][k]);
                    d[i][k] += rstd2 * (dy[k] * f[k] - mm * coef);
                }
            }
            if (p.dres) Raw<TR, kVec>::st(p.dres, row * p.dim + c, d[i]);
            float n[kVec], z[kVec], w[kVec], sc[kVec];
            xr[i].get(n);
            if (p.gate != kGateNone) zr[i].get(z);
            if (before) {
#pragma unroll
                for (int k = 0; k < kVec; ++k) n[k] *= silu_f32(z[k]);
            }
#pragma unroll
            for (int k = 0; k < kVec; ++k) w[k] = sc[k] = 1.f;
            if (p.weight) ld_weight<kVec>(p.weight, c, w);
            if (p.res_scale) ld_weight<kVec>(p.res_scale, c, sc);
#pragma unroll
            for (int k = 0; k < kVec; ++k) n[k] *= rstd;
            if (after) {
                float dz[kVec];
#pragma unroll
                for (int k = 0; k < kVec; ++k) {
                    const float sig = sigmoid_f32(z[k]);
                    dz[k] = d[i][k] * sc[k] * (n[k] * w[k]) * sig * (1.f + z[k] * (1.f - sig));
                    d[i][k] *= z[k] * sig;
                }
                Raw<T, kVec>::st(p.dz, row * p.dim + c, dz);
            }
#pragma unroll
            for (int k = 0; k < kVec; ++k) {
                ab[i][k] = fmaf(d[i][k], n[k], ab[i][k]);
                d[i][k] *= sc[k] * w[k];
                s_dn[0] = fmaf(d[i][k], n[k], s_dn[0]);
            }
        }
        if (kRing) {
            const long long next = base + gridDim.x, later = base + (long long)p.stages * gridDim.x;
            const int was = stage;
            if (++stage == p.stages) {
                stage = 0;
                phase ^= 1;
            }
            float two[2] = {s_dn[0], 0.f};
            if (next < p.rows) {
                if (!mbar_wait(&full[stage], phase, &kNoAbortRow, kRowWaitNs)) failed[odd] = 1;
                if (p.weight)
                    two[1] = stage_sum<T, kVec, kNV>(p, dyn + (size_t)stage * p.stage_bytes,
                                                     grp < p.groups, grp, lane, m.tg, gs);
            }
            if (p.weight) sum_over(two, m.tg, first_g, red[2]);
            if (!p.weight || m.tg <= 32) __syncthreads();  // else the sum's barrier has been
            if (*(volatile int *)&failed[odd]) {
                row_copy_failed(p, full, stage, phase, next, p.stages - 1);
                return;
            }
            if (t == 0 && later < p.rows) fetch_row<T, TR>(p, at, &full[was], later, true);
            s_dn[0] = two[0];
            first[0] = two[1];
        } else if (p.weight) {
            sum_over(s_dn, m.tg, first_g, red[2]);
        }
        odd ^= 1;
        const float cg = s_dn[0] * inv_gs;
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            const int e = (i * m.tg + lane) * kVec;
            if (!live || e >= gs) continue;
            const long long c = (long long)grp * gs + e;
            float x[kVec], z[kVec];
            xr[i].get(x);
            if (before) zr[i].get(z);
            float dz[kVec];
#pragma unroll
            for (int k = 0; k < kVec; ++k) {
                float a = x[k], sig = 0.f;
                if (before) {
                    sig = sigmoid_f32(z[k]);
                    a *= z[k] * sig;
                }
                if (p.weight) d[i][k] = rstd * (d[i][k] - a * rstd * cg);
                if (before) {
                    dz[k] = d[i][k] * x[k] * sig * (1.f + z[k] * (1.f - sig));
                    d[i][k] *= z[k] * sig;
                }
            }
            if (before) Raw<T, kVec>::st(p.dz, row * p.dim + c, dz);
            Raw<T, kVec>::st(p.dx, row * p.dim + c, d[i]);
        }
    }
    // the block's column sums; its row slots add theirs in turn
    float *part = p.partial + (long long)blockIdx.x * 2 * p.dim;
    if (m.rows_per > 1) {
        for (int s = 0; s < m.rows_per; ++s) {
            if (sub == s && grp < p.groups) {
#pragma unroll
                for (int i = 0; i < kNV; ++i) {
                    const int e = (i * m.tg + lane) * kVec;
                    if (e >= gs) continue;
#pragma unroll
                    for (int k = 0; k < kVec; ++k) {
                        const int c = grp * gs + e + k;
                        sums[c] = (s ? sums[c] : 0.f) + ab[i][k];
                        sums[p.dim + c] = (s ? sums[p.dim + c] : 0.f) + an[i][k];
                    }
                }
            }
            __syncthreads();
        }
        for (int c = t; c < 2 * p.dim; c += blockDim.x) part[c] = sums[c];
        return;
    }
    if (grp < p.groups) {
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            const int e = (i * m.tg + lane) * kVec;
            if (e >= gs) continue;
            const int c = grp * gs + e;
            if (p.weight || p.res_scale) Raw<float, kVec>::st(part, c, ab[i]);
            if (p.next_weight) Raw<float, kVec>::st(part + p.dim, c, an[i]);
        }
    }
}

// Column sums over the n blocks' partials: 32 columns a block, 32 slices.
__global__ void __launch_bounds__(1024)
block_norm_reduce_kernel(const BlockNormParams p, int n) {
    __shared__ float s[32][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, which = blockIdx.y;
    if (which ? !p.dnext_weight : !p.dweight && !p.dres_scale) return;
    float v = 0.f;
    if (c < p.dim) {
#pragma unroll 8
        for (int k = w; k < n; k += 32) v += p.partial[((long long)k * 2 + which) * p.dim + c];
    }
    s[w][lane] = v;
    __syncthreads();
    float u = s[lane][w];  // column w of the 32, slice `lane`
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) u += __shfl_xor_sync(0xffffffffu, u, m);
    const int o = blockIdx.x * 32 + w;
    if (lane != 0 || o >= p.dim) return;
    if (which) {
        p.dnext_weight[o] = u;
    } else {
        if (p.dweight) p.dweight[o] = p.res_scale ? u * p.res_scale[o] : u;
        if (p.dres_scale) p.dres_scale[o] = p.weight ? u * p.weight[o] : u;
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

// The ring for a block's rows: stage layout, and as many stages (up to eight) as
// `room` bytes hold; 0 where fewer than two fit or a block has fewer than
// `enough` rows to bring.
int plan_ring(BlockNormParams *p, size_t es, size_t rs, bool bwd, long long blocks, int room) {
    const int nt = (int)(p->dim * es), nr = (int)(p->dim * rs);
    int off = nt;
    auto take = [&off](bool have, int n) {
        const int at = off;
        if (have) off += n;
        return at;
    };
    p->off_z = take(p->gate != kGateNone, nt);
    p->off_res = take(p->res && (!bwd || p->next_weight), nr);
    p->off_dy = take(bwd && p->next_weight, nt);
    p->off_dout = take(bwd && p->dout, nr);
    p->stage_bytes = (off + 127) / 128 * 128;
    p->stages = std::min(room / p->stage_bytes, kMaxStages);
    if (p->stages < 2 || p->rows < 4 * blocks) p->stages = 0;
    return p->stages;
}

// A ring may take kRoom bytes whatever this call's stages come to: the opt-in belongs to
// the function and the device, so a call's own size set here would shrink it under a
// launch that another host thread is about to make with more. Set once per device.
template <int kRoom, typename Kernel>
cudaError_t allow_ring(Kernel kernel, std::atomic<unsigned long long> &configured) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (configured.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRoom);
    if (e == cudaSuccess) configured.fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

template <typename T, typename TR, int kVec, int kNV, int kThreads, int kBlocks>
cudaError_t fwd(const BlockNormParams &params, const Map &m, cudaStream_t stream) {
    BlockNormParams p = params;
    const int threads = m.row_threads * m.rows_per;
    if constexpr (kVec == 8) {
        // two blocks an SM, 100 KB of rows on their way to each
        constexpr int kRoom = 100 << 10;
        const long long blocks = 2ll * sm_count();
        if (m.rows_per == 1 && plan_ring(&p, sizeof(T), sizeof(TR), false, blocks, kRoom)) {
            auto k = block_norm_fwd_kernel<T, TR, kVec, kNV, kThreads, kBlocks, true>;
            static std::atomic<unsigned long long> configured{0};
            const cudaError_t e = allow_ring<kRoom>(k, configured);
            if (e != cudaSuccess) return e;
            k<<<(unsigned)blocks, threads, p.stages * p.stage_bytes, stream>>>(p, m);
            return cudaGetLastError();
        }
    }
    const long long blocks = (p.rows + m.rows_per - 1) / m.rows_per;
    block_norm_fwd_kernel<T, TR, kVec, kNV, kThreads, kBlocks, false>
        <<<(unsigned)blocks, threads, 0, stream>>>(p, m);
    return cudaGetLastError();
}

// The kernel with the fewest elements a thread that covers a row, since the sums and the
// row itself are registers: vectors of 8 where the rows allow, else single elements. The
// thread limits are what the registers leave: 640 threads twice an SM at 48 registers
// (8 elements, up to 5120 columns), 512 to 1024 with more elements else. In the gradient
// 8 elements take 96 registers: 320 threads twice (up to 2560 columns) or 640 once an SM,
// and 16 or 32 elements beyond. Its kernels spill: 100 to 330 bytes a thread at 8
// elements, 0.4 to 1.1 KB at 16, up to 4 KB at 32 (and so do rows of 32 single elements
// a thread forward, 1.1 KB). Measured, 41.9 M elements of bfloat16 with a float32 residual and all
// parts, as shares of the copy rate, forward / gradient: 1536 columns 53 / 35%, 2560
// 68 / 50%, 4096 81 / 40%, 5120 86 / 46%, 8192 55 / 34%.
template <typename T, typename TR>
cudaError_t fwd_typed(const BlockNormParams &p, cudaStream_t stream) {
    Map m;
    if (use_vec(p)) {
        if (fits(p, 8, 1, 640, &m)) return fwd<T, TR, 8, 1, 640, 2>(p, m, stream);
        if (fits(p, 8, 2, 640, &m)) return fwd<T, TR, 8, 2, 640, 1>(p, m, stream);
        if (fits(p, 8, 4, 512, &m)) return fwd<T, TR, 8, 4, 512, 1>(p, m, stream);
    }
    if (fits(p, 1, 8, 512, &m)) return fwd<T, TR, 1, 8, 512, 2>(p, m, stream);
    if (fits(p, 1, 32, 1024, &m)) return fwd<T, TR, 1, 32, 1024, 1>(p, m, stream);
    return cudaErrorInvalidValue;
}

int blocks_of(long long rows, int threads) {
    const long long most = (long long)sm_count() * std::max(2, 1024 / std::max(threads, 128));
    return (int)std::max<long long>(1, std::min(rows, most));
}

template <typename T, typename TR, int kVec, int kNV, int kThreads, int kBlocks>
cudaError_t bwd(const BlockNormParams &params, const Map &m, cudaStream_t stream) {
    BlockNormParams p = params;
    const long long want = (p.rows + m.rows_per - 1) / m.rows_per;
    const int threads = m.row_threads * m.rows_per;
    // the workspace has room for so many
    const long long room = block_norm_bwd_blocks(p.rows, p.dim);
    long long blocks = std::min({want, room, (long long)blocks_of(p.rows, threads)});
    bool ring = false;
    if constexpr (kVec == 8) {
        constexpr int kRoom = kBlocks == 2 ? 100 << 10 : 200 << 10;
        const long long two = (long long)kBlocks * sm_count();
        if (m.rows_per == 1 && two <= blocks &&
            plan_ring(&p, sizeof(T), sizeof(TR), true, two, kRoom)) {
            ring = true;
            blocks = two;
            auto k = block_norm_bwd_kernel<T, TR, kVec, kNV, kThreads, kBlocks, true>;
            static std::atomic<unsigned long long> configured{0};
            const cudaError_t e = allow_ring<kRoom>(k, configured);
            if (e != cudaSuccess) return e;
            k<<<(unsigned)blocks, threads, p.stages * p.stage_bytes, stream>>>(p, m);
        }
    }
    if (!ring) {
        const int smem = m.rows_per > 1 ? 2 * p.dim * (int)sizeof(float) : 0;
        block_norm_bwd_kernel<T, TR, kVec, kNV, kThreads, kBlocks, false>
            <<<(unsigned)blocks, threads, smem, stream>>>(p, m);
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !(p.weight || p.res_scale || p.next_weight)) return e;
    block_norm_reduce_kernel<<<dim3((unsigned)((p.dim + 31) / 32), 2), 1024, 0, stream>>>(
        p, (int)blocks);
    return cudaGetLastError();
}

template <typename T, typename TR>
cudaError_t bwd_typed(const BlockNormParams &p, cudaStream_t stream) {
    Map m;
    if (use_vec(p)) {
        if (fits(p, 8, 1, 320, &m)) return bwd<T, TR, 8, 1, 320, 2>(p, m, stream);
        if (fits(p, 8, 1, 640, &m)) return bwd<T, TR, 8, 1, 640, 1>(p, m, stream);
        if (fits(p, 8, 2, 512, &m)) return bwd<T, TR, 8, 2, 512, 1>(p, m, stream);
        if (fits(p, 8, 4, 512, &m)) return bwd<T, TR, 8, 4, 512, 1>(p, m, stream);
    }
    if (fits(p, 1, 4, 512, &m)) return bwd<T, TR, 1, 4, 512, 2>(p, m, stream);
    if (fits(p, 1, 16, 512, &m)) return bwd<T, TR, 1, 16, 512, 1>(p, m, stream);
    if (fits(p, 1, 32, 1024, &m)) return bwd<T, TR, 1, 32, 1024, 1>(p, m, stream);
    return cudaErrorInvalidValue;
}

}  // namespace

// Blocks of the gradient, each with its column sums: about a thousand threads an SM of
// the fewest that a row of this width gets (8 elements each, up to 512 threads), two
// blocks at least. 16384 columns: 39 MB of sums (155 if sized for 128 threads).
int block_norm_bwd_blocks(long long rows, int dim) {
    return blocks_of(rows, std::min((dim + 7) / 8, 512));
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
