// linattn_tc.cu -- linear attention with a decay for each head on the
// fifth-generation tensor cores: the sweep of linattn_params.cuh for bfloat16
// I/O, one persistent pass over the tokens with the state kept on the chip.
//
// Per (batch row, head), chunks of 64 tokens (formulas in linattn.cu). The
// state S is held transposed, value column d on tensor-memory lane d:
//   scores   Q Kᵀ                           64 (of 128) × 64 × D
//   Y        (Q S_in)ᵀ = S_inᵀ Qᵀ           128 × 64 × D, and on top of it
//            (P V)ᵀ = Vᵀ Pᵀ                 128 × 64 × 64
//   U        Σ_j c_j·v_j k_jᵀ = (c ◦ V)ᵀ K  128 × D × 64
//   y = r ◦ Y,   S ← exp(G_end)·S + U
// A pair's weight exp(A_row − A_col) is split: P takes 1/exp(A_col), the output
// r = exp(A_row), so that P costs a product per score and the two products one
// accumulator; both are taken about the middle of the chunk's decay, the entering
// state too, so that none goes beyond 2^±30. The gradient keeps the row factor in P
// and the products apart: its sweeps for dq and dk must make the same weights, to
// about 2^-20 (their dot products cancel in the log decays' gradient). So does, with
// an exponential per score, a chunk whose factors span more than 2^60 (a reset, a few
// tokens of strong decay).
// Q, K, V (and in the gradient the operand of the dot product) come by TMA into
// a ring of stages, 128-byte swizzled; P is written to shared memory; S_in and
// c ◦ V are A operands in tensor memory. Warps (20, one block an SM):
//   0-1    P: scores from tensor memory, weighted, to bfloat16
//   2      TMA producer, and each chunk's prefix sums of the log decays
//   3      issues every MMA (one thread)
//   4-7    c ◦ V: lane d reads column d of V, scales and splits it
//   8-15   state: half of a row's D columns per warp group, float32 registers
//   16-19  outputs: y to shared memory, TMA store; the gradient's dot products
// Precision: P and (in the forward pass) S_in are rounded once to bfloat16, an
// error of the output's own rounding on each of many terms; c ◦ V is split
// into three bfloat16 parts, so that the state, a float32 result that is
// carried over the whole sequence, keeps 24 bits. The gradient needs its
// products with S_in to about 16 bits instead (its log decays' gradient sums
// q·dq − k·dk, which cancel), so there S_in is a high/low pair and c ◦ V two
// parts (17 bits): both fill the 512 columns of tensor memory. The last state of the
// sweep for dv is a float32 result where the first state's gradient is asked for:
// there c ◦ V has three parts too, the third in the scores' columns.
//
// Bound: a chunk's chain of scores, P, output product and store, and of c ◦ V, U and
// state: 2.6 µs a chunk at D = 128 (3.5 in the gradient, 1.7 in the pass over states)
// where the MMAs alone take 0.9; 2 × 4096 tokens of 32 heads of 128: 118 µs (1786 on
// the CUDA cores), 65536 tokens of 16 heads 460 µs. Chunks of 128 tokens would double
// the work on P, the largest of the roles' shares. The forward full pass at D = 128 keeps
// 76 bytes a thread in local memory beside its 96 registers.
#include "linattn_params.cuh"
#include "umma_util.cuh"

#include <algorithm>

#include <math_constants.h>

namespace selscan {
namespace {

typedef __nv_bfloat16 bf16;

constexpr int kC = kLaChunk;
constexpr long long kWaitClocks = 4000000000ll;  // every wait gives up after about 2 s
constexpr int kStatusLinattnWait = 6;         // device error code
constexpr int kThr = 640;
constexpr float kRange = 60.f;                // |log2| a chunk's split factors may span
constexpr int kWarpTma = 2, kWarpMma = 3;
constexpr int kMaps = 8;

template <bool kV> struct Flag {
    static constexpr bool value = kV;
};
typedef Flag<true> Yes;
typedef Flag<false> No;

struct TcMaps {
    CUtensorMap m[kMaps];
};

// ---- tensor memory -------------------------------------------------------------
// 8 consecutive columns of this thread's lane.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
    uint32_t r[8];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(r[k]);
}
// 16 lanes × 32 columns in fragments: thread t holds, for the c-th 8 columns,
// lane t/4 columns 2·(t%4), + 1 in v[4c], v[4c+1] and lane t/4 + 8 in v[4c+2],
// v[4c+3].
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(r[k]);
}
// 16 lanes × 16 columns from fragments: lane t/4 column 4c + t%4 in r[2c], lane
// t/4 + 8 in r[2c+1] (completed by tmem_st_wait).
__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
                   "r"(r[6]), "r"(r[7])
                 : "memory");
}
// Four transposed 8×8 matrices of 16-bit elements from / to shared memory;
// thread t gives the address of row t%8 of matrix t/8.
__device__ __forceinline__ void ldmatrix_t(const void *row, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_addr(row))
                 : "memory");
}
__device__ __forceinline__ void stmatrix_t(void *row, uint32_t a, uint32_t b, uint32_t c,
                                           uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};"
                 ::"r"(smem_addr(row)), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}
__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }
// Two floats at a time: half the instructions, of which the roles' loops have more than
// the instruction caches like.
__device__ __forceinline__ uint64_t pair(float x, float y) {
    uint64_t p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
    return p;
}
__device__ __forceinline__ void unpair(uint64_t p, float &x, float &y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// 4 columns of this thread's lane (completed by tmem_st_wait).
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t (&r)[4]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};"
                 ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// D (tensor memory) = A (tensor memory, lane = row, two K elements a column) · B (shared memory).
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b,
                                             uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Waits for the phase of `bar` with the given parity; false once *abort is set
// or the time is up. Timed by the SM's clock: a wait stands between two MMAs
// here, and reading the global timer at its start was measured to delay the
// waiting thread by about a microsecond.
__device__ __forceinline__ bool try_wait_hint(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity), "r"(20000u)  // may sleep up to 20 us
        : "memory");
    return ok != 0;
}
// Out of line: the roles' loops share the instruction caches.
__device__ __noinline__ bool wait_bar_slow(uint64_t *bar, uint32_t parity, const int *abort) {
    const long long start = clock64();
    for (;;) {
        if (try_wait_hint(bar, parity)) return true;
        if (*reinterpret_cast<const volatile int *>(abort)) return false;
        if (clock64() - start > kWaitClocks) return false;
    }
}
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, const int *abort) {
    return mbar_try_wait(bar, parity) || wait_bar_slow(bar, parity, abort);
}

// One lane of the warp, always the same. Asked for where it is used, with the warp
// brought together: kept in a register over divergent code, the answer was
// measured to be worked out anew there, with two lanes issuing.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// ---- TMA -------------------------------------------------------------------------
__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, uint64_t *bar,
                                            int c0, int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(c0), "r"(c1), "r"(c2),
        "r"(c3)
        : "memory");
}
__device__ __forceinline__ void tma_store_4d(const CUtensorMap *map, const void *src, int c0,
                                             int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];"
        ::"l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(src)), "r"(c0), "r"(c1), "r"(c2),
          "r"(c3)
        : "memory");
}

// Byte offset of (token j, column d) in a tile of 64-column slabs of 64 rows,
// 128-byte swizzled.
__device__ __forceinline__ uint32_t tile_off(int j, int d) {
    return (uint32_t)((d >> 6) * (kC * 128) + j * 128 + ((((d >> 3) & 7) ^ (j & 7)) << 4) +
                      (d & 7) * 2);
}

// ---- sizes -------------------------------------------------------------------------
// Tensor-memory columns. The pass over the segments' own states holds U and
// c ◦ V twice instead of the rest. The full forward pass holds c ◦ V twice too: at
// D = 128 the second copy's first two parts lie where Ye does, which only a strong
// chunk uses, and the third in the last columns.
template <int D, bool kBwd, bool kFull> struct Cols {
    static constexpr uint32_t S = 0, Yi = 64, Ye = 128, U = kFull ? 192 : 0;
    static constexpr uint32_t St = 192 + D;
    // A gradient's sweep has two parts of c ◦ V or, where its last state is a result
    // (`fine`), three: at D = 128 the third lies where S does, once S has been read.
    static constexpr uint32_t StParts = kBwd ? 2 : 1;
    static constexpr bool VpOnS = kFull && kBwd && D == 128;
    static __device__ __forceinline__ int vp_parts(bool fine) { return kBwd && !fine ? 2 : 3; }
    static constexpr int UBufs = kFull ? 1 : 2, VpBufs = kFull && kBwd ? 1 : 2;
    static constexpr bool VpOnYe = kFull && !kBwd && D == 128;
    static constexpr uint32_t VpNext = 96;
    static constexpr uint32_t Vp = kFull ? St + StParts * (D / 2) : 2 * D;
    static __device__ __forceinline__ uint32_t vp(int buf, int part) {
        if (VpOnYe && buf) return part < 2 ? Ye + 32 * part : Vp + VpNext;
        if (VpOnS && part == 2) return S;
        return Vp + buf * VpNext + part * 32;
    }
    static_assert(Vp + (VpOnYe ? VpNext + 32 : VpOnS ? 64 : VpBufs * VpNext) <= 512,
                  "tensor memory");
};

// What is special about a chunk.
struct __align__(8) Kind {
    unsigned char strong;  // the factors of P leave float32's comfortable range
    unsigned char resets;  // may hold some: it is strong and (forward) does
    unsigned char none[2];
    unsigned char odd[4];  // bit 0: V holds a value that is not finite, by 32 columns; bit 1:
                           // the row's length ends in it
};
// A chunk's resets, tokens whose factor the exponentials flush to zero, as bits: the
// first token that token r still sees forward in time, and the one after the last that
// it sees backwards.
constexpr double kCutLog2 = -126.0;
__device__ __forceinline__ int after_cut(uint64_t cuts, int r) {
    const uint64_t upto = cuts & (~0ull >> (63 - r));
    return upto ? 63 - __clzll(upto) : 0;
}
__device__ __forceinline__ int before_cut(uint64_t cuts, int r) {
    const uint64_t from = r < 63 ? cuts >> (r + 1) : 0;
    return from ? r + __ffsll(from) : 64;
}
// Bit n to bit 2·n.
__device__ __forceinline__ uint64_t spread(uint32_t bits) {
    uint64_t out = 0;
    for (; bits; bits &= bits - 1) out |= 1ull << 2 * (__ffs(bits) - 1);
    return out;
}
// Rows [*from, *to) of a chunk that the state leaving takes.
__device__ __forceinline__ void kept_rows(uint64_t cuts, bool rev, int *from, int *to) {
    *from = rev ? 0 : after_cut(cuts, 63);
    *to = rev && cuts ? __ffsll(cuts) - 1 : 64;
}

template <int D, bool kBwd, bool kFull> struct TcSmem {
    static constexpr bool kCentred = kFull && !kBwd;
    static constexpr int kTiles = !kFull ? 2 : kBwd ? 4 : 3;  // (q,) k, v (, dot)
    static constexpr int kK = kFull ? 1 : 0, kV = kK + 1;     // places of k and v
    static constexpr int kStages = kFull ? 3 : 6;
    static constexpr int kSlots = kFull ? 6 : 8;              // ring of the chunks' decay factors
    bf16 tile[kStages][kTiles][kC * D];
    bf16 P[kFull ? kC * kC : 8];
    bf16 out[kFull ? kC * D : 8];   // y on its way out: swizzled slabs of 64 columns
    float A[kSlots][kC];            // log2 of the row factors without their scale
    float rowf[kSlots][kC];
    float colf[kSlots][kC];         // column factors of P; in a strong chunk those of A's rounding
    float colw[kSlots][kC];
    float decay[kSlots];
    float scale[kCentred ? kSlots : 1];  // of the state entering, 2^(the factors' middle)
    Kind kind[kSlots];
    uint64_t cuts[kSlots];          // of strong chunks; others have none
    uint64_t reached[kFull ? D : 1];  // an odd chunk's tokens that such values reach, by column
    int odds[4];                    // chunks that were odd, by 32 columns
    float red[4][kC];
    uint64_t full[kStages], empty[kStages], factors[kSlots];
    uint64_t vp_full[2], vp_empty[2], u_full[2], u_empty[2];
    uint64_t s_full, s_empty, p_full, p_empty, st_full, st_empty;
    uint64_t o_full, o_empty, drain;
    uint64_t odd_read[4];           // the last odd chunk's `reached` is read, by 32 columns
    uint64_t ye_read[4];            // VpOnYe: the strong chunks' outputs are read, in turn
    uint64_t v_sync[2], o_sync;     // the warps of c ◦ V, the output warps
    uint32_t tmem;
    int abort;
};

// 32 columns of a row of P as packed bfloat16: scores times f_j (kRow: times
// `row` too); in a strong chunk times row·f_j·2^(a − A_j). Zero outside columns
// lo .. hi, whatever the score. Selects, not branches.
template <bool kRow, bool kStrong>
__device__ __forceinline__ void score_weights(const float (&v)[32], const float *f, const float *A,
                                              float row, float a, int lo, int hi,
                                              uint32_t (&out)[16]) {
#pragma unroll
    for (int e4 = 0; e4 < 8; ++e4) {
        const float4 f4 = *reinterpret_cast<const float4 *>(f + 4 * e4);
        float h[4] = {}, x[4];
        if (kStrong) {
            const float4 h4 = *reinterpret_cast<const float4 *>(A + 4 * e4);
            h[0] = h4.x; h[1] = h4.y; h[2] = h4.z; h[3] = h4.w;
        }
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            const int j = 4 * e4 + e;
            uint64_t w = e ? pair(f4.z, f4.w) : pair(f4.x, f4.y);
            if (kStrong) w = mul2(w, pair(ex2_approx(a - h[e]), ex2_approx(a - h[e + 1])));
            if (kRow || kStrong) w = mul2(w, pair(row, row));
            w = mul2(w, pair(v[j], v[j + 1]));
            unpair(w, x[e], x[e + 1]);
            x[e] = j >= lo && j <= hi ? x[e] : 0.f;
            x[e + 1] = j + 1 >= lo && j + 1 <= hi ? x[e + 1] : 0.f;
        }
        out[2 * e4] = pack_bf16x2(x[0], x[1]);
        out[2 * e4 + 1] = pack_bf16x2(x[2], x[3]);
    }
}

// A chunk's outputs of 32 value columns from d0 on (this warp's lanes): y = r ◦ Y,
// or Y + r ◦ Ye where the two products are kept apart (kTwo; kReset: where r is
// zero, a reset, Ye does not count whatever it is). The accumulators are given
// back (`done`) as soon as the last is read. The outputs go into the staging rows
// (kF32: to float32 rows in memory, nl of them of dv columns), and with kDot
// their products with the dot operand, summed over the columns, into `red`. In
// fragments, so that the transposition to token rows is stmatrix's, and a sum
// over 32 columns is four additions and a ninth of a shuffle per token (with a
// lane per column a chunk took 720 instructions and 6000 clocks with the dot
// products).
template <bool kF32, bool kDot, bool kTwo, bool kReset, typename Done>
__device__ __forceinline__ void output_rows(uint32_t t_y, uint32_t t_ye, bf16 *out,
                                            const bf16 *dot, float *red, const float *rowf, int d0,
                                            float *y, long long y_row, int nl, int dv,
                                            const Done &done) {
    const int t = threadIdx.x & 31, r = t >> 2, c2 = 2 * (t & 3);
    char *orow = reinterpret_cast<char *>(out);
    const char *drow = reinterpret_cast<const char *>(dot);
    // rolled by 32 tokens: the loop bodies of the five roles share the instruction caches
#pragma unroll 1
    for (int th = 0; th < 2; ++th) {
        float v[2][16];  // the warp's two halves of 16 columns
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const uint32_t at = ((uint32_t)(16 * hh) << 16) + 32 * th;
            tmem_ld_frag(t_y + at, v[hh]);
            float ye[16];
            if (kTwo) tmem_ld_frag(t_ye + at, ye);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float2 f = *reinterpret_cast<const float2 *>(rowf + 32 * th + 8 * c + c2);
                const uint64_t f2 = pair(f.x, f.y);
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                    float *x = v[hh] + 4 * c + k;
                    if (!kTwo) {
                        unpair(mul2(pair(x[0], x[1]), f2), x[0], x[1]);
                    } else if (!kReset) {
                        unpair(fma2(f2, pair(ye[4 * c + k], ye[4 * c + k + 1]), pair(x[0], x[1])),
                               x[0], x[1]);
                    } else {
                        if (f.x != 0.f) x[0] = fmaf(f.x, ye[4 * c + k], x[0]);
                        if (f.y != 0.f) x[1] = fmaf(f.y, ye[4 * c + k + 1], x[1]);
                    }
                }
            }
        }
        if (th == 1) done();
        float acc[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = 0.f;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const float(&x)[16] = v[hh];
            if (kF32) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int j = 32 * th + 8 * (e >> 2) + c2 + (e & 1);
                    const int d = d0 + 16 * hh + r + 8 * ((e >> 1) & 1);
                    if (j < nl && d < dv) y[j * y_row + d] = x[e];
                }
            }
#pragma unroll
            for (int cp = 0; cp < 2; ++cp) {
                const uint32_t off = tile_off(32 * th + 16 * cp + 8 * (t >> 4) + (t & 7),
                                              d0 + 16 * hh + (t & 8));
                const float *u = x + 8 * cp;
                if (!kF32)
                    stmatrix_t(orow + off, pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3]),
                               pack_bf16x2(u[4], u[5]), pack_bf16x2(u[6], u[7]));
                if (kDot) {
                    uint32_t q[4];
                    ldmatrix_t(drow + off, q);
                    float *s = acc + 4 * cp;
                    s[0] = fmaf(u[0], bf_lo(q[0]), fmaf(u[2], bf_lo(q[1]), s[0]));
                    s[1] = fmaf(u[1], bf_hi(q[0]), fmaf(u[3], bf_hi(q[1]), s[1]));
                    s[2] = fmaf(u[4], bf_lo(q[2]), fmaf(u[6], bf_lo(q[3]), s[2]));
                    s[3] = fmaf(u[5], bf_hi(q[2]), fmaf(u[7], bf_hi(q[3]), s[3]));
                }
            }
        }
        if (kDot) {
            // over the 8 lanes of a column group: halves are exchanged and added,
            // lane group r keeps token 8·(r / 2) + c2 + r % 2
#pragma unroll
            for (int m = 4; m > 0; m >>= 1) {
                const bool up = (r & m) != 0;
#pragma unroll
                for (int k = 0; k < m; ++k) {
                    const float send = up ? acc[k] : acc[k + m];
                    const float keep = up ? acc[k + m] : acc[k];
                    acc[k] = keep + __shfl_xor_sync(0xffffffffu, send, 4 * m);
                }
            }
            red[32 * th + 8 * (r >> 1) + c2 + (r & 1)] = acc[0];
        }
    }
}

// ---- values that are not finite ------------------------------------------------------
// The products run over pairs that do not count (a later token, one that a reset cuts
// off) with a weight of zero, and zero times a value that is not finite would. So such
// values leave the operands, and what they do reach is marked by hand. Out of line, and
// only for the chunks that need it.

// v·0 + sums, pairs of bfloat16: stays zero while every v is finite.
__device__ __forceinline__ void add_odd(uint32_t &sums, uint32_t v) {
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sums) : "r"(v), "r"(0u));
}
__device__ __forceinline__ bool holds_odd(uint32_t sums) { return (sums & 0x7FFF7FFFu) != 0; }

// c ◦ V of 32 tokens × 16 columns as bfloat16 parts. kOdd: V may be infinite, which the
// first part takes alone, and counts in rows [from, to) only.
template <bool kOdd>
__device__ __forceinline__ void cv_parts(const char *tile, const float *w, int th, int hh, int d0,
                                         int nvp, int from, int to, uint32_t (&part)[3][8],
                                         uint32_t &odd) {
    const int lane = threadIdx.x & 31, r8 = lane >> 4, c2 = 2 * (lane & 3);
#pragma unroll
    for (int cp = 0; cp < 2; ++cp) {
        uint32_t v[4];
        ldmatrix_t(tile + tile_off(32 * th + 16 * cp + 8 * r8 + (lane & 7), d0 + 16 * hh + (lane & 8)),
                   v);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int j = 32 * th + 16 * cp + 8 * (k >> 1) + c2;
            const float2 f = *reinterpret_cast<const float2 *>(w + j);
            float x0, x1;
            unpair(mul2(pair(f.x, f.y), pair(bf_lo(v[k]), bf_hi(v[k]))), x0, x1);
            if (kOdd) {
                x0 = j >= from && j < to ? x0 : 0.f;
                x1 = j + 1 >= from && j + 1 < to ? x1 : 0.f;
            } else {
                add_odd(odd, v[k]);
            }
#pragma unroll
            for (int e = 0; e < 3; ++e) {
                if (e >= nvp) break;
                // all parts but the last by truncation (no conversion)
                const uint32_t u =
                    e + 1 < nvp ? __byte_perm(__float_as_uint(x0), __float_as_uint(x1), 0x7632)
                                : pack_bf16x2(x0, x1);
                part[e][4 * cp + k] = u;
                const bool odd0 = kOdd && !(fabsf(x0) < CUDART_INF_F),
                           odd1 = kOdd && !(fabsf(x1) < CUDART_INF_F);
                unpair(fma2(pair(bf_lo(u), bf_hi(u)), pair(-1.f, -1.f), pair(x0, x1)), x0, x1);
                if (odd0) x0 = 0.f;
                if (odd1) x1 = 0.f;
            }
        }
    }
}

// The end of c ◦ V for a chunk that may hold resets or, by every warp that meets one in
// V, values that are not finite. False where a wait gave up.
//   K: rows that the state leaving does not take are cleared where they hold such a
//     value, once the chunk's scores have been made of them. The 128 threads of c ◦ V
//     share the rows.
//   V (`odd`: this lane met one): c ◦ V of the warp's 32 columns again; in the full pass
//     such values then leave V, and the tokens that they reach are marked.
template <int D, bool kBwd, bool kFull>
__device__ __noinline__ bool odd_chunk(TcSmem<D, kBwd, kFull> &S, int i, bool rev, bool fine,
                                       bool odd) {
    typedef TcSmem<D, kBwd, kFull> Smem;
    typedef Cols<D, kBwd, kFull> C;
    const int s = i % Smem::kStages, sl = i % Smem::kSlots, lane = threadIdx.x & 31;
    const int tg = threadIdx.x & 127, g = tg >> 5, d0 = 32 * g;
    auto wait = [&](uint64_t *bar, int parity) -> bool {
        return __all_sync(0xffffffffu, wait_bar(bar, parity & 1, &S.abort));
    };
    const uint64_t cuts = S.kind[sl].strong ? S.cuts[sl] : 0;
    int from, to;
    kept_rows(cuts, rev, &from, &to);
    if (cuts) {
        char *tile = reinterpret_cast<char *>(S.tile[s][Smem::kK]);
        uint32_t sums[4] = {0, 0, 0, 0};
#pragma unroll
        for (int it = 0; it < D / 16; ++it) {
            const int e = tg + 128 * it, j = e / (D / 8);
            uint4 u = *reinterpret_cast<const uint4 *>(tile + tile_off(j, 8 * (e % (D / 8))));
            if (j >= from && j < to) u = make_uint4(0, 0, 0, 0);
            add_odd(sums[0], u.x);
            add_odd(sums[1], u.y);
            add_odd(sums[2], u.z);
            add_odd(sums[3], u.w);
        }
        const bool found = holds_odd(sums[0] | sums[1] | sums[2] | sums[3]);
        if (__any_sync(0xffffffffu, found)) {
            if (kFull && !wait(&S.s_full, i)) return false;
#pragma unroll 1
            for (int e = tg; found && e < kC * (D / 8); e += 128) {
                const int j = e / (D / 8);
                if (j < from || j >= to)
                    *reinterpret_cast<uint4 *>(tile + tile_off(j, 8 * (e % (D / 8)))) =
                        make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
        }
    }
    if (d0 >= D || !__any_sync(0xffffffffu, odd)) return true;
    char *tile = reinterpret_cast<char *>(S.tile[s][Smem::kV]);
    const int nvp = C::vp_parts(fine);
    const uint32_t taddr = S.tmem + ((uint32_t)d0 << 16);
    tmem_st_wait();  // the same places are written again
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
        const int th = q >> 1, hh = q & 1;
        uint32_t part[3][8], none = 0;
        cv_parts<true>(tile, S.colw[sl], th, hh, d0, nvp, from, to, part, none);
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < nvp)
                tmem_st_frag(taddr + ((uint32_t)(16 * hh) << 16) + C::vp(i % C::VpBufs, e) + 16 * th,
                             part[e]);
    }
    if (!kFull) return true;
    const int before = S.odds[g];
    // the last odd chunk's outputs have read `reached` (and every lane the tile)
    if (before > 0 && !wait(&S.odd_read[g], before - 1)) return false;
    __syncwarp();
    const int d = d0 + lane;
    uint64_t reached = 0;
    bool hit = false;
    for (int k = 0; k < kC; ++k) {
        const int j = rev ? kC - 1 - k : k;
        const bool cut = cuts >> j & 1;
        unsigned short *at = reinterpret_cast<unsigned short *>(tile + tile_off(j, d));
        if (!rev && cut) hit = false;
        if ((*at & 0x7F80) == 0x7F80) {
            *at = 0;
            hit = true;
        }
        if (hit) reached |= 1ull << j;
        if (rev && cut) hit = false;
    }
    S.reached[d] = reached;
    if (kBwd)  // their dot products too
        for (int j = 0; j < kC; ++j)
            if (reached >> j & 1)
                *reinterpret_cast<unsigned short *>(
                    reinterpret_cast<char *>(S.tile[s][Smem::kTiles - 1]) + tile_off(j, d)) = 0x7FFF;
    if (lane == 0) {
        S.odds[g] = before + 1;
        S.kind[sl].odd[g] |= 1;
    }
    fence_proxy_async_smem();
    __syncwarp();
    return true;
}

// A chunk's output rows put right before they are stored, by the warp that stores: the
// tokens that values reach which are not finite become NaN, rows behind the row's length
// zero (they came out as the state's products with zero operands). In the staging rows
// or in the float32 rows in memory.
template <int D, bool kBwd, bool kFull>
__device__ __noinline__ void odd_rows(TcSmem<D, kBwd, kFull> &S, const LinattnParams &p,
                                      const SweepArgs &a, int b, int h, int len, int t0, int sl) {
    const int lane = threadIdx.x & 31, nq = min(kC, len - t0),
              nl = (int)min((long long)kC, p.seqlen - t0);
    float *y = kBwd && a.y_f32 ? static_cast<float *>(a.y) +
                                     (((long long)b * p.seqlen + t0) * p.heads + h) * a.dv
                               : nullptr;
    for (int g = 0; g < D / 32; ++g) {
        const bool odd = S.kind[sl].odd[g] & 1;
        const int d = 32 * g + lane;
        const uint64_t reached = odd ? S.reached[d] : 0;
        for (int j = odd ? 0 : nq; j < kC; ++j) {
            const bool nan = j < nq && ((reached >> j) & 1);
            if (!nan && j < nq) continue;
            if (!y)
                *reinterpret_cast<unsigned short *>(reinterpret_cast<char *>(S.out) +
                                                    tile_off(j, d)) = nan ? 0x7FFF : 0;
            else if (j < nl && d < a.dv)
                y[(long long)j * p.heads * a.dv + d] = nan ? CUDART_NAN_F : 0.f;
        }
        __syncwarp();
        if (odd && lane == 0) mbar_arrive(&S.odd_read[g]);
    }
    fence_proxy_async_smem();
    __syncwarp();
}

// One block: one (sweep, batch row, head, segment). kFull false: only the
// segment's own state, from zero. kFine: some sweeps have three parts of c ◦ V (one
// kernel for both cost the gradient without them 224 → 257 µs on 2 × 4096 tokens of
// 16 heads of 128, in registers and code).
template <int D, bool kBwd, bool kFull, bool kFine>
__global__ void __launch_bounds__(kThr, 1)
linattn_tc_kernel(const __grid_constant__ LinattnParams p, const __grid_constant__ TcMaps maps) {
    typedef TcSmem<D, kBwd, kFull> Smem;
    typedef Cols<D, kBwd, kFull> C;
    constexpr int kStages = Smem::kStages, kSlots = Smem::kSlots;
    constexpr bool kCentred = Smem::kCentred;
    extern __shared__ __align__(128) unsigned char smem_raw[];
    // 1024-byte aligned: the 128-byte swizzle pattern is taken from address bits 7..9
    Smem &S = *reinterpret_cast<Smem *>(smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023));
    const int order = p.order0 + (int)(blockIdx.x % p.orders);  // in the sweep's direction
    const long long id = blockIdx.x / p.orders;
    if (kFull && p.nseg > 1 && order == 0) linattn_let_states_start();
    const SweepArgs &a = p.sweep[id % p.nsweeps];
    const long long bh = id / p.nsweeps;
    const int b = (int)(bh / p.heads), h = (int)(bh % p.heads);
    const bool rev = a.reverse != 0;
    const int seg = rev ? p.nseg - 1 - order : order;
    const int len = p.seqlens ? (int)min((long long)max(__ldg(p.seqlens + b), 0), p.seqlen)
                              : (int)p.seqlen;
    int c_first, c_end;
    linattn_segment(p, rev, order, &c_first, &c_end);
    const int c_live = max(c_first, min(c_end, (len + kC - 1) / kC));  // chunks with tokens
    const int n = c_live - c_first;
    auto chunk_of = [&](int i) { return rev ? c_live - 1 - i : c_first + i; };
    const int t = threadIdx.x, lane = t & 31, warp = __shfl_sync(0xffffffffu, t >> 5, 0);
    const bool has_dot = kBwd && kFull && a.dot_out != nullptr;
    const bool fine = kFine && a.fine_state != 0;
    const int nvp = C::vp_parts(fine);

    if (warp == kWarpTma) tmem_alloc(&S.tmem, 512);
    if (t == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&S.full[s], 2);
            mbar_init(&S.empty[s], has_dot ? 5 : 1);  // the MMAs (and the dot operand's readers)
        }
        mbar_init(&S.s_full, 1);
        mbar_init(&S.s_empty, 2);
        mbar_init(&S.p_full, 2);
        mbar_init(&S.p_empty, 1);
        for (int k = 0; k < 2; ++k) {
            mbar_init(&S.vp_full[k], 4);
            mbar_init(&S.vp_empty[k], 1);
            mbar_init(&S.u_full[k], 1);
            mbar_init(&S.u_empty[k], 8);
            mbar_init(&S.v_sync[k], 4);
        }
        for (int k = 0; k < kSlots; ++k) mbar_init(&S.factors[k], 1);
        mbar_init(&S.st_full, 8);
        mbar_init(&S.st_empty, 1);
        mbar_init(&S.drain, 1);
        mbar_init(&S.o_full, 1);
        mbar_init(&S.o_empty, 4);
        for (int k = 0; k < 4; ++k) {
            mbar_init(&S.ye_read[k], 4);
            mbar_init(&S.odd_read[k], 1);
            S.odds[k] = 0;
        }
        mbar_init(&S.o_sync, 4);
        S.abort = 0;
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;  // this warp's lanes
    // A wait of a whole warp; false once any role has given up.
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, wait_bar(bar, parity & 1, &S.abort));
    };
    auto arrive = [&](uint64_t *bar) {  // by one lane for the warp
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    bool ok = true;
    // Chunk i's factors stand in slot i % kSlots. They are written once the MMAs of
    // chunk i − kStages are done. Full pass: those of chunk i − 3 wait for the outputs
    // of chunk i − 4, so six slots do; states: those of chunk i − 6 for the state of
    // chunk i − 8. Roles that hold no stage wait for the slot's barrier: a stage's
    // could be two phases on by then.
    constexpr int kUBufs = C::UBufs, kVBufs = C::VpBufs;
    if (warp < 4) {
        if (warp == kWarpTma) {
            // ---- producer: tiles by TMA, decays by the warp -----------------------------
            const CUtensorMap *mq = &maps.m[a.map[0]], *mk = &maps.m[a.map[1]],
                              *mv = &maps.m[a.map[2]], *md = &maps.m[a.map[3]];
            const int hq = h / a.q_group, hk = h / a.k_group, hv = h / a.v_group,
                      hd = has_dot ? h / a.dot_group : 0;
            const float gh = p.g ? 0.f : p.g_head ? __ldg(p.g_head + h) : 0.f;
            auto raw = [&](int i, int e) -> float {  // the log decay of token 2·lane + e of chunk i
                const int tok = chunk_of(i) * kC + 2 * lane + e;
                if (i >= n || tok >= len) return 0.f;
                return p.g ? ldg_f32(static_cast<const bf16 *>(p.g) +
                                     ((long long)b * p.seqlen + tok) * p.heads + h)
                           : gh;
            };
            float r0 = raw(0, 0), r1 = raw(0, 1);
            double seg_log2 = 0.0;
            int issued = 0;
            for (int i = 0; i < n; ++i) {
                const int s = i % kStages;
                ok = wait(&S.empty[s], ((i / kStages) & 1) ^ 1);
                if (!ok) break;
                const int t0 = chunk_of(i) * kC;
                if (lane == 0) {
                    constexpr int kSlabs = D / 64;
                    constexpr uint32_t kBytes = kSlabs * kC * 128;
                    mbar_arrive_expect_tx(&S.full[s],
                                          kBytes * (kFull ? (has_dot ? 4 : 3) : 2));
#pragma unroll
                    for (int sl = 0; sl < kSlabs; ++sl) {
                        if (kFull)
                            tma_load_4d(&S.tile[s][0][sl * kC * 64], mq, &S.full[s], sl * 64, hq, t0, b);
                        tma_load_4d(&S.tile[s][Smem::kK][sl * kC * 64], mk, &S.full[s], sl * 64, hk, t0,
                                    b);
                        tma_load_4d(&S.tile[s][Smem::kV][sl * kC * 64], mv, &S.full[s], sl * 64, hv, t0,
                                    b);
                        if (has_dot)
                            tma_load_4d(&S.tile[s][Smem::kTiles - 1][sl * kC * 64], md, &S.full[s],
                                        sl * 64, hd, t0, b);
                    }
                }
                issued = i + 1;
                double g0 = (double)r0 * 1.4426950408889634, g1 = (double)r1 * 1.4426950408889634;
                r0 = raw(i + 1, 0);
                r1 = raw(i + 1, 1);
                g0 = g0 < kLaResetLog2 ? kLaResetLog2 : g0;
                g1 = g1 < kLaResetLog2 ? kLaResetLog2 : g1;
                double sum = g0 + g1;
#pragma unroll
                for (int m = 1; m < 32; m <<= 1) {
                    const double o = __shfl_up_sync(0xffffffffu, sum, m);
                    if (lane >= m) sum += o;
                }
                const double end = __shfl_sync(0xffffffffu, sum, 31);
                // A: the log2 of what separates a token from the state entering (in the sweep's
                // direction); a pair's weight is 2^(A_row − A_col)
                const double G[2] = {sum - g1, sum};
                double exact[2];
                float A[2], row[2], colf[2], colw[2];
                bool far = false;
                // Forward, the factors are taken about the middle of the chunk's decay: each
                // keeps within 2^±30 (backwards P takes both, and no more than their product).
                float at = 0.f;
                if (kCentred) {
                    at = rintf(0.5f * (float)end);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        far = far || !(fabsf((float)G[e] - at) <= 0.5f * kRange);
                    far = __any_sync(0xffffffffu, far);
                    if (far) at = 0.f;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    exact[e] = rev ? end - G[e] : G[e];
                    A[e] = (float)exact[e];
                    if (!kCentred) far = far || !(fabsf(A[e]) <= kRange);
                    row[e] = a.row_scale * ex2_approx(kCentred ? A[e] - at : A[e]);
                    colf[e] = a.col_scale * ex2_approx(kCentred ? at - A[e] : -A[e]);
                    colw[e] = a.col_scale * ex2_approx((float)(rev ? G[e] : end - G[e]));
                }
                // the total too: a reset on a chunk's first token is in no A backwards
                if (!kCentred) far = __any_sync(0xffffffffu, far || !(fabsf((float)end) <= kRange));
                uint32_t cut0 = 0, cut1 = 0;
                if (far) {
                    // A strong chunk's weights are 2^(A_row − A_col) from A as it is rounded
                    // (a step of 2^-10 behind many resets, where it passes 2^13; the
                    // difference itself is exact there) and the factors of what it lost.
                    colf[0] = ex2_approx((float)((double)A[0] - exact[0]));
                    colf[1] = ex2_approx((float)((double)A[1] - exact[1]));
                    cut0 = __ballot_sync(0xffffffffu, g0 < kCutLog2);
                    cut1 = __ballot_sync(0xffffffffu, g1 < kCutLog2);
                    if (lane == 0) S.cuts[i % kSlots] = spread(cut0) | spread(cut1) << 1;
                }
                const int sl = i % kSlots;
                *reinterpret_cast<float2 *>(&S.A[sl][2 * lane]) = make_float2(A[0], A[1]);
                *reinterpret_cast<float2 *>(&S.rowf[sl][2 * lane]) = make_float2(row[0], row[1]);
                *reinterpret_cast<float2 *>(&S.colf[sl][2 * lane]) = make_float2(colf[0], colf[1]);
                *reinterpret_cast<float2 *>(&S.colw[sl][2 * lane]) = make_float2(colw[0], colw[1]);
                if (lane == 0) {
                    S.decay[sl] = ex2_approx((float)end);
                    *reinterpret_cast<uint2 *>(&S.kind[sl]) =
                        make_uint2(far ? 1u | (!kCentred || (cut0 | cut1) ? 256u : 0u) : 0u,
                                   len - t0 < kC && len < p.seqlen ? 0x02020202u : 0u);
                    if (kCentred) S.scale[sl] = ex2_approx(at);
                }
                seg_log2 += end;
                arrive(&S.full[s]);
                if (lane == 0) mbar_arrive(&S.factors[sl]);
            }
            if ((!kFull || (p.nseg > 1 && order == 0)) && lane == 0)
                a.seg_decay[bh * p.nseg + seg] = kFull ? 0.f : ex2_approx((float)seg_log2);
            if (!ok) {  // copies still in flight land before the block goes
                const int none = 0;
                for (int i = max(0, issued - kStages); i < issued; ++i)
                    wait_bar(&S.full[i % kStages], (i / kStages) & 1, &none);
            }
        } else if (warp == kWarpMma) {
            // ---- MMA issuer ---------------------------------------------------------------
            // The warp waits (a lane per barrier, so that several waits cost one), an elected
            // lane issues. Descriptors are a tile's first plus an offset in 16-byte units:
            // an MMA of 64 columns is bound by its issue (about 50 clocks), so that its
            // loops can be rolled for the instruction caches' sake (2 × 4096 tokens of 32
            // heads of 128: 130 → 121 µs).
            constexpr uint32_t id_s = idesc_bf16(128, 64, 0, 0);   // Q (K-major), K (K-major)
            constexpr uint32_t id_yi = idesc_bf16(128, 64, 1, 0);  // Vᵀ (M-major), P (K-major)
            constexpr uint32_t id_ye = idesc_bf16(128, 64, 0, 0);  // S (tensor memory), Q
            constexpr uint32_t id_u = idesc_bf16(128, D, 0, 1);    // c ◦ V (tensor memory), K (N-major)
            constexpr uint32_t kSlab = kC * 128;
            auto wait3 = [&](uint64_t *b0, uint32_t p0, uint64_t *b1, uint32_t p1, uint64_t *b2,
                             uint32_t p2) -> bool {
                bool done = true;
                if (lane < 3)
                    done = wait_bar(lane == 0 ? b0 : lane == 1 ? b1 : b2,
                                    (lane == 0 ? p0 : lane == 1 ? p1 : p2) & 1, &S.abort);
                ok = __all_sync(0xffffffffu, done);
                tc_fence_after();
                return ok;
            };
            auto wait2 = [&](uint64_t *b0, uint32_t p0, uint64_t *b1, uint32_t p1) -> bool {
                return wait3(b0, p0, b1, p1, b1, p1);
            };
            // K-major: steps of 16 columns inside slabs of 64; M- or N-major: steps of 16
            // tokens, two 8-row atoms
            auto kstep = [](int x) { return (uint64_t)(((x >> 2) * kSlab + (x & 3) * 32) >> 4); };
            constexpr uint64_t kTok = 2048 >> 4;
            auto scores = [&](int i) {  // rows 64 .. 127 of A are whatever follows the tile
                const int s = i % kStages;
                const uint64_t q = umma_desc_sw128(smem_addr(S.tile[s][0]), 16, 1024),
                               k = umma_desc_sw128(smem_addr(S.tile[s][Smem::kK]), 16, 1024);
                if (!wait2(&S.full[s], i / kStages, &S.s_empty, (i & 1) ^ 1)) return;
                if (elect_one()) {
#pragma unroll 1
                    for (int x = 0; x < D / 16; ++x)
                        umma_bf16(tmem + C::S, q + kstep(x), k + kstep(x), id_s, x > 0);
                    umma_commit(&S.s_full);
                }
                __syncwarp();
            };
            if (kFull && n > 0) scores(0);
            for (int i = 0; ok && i < n; ++i) {
                const int s = i % kStages;
                const uint64_t k = umma_desc_sw128(smem_addr(S.tile[s][Smem::kK]), kSlab, 1024);
                const int ub = i % kUBufs, vb = i % kVBufs;
                // U: both operands' K is the token. Its tiles have landed: c ◦ V was made from them.
                if (!wait2(&S.vp_full[vb], i / kVBufs, &S.u_empty[ub], ((i / kUBufs) & 1) ^ 1)) break;
                if (elect_one()) {
                    const uint32_t u = tmem + C::U + ub * D;
#pragma unroll
                    for (int part = 0; part < 3; ++part) {
                        if (part >= nvp) break;
#pragma unroll 1
                        for (int x = 0; x < kC / 16; ++x)
                            umma_bf16_ts(u, tmem + C::vp(vb, part) + x * 8, k + x * kTok,
                                         id_u, part > 0 || x > 0);
                    }
                    umma_commit(&S.u_full[ub]);
                    if (kVBufs != kUBufs) umma_commit(&S.vp_empty[vb]);
                    if (!kFull) umma_commit(&S.empty[s]);
                }
                __syncwarp();
                if (!kFull) continue;
                if (i + 1 < n) {
                    // U reads c ◦ V's third part from where the scores go
                    if (C::VpOnS && fine && !wait2(&S.u_full[ub], i, &S.u_full[ub], i)) break;
                    scores(i + 1);
                }
                // Ye = S_inᵀ Qᵀ and Yi = Vᵀ Pᵀ, the second on top of the first where the row
                // factors stand in the outputs
                const bool two = kBwd || S.kind[i % kSlots].strong != 0;
                const uint32_t yi = tmem + C::Yi, ye = two ? tmem + C::Ye : yi;
                const uint64_t q = umma_desc_sw128(smem_addr(S.tile[s][0]), 16, 1024);
                const uint64_t v = umma_desc_sw128(smem_addr(S.tile[s][Smem::kV]), kSlab, 1024),
                               pp = umma_desc_sw128(smem_addr(S.P), 16, 1024);
                if (!ok || !wait3(&S.o_empty, (i & 1) ^ 1, &S.st_full, i, &S.p_full, i)) break;
                // U reads c ◦ V from where this Ye goes
                if (C::VpOnYe && two && vb && !wait2(&S.vp_empty[vb], i / kVBufs, &S.p_full, i)) break;
                if (elect_one()) {
#pragma unroll
                    for (int part = 0; part < (int)C::StParts; ++part)
#pragma unroll 1
                        for (int x = 0; x < D / 16; ++x)
                            umma_bf16_ts(ye, tmem + C::St + part * (D / 2) + x * 8, q + kstep(x), id_ye,
                                         part > 0 || x > 0);
                    umma_commit(&S.st_empty);
#pragma unroll 1
                    for (int x = 0; x < kC / 16; ++x)
                        umma_bf16(yi, v + x * kTok, pp + kstep(x), id_yi, !two || x > 0);
                    umma_commit(&S.o_full);
                    umma_commit(&S.p_empty);
                    umma_commit(&S.empty[s]);
                }
                __syncwarp();
            }
            if (!ok) {  // MMAs in flight end before tensor memory is given back
                const int none = 0;
                if (elect_one()) {
                    umma_commit(&S.drain);
                    wait_bar(&S.drain, 0, &none);
                }
                __syncwarp();
            }
        } else {
            // ---- P: weights of the products inside the chunk, a row per lane ---------------
            if (kFull) {
                const int r = 32 * warp + lane;
                for (int i = 0; i < n; ++i) {
                    const int nq = min(kC, len - chunk_of(i) * kC), sl = i % kSlots;
                    ok = wait(&S.factors[sl], i / kSlots);
                    if (!ok) break;
                    const bool strong = S.kind[sl].strong != 0;
                    const float rf = S.rowf[sl][r], ar = S.A[sl][r];
                    // in a strong chunk: the reciprocal of a factor within 2^-11.5 of one, to 2^-23
                    const float low = a.p_scale * (2.f - S.colf[sl][r]);
                    int lo = rev ? r : 0, hi = r >= nq ? -1 : rev ? nq - 1 : r;
                    if (strong) {  // what stands beyond a reset does not count
                        if (rev)
                            hi = min(hi, before_cut(S.cuts[sl], r) - 1);
                        else
                            lo = after_cut(S.cuts[sl], r);
                    }
                    ok = wait(&S.s_full, i);
                    if (!ok) break;
                    tc_fence_after();
                    char *row = reinterpret_cast<char *>(S.P) + r * 128;
                    uint32_t out[16];
                    auto block = [&](int half, bool last) {
                        float v[32];
                        tmem_ld32(tmem + lanes + C::S + 32 * half, v);
                        if (last) {
                            tc_fence_before();
                            arrive(&S.s_empty);  // the next chunk's scores may come
                        }
                        const float *f = S.colf[sl] + 32 * half;
                        if (strong)
                            score_weights<true, true>(v, f, S.A[sl] + 32 * half, low, ar,
                                                      lo - 32 * half, hi - 32 * half, out);
                        else
                            score_weights<kBwd, false>(v, f, nullptr, rf, 0.f, lo - 32 * half,
                                                       hi - 32 * half, out);
                    };
                    // the block off the diagonal (of the warp that has one, else zeros), then
                    // the one on it
                    const bool off = warp == (rev ? 0 : 1);
#pragma unroll 1
                    for (int k = 0; k < 2; ++k) {
                        const int half = k ? warp : 1 - warp;
                        if (k || off) {
                            block(half, k == 1);
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; ++e) out[e] = 0;
                        }
                        if (k == 0) {
                            ok = wait(&S.p_empty, (i & 1) ^ 1);
                            if (!ok) break;
                        }
#pragma unroll
                        for (int c8 = 0; c8 < 4; ++c8)
                            *reinterpret_cast<uint4 *>(row + (((4 * half + c8) ^ (r & 7)) << 4)) =
                                make_uint4(out[4 * c8], out[4 * c8 + 1], out[4 * c8 + 2],
                                           out[4 * c8 + 3]);
                    }
                    if (!ok) break;
                    fence_proxy_async_smem();
                    arrive(&S.p_full);
                }
            }
        }
    } else if (warp < 8 || (!kFull && warp >= 16)) {
        // ---- c ◦ V as bfloat16 parts, column d of V on lane d --------------------------
        // In the pass over the segments' own states the output warps take every other chunk.
        const int group = warp >= 16 ? 1 : 0, tg = t - (group ? 512 : 128);
        const int d0 = 32 * (warp & 3);
        uint32_t syncs = 0;
        int strongs = 0;
        for (int i = group; i < n; i += kFull ? 1 : 2) {
            const int s = i % kStages, vb = i % kVBufs, use = i / kVBufs;
            const int nq = min(kC, len - chunk_of(i) * kC);
            ok = wait(&S.full[s], i / kStages);
            if (!ok) break;
            if (nq < kC && len < p.seqlen) {
                // what stands behind the row's length may be anything: zero it
                for (int e = tg; e < (kC - nq) * (D / 8); e += 128) {
                    const uint32_t off = tile_off(nq + e / (D / 8), 8 * (e % (D / 8)));
#pragma unroll 1
                    for (int x = 0; x < Smem::kTiles; ++x)
                        *reinterpret_cast<uint4 *>(reinterpret_cast<char *>(S.tile[s][x]) + off) =
                            make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                arrive(&S.v_sync[group]);
                ok = wait(&S.v_sync[group], syncs++);
                if (!ok) break;
            }
            const char *tile = reinterpret_cast<const char *>(S.tile[s][Smem::kV]);
            const int sl = i % kSlots;
            const float *w = S.colw[sl];
            const bool resets = S.kind[sl].resets != 0;
            uint32_t odd = 0;  // NaN where V is not finite
            // rolled: the loop bodies of the five roles share the instruction caches. The
            // first quarter is made while U still reads the previous parts.
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {  // 32 tokens × 16 columns
                const int th = q >> 1, hh = q & 1;
                uint32_t part[3][8];
                if (d0 < D) cv_parts<false>(tile, w, th, hh, d0, nvp, 0, kC, part, odd);
                if (q == 0 && use > 0) {
                    // U has read what stands there
                    ok = wait(kVBufs == kUBufs ? &S.u_full[vb] : &S.vp_empty[vb], use - 1);
                    if (!ok) break;
                    tc_fence_after();
                }
                if (C::VpOnS && fine && q == 0) {
                    ok = wait(&S.s_empty, i);  // the chunk's scores have been read
                    if (!ok) break;
                    tc_fence_after();
                }
                if (C::VpOnYe && q == 0 && vb) {
                    // The last strong chunk's Ye has been read. U(i − 2) is done, so the
                    // outputs of chunk i − 4 are: o_empty could be two phases behind, one of
                    // four barriers that strong chunks take in turn is one behind at most.
                    const int before = strongs;
                    strongs += (S.kind[(i - 1) % kSlots].strong != 0) +
                               (i > 1 && S.kind[(i - 2) % kSlots].strong != 0);
                    if (strongs > before) {
                        ok = wait(&S.ye_read[(strongs - 1) & 3], (strongs - 1) >> 2);
                        if (!ok) break;
                        tc_fence_after();
                    }
                }
                if (d0 < D) {
#pragma unroll
                    for (int e = 0; e < 3; ++e)
                        if (e < nvp)
                            tmem_st_frag(tmem + lanes + ((uint32_t)(16 * hh) << 16) +
                                             C::vp(vb, e) + 16 * th,
                                         part[e]);
                }
            }
            if (!ok) break;
            if (__any_sync(0xffffffffu, resets || holds_odd(odd))) {
                ok = odd_chunk(S, i, rev, fine, holds_odd(odd));
                if (!ok) break;
            }
            if (d0 < D) tmem_st_wait();
            tc_fence_before();
            arrive(&S.vp_full[vb]);
        }
    } else if (warp < 16) {
        // ---- state: lane d, columns half·D/2 .. ------------------------------------------
        constexpr int kH = D / 2;
        const int d = 32 * (warp & 3) + lane, half = (warp - 8) >> 2;
        const long long elems = (long long)a.dk * a.dv;
        float st[kH];
        {
            const float *src = nullptr;
            bool tr = false;
            if (kFull && order > 0) {
                src = a.seg_state + (bh * p.nseg + seg) * elems;
            } else if (kFull && a.h_init) {
                src = a.h_init + bh * elems;
                tr = a.h_init_t != 0;
            }
            const int step = tr ? 1 : a.dv, cols = src && d < a.dv ? a.dk - half * kH : 0;
            if (src) src += (tr ? d * a.dk : d) + half * kH * step;
#pragma unroll
            for (int k = 0; k < kH; ++k) st[k] = k < cols ? src[k * step] : 0.f;
        }
        for (int i = 0; i < n; ++i) {
            const int buf = i % kUBufs, use = i / kUBufs;
            if (kFull) {
                ok = (!kCentred || wait(&S.factors[i % kSlots], i / kSlots)) &&
                     wait(&S.st_empty, (i & 1) ^ 1);
                if (!ok) break;
                tc_fence_after();
                const float f = kCentred ? S.scale[i % kSlots] : 1.f;
                if (d < D) {
#pragma unroll
                    for (int k8 = 0; k8 < kH / 8; ++k8) {
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float x0 = st[8 * k8 + 2 * e], x1 = st[8 * k8 + 2 * e + 1];
                            if (kCentred) unpair(mul2(pair(x0, x1), pair(f, f)), x0, x1);
                            hi[e] = pack_bf16x2(x0, x1);
                            if (kBwd) lo[e] = pack_bf16x2(x0 - bf_lo(hi[e]), x1 - bf_hi(hi[e]));
                        }
                        const uint32_t at = tmem + lanes + C::St + half * (kH / 2) + 4 * k8;
                        tmem_st4(at, hi);
                        if (kBwd) tmem_st4(at + D / 2, lo);
                    }
                    tmem_st_wait();
                }
                tc_fence_before();
                arrive(&S.st_full);
            }
            ok = (kCentred || wait(&S.factors[i % kSlots], i / kSlots)) && wait(&S.u_full[buf], use);
            if (!ok) break;
            tc_fence_after();
            const float dec = S.decay[i % kSlots];
            if (d < D) {
#pragma unroll
                for (int k8 = 0; k8 < kH / 8; ++k8) {
                    float u[8];
                    tmem_ld8(tmem + lanes + C::U + buf * D + half * kH + 8 * k8, u);
                    if (dec == 0.f) {  // a reset: the old state does not count
#pragma unroll
                        for (int e = 0; e < 8; ++e) st[8 * k8 + e] = u[e];
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            st[8 * k8 + e] = fmaf(dec, st[8 * k8 + e], u[e]);
                    }
                }
            }
            tc_fence_before();
            arrive(&S.u_empty[buf]);
        }
        float *dst = nullptr;
        bool tr = false;
        if (!kFull || (p.nseg > 1 && order == 0)) {
            dst = a.seg_state + (bh * p.nseg + seg) * elems;
        } else if (a.h_final && order == p.nseg - 1) {
            dst = a.h_final + bh * elems;
            tr = a.h_final_t != 0;
        }
        if (dst) {
            const int step = tr ? 1 : a.dv, cols = d < a.dv ? a.dk - half * kH : 0;
            dst += (tr ? d * a.dk : d) + half * kH * step;
#pragma unroll
            for (int k = 0; k < kH; ++k)
                if (k < cols) dst[k * step] = st[k];
        }
    } else {
        if (kFull) {
            // ---- outputs: lane d, a column per token -----------------------------------------
            const int d0 = 32 * (warp & 3);
            const int tl = t - 512;  // 0 .. 127
            const CUtensorMap *my = &maps.m[a.map_y];
            const bool f32 = kBwd && a.y_f32;
            uint32_t syncs = 0;
            int strongs = 0;
            for (int i = 0; i < n; ++i) {
                const int s = i % kStages;
                const int t0 = chunk_of(i) * kC, nq = min(kC, len - t0);
                ok = wait(&S.factors[i % kSlots], i / kSlots) && wait(&S.o_full, i);
                if (!ok) break;
                tc_fence_after();
                if (tl == 0) bulk_wait_read<0>();  // the previous chunk's store has read the staging
                arrive(&S.o_sync);
                ok = wait(&S.o_sync, syncs++);
                if (!ok) break;
                if (d0 < D) {
                    // float32 rows (the heads' parts of a shared gradient) go straight to memory
                    const int nl = (int)min((long long)kC, p.seqlen - t0);
                    const long long y_row = (long long)p.heads * a.dv;
                    float *yf = f32 ? static_cast<float *>(a.y) +
                                          ((long long)b * p.seqlen + t0) * y_row + h * a.dv
                                    : nullptr;
                    const bf16 *dot = S.tile[s][Smem::kTiles - 1];
                    const uint32_t t_y = tmem + lanes + C::Yi, t_ye = tmem + lanes + C::Ye;
                    const int sl = i % kSlots;
                    const bool strong = S.kind[sl].strong != 0;
                    auto done = [&]() {  // the next chunk's products may come
                        tc_fence_before();
                        arrive(&S.o_empty);
                        if (C::VpOnYe && strong) arrive(&S.ye_read[strongs++ & 3]);
                    };
                    auto rows = [&](auto is_f32, auto is_dot) {
                        constexpr bool kF32 = decltype(is_f32)::value, kDot = decltype(is_dot)::value;
                        if (strong)
                            output_rows<kF32, kDot, true, true>(t_y, t_ye, S.out, dot, S.red[warp & 3],
                                                                S.rowf[sl], d0, yf, y_row, nl, a.dv,
                                                                done);
                        else
                            output_rows<kF32, kDot, kBwd, false>(t_y, t_ye, S.out, dot,
                                                                 S.red[warp & 3], S.rowf[sl], d0, yf,
                                                                 y_row, nl, a.dv, done);
                    };
                    if constexpr (kBwd) {
                        if (has_dot && f32)
                            rows(Yes(), Yes());
                        else if (has_dot)
                            rows(No(), Yes());
                        else if (f32)
                            rows(Yes(), No());
                        else
                            rows(No(), No());
                    } else {
                        rows(No(), No());
                    }
                } else {
                    arrive(&S.o_empty);
                }
                if (has_dot) arrive(&S.empty[s]);
                fence_proxy_async_smem();
                arrive(&S.o_sync);
                ok = wait(&S.o_sync, syncs++);
                if (!ok) break;
                if (warp == 16 && *reinterpret_cast<const uint32_t *>(S.kind[i % kSlots].odd))
                    odd_rows(S, p, a, b, h, len, t0, i % kSlots);
                if (tl == 0 && !f32) {
                    for (int c = 0; c < a.dv; c += 64)
                        tma_store_4d(my, S.out + (c >> 6) * (kC * 64), c, h, t0, b);
                    bulk_commit();
                }
                if (kBwd && has_dot && tl < nq) {
                    float sum = 0.f;
#pragma unroll
                    for (int w = 0; w < D / 32; ++w) sum += S.red[w][tl];
                    a.dot_out[bh * p.seqlen + t0 + tl] = sum;
                }
            }
            if (tl == 0) bulk_wait<0>();  // the last stores are out before the block ends
            // chunks without a token: zeros
            const long long row0 = (long long)b * p.seqlen;
            for (long long tok = (long long)c_live * kC; tok < min((long long)c_end * kC, p.seqlen);
                 ++tok) {
                const long long off = ((row0 + tok) * p.heads + h) * a.dv + tl;
                if (tl >= a.dv) break;
                if (f32)
                    static_cast<float *>(a.y)[off] = 0.f;
                else
                    static_cast<bf16 *>(a.y)[off] = __float2bfloat16_rn(0.f);
            }
        }
    }

    if (!ok && lane == 0) {  // the others stop waiting too
        *reinterpret_cast<volatile int *>(&S.abort) = 1;
        if (p.status) atomicCAS(p.status, 0, kStatusLinattnWait);
    }
    // The block's barrier takes a warp as arrived once one of its lanes is: a lane that
    // still issues or stores comes first.
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kWarpTma) tmem_dealloc(tmem, 512);
    if (!kFull && blockIdx.x == gridDim.x - 1) linattn_wait_for_first();
}

// ---- host ---------------------------------------------------------------------------
// [batch][seqlen][heads][dim] with `row` elements between tokens: boxes of 64
// tokens and 64 columns.
bool make_map(CUtensorMap *m, const void *base, long long batch, long long seqlen, int heads,
              int dim, long long row) {
    auto fn = tma_encode();
    if (!fn) return false;
    cuuint64_t gdim[4] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)seqlen, (cuuint64_t)batch};
    cuuint64_t gstride[3] = {(cuuint64_t)dim * 2, (cuuint64_t)row * 2,
                             (cuuint64_t)(seqlen * row) * 2};
    cuuint32_t box[4] = {64, 1, (cuuint32_t)kC, 1};
    cuuint32_t estride[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), gdim, gstride, box,
              estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kBwd, bool kFine>
cudaError_t launch(const LinattnParams &p, const TcMaps &maps, cudaStream_t stream) {
    const int smem = (int)sizeof(TcSmem<D, kBwd, true>) + 1024;
    const int smem_own = (int)sizeof(TcSmem<D, kBwd, false>) + 1024;
    static_assert(sizeof(TcSmem<D, kBwd, true>) + 1024 <= 232448, "shared memory");
    auto full = linattn_tc_kernel<D, kBwd, true, kFine>;
    auto state = linattn_tc_kernel<D, kBwd, false, kFine>;
    cudaError_t e = cudaFuncSetAttribute(full, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(state, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_own);
    if (e != cudaSuccess) return e;
    return linattn_launch(full, state, kThr, smem, smem_own, p.batch * p.heads * p.nsweeps, p,
                          stream, maps);
}

}  // namespace

bool linattn_tc_rows(const void *ptr, long long row, int dim, long long seqlen) {
    return dim % 8 == 0 && row % 8 == 0 && (reinterpret_cast<uintptr_t>(ptr) & 15) == 0 &&
           seqlen < (1ll << 30) && seqlen * row < (1ll << 38);
}

cudaError_t launch_linattn_tc(const LinattnParams &params, cudaStream_t stream) {
    LinattnParams p = params;
    TcMaps maps{};
    int n = 0;
    // one map per distinct operand
    struct Key {
        const void *ptr;
        long long row;
        int dim, heads;
    } keys[kMaps];
    auto operand = [&](const void *ptr, long long row, int dim, int group) -> int {
        const int heads = p.heads / group;
        for (int i = 0; i < n; ++i)
            if (keys[i].ptr == ptr && keys[i].row == row && keys[i].dim == dim &&
                keys[i].heads == heads)
                return i;
        if (n >= kMaps || !make_map(&maps.m[n], ptr, p.batch, p.seqlen, heads, dim, row))
            return -1;
        keys[n] = Key{ptr, row, dim, heads};
        return n++;
    };
    int most = 0;
    for (int s = 0; s < p.nsweeps; ++s) {
        SweepArgs &a = p.sweep[s];
        a.map[0] = operand(a.q, a.q_row, a.dk, a.q_group);
        a.map[1] = operand(a.k, a.k_row, a.dk, a.k_group);
        a.map[2] = operand(a.v, a.v_row, a.dv, a.v_group);
        a.map[3] = a.dot ? operand(a.dot, a.dot_row, a.dv, a.dot_group) : 0;
        if (a.map[0] < 0 || a.map[1] < 0 || a.map[2] < 0 || a.map[3] < 0) return cudaErrorInvalidValue;
        most = std::max(most, std::max(a.dk, a.dv));
    }
    for (int s = 0; s < p.nsweeps; ++s) {
        SweepArgs &a = p.sweep[s];
        if (a.y_f32) continue;  // stored without TMA
        if (n >= kMaps || !make_map(&maps.m[n], a.y, p.batch, p.seqlen, p.heads, a.dv,
                                    (long long)p.heads * a.dv))
            return cudaErrorInvalidValue;
        keys[n] = Key{nullptr, 0, 0, 0};
        a.map_y = n++;
    }
    if (p.nsweeps == 1)
        return most <= 64 ? launch<64, false, false>(p, maps, stream)
                          : launch<128, false, false>(p, maps, stream);
    bool fine = false;
    for (int i = 0; i < p.nsweeps; ++i) fine = fine || p.sweep[i].fine_state;
    if (fine)
        return most <= 64 ? launch<64, true, true>(p, maps, stream)
                          : launch<128, true, true>(p, maps, stream);
    return most <= 64 ? launch<64, true, false>(p, maps, stream)
                      : launch<128, true, false>(p, maps, stream);
}

}  // namespace selscan
