// api_util.cuh -- argument checks shared by the C entry points: alignment,
// overlapping buffers, sizes, and the error bookkeeping behind
// SELSCAN_ERR_CUDA.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace selscan {

// Records the error for selscan_last_cuda_error and returns SELSCAN_ERR_CUDA.
int cuda_fail(cudaError_t e);

inline bool misaligned(const void *p, size_t a) {
    return p != nullptr && (reinterpret_cast<uintptr_t>(p) % a) != 0;
}

// Half-open byte ranges [a, a + na) and [b, b + nb) intersect.
inline bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
    if (a == nullptr || b == nullptr || na == 0 || nb == 0) return false;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a);
    const uintptr_t pb = reinterpret_cast<uintptr_t>(b);
    return pa < pb + nb && pb < pa + na;
}

// a · b ≤ limit for non-negative a, b, without overflow.
inline bool mul_le(int64_t a, int64_t b, int64_t limit) {
    return a == 0 || b <= limit / a;
}

constexpr int64_t kMaxElems = (int64_t)1 << 40;  // per tensor

inline int sm_count() {
    static int cached[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 148;
    if (dev < 64 && cached[dev] > 0) return cached[dev];
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        sms <= 0)
        sms = 148;
    if (dev < 64) cached[dev] = sms;
    return sms;
}

inline int64_t round_up(int64_t a, int64_t m) { return (a + m - 1) / m * m; }

struct Span {
    const void *p;
    size_t n;
};

inline bool any_overlap(const Span *outs, int no, const Span *ins, int ni) {
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni; ++j)
            if (overlaps(outs[i].p, outs[i].n, ins[j].p, ins[j].n)) return true;
        for (int j = i + 1; j < no; ++j)
            if (overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return true;
    }
    return false;
}

}  // namespace selscan
