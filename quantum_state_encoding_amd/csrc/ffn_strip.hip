// Products of few rows: A B^T (and the gated block) for m up to 32.
//
// The rows of B are read once and bound the time, so a workgroup takes 16 of
// them (16 of each projection) and all of A, its waves take the 128-byte
// steps of k in turn, straight from memory into the matrix instructions'
// registers, and one sum over the waves in LDS, in a fixed order, joins them.
//
// Memory bounds it, for one token the time to start too: e4m3 m 1 n 4096 k
// 16384 takes 13.4 us (5.0 TB/s; a large copy reaches 5.15), gated bf16 m 8
// n 16384 k 4096 47 us (5.7 TB/s: reads alone are faster than a copy).
#include <hip/hip_runtime.h>

#include "ffn_strip.h"

namespace qse {
namespace {

template <int TYPE, int MT, int W, int U, int EP, int SM, bool ODD = false>
hipError_t run(const ProductArgs& p, hipStream_t stream)
{
    constexpr int P = EP == kEpStore ? 1 : 2;
    constexpr size_t kLds = (size_t)W * P * MT * 4 * 64 * 4;
    static_assert(kLds <= 65536, "dynamic LDS without an attribute");
    hipLaunchKernelGGL((strip_kernel<TYPE, MT, W, U, EP, SM, ODD>), dim3((unsigned)((p.n + 15) / 16)),
                       dim3(64 * W), kLds, stream, p);
    return hipGetLastError();
}

// Waves and steps in flight: sixteen waves pay for a long k alone, from 8192 on,
// where every wave has its four steps (microseconds in a graph with eight and
// sixteen, e4m3, m 1, cold weights: n 4096 k 4096 6.1 and 6.3, 8192 10.0 and 8.9,
// 12288 13.8 and 13.3, 16384 18.8 and 16.6; n 8192 9.2 and 10.9, 15.9 and 15.4,
// 23.3 and 24.3, 32.7 and 30.1; f16 results alike), and only where their four
// steps fit 128 registers: not with a scale for each row of B (22 spill).
template <int TYPE, int EP, int SM>
hipError_t pick(const ProductArgs& p, hipStream_t stream)
{
    if constexpr (SM == 0) {
        const uintptr_t any = (uintptr_t)p.a | (uintptr_t)p.b0 | (uintptr_t)p.b1 |
                              (uintptr_t)p.lda | (uintptr_t)p.ldb0 | (uintptr_t)p.ldb1;
        if (any & 3)
            return p.m > 16 ? run<TYPE, 2, 8, 2, EP, SM, true>(p, stream)
                            : run<TYPE, 1, 8, 4, EP, SM, true>(p, stream);
    }
    if (p.m > 16)
        return run<TYPE, 2, 8, 2, EP, SM>(p, stream);
    if constexpr (EP == kEpStore && SM == 1) {
        if (p.kbytes >= 64 * kStep)
            return run<TYPE, 1, 16, 4, EP, SM>(p, stream);
    }
    return run<TYPE, 1, 8, 4, EP, SM>(p, stream);
}

}  // namespace

hipError_t launch_strip(const ProductArgs& p, int type, int ep, bool row_scales,
                        hipStream_t stream)
{
    if (type == kTE4m3 && p.ctype != kTBf16) {
        if (ep == kEpGate)
            return pick<kTE4m3Exact, kEpGate, 1>(p, stream);
        return row_scales ? pick<kTE4m3Exact, kEpStore, 2>(p, stream)
                          : pick<kTE4m3Exact, kEpStore, 1>(p, stream);
    }
    if (type == kTE4m3) {
        if (ep == kEpGate)
            return pick<kTE4m3, kEpGate, 1>(p, stream);
        return row_scales ? pick<kTE4m3, kEpStore, 2>(p, stream)
                          : pick<kTE4m3, kEpStore, 1>(p, stream);
    }
    if (type == kTBf16)
        return pick<kTBf16, kEpGate, 0>(p, stream);
    return pick<kTF16, kEpGate, 0>(p, stream);
}

}  // namespace qse
