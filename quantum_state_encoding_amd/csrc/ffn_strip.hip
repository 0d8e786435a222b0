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

#include "ffn_device.h"

namespace qse {
namespace {

constexpr int kStep = 128;   // bytes of k per step

// Sixteen bytes at `at` of a row of len bytes, 0 past its end.  e4m3 rows are
// 16-byte aligned, so a chunk that holds a byte of the row is in its page;
// those of 16-bit types are read from the row's last 16 bytes.
template <int TYPE>
__device__ __forceinline__ v4i load16_tail(const char* row, int64_t at, int64_t len)
{
    if constexpr (TYPE == kTBf16 || TYPE == kTF16) {
        if (len < 16)
            return chunk_of_short_row(row, at == 0 ? (int)len : 0);
        const int64_t from = at < len - 16 ? at : len - 16;
        const int by = (int)((uintptr_t)(row + from) & 2);
        return drop(moved(load_around(row + from), by), (int)(at - from));
    } else {
        v4i v = load16(row + (at < len ? at : (len - 1) & ~(int64_t)15));
        const int left = (int)(len - at);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int b = left - 4 * w;
            v[w] = b >= 4 ? v[w] : b <= 0 ? 0 : v[w] & ((1 << (8 * b)) - 1);
        }
        return v;
    }
}

// ODD: 16-bit rows at addresses that are not multiples of 4.
template <int TYPE, int MT, int W, int U, int EP, int SM, bool ODD>
__global__ __launch_bounds__(64 * W) void strip_kernel(const ProductArgs p)
{
    constexpr int P = EP == kEpStore ? 1 : 2;    // projections
    extern __shared__ __align__(16) unsigned char lds[];
    float* red = (float*)lds;                    // [W][P][MT][4][64]
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int q = lane >> 4, l16 = lane & 15;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int64_t nl = n0 + l16 < p.n ? n0 + l16 : p.n - 1;   // past the end: the last row
    const char* bp[P];
    bp[0] = (const char*)p.b0 + nl * p.ldb0 + q * 16;
    if constexpr (P == 2)
        bp[1] = (const char*)p.b1 + nl * p.ldb1 + q * 16;
    const char* ap[MT];
    int mr[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        mr[i] = i * 16 + l16 < p.m ? i * 16 + l16 : (int)p.m - 1;
        ap[i] = (const char*)p.a + mr[i] * p.lda + q * 16;
    }
    int64_t sbn[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int64_t n = n0 + q * 4 + r < p.n ? n0 + q * 4 + r : p.n - 1;
        sbn[r] = SM == 1 ? n / kFfnBlock : n;
    }
    v4f acc[P][MT];
#pragma unroll
    for (int j = 0; j < P; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i)
            acc[j][i] = v4f{0.f, 0.f, 0.f, 0.f};

    // A step: both operands and their scales; all loads of the steps in flight
    // are issued before the first is used.
    struct Step {
        v4i b[P][2], a[MT][2];
        unsigned blast[ODD ? P : 1][2], alast[ODD ? MT : 1][2];
        float sb[SM ? P : 1][SM == 2 ? 4 : 1], sa[SM ? MT : 1];
    };
    auto fetch = [](v4i& v, unsigned& last, const char* at) __attribute__((always_inline)) {
        if constexpr (ODD) {
            const Around a = load_around(at);
            v = a.w;
            last = a.last;
        } else {
            v = load16(at);
        }
    };
    auto load_scales = [&](Step& t, int64_t kt) __attribute__((always_inline)) {
        if constexpr (SM != 0) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
                t.sa[i] = p.sa[kt * p.m + mr[i]];
#pragma unroll
            for (int j = 0; j < P; ++j)
#pragma unroll
                for (int r = 0; r < (SM == 2 ? 4 : 1); ++r)
                    t.sb[j][r] = (j ? p.sb1 : p.sb0)[kt * p.sb_n + sbn[r]];
        }
    };
    auto add = [&](const Step& t) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < P; ++j)
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                if constexpr (SM == 0) {
                    acc[j][i] = matrix_step<TYPE>(t.b[j], t.a[i], acc[j][i]);
                } else {
                    const v4f v = matrix_step<TYPE>(t.b[j], t.a[i], v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        acc[j][i][r] = __builtin_fmaf(v[r], t.sa[i] * t.sb[j][SM == 2 ? r : 0],
                                                      acc[j][i][r]);
                }
            }
    };

    const int64_t full = p.kbytes / kStep;
    int64_t kt = wave;
    for (; kt + (U - 1) * W < full; kt += U * W) {
        Step t[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int j = 0; j < P; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    fetch(t[u].b[j][h], t[u].blast[ODD ? j : 0][h],
                          bp[j] + (kt + u * W) * kStep + h * 64);
            load_scales(t[u], kt + u * W);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    fetch(t[u].a[i][h], t[u].alast[ODD ? i : 0][h],
                          ap[i] + (kt + u * W) * kStep + h * 64);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if constexpr (ODD) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int j = 0; j < P; ++j)
                        t[u].b[j][h] = moved(Around{t[u].b[j][h], t[u].blast[j][h]},
                                             (int)(uintptr_t)bp[j] & 2);
#pragma unroll
                    for (int i = 0; i < MT; ++i)
                        t[u].a[i][h] = moved(Around{t[u].a[i][h], t[u].alast[i][h]},
                                             (int)(uintptr_t)ap[i] & 2);
                }
            }
            add(t[u]);
        }
    }
    for (; kt * kStep < p.kbytes; kt += W) {
        Step t;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < P; ++j)
                t.b[j][h] = load16_tail<TYPE>(bp[j] - q * 16, kt * kStep + h * 64 + q * 16, p.kbytes);
#pragma unroll
            for (int i = 0; i < MT; ++i)
                t.a[i][h] = load16_tail<TYPE>(ap[i] - q * 16, kt * kStep + h * 64 + q * 16, p.kbytes);
        }
        load_scales(t, kt);
        add(t);
    }

#pragma unroll
    for (int j = 0; j < P; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                red[(((wave * P + j) * MT + i) * 4 + r) * 64 + lane] = acc[j][i][r];
    __syncthreads();
    const bool bf = p.ctype == kTBf16;
    for (int t = threadIdx.x; t < MT * 256; t += 64 * W) {
        // results of one row of A side by side: n on the lowest bits
        const int nn = t & 15, mm = t >> 4;
        const int i = mm >> 4, at = (nn >> 2) * 16 + (mm & 15), r = nn & 3;
        float s[P];
#pragma unroll
        for (int j = 0; j < P; ++j) {
            s[j] = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w)
                s[j] += red[(((w * P + j) * MT + i) * 4 + r) * 64 + at];
        }
        const int64_t n = n0 + nn;
        if (mm >= p.m || n >= p.n)
            continue;
        float v = s[0];
        if constexpr (EP == kEpGate) {
            float d;
            if constexpr (TYPE == kTE4m3Exact)
                v = activation_exact(p.act, s[0]);
            else
                activation(p.act, s[0], v, d);
            v *= s[P - 1];
        }
        const int64_t o = mm * p.ldc + n;
        if (p.ctype == kTF32)
            ((float*)p.c)[o] = v;
        else
            ((unsigned short*)p.c)[o] = to16(v, bf);
    }
}

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
