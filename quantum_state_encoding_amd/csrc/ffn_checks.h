// Checks of arguments that the feed-forward entry points share (ffn_api.cpp,
// experts_api.cpp).  Internal.
#pragma once

#include <hip/hip_runtime_api.h>

#include "../../include/fwt_experts.h"
#include "ffn_internal.h"
#include "fwt_internal.h"

namespace {

inline int64_t size_of(int type)
{
    return type == FWT_FP32 ? 4 : type == FWT_E4M3 || type == FWT_INT8 ? 1 : 2;
}

inline bool is16(int type) { return type == FWT_BF16 || type == FWT_F16; }

inline bool is_out(int type) { return is16(type) || type == FWT_FP32; }

// A strided array in device memory: rows x cols elements of `size` bytes.
struct Array {
    const void* p;
    int64_t rows, cols, ld, size;
    bool written;
    // bytes from the first element to past the last
    size_t span() const
    {
        return rows <= 0 ? 0 : (size_t)((rows - 1) * ld + cols) * (size_t)size;
    }
};

constexpr int64_t kMaxDim = (int64_t)1 << 30;

// Whether a product has too many tiles of 128 x 64 for one launch (larger and
// smaller tiles are chosen where theirs fit).
inline bool too_many(int64_t m, int64_t n)
{
    return ((m + 127) / 128) * ((n + 63) / 64) >= qse::kFfnMaxTiles;
}

// The array must have a sane stride, ...
inline int check_stride(const Array& a)
{
    if (!a.p || a.ld < a.cols)
        return FWT_EINVAL;
    if (a.ld > ((int64_t)1 << 40) || (a.rows > 1 && a.ld > INT64_MAX / 8 / a.rows))
        return FWT_EINVAL;
    return (uintptr_t)a.p & (uintptr_t)(a.size - 1) ? FWT_EALIGN : FWT_OK;
}

// ... and lie in one device allocation.
inline int check_memory(const Array& a)
{
    hipDeviceptr_t base = nullptr;
    size_t size = 0;
    const hipError_t e = hipMemGetAddressRange(&base, &size, (hipDeviceptr_t)a.p);
    if (e != hipSuccess) {
        const int st = qse::hip_status(e);
        (void)hipGetLastError();
        return e == hipErrorNoDevice || e == hipErrorNotInitialized ||
                       e == hipErrorInsufficientDriver
                   ? st
                   : FWT_EINVAL;
    }
    const uintptr_t b = (uintptr_t)base, p = (uintptr_t)a.p;
    if (p < b || p - b > size || size - (p - b) < a.span())
        return FWT_EINVAL;
    return FWT_OK;
}

inline bool overlap(const Array& a, const Array& b)
{
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return x < y + b.span() && y < x + a.span();
}

// Every array's stride, what is written against all others, the memory; then
// the stream.  (size 0: an array that this call does not have)
template <int N>
inline int check_call(const Array (&arrays)[N], hipStream_t stream)
{
    for (const Array& a : arrays) {
        const int rc = a.size ? check_stride(a) : FWT_OK;
        if (rc != FWT_OK)
            return rc;
    }
    for (const Array& a : arrays)
        if (a.size && a.written)
            for (const Array& b : arrays)
                if (&a != &b && b.size && overlap(a, b))
                    return FWT_EINVAL;
    for (const Array& a : arrays) {
        const int rc = a.size ? check_memory(a) : FWT_OK;
        if (rc != FWT_OK)
            return rc;
    }
    if (stream) {
        int cur = 0;
        hipDevice_t sdev = 0;
        hipError_t e = hipGetDevice(&cur);
        if (e == hipSuccess)
            e = hipStreamGetDevice(stream, &sdev);
        if (e != hipSuccess)
            return qse::hip_status(e);
        if ((int)sdev != cur)
            return FWT_EINVAL;
    }
    return FWT_OK;
}

inline bool dims_ok(int64_t m, int64_t n, int64_t k)
{
    return m >= 0 && n >= 0 && k >= 1 && m <= kMaxDim && n <= kMaxDim && k <= kMaxDim;
}

inline int64_t blocks(int64_t k) { return (k + qse::kFfnBlock - 1) / qse::kFfnBlock; }

inline bool aligned16(const void* p, int64_t stride_bytes)
{
    return (((uintptr_t)p | (uintptr_t)stride_bytes) & 15u) == 0;
}

inline int status(hipError_t e) { return e == hipSuccess ? FWT_OK : qse::hip_status(e); }

constexpr Array kNone{nullptr, 0, 0, 0, 0, false};

}  // namespace
