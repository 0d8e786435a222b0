// C ABI of the feed-forward operators (include/fwt_ffn.h): argument checks
// and the choice of kernels.
#include "../../include/fwt_ffn.h"

#include <hip/hip_runtime_api.h>

#include "ffn_internal.h"
#include "fwt_internal.h"

using qse::ProductArgs;
using qse::RotateArgs;

namespace {

int64_t size_of(int type)
{
    return type == FWT_FP32 ? 4 : type == FWT_E4M3 ? 1 : 2;
}

bool is16(int type) { return type == FWT_BF16 || type == FWT_F16; }

bool is_out(int type) { return is16(type) || type == FWT_FP32; }

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
bool too_many(int64_t m, int64_t n)
{
    return ((m + 127) / 128) * ((n + 63) / 64) >= qse::kFfnMaxTiles;
}

// The array must have a sane stride, ...
int check_stride(const Array& a)
{
    if (!a.p || a.ld < a.cols)
        return FWT_EINVAL;
    if (a.ld > ((int64_t)1 << 40) || (a.rows > 1 && a.ld > INT64_MAX / 8 / a.rows))
        return FWT_EINVAL;
    return (uintptr_t)a.p & (uintptr_t)(a.size - 1) ? FWT_EALIGN : FWT_OK;
}

// ... and lie in one device allocation.
int check_memory(const Array& a)
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

bool overlap(const Array& a, const Array& b)
{
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return x < y + b.span() && y < x + a.span();
}

// Every array's stride, what is written against all others, the memory; then
// the stream.  (size 0: an array that this call does not have)
template <int N>
int check_call(const Array (&arrays)[N], hipStream_t stream)
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

bool dims_ok(int64_t m, int64_t n, int64_t k)
{
    return m >= 0 && n >= 0 && k >= 1 && m <= kMaxDim && n <= kMaxDim && k <= kMaxDim;
}

int64_t blocks(int64_t k) { return (k + qse::kFfnBlock - 1) / qse::kFfnBlock; }

bool aligned16(const void* p, int64_t stride_bytes)
{
    return (((uintptr_t)p | (uintptr_t)stride_bytes) & 15u) == 0;
}

int status(hipError_t e) { return e == hipSuccess ? FWT_OK : qse::hip_status(e); }

constexpr Array kNone{nullptr, 0, 0, 0, 0, false};

// 16-bit elements of a row padded to whole 16-byte chunks.
int64_t pad8(int64_t n) { return (n + 7) & ~(int64_t)7; }

// Scratch that a product's shares of a long contraction need.
size_t shares_of(int64_t m, int64_t n, int64_t k, int type, int ctype, int epilogue, bool row,
                 int parts = 1)
{
    ProductArgs p{};
    p.m = m;
    p.n = n;
    p.kbytes = k * size_of(type);
    p.ctype = ctype;
    p.parts = parts;
    return qse::product_workspace(p, type, epilogue, row);
}

// The backward pass's scratch: dg beside du, m rows of 2 pad8(n) 16-bit
// elements, behind it their range, and the shares of one product at a time.
size_t backward_range(int64_t m, int64_t n)
{
    return ((size_t)m * 4 * (size_t)pad8(n) + 255) & ~(size_t)255;
}
size_t backward_sums(int64_t m, int64_t n) { return backward_range(m, n) + 256; }
static_assert(sizeof(qse::GradRange) <= 256, "behind it the shares, aligned");
size_t backward_scratch(int64_t m, int64_t n, int64_t k)
{
    size_t most = shares_of(m, n, k, FWT_BF16, FWT_BF16, qse::kEpGateGrad, false);
    const size_t dx = shares_of(m, k, n, FWT_BF16, FWT_BF16, qse::kEpStore, false, 2);
    const size_t dw = shares_of(2 * pad8(n), k, m, FWT_BF16, FWT_BF16, qse::kEpStoreT, false);
    most = most > dx ? most : dx;
    return backward_sums(m, n) + (most > dw ? most : dw);
}

}  // namespace

extern "C" {

int fwt_rotate_quantize_workspace(int64_t m, int64_t k, int bits, fwt_scales scales,
                                  int transposed, size_t* bytes)
{
    if (!bytes || !dims_ok(m, 0, k) || bits < 0 ||
        bits > (transposed ? qse::kFfnMaxBitsT : qse::kFfnMaxBits) ||
        (scales != FWT_SCALES_ROW && scales != FWT_SCALES_TILE))
        return FWT_EINVAL;
    *bytes = qse::rotate_workspace(m, k, bits, scales == FWT_SCALES_TILE, transposed != 0);
    return FWT_OK;
}

int fwt_rotate_quantize(const void* x, fwt_ffn_dtype dtype, int64_t m, int64_t k, int64_t ldx,
                        int transposed, int bits, fwt_scales scales, void* codes,
                        int64_t ldcodes, float* s, void* ws, size_t ws_bytes, hipStream_t stream)
{
    size_t need = 0;
    const int rc0 = fwt_rotate_quantize_workspace(m, k, bits, scales, transposed, &need);
    if (rc0 != FWT_OK)
        return rc0;
    if (!is_out(dtype) || (k & (((int64_t)1 << bits) - 1)))
        return FWT_EINVAL;
    if (m == 0)
        return FWT_OK;
    const bool tile = scales == FWT_SCALES_TILE;
    if (!x || !codes || !s || (need && (!ws || ws_bytes < need)))
        return FWT_EINVAL;
    if (!aligned16(codes, ldcodes) || (need && !aligned16(ws, 0)))
        return FWT_EALIGN;
    // threads of a launch: 8 a block, or 1024 for 128 rows of one
    if (m * blocks(k) >= ((int64_t)1 << 29) ||
        ((tile || transposed) && (blocks(m) > 65535 || blocks(k) >= ((int64_t)1 << 22))))
        return FWT_EUNSUPPORTED;
    const Array arrays[] = {
        {x, transposed ? k : m, transposed ? m : k, ldx, size_of(dtype), false},
        {codes, m, (k + 15) & ~(int64_t)15, ldcodes, 1, true},
        {s, blocks(k), tile ? blocks(m) : m, tile ? blocks(m) : m, 4, true},
        need ? Array{ws, 1, (int64_t)need, (int64_t)need, 1, true} : kNone,
    };
    const int rc = check_call(arrays, stream);
    if (rc != FWT_OK)
        return rc;
    RotateArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.m = m;
    a.k = k;
    a.bits = bits;
    a.q = (uint8_t*)codes;
    a.ldq = ldcodes;
    a.s = s;
    a.amax = (float*)ws;
    return status(qse::launch_rotate(a, (int)dtype, tile, transposed != 0, stream));
}

int fwt_scaled_matmul_workspace(int64_t m, int64_t n, int64_t k, fwt_scales b_kind,
                                fwt_ffn_dtype ctype, size_t* bytes)
{
    if (!bytes || !dims_ok(m, n, k) || !is_out(ctype) ||
        (b_kind != FWT_SCALES_ROW && b_kind != FWT_SCALES_TILE))
        return FWT_EINVAL;
    *bytes = m == 0 || n == 0 ? 0
                              : shares_of(m, n, k, FWT_E4M3, ctype, qse::kEpStore,
                                          b_kind == FWT_SCALES_ROW);
    return FWT_OK;
}

int fwt_scaled_matmul(const void* a, int64_t lda, const float* a_scales, const void* b,
                      int64_t ldb, const float* b_scales, fwt_scales b_kind, int64_t m,
                      int64_t n, int64_t k, void* c, fwt_ffn_dtype ctype, int64_t ldc, void* ws,
                      size_t ws_bytes, hipStream_t stream)
{
    size_t need = 0;
    const int rc0 = fwt_scaled_matmul_workspace(m, n, k, b_kind, ctype, &need);
    if (rc0 != FWT_OK)
        return rc0;
    if (m == 0 || n == 0)
        return FWT_OK;
    if (!ws)
        need = 0;
    if (ws_bytes < need)
        return FWT_EINVAL;
    if (need && !aligned16(ws, 0))
        return FWT_EALIGN;
    if (!a || !b || !c || !a_scales || !b_scales)
        return FWT_EINVAL;
    if (!aligned16(a, lda) || !aligned16(b, ldb))
        return FWT_EALIGN;
    if (lda >= qse::kFfnMaxStride || ldb >= qse::kFfnMaxStride || too_many(m, n))
        return FWT_EUNSUPPORTED;
    const int64_t sbn = b_kind == FWT_SCALES_ROW ? n : blocks(n);
    const Array arrays[] = {
        {a, m, k, lda, 1, false},
        {b, n, k, ldb, 1, false},
        {a_scales, blocks(k), m, m, 4, false},
        {b_scales, blocks(k), sbn, sbn, 4, false},
        {c, m, n, ldc, size_of(ctype), true},
        need ? Array{ws, 1, (int64_t)need, (int64_t)need, 1, true} : kNone,
    };
    const int rc = check_call(arrays, stream);
    if (rc != FWT_OK)
        return rc;
    ProductArgs p{};
    p.a = a;
    p.b0 = b;
    p.lda = lda;
    p.ldb0 = ldb;
    p.m = m;
    p.n = n;
    p.kbytes = k;
    p.parts = 1;
    p.sa = a_scales;
    p.sb0 = b_scales;
    p.sb_n = sbn;
    p.c = c;
    p.ldc = ldc;
    p.ctype = (int)ctype;
    p.may_split = need != 0;
    p.partial = ws;
    return status(qse::launch_product(p, FWT_E4M3, qse::kEpStore, b_kind == FWT_SCALES_ROW, stream));
}

int fwt_gated_ffn_workspace(fwt_ffn_dtype dtype, int64_t m, int64_t n, int64_t k,
                            fwt_ffn_dtype htype, size_t* bytes)
{
    const bool f8 = dtype == FWT_E4M3;
    if (!bytes || !dims_ok(m, n, k) || (!f8 && !is16(dtype)) ||
        (f8 ? !is_out(htype) : htype != dtype))
        return FWT_EINVAL;
    *bytes = m == 0 || n == 0 ? 0 : shares_of(m, n, k, dtype, htype, qse::kEpGate, false);
    return FWT_OK;
}

int fwt_gated_ffn(const void* x, int64_t ldx, const float* x_scales, const void* gate,
                  int64_t ldgate, const float* gate_scales, const void* up, int64_t ldup,
                  const float* up_scales, fwt_ffn_dtype dtype, int64_t m, int64_t n, int64_t k,
                  fwt_activation act, void* h, fwt_ffn_dtype htype, int64_t ldh, void* ws,
                  size_t ws_bytes, hipStream_t stream)
{
    const bool f8 = dtype == FWT_E4M3;
    size_t need = 0;
    const int rc0 = fwt_gated_ffn_workspace(dtype, m, n, k, htype, &need);
    if (rc0 != FWT_OK)
        return rc0;
    if (act != FWT_SILU && act != FWT_GELU)
        return FWT_EINVAL;
    if (m == 0 || n == 0)
        return FWT_OK;
    if (!ws)
        need = 0;
    if (ws_bytes < need)
        return FWT_EINVAL;
    if (need && !aligned16(ws, 0))
        return FWT_EALIGN;
    if (!x || !gate || !up || !h || f8 != (x_scales != nullptr) ||
        f8 != (gate_scales != nullptr) || f8 != (up_scales != nullptr))
        return FWT_EINVAL;
    const int64_t sz = size_of(dtype);
    if (f8 && (!aligned16(x, ldx) || !aligned16(gate, ldgate) || !aligned16(up, ldup)))
        return FWT_EALIGN;
    if (ldx * sz >= qse::kFfnMaxStride || ldgate * sz >= qse::kFfnMaxStride ||
        ldup * sz >= qse::kFfnMaxStride || too_many(m, n))
        return FWT_EUNSUPPORTED;
    const Array arrays[] = {
        {x, m, k, ldx, sz, false},
        {gate, n, k, ldgate, sz, false},
        {up, n, k, ldup, sz, false},
        {h, m, n, ldh, size_of(htype), true},
        f8 ? Array{x_scales, blocks(k), m, m, 4, false} : kNone,
        f8 ? Array{gate_scales, blocks(k), blocks(n), blocks(n), 4, false} : kNone,
        f8 ? Array{up_scales, blocks(k), blocks(n), blocks(n), 4, false} : kNone,
        need ? Array{ws, 1, (int64_t)need, (int64_t)need, 1, true} : kNone,
    };
    const int rc = check_call(arrays, stream);
    if (rc != FWT_OK)
        return rc;
    ProductArgs p{};
    p.a = x;
    p.b0 = gate;
    p.b1 = up;
    p.lda = ldx * sz;
    p.ldb0 = ldgate * sz;
    p.ldb1 = ldup * sz;
    p.m = m;
    p.n = n;
    p.kbytes = k * sz;
    p.sa = x_scales;
    p.sb0 = gate_scales;
    p.sb1 = up_scales;
    p.sb_n = blocks(n);
    p.c = h;
    p.ldc = ldh;
    p.ctype = (int)htype;
    p.act = (int)act;
    p.may_split = need != 0;
    p.partial = ws;
    return status(qse::launch_product(p, (int)dtype, qse::kEpGate, false, stream));
}

int fwt_gated_ffn_backward_workspace(int64_t m, int64_t n, int64_t k, size_t* bytes)
{
    if (!bytes || !dims_ok(m, n, k))
        return FWT_EINVAL;
    *bytes = m == 0 || n == 0 ? 0 : backward_scratch(m, n, k);
    return FWT_OK;
}

int fwt_gated_ffn_backward(const void* x, int64_t ldx, const void* gate, int64_t ldgate,
                           const void* up, int64_t ldup, const void* dh, int64_t lddh,
                           fwt_ffn_dtype dtype, int64_t m, int64_t n, int64_t k,
                           fwt_activation act, void* dx, int64_t lddx, void* dgate,
                           int64_t lddgate, void* dup, int64_t lddup, void* ws, size_t ws_bytes,
                           hipStream_t stream)
{
    size_t need = 0;
    const int rc0 = fwt_gated_ffn_backward_workspace(m, n, k, &need);
    if (rc0 != FWT_OK)
        return rc0;
    if (!is16(dtype) || (act != FWT_SILU && act != FWT_GELU))
        return FWT_EINVAL;
    if (m == 0 && n == 0)
        return FWT_OK;
    const bool sums = m != 0 && n != 0;   // otherwise what is written is zeros
    if (sums && (!x || !gate || !up || !dh || !ws || ws_bytes < need))
        return FWT_EINVAL;
    if ((m && !dx) || (n && (!dgate || !dup)))
        return FWT_EINVAL;
    if (sums && !aligned16(ws, 0))
        return FWT_EALIGN;
    if (ldx * 2 >= qse::kFfnMaxStride || ldgate * 2 >= qse::kFfnMaxStride ||
        ldup * 2 >= qse::kFfnMaxStride || pad8(n) * 4 >= qse::kFfnMaxStride ||
        too_many(m, n) || too_many(m, k) || too_many(2 * pad8(n), k))
        return FWT_EUNSUPPORTED;
    const Array arrays[] = {
        sums ? Array{x, m, k, ldx, 2, false} : kNone,
        sums ? Array{gate, n, k, ldgate, 2, false} : kNone,
        sums ? Array{up, n, k, ldup, 2, false} : kNone,
        sums ? Array{dh, m, n, lddh, 2, false} : kNone,
        m ? Array{dx, m, k, lddx, 2, true} : kNone,
        n ? Array{dgate, n, k, lddgate, 2, true} : kNone,
        n ? Array{dup, n, k, lddup, 2, true} : kNone,
        sums ? Array{ws, 1, (int64_t)need, (int64_t)need, 1, true} : kNone,
    };
    const int rc = check_call(arrays, stream);
    if (rc != FWT_OK)
        return rc;
    if (!sums) {
        hipError_t e = m ? qse::launch_zero16(dx, lddx, m, k, stream)
                         : qse::launch_zero16(dgate, lddgate, n, k, stream);
        if (e == hipSuccess && n)
            e = qse::launch_zero16(dup, lddup, n, k, stream);
        return status(e);
    }
    // dg and du, from the two products
    const int64_t np = pad8(n);
    ProductArgs p{};
    p.a = x;
    p.b0 = gate;
    p.b1 = up;
    p.lda = ldx * 2;
    p.ldb0 = ldgate * 2;
    p.ldb1 = ldup * 2;
    p.m = m;
    p.n = n;
    p.kbytes = k * 2;
    p.c = ws;
    p.ldc = 2 * np;
    p.part_c = np;
    p.ctype = (int)dtype;
    p.dh = dh;
    p.lddh = lddh;
    p.act = (int)act;
    p.may_split = 1;
    p.partial = (char*)ws + backward_sums(m, n);
    hipError_t e = hipSuccess;
    if (dtype == FWT_F16) {
        p.range = (qse::GradRange*)((char*)ws + backward_range(m, n));
        e = qse::launch_zero16(p.range, 0, 1, sizeof(qse::GradRange) / 2, stream);
    }
    if (e == hipSuccess)
        e = qse::launch_product(p, (int)dtype, qse::kEpGateGrad, false, stream);
    if (e == hipSuccess && dtype == FWT_F16) {
        // once more with a factor, if they are out of range; otherwise the
        // launch ends at once (both launches: m 64 n 4096 k 1024 31.3 us
        // without, 34.9 with them; m 4096 n 8192 k 4096 1347 and 1349)
        p.again = 1;
        e = qse::launch_product(p, (int)dtype, qse::kEpGateGrad, false, stream);
    }
    if (e != hipSuccess)
        return status(e);
    // dx = dg gate + du up: the contraction runs over n of gate, then of up
    ProductArgs d{};
    d.a = ws;
    d.lda = 4 * np;
    d.b0 = gate;
    d.b1 = up;
    d.ldb0 = ldgate * 2;
    d.ldb1 = ldup * 2;
    d.m = m;
    d.n = k;
    d.kbytes = 2 * n;
    d.parts = 2;
    d.part_a = 2 * np;
    d.c = dx;
    d.ldc = lddx;
    d.ctype = (int)dtype;
    d.range = p.range;
    d.may_split = 1;
    d.partial = p.partial;
    e = qse::launch_product(d, (int)dtype, qse::kEpStore, false, stream);
    if (e != hipSuccess)
        return status(e);
    // [dgate; dup] = [dg du]^T x
    ProductArgs g{};
    g.a = ws;
    g.lda = 4 * np;
    g.b0 = x;
    g.ldb0 = ldx * 2;
    g.m = 2 * np;
    g.n = k;
    g.kbytes = 2 * m;
    g.c = dgate;
    g.c1 = dup;
    g.split = np;
    g.split_rows = n;
    g.ldc = lddgate;
    g.ldc1 = lddup;
    g.ctype = (int)dtype;
    g.range = p.range;
    g.may_split = 1;
    g.partial = p.partial;
    e = qse::launch_product(g, (int)dtype, qse::kEpStoreT, false, stream);
    return status(e);
}

}  // extern "C"
