// C ABI of the 8-bit integer products and of the products grouped by expert
// (include/fwt_experts.h): argument checks and the choice of kernels.
#include "../../include/fwt_experts.h"

#include <hip/hip_runtime_api.h>

#include "ffn_checks.h"
#include "ffn_internal.h"
#include "fwt_internal.h"

using qse::GroupArgs;
using qse::ProductArgs;

static_assert(FWT_INT8 == (int)qse::kTI8, "types");

namespace {

constexpr int64_t kMaxInt8K = (int64_t)1 << 17;      // sums of 128^2 stay in 32 bits
constexpr int64_t kMaxExperts = (int64_t)1 << 16;

// Row tiles of 128 that m rows of so many groups may have, and whether those
// of 64 columns are too many for a launch.
bool too_many_grouped(int64_t m, int64_t n, int64_t groups)
{
    const int64_t r = groups < m ? groups : m;
    const int64_t tn = (n + 63) / 64;
    return (m + r * 127) / 128 > qse::kFfnMaxTiles / tn ||
           (m + r * 127) / 128 * tn >= qse::kFfnMaxTiles;
}

// An array for each expert, rows x cols: a sane row stride, ...
bool rows_ok(int64_t rows, int64_t ld, int64_t cols)
{
    return ld >= cols && ld <= ((int64_t)1 << 40) && ld <= INT64_MAX / 8 / rows;
}

// ... and all of them as one array with a row for each (check_call sees to the
// stride between experts).
Array experts_array(const void* p, int64_t experts, int64_t rows, int64_t ld, int64_t cols,
                    int64_t stride, int64_t size, bool written)
{
    return Array{p, experts, (rows - 1) * ld + cols,
                 experts > 1 ? stride : (rows - 1) * ld + cols, size, written};
}

GroupArgs groups(const int32_t* ends, int64_t experts, int64_t m)
{
    GroupArgs g{};
    g.ends = ends;
    g.experts = (int)experts;
    g.rows = m;
    return g;
}

ProductArgs sizes(int64_t m, int64_t n, int64_t kbytes)
{
    ProductArgs p{};
    p.m = m;
    p.n = n;
    p.kbytes = kbytes;
    p.parts = 1;
    return p;
}

// Tiles of 128 x 64 of the gradients of all experts' weights.
bool too_many_weights(int64_t experts, int64_t n, int64_t k)
{
    const int64_t tiles = ((n + 127) / 128) * ((k + 63) / 64);
    return too_many(n, k) || tiles * experts >= qse::kFfnMaxTiles;
}

// Copies of operands into rows of multiples of 16 bytes, in scratch behind the sums:
// where those rows' products and the copies take less time.  Rows of fewer than 64
// elements or of 2^20 and more, and operands of more than 1 GiB together, are left as
// they are, and those of calls of less than 60 us, where the model is too coarse for
// what there is to gain (gradients, bf16: m 2523 e 3 n 846 k 627 38.7 us, 41.9 with
// copies; m 8000 e 4 n 2001 k 2001 276 and 215; m 16000 e 8 n 4001 k 4095, forward, 731
// and 649).
constexpr int64_t kMinCopied = 64, kMaxCopied = (int64_t)1 << 20, kMaxCopies = (int64_t)1 << 30;

bool worth_copies(int64_t bytes, double now, double without)
{
    return without > 60.0 && now + qse::row_copies_cost(bytes) < without;
}

bool may_copy(int64_t cols) { return cols >= kMinCopied && cols < kMaxCopied; }

size_t aligned256(size_t n) { return (n + 255) & ~(size_t)255; }

// Bytes of a copy, 0 for rows that need none, more than kMaxCopies for any more than that.
int64_t copy_bytes(int64_t rows, int64_t cols)
{
    if (cols % 8 == 0)
        return 0;
    const int64_t row = qse::padded_row(cols);
    return rows > kMaxCopies / row ? kMaxCopies + 1 : rows * row;
}

// How an operand lies: 0 at multiples of 16 bytes, 1 of 4, 2 others.
int level_of(const void* p, int64_t ld, int64_t stride)
{
    const uintptr_t a = (uintptr_t)p | 2 * (uintptr_t)ld | 2 * (uintptr_t)stride;
    return (a & 15) == 0 ? 0 : (a & 3) == 0 ? 1 : 2;
}

int larger(int a, int b) { return a > b ? a : b; }

// dx and dw of the sizes, at these levels.
double backward_cost(int64_t experts, int64_t m, int64_t n, int64_t k, int dx, int dw)
{
    GroupArgs g = groups(nullptr, experts, m);
    double cost = 0;
    if (dx >= 0) {
        ProductArgs p = sizes(m, k, 2 * n);
        p.may_split = 1;
        cost += qse::grouped_cost(p, g, true, dx);
    }
    if (dw >= 0) {
        ProductArgs p = sizes(n, k, 2 * m);
        p.may_split = 1;
        cost += qse::grouped_t_cost(p, g, dw);
    }
    return cost;
}
double forward_cost(int64_t experts, int64_t m, int64_t n, int64_t k, int level)
{
    ProductArgs p = sizes(m, n, 2 * k);
    p.may_split = 1;
    return qse::grouped_cost(p, groups(nullptr, experts, m), false, level);
}

// Bytes of scratch for copies, 0 where none are made.
int64_t forward_copies(int64_t experts, int64_t m, int64_t n, int64_t k)
{
    const int64_t bytes = copy_bytes(m, k) + copy_bytes(experts * n, k);
    return may_copy(k) && bytes && bytes <= kMaxCopies &&
                   worth_copies(bytes, forward_cost(experts, m, n, k, 0),
                                forward_cost(experts, m, n, k, 2))
               ? bytes
               : 0;
}
int64_t backward_copies(int64_t experts, int64_t m, int64_t n, int64_t k)
{
    const int64_t bytes = copy_bytes(m + experts * n, k) + copy_bytes(m, n);
    return may_copy(k) && may_copy(n) && bytes && bytes <= kMaxCopies &&
                   worth_copies(bytes, backward_cost(experts, m, n, k, 0, 0),
                                backward_cost(experts, m, n, k, 2, 2))
               ? bytes
               : 0;
}

// The copies of a call.
struct Copies {
    qse::RowCopy at[3];
    int count = 0;
    int64_t bytes = 0;
    bool room = true;        // for each that is wanted
    // a misaligned operand of `rows` (`each` of an expert) by cols: its number, or -1
    int want(int level, int64_t rows, int64_t cols, int64_t each, const void* src, int64_t ld,
             int64_t stride)
    {
        if (level == 0)
            return -1;
        room = room && copy_bytes(rows, cols);
        at[count] = qse::RowCopy{src,  nullptr, (int64_t)(2 * (uint64_t)ld), (int64_t)(2 * (uint64_t)stride),
                                 rows, cols,    each};
        bytes += copy_bytes(rows, cols);
        return count++;
    }
    void none()
    {
        count = 0;
        bytes = 0;
    }
    // that operand's copy, its rows' and its experts' strides in elements
    void use(int i, const void*& src, int64_t& ld, int64_t& stride) const
    {
        if (i < 0 || !count)
            return;
        src = at[i].dst;
        ld = qse::padded_row(at[i].cols) / 2;
        stride = at[i].each * ld;
    }
    hipError_t make(void* ws, const GroupArgs& g, hipStream_t stream)
    {
        char* next = (char*)ws;
        for (int i = 0; i < count; ++i) {
            at[i].dst = next;
            next += copy_bytes(at[i].rows, at[i].cols);
        }
        return qse::launch_row_copies(at, count, g, stream);
    }
};

// What of these operands is copied, if anything; stride_w 0 for one expert.
struct ForwardCopies : Copies {
    int x, w;
    ForwardCopies(const void* px, int64_t ldx, const void* pw, int64_t ldw, int64_t stride_w,
                  int64_t experts, int64_t m, int64_t n, int64_t k)
    {
        const int lx = level_of(px, ldx, 0), lw = level_of(pw, ldw, stride_w);
        x = want(lx, m, k, 0, px, ldx, 0);
        w = want(lw, experts * n, k, n, pw, ldw, stride_w);
        if (!count || !room || !forward_copies(experts, m, n, k) ||
            !worth_copies(bytes, forward_cost(experts, m, n, k, 0),
                          forward_cost(experts, m, n, k, larger(lx, lw))))
            none();
    }
};
struct BackwardCopies : Copies {
    int dy, x, w;
    BackwardCopies(const void* px, int64_t ldx, const void* pw, int64_t ldw, int64_t stride_w,
                   const void* pdy, int64_t lddy, int64_t experts, int64_t m, int64_t n, int64_t k,
                   bool rows, bool weights)
    {
        const int lx = weights ? level_of(px, ldx, 0) : 0;
        const int lw = rows ? level_of(pw, ldw, stride_w) : 0;
        const int ld = level_of(pdy, lddy, 0);
        dy = want(ld, m, n, 0, pdy, lddy, 0);
        x = want(lx, m, k, 0, px, ldx, 0);
        w = want(lw, experts * n, k, n, pw, ldw, stride_w);
        if (!count || !room || !backward_copies(experts, m, n, k) ||
            !worth_copies(bytes,
                          backward_cost(experts, m, n, k, rows ? 0 : -1, weights ? 0 : -1),
                          backward_cost(experts, m, n, k, rows ? larger(ld, lw) : -1,
                                        weights ? larger(ld, lx) : -1)))
            none();
    }
};

// Scratch: the sums, then the copies.
size_t with_copies(size_t sums, int64_t copies)
{
    return copies ? aligned256(sums) + copies : sums;
}

// Sums of the forward call; whether there is work that is not refused.
bool forward_runs(int64_t experts, int64_t m, int64_t n)
{
    return m != 0 && n != 0 && experts <= kMaxExperts && !too_many_grouped(m, n, experts + 1);
}
size_t forward_need(int dtype, int64_t experts, int64_t m, int64_t n, int64_t k)
{
    GroupArgs g = groups(nullptr, experts, m);
    g.zero_rest = 1;
    return qse::grouped_workspace(sizes(m, n, k * size_of(dtype)), g, dtype, false);
}

// dx = dy w_e (contraction over n) and dw_e = dy^T x (over the rows).
size_t backward_need(int64_t experts, int64_t m, int64_t n, int64_t k)
{
    GroupArgs g = groups(nullptr, experts, m);
    const size_t dw = qse::grouped_t_workspace(sizes(n, k, 2 * m), g, FWT_BF16);
    g.zero_rest = 1;
    const size_t dx = qse::grouped_workspace(sizes(m, k, 2 * n), g, FWT_BF16, true);
    return dx > dw ? dx : dw;
}
bool backward_runs(int64_t experts, int64_t m, int64_t n, int64_t k)
{
    return m != 0 && n != 0 && experts <= kMaxExperts && !too_many_grouped(m, k, experts + 1) &&
           !too_many_weights(experts, n, k);
}

}  // namespace

extern "C" {

int fwt_rotate_quantize_int8(const void* x, fwt_ffn_dtype dtype, int64_t m, int64_t k,
                             int64_t ldx, int bits, void* codes, int64_t ldcodes, float* s,
                             hipStream_t stream)
{
    if (!dims_ok(m, 0, k) || bits < 0 || bits > qse::kFfnMaxBits || !is_out(dtype) ||
        (k & (((int64_t)1 << bits) - 1)))
        return FWT_EINVAL;
    if (m == 0)
        return FWT_OK;
    if (!x || !codes || !s)
        return FWT_EINVAL;
    if (!aligned16(codes, ldcodes))
        return FWT_EALIGN;
    if (qse::quantize8_groups(m, k) >= qse::kFfnMaxTiles)
        return FWT_EUNSUPPORTED;
    const Array arrays[] = {
        {x, m, k, ldx, size_of(dtype), false},
        {codes, m, (k + 15) & ~(int64_t)15, ldcodes, 1, true},
        {s, 1, m, m, 4, true},
    };
    const int rc = check_call(arrays, stream);
    if (rc != FWT_OK)
        return rc;
    qse::Quantize8Args a{};
    a.x = x;
    a.ldx = ldx;
    a.m = m;
    a.k = k;
    a.bits = bits;
    a.q = (int8_t*)codes;
    a.ldq = ldcodes;
    a.s = s;
    return status(qse::launch_quantize8(a, (int)dtype, stream));
}

int fwt_int8_matmul_workspace(int64_t m, int64_t n, int64_t k, fwt_ffn_dtype ctype,
                              size_t* bytes)
{
    if (!bytes || !dims_ok(m, n, k) || !is_out(ctype))
        return FWT_EINVAL;
    *bytes = m == 0 || n == 0 ? 0 : qse::int8_workspace(sizes(m, n, k));
    return FWT_OK;
}

int fwt_int8_matmul(const void* a, int64_t lda, const float* a_scales, const void* b,
                    int64_t ldb, const float* b_scales, int64_t m, int64_t n, int64_t k, void* c,
                    fwt_ffn_dtype ctype, int64_t ldc, void* ws, size_t ws_bytes,
                    hipStream_t stream)
{
    size_t need = 0;
    const int rc0 = fwt_int8_matmul_workspace(m, n, k, ctype, &need);
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
    if (k >= kMaxInt8K || lda >= qse::kFfnMaxStride || ldb >= qse::kFfnMaxStride ||
        too_many(m, n))
        return FWT_EUNSUPPORTED;
    const Array arrays[] = {
        {a, m, k, lda, 1, false},
        {b, n, k, ldb, 1, false},
        {a_scales, 1, m, m, 4, false},
        {b_scales, 1, n, n, 4, false},
        {c, m, n, ldc, size_of(ctype), true},
        need ? Array{ws, 1, (int64_t)need, (int64_t)need, 1, true} : kNone,
    };
    const int rc = check_call(arrays, stream);
    if (rc != FWT_OK)
        return rc;
    ProductArgs p = sizes(m, n, k);
    p.a = a;
    p.b0 = b;
    p.lda = lda;
    p.ldb0 = ldb;
    p.sa = a_scales;
    p.sb0 = b_scales;
    p.c = c;
    p.ldc = ldc;
    p.ctype = (int)ctype;
    p.may_split = need != 0;
    p.partial = ws;
    return status(qse::launch_int8(p, stream));
}

int fwt_grouped_matmul_workspace(int dtype, int64_t experts, int64_t m, int64_t n, int64_t k,
                                 size_t* bytes)
{
    if (!bytes || !dims_ok(m, n, k) || experts < 1 ||
        (!is16(dtype) && dtype != FWT_INT8))
        return FWT_EINVAL;
    *bytes = 0;
    if (forward_runs(experts, m, n))
        *bytes = with_copies(forward_need(dtype, experts, m, n, k),
                             is16(dtype) ? forward_copies(experts, m, n, k) : 0);
    return FWT_OK;
}

int fwt_grouped_matmul_workspace_for(const void* x, int64_t ldx, const void* w, int64_t ldw,
                                     int64_t stride_w, int64_t experts, int dtype, int64_t m,
                                     int64_t n, int64_t k, size_t* bytes)
{
    if (!bytes || !dims_ok(m, n, k) || experts < 1 ||
        (!is16(dtype) && dtype != FWT_INT8))
        return FWT_EINVAL;
    *bytes = 0;
    if (!forward_runs(experts, m, n))
        return FWT_OK;
    *bytes = forward_need(dtype, experts, m, n, k);
    if (is16(dtype))
        *bytes = with_copies(*bytes, ForwardCopies(x, ldx, w, ldw, experts > 1 ? stride_w : 0,
                                                   experts, m, n, k)
                                         .bytes);
    return FWT_OK;
}

int fwt_grouped_matmul(const void* x, int64_t ldx, const float* x_scales, const void* w,
                       int64_t ldw, int64_t stride_w, const float* w_scales,
                       const int32_t* ends, int64_t experts, int dtype, int64_t m, int64_t n,
                       int64_t k, void* y, fwt_ffn_dtype ytype, int64_t ldy, int zero_rest,
                       void* ws, size_t ws_bytes, hipStream_t stream)
{
    size_t need = 0;
    const int rc0 = fwt_grouped_matmul_workspace_for(x, ldx, w, ldw, stride_w, experts, dtype, m, n,
                                                     k, &need);
    if (rc0 != FWT_OK)
        return rc0;
    const bool i8 = dtype == FWT_INT8;
    if (i8 ? !is_out(ytype) : (int)ytype != dtype)
        return FWT_EINVAL;
    if (m == 0 || n == 0)
        return FWT_OK;
    if (!ws)
        need = 0;
    if (ws_bytes < need)
        return FWT_EINVAL;
    if (need && !aligned16(ws, 0))
        return FWT_EALIGN;
    if (!x || !w || !y || !ends || i8 != (x_scales != nullptr) || i8 != (w_scales != nullptr))
        return FWT_EINVAL;
    const int64_t sz = size_of(dtype);
    if (i8 && (!aligned16(x, ldx) || !aligned16(w, ldw) || (experts > 1 && (stride_w & 15))))
        return FWT_EALIGN;
    if (experts > kMaxExperts || too_many_grouped(m, n, experts + 1) ||
        ldx * sz >= qse::kFfnMaxStride || ldw * sz >= qse::kFfnMaxStride ||
        (i8 && k >= kMaxInt8K))
        return FWT_EUNSUPPORTED;
    if (!rows_ok(n, ldw, k))
        return FWT_EINVAL;
    const Array arrays[] = {
        {x, m, k, ldx, sz, false},
        experts_array(w, experts, n, ldw, k, stride_w, sz, false),
        {ends, 1, experts, experts, 4, false},
        {y, m, n, ldy, size_of(ytype), true},
        i8 ? Array{x_scales, 1, m, m, 4, false} : kNone,
        i8 ? Array{w_scales, experts, n, n, 4, false} : kNone,
        need ? Array{ws, 1, (int64_t)need, (int64_t)need, 1, true} : kNone,
    };
    const int rc = check_call(arrays, stream);
    if (rc != FWT_OK)
        return rc;
    GroupArgs g = groups(ends, experts, m);
    if (need && !i8) {
        int64_t none = 0, between = experts > 1 ? stride_w : 0;
        ForwardCopies c(x, ldx, w, ldw, between, experts, m, n, k);
        if (c.count) {
            const hipError_t e = c.make((char*)ws + (need - c.bytes), g, stream);
            if (e != hipSuccess)
                return status(e);
            c.use(c.x, x, ldx, none);
            c.use(c.w, w, ldw, between);
            stride_w = between;
        }
    }
    ProductArgs p = sizes(m, n, k * sz);
    p.a = x;
    p.lda = ldx * sz;
    p.b0 = w;
    p.ldb0 = ldw * sz;
    p.sa = x_scales;
    p.sb0 = w_scales;
    p.c = y;
    p.ldc = ldy;
    p.ctype = (int)ytype;
    p.may_split = need != 0;
    p.partial = ws;
    g.stride_b = experts > 1 ? stride_w * sz : 0;
    g.zero_rest = zero_rest != 0;
    return status(qse::launch_grouped(p, g, dtype, false, stream));
}

int fwt_grouped_matmul_backward_workspace(int64_t experts, int64_t m, int64_t n, int64_t k,
                                          size_t* bytes)
{
    if (!bytes || !dims_ok(m, n, k) || experts < 1)
        return FWT_EINVAL;
    *bytes = 0;
    if (backward_runs(experts, m, n, k))
        *bytes = with_copies(backward_need(experts, m, n, k), backward_copies(experts, m, n, k));
    return FWT_OK;
}

int fwt_grouped_matmul_backward_workspace_for(const void* x, int64_t ldx, const void* w,
                                              int64_t ldw, int64_t stride_w, int64_t experts,
                                              const void* dy, int64_t lddy, int64_t m, int64_t n,
                                              int64_t k, int dx, int dw, size_t* bytes)
{
    if (!bytes || !dims_ok(m, n, k) || experts < 1)
        return FWT_EINVAL;
    *bytes = 0;
    if (backward_runs(experts, m, n, k) && (dx || dw))
        *bytes = with_copies(backward_need(experts, m, n, k),
                             BackwardCopies(x, ldx, w, ldw, experts > 1 ? stride_w : 0, dy, lddy,
                                            experts, m, n, k, dx != 0, dw != 0)
                                 .bytes);
    return FWT_OK;
}

int fwt_grouped_matmul_backward(const void* x, int64_t ldx, const void* w, int64_t ldw,
                                int64_t stride_w, const int32_t* ends, int64_t experts,
                                const void* dy, int64_t lddy, fwt_ffn_dtype dtype, int64_t m,
                                int64_t n, int64_t k, void* dx, int64_t lddx, void* dw,
                                int64_t lddw, int64_t stride_dw, void* ws, size_t ws_bytes,
                                hipStream_t stream)
{
    size_t need = 0;
    const int rc0 = fwt_grouped_matmul_backward_workspace_for(
        x, ldx, w, ldw, stride_w, experts, dy, lddy, m, n, k, dx != nullptr, dw != nullptr, &need);
    if (rc0 != FWT_OK)
        return rc0;
    if (!is16(dtype))
        return FWT_EINVAL;
    const bool rows = m != 0 && dx, weights = n != 0 && dw;
    if (!rows && !weights)
        return FWT_OK;
    if (!ws)
        need = 0;
    if (ws_bytes < need)
        return FWT_EINVAL;
    if (need && !aligned16(ws, 0))
        return FWT_EALIGN;
    const bool sums = m != 0 && n != 0;      // otherwise what is written is zeros
    if (!ends || (sums && (!dy || (rows && !w) || (weights && !x))))
        return FWT_EINVAL;
    if (experts > kMaxExperts || (m && too_many_grouped(m, k, experts + 1)) ||
        (n && too_many_weights(experts, n, k)) || ldx * 2 >= qse::kFfnMaxStride ||
        ldw * 2 >= qse::kFfnMaxStride || lddy * 2 >= qse::kFfnMaxStride)
        return FWT_EUNSUPPORTED;
    if (n && ((sums && rows && !rows_ok(n, ldw, k)) || (weights && !rows_ok(n, lddw, k))))
        return FWT_EINVAL;
    const Array arrays[] = {
        sums && weights ? Array{x, m, k, ldx, 2, false} : kNone,
        sums && rows ? experts_array(w, experts, n, ldw, k, stride_w, 2, false) : kNone,
        sums ? Array{dy, m, n, lddy, 2, false} : kNone,
        {ends, 1, experts, experts, 4, false},
        rows ? Array{dx, m, k, lddx, 2, true} : kNone,
        weights ? experts_array(dw, experts, n, lddw, k, stride_dw, 2, true) : kNone,
        need ? Array{ws, 1, (int64_t)need, (int64_t)need, 1, true} : kNone,
    };
    const int rc = check_call(arrays, stream);
    if (rc != FWT_OK)
        return rc;
    GroupArgs g = groups(ends, experts, m);
    hipError_t e = hipSuccess;
    if (need && sums) {
        int64_t none = 0, between = experts > 1 ? stride_w : 0;
        BackwardCopies c(x, ldx, w, ldw, between, dy, lddy, experts, m, n, k, rows, weights);
        if (c.count) {
            e = c.make((char*)ws + (need - c.bytes), g, stream);
            if (e != hipSuccess)
                return status(e);
            c.use(c.dy, dy, lddy, none);
            c.use(c.x, x, ldx, none);
            c.use(c.w, w, ldw, between);
            stride_w = between;
        }
    }
    if (rows && !sums) {
        e = qse::launch_zero16(dx, lddx, m, k, stream);
    } else if (rows) {
        // the contraction runs over n, which w has as its rows
        ProductArgs p = sizes(m, k, 2 * n);
        p.a = dy;
        p.lda = 2 * lddy;
        p.b0 = w;
        p.ldb0 = 2 * ldw;
        p.c = dx;
        p.ldc = lddx;
        p.ctype = (int)dtype;
        p.may_split = need != 0;
        p.partial = ws;
        GroupArgs d = g;
        d.stride_b = experts > 1 ? 2 * stride_w : 0;
        d.zero_rest = 1;
        e = qse::launch_grouped(p, d, (int)dtype, true, stream);
    }
    if (e != hipSuccess || !weights)
        return status(e);
    ProductArgs p = sizes(n, k, 2 * m);
    p.a = dy;
    p.lda = 2 * lddy;
    p.b0 = x;
    p.ldb0 = 2 * ldx;
    p.c = dw;
    p.ldc = lddw;
    p.ctype = (int)dtype;
    p.may_split = need != 0;
    p.partial = ws;
    g.stride_c = experts > 1 ? stride_dw : 0;
    return status(qse::launch_grouped_t(p, g, (int)dtype, stream));
}

}  // extern "C"
