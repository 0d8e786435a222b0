// Device helpers of the feed-forward kernels: matrix-instruction operands,
// loads straight into LDS, rounding and activations.  Internal.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "ffn_internal.h"

namespace qse {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

// Four sums of a matrix instruction.
template <int TYPE>
using Sums = std::conditional_t<TYPE == kTI8, v4i, v4f>;

constexpr int kStep = 128;   // bytes of k that a product takes at a time

constexpr unsigned kRsrcFlags = 0x00020000;   // raw 32-bit buffer

// A raw buffer descriptor: bytes at base, reads past them give 0.
__device__ __forceinline__ v4i make_rsrc(const void* base, uint64_t bytes)
{
    const uint64_t p = (uint64_t)base;
    v4i r;
    r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)p);
    r[1] = __builtin_amdgcn_readfirstlane((int)((uint32_t)(p >> 32) & 0xffffu));
    r[2] = __builtin_amdgcn_readfirstlane(
        (int)(uint32_t)(bytes > 0xffffffffull ? 0xffffffffull : bytes));
    r[3] = (int)kRsrcFlags;
    return r;
}

// Sixteen bytes a lane from rsrc[voff + soff] to LDS at lds + 16 * lane,
// with no register in between.  The compiler does not count these: wait
// with wait_vm() before the data are used.
__device__ __forceinline__ void load_to_lds(v4i rsrc, unsigned lds, unsigned voff, unsigned soff)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
                 : "memory", "m0");
}
// The same, four bytes a lane.
__device__ __forceinline__ void load4_to_lds(v4i rsrc, unsigned lds, unsigned voff)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(rsrc)
                 : "memory", "m0");
}
// Waits until at most the last N memory operations of the wave are unfinished.
template <int N>
__device__ __forceinline__ void wait_vm()
{
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

// Eight e4m3 codes as f16, which holds every one of them exactly.
__device__ __forceinline__ v8h widen(int lo, int hi)
{
    typedef _Float16 v2h __attribute__((ext_vector_type(2)));
    const v2h p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
    const v2h p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
    const v2h p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
    const v2h p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
    return v8h{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// 8-bit integers (kTI8) are two instructions of 64 elements with 32-bit integer
// sums: nothing is lost.
__device__ __forceinline__ v4i matrix_step_i8(const v4i* a, const v4i* b, v4i acc)
{
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[0], b[0], acc, 0, 0, 0);
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a[1], b[1], acc, 0, 0, 0);
}

// acc += a b over 32 bytes of each operand's row: one matrix instruction of
// 128 e4m3 elements, or two of 32 16-bit ones (a and b: [0] and [1]).
//
// The 8-bit instruction cuts each product, towards zero, to a step of 2^-13
// of the largest of its eight neighbours along k (between the eights it keeps
// 32 bits): seven of them lose up to 7 * 2^-13 = 8.5e-4 of that largest one,
// and with products of one sign the result loses as much (6.5e-4 measured with
// one large product in each eight; zero-mean Gaussian codes lose 1.4e-5 in
// norm).  That is 0.22 of half a step of bf16, whose results take it, but 1.75
// of f16's.  kTE4m3Exact, for f16 and fp32 results, widens the codes for the
// f16 instruction, whose products and sums lose nothing but fp32's rounding,
// at half its rate.  (The 8-bit 16x16x32 instruction cuts as the 128 one does.)
template <int TYPE>
__device__ __forceinline__ v4f matrix_step(const v4i* a, const v4i* b, v4f acc)
{
    if constexpr (TYPE == kTE4m3) {
        const v8i x = __builtin_shufflevector(a[0], a[1], 0, 1, 2, 3, 4, 5, 6, 7);
        const v8i y = __builtin_shufflevector(b[0], b[1], 0, 1, 2, 3, 4, 5, 6, 7);
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc, 0, 0, 0, 0, 0, 0);
    } else if constexpr (TYPE == kTE4m3Exact) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int w = 0; w < 4; w += 2)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen(a[h][w], a[h][w + 1]),
                                                             widen(b[h][w], b[h][w + 1]), acc, 0,
                                                             0, 0);
        return acc;
    } else if constexpr (TYPE == kTBf16) {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a[0]),
                                                      __builtin_bit_cast(v8bf, b[0]), acc, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            __builtin_bit_cast(v8bf, a[1]), __builtin_bit_cast(v8bf, b[1]), acc, 0, 0, 0);
    } else {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a[0]),
                                                     __builtin_bit_cast(v8h, b[0]), acc, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(
            __builtin_bit_cast(v8h, a[1]), __builtin_bit_cast(v8h, b[1]), acc, 0, 0, 0);
    }
}

// An integer sum times its row's scale and its column's, one after the other (the
// scales' product alone may leave the range that the result is in), rounded after
// each in every kernel: the last product and the rounding to f16 are not to
// become one instruction.
__device__ __forceinline__ float scaled(int sum, float sa, float sb)
{
    float v = (float)sum * sa * sb;
    asm("" : "+v"(v));       // (v_fma_mixlo_f16 otherwise, with contraction off too)
    return v;
}

// Half of such a step, of 16-bit types and 8-bit integers: 16 bytes a lane.
template <int TYPE>
__device__ __forceinline__ Sums<TYPE> half_step(v4i a, v4i b, Sums<TYPE> acc)
{
    if constexpr (TYPE == kTI8)
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, acc, 0, 0, 0);
    else if constexpr (TYPE == kTBf16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a),
                                                       __builtin_bit_cast(v8bf, b), acc, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a),
                                                      __builtin_bit_cast(v8h, b), acc, 0, 0, 0);
}

// Sixteen bytes at any address.
__device__ __forceinline__ v4i load16(const char* p)
{
    struct __attribute__((packed)) Any {
        v4i v;
    };
    return ((const Any*)p)->v;
}

// The same of 16-bit elements at odd addresses too: a load that is not
// 4-byte aligned takes three times as long, so the words around it are loaded,
// w and the one that holds its last element, and moved by `by` = address & 2
// later.  For a strip's operands (gated bf16 m 8: n 8000 k 4097 68 us with
// such loads, 33 so; k 4098 28); in the tiles, whose loads share the CU with
// more, the second load costs more than it saves (f16 m 1021 n 5501 k 2047:
// 75 and 84 us).
struct Around {
    v4i w;
    unsigned last;
};
__device__ __forceinline__ Around load_around(const char* p)
{
    struct __attribute__((packed, aligned(4))) Words {
        v4i v;
    };
    const uintptr_t at = (uintptr_t)p & ~(uintptr_t)3;
    return Around{((const Words*)at)->v, *(const unsigned*)(at + 12 + 2 * ((uintptr_t)p & 2))};
}
__device__ __forceinline__ v4i moved(const Around& a, int by)
{
    return v4i{(int)__builtin_amdgcn_alignbyte((unsigned)a.w[1], (unsigned)a.w[0], by),
               (int)__builtin_amdgcn_alignbyte((unsigned)a.w[2], (unsigned)a.w[1], by),
               (int)__builtin_amdgcn_alignbyte((unsigned)a.w[3], (unsigned)a.w[2], by),
               (int)__builtin_amdgcn_alignbyte(a.last, (unsigned)a.w[3], by)};
}

// A 16-byte chunk of 16-bit elements that ends `past` bytes behind its row is
// read `past` bytes earlier, from the row's last 16: moved to its place, with
// zeros behind the row.
__device__ __forceinline__ v4i drop(v4i v, int past)
{
    if (past & 8)
        v = v4i{v[2], v[3], 0, 0};
    if (past & 4)
        v = v4i{v[1], v[2], v[3], 0};
    if (past & 2)
        v = v4i{(int)__builtin_amdgcn_alignbyte((unsigned)v[1], (unsigned)v[0], 2),
                (int)__builtin_amdgcn_alignbyte((unsigned)v[2], (unsigned)v[1], 2),
                (int)__builtin_amdgcn_alignbyte((unsigned)v[3], (unsigned)v[2], 2),
                (int)((unsigned)v[3] >> 16)};
    return past >= 16 ? v4i{0, 0, 0, 0} : v;
}

// A chunk `left` bytes before its row's end element by element, which rows of
// fewer than 16 bytes need.
__device__ __forceinline__ v4i chunk_of_short_row(const char* p, int left)
{
    v4i v = v4i{0, 0, 0, 0};
#pragma unroll 1
    for (int e = 0; 2 * e < left && e < 8; ++e) {
        const int u = (int)((unsigned)((const unsigned short*)p)[e] << (16 * (e & 1)));
        if (e < 2)
            v[0] |= u;
        else if (e < 4)
            v[1] |= u;
        else if (e < 6)
            v[2] |= u;
        else
            v[3] |= u;
    }
    return v;
}

// Round to nearest even in 16 bits; the type is uniform.
__device__ __forceinline__ unsigned short to16(float v, bool bf)
{
    if (bf)
        return __builtin_bit_cast(unsigned short, (__bf16)v);
    return __builtin_bit_cast(unsigned short, (_Float16)v);
}
__device__ __forceinline__ float from16(unsigned short u, bool bf)
{
    if (bf)
        return __uint_as_float((unsigned)u << 16);
    return (float)__builtin_bit_cast(_Float16, u);
}

// Four results to c[at ..], the first cnt of which exist; four at once, at
// any address (m 3855 n 4469 k 155, fp32: 63 us with four stores, 56 turned
// in LDS for stores of neighbours, 39 like this).
__device__ __forceinline__ void store4(void* c, int64_t at, v4f v, int type, int cnt)
{
    if (type == kTF32) {
        struct __attribute__((packed)) Any {
            v4f v;
        };
        float* p = (float*)c + at;
        if (cnt == 4) {
            ((Any*)p)->v = v;
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k < cnt)
                    p[k] = v[k];
        }
        return;
    }
    typedef unsigned short v4h __attribute__((ext_vector_type(4)));
    struct __attribute__((packed)) Any {
        v4h v;
    };
    v4h h;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        h[k] = to16(v[k], type == kTBf16);
    unsigned short* p = (unsigned short*)c + at;
    if (cnt == 4) {
        ((Any*)p)->v = h;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < cnt)
                p[k] = h[k];
    }
}

// Sixteen bytes to any address.
__device__ __forceinline__ void put16(void* p, v4i v)
{
    struct __attribute__((packed)) Any {
        v4i v;
    };
    ((Any*)p)->v = v;
}

// Eight neighbours.
__device__ __forceinline__ v4i pack8(v4f u, v4f v, int type)
{
    typedef unsigned short v8s __attribute__((ext_vector_type(8)));
    v8s h;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        h[k] = to16(u[k], type == kTBf16);
        h[k + 4] = to16(v[k], type == kTBf16);
    }
    return __builtin_bit_cast(v4i, h);
}
__device__ __forceinline__ void store8(void* c, int64_t at, v4f u, v4f v, int type, int cnt)
{
    if (type != kTF32 && cnt == 8) {
        put16((unsigned short*)c + at, pack8(u, v, type));
        return;
    }
    store4(c, at, u, type, cnt < 4 ? cnt : 4);
    if (cnt > 4)
        store4(c, at + 4, v, type, cnt - 4);
}

// f16 gradients between two products.  dg and du are rounded to f16 for the
// matrix cores, whose range (65504 down to steps of 2^-24) the products' results
// need not share: where the largest of them is past it, or so small that half a
// step is more than 2^-13 of it, both are stored times 2^-e with the largest
// near 2^14, and the products that read them multiply their sums by 2^e (both
// exact).  Otherwise e is 0.
constexpr float kRangeHigh = 65504.0f, kRangeLow = 0x1p-12f;

// A lane's largest finite magnitude (bits, not 0) into the range.
__device__ __forceinline__ void note_range(GradRange* r, unsigned top)
{
    // most store one and the same word; a maximum has no order
    if (top >= __float_as_uint(kRangeLow) && top <= __float_as_uint(kRangeHigh))
        r->within = 1;
    else
        atomicMax(&r->top, top);
}
__device__ __forceinline__ int range_exponent(const GradRange* r)
{
    const unsigned top = r->top;
    if (top == 0 || (top <= __float_as_uint(kRangeHigh) && r->within))
        return 0;
    const int e = (int)(top >> 23) - 127 - 14;      // (a subnormal: -141)
    return e > -100 ? e : -100;
}
__device__ __forceinline__ float power_of_two(int e)
{
    return __uint_as_float((unsigned)(e + 127) << 23);
}

// Four 16-bit values from p[at ..], 0 past cnt.
typedef unsigned short v4h __attribute__((ext_vector_type(4)));
__device__ __forceinline__ v4h load4(const void* p, int64_t at, int cnt)
{
    struct __attribute__((packed)) Any {
        v4h v;
    };
    const unsigned short* s = (const unsigned short*)p + at;
    v4h h = v4h{0, 0, 0, 0};
    if (cnt == 4) {
        h = ((const Any*)s)->v;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < cnt)
                h[k] = s[k];
    }
    return h;
}

// act(g) and its derivative in 32 bits.  silu: g s and s (1 + g (1 - s))
// with s = 1 / (1 + e^-g); for e^-g past the fp32 range s is 0.  gelu: g P
// and P + g e^(-g^2/2) / sqrt(2 pi) with P the normal distribution
// function, from erfc so that the lower tail keeps its relative precision.
// The hardware's exponential and reciprocal (about one unit in the last place
// of fp32, of an argument that is rounded: 2^-23 |g| or g^2 of the result) are
// far below the 16-bit rounding of the result; an fp32 result takes
// activation_exact.
__device__ __forceinline__ void activation(int act, float g, float& f, float& d)
{
    if (act == 0) {
        const float e = __builtin_amdgcn_exp2f(g * -1.44269504f);
        const float s = __builtin_amdgcn_rcpf(1.0f + e);
        f = g * s;
        d = s + f * (1.0f - s);
    } else {
        const float p = 0.5f * erfcf(g * -0.70710678f);
        f = g * p;
        d = p + g * 0.39894228f * __builtin_amdgcn_exp2f(g * g * -0.72134752f);
    }
}

// act(g) to a few units in the last place of fp32 at any g.  silu: with
// z = e^-|g|, which does not overflow, s is 1 / (1 + z) or z / (1 + z).  gelu:
// the argument of erfc is rounded to t, and r is what that lost; near t erfc
// changes by -2 / sqrt(pi) e^(-t^2) r, which in the lower tail is 2 t r of it.
__device__ __forceinline__ float activation_exact(int act, float g)
{
    if (act == 0) {
        const float z = expf(-__builtin_fabsf(g));
        return g * ((g < 0.0f ? z : 1.0f) / (1.0f + z));
    }
    constexpr float kHigh = 0.707106769f, kLow = 1.21016171e-8f;   // their sum: 2^(-1/2)
    const float t = g * -kHigh;
    float p = erfcf(t);
    const float r = __builtin_fmaf(g, -kHigh, -t) - g * kLow;
    if (t > 0.0f && t < 20.0f)
        p -= 1.12837917f * expf(-t * t) * r;
    return g * (0.5f * p);
}

}  // namespace
}  // namespace qse
