// The layouts in which a Walsh-Hadamard rotation's stages run, as ffn_rotate.hip
// describes them, for it and for ffn_quantize8.hip.  Internal.
#pragma once

#include <hip/hip_runtime.h>

#include "ffn_device.h"
#include "fwt_device.h"

namespace qse {
namespace {

template <int TYPE>
__device__ __forceinline__ float element(const void* x, int64_t i)
{
    if constexpr (TYPE == kTF32)
        return ((const float*)x)[i];
    else
        return from16(((const unsigned short*)x)[i], TYPE == kTBf16);
}

// Sixteen elements from x[at], the first `left` of which exist (0 after).
template <int TYPE>
__device__ __forceinline__ void load_elements(const void* x, int64_t at, int left, float (&v)[16])
{
    if (left >= 16) {
        struct __attribute__((packed)) Any {
            v4i w[TYPE == kTF32 ? 4 : 2];
        };
        const Any a = *(const Any*)((const char*)x + at * (TYPE == kTF32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if constexpr (TYPE == kTF32)
                v[i] = __int_as_float(a.w[i >> 2][i & 3]);
            else
                v[i] = from16((unsigned short)((unsigned)a.w[i >> 3][(i >> 1) & 3] >> (16 * (i & 1))),
                              TYPE == kTBf16);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[i] = i < left ? element<TYPE>(x, at + i) : 0.0f;
    }
}

// Stages on register bits [LO, HI) of 32 values.
template <int LO, int HI>
__device__ __forceinline__ void stages32(float (&v)[32])
{
#pragma unroll
    for (int b = LO; b < HI; ++b)
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (!(i & (1 << b)))
                butterfly(v[i], v[i | (1 << b)]);
}

// Layout A, from memory to LDS.
template <int BITS>
__device__ __forceinline__ void layout_a32(const float* x, float* lds, int t)
{
    constexpr int kNear = 1 << (15 - BITS), kSegs = 1 << (BITS - 10);
    struct __attribute__((packed)) Near {
        float w[kNear];
    };
    typedef float v2f __attribute__((ext_vector_type(2)));
    float v[32];
#pragma unroll
    for (int g = 0; g < kSegs; ++g) {
        const Near n = *(const Near*)(x + t * kNear + g * 1024);
#pragma unroll
        for (int i = 0; i < kNear; ++i)
            v[g * kNear + i] = n.w[i];
    }
    stages32<0, 5>(v);
    const int a0 = t * kNear, am = ((a0 >> 6) & 7) << 2;
#pragma unroll
    for (int i = 0; i < kNear; i += 2) {
        float* const even = lds + ((a0 + i) ^ am);
        float* const odd = lds + ((a0 + i) ^ am ^ 32);
#pragma unroll
        for (int g = 0; g < kSegs; ++g)
            *(v2f*)(((g ^ (g >> 1)) & 1 ? odd : even) + g * 1024) =
                v2f{v[g * kNear + i], v[g * kNear + i + 1]};
    }
}

// H_32 as the first operand of two 16-bit matrix instructions (rows 0 .. 15 and
// 16 .. 31): lane (q, l) holds inputs 8 q .. 8 q + 7 of row l (and 16 + l),
// (-1)^popcount(row AND input).  Products by +-1 are exact, sums are fp32.
template <int TYPE>
__device__ __forceinline__ void hadamard32(int lane, v4i (&h)[2])
{
    const int q = lane >> 4, l16 = lane & 15;
    // signs of two inputs at a time: bits 0-2 of the input are in the word
    const unsigned one = TYPE == kTBf16 ? 0x3f803f80u : 0x3c003c00u;
    const auto sign = [](int bit) { return bit ? 0x80008000u : 0u; };
    const unsigned w0 = one ^ sign((l16 >> 3) & q & 1) ^ (l16 & 1 ? 0x80000000u : 0u);
    const unsigned s1 = sign(l16 & 2), s2 = sign(l16 & 4);
    h[0] = v4i{(int)w0, (int)(w0 ^ s1), (int)(w0 ^ s2), (int)(w0 ^ s1 ^ s2)};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        h[1][i] = (int)((unsigned)h[0][i] ^ sign(q >> 1));
}

// Their products with 32 inputs of 16 places: lane (q, l) holds inputs 8 q ..
// of place l, and gets rows 4 q .. 4 q + 3 of it.
template <int TYPE>
__device__ __forceinline__ v4f times(v4i h, v4i in)
{
    const v4f zero = v4f{0.f, 0.f, 0.f, 0.f};
    if constexpr (TYPE == kTBf16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, h),
                                                       __builtin_bit_cast(v8bf, in), zero, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, h),
                                                      __builtin_bit_cast(v8h, in), zero, 0, 0, 0);
}

// The same for 16-bit inputs, 16 places at a time.
template <int TYPE, int BITS>
__device__ __forceinline__ void layout_a16(const unsigned short* x, float* lds, int t)
{
    constexpr int kNear = 1 << (15 - BITS);
    constexpr int kRun = kNear < 8 ? kNear : 8;     // neighbours of a load
    const int lane = t & 63, q = lane >> 4, l16 = lane & 15, place0 = t - lane;
    v4i in[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const unsigned short* at = x + (place0 + c * 16 + l16) * kNear + q * 8 / kNear * 1024 +
                                   q * 8 % kNear;
        struct __attribute__((packed)) Run {
            unsigned short w[kRun];
        };
        struct All {
            Run r[8 / kRun];
        } all;
#pragma unroll
        for (int r = 0; r < 8 / kRun; ++r)
            all.r[r] = *(const Run*)(at + r * 1024);
        in[c] = __builtin_bit_cast(v4i, all);
    }
    v4i h[2];
    hadamard32<TYPE>(lane, h);
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const v4f d = times<TYPE>(h[e], in[c]);
            // rows 16 e + 4 q .. + 3: neighbours within kNear, then segments
            constexpr int kWide = kNear < 4 ? kNear : 4;
            typedef float Piece __attribute__((ext_vector_type(kWide)));
#pragma unroll
            for (int r = 0; r < 4; r += kWide) {
                const int out = e * 16 + q * 4 + r;
                const int seg = out / kNear;
                const int i = (place0 + c * 16 + l16) * kNear + out % kNear;
                float* at = lds + seg * 1024 +
                            (i ^ (((i >> 6) & 7) << 2) ^ (((seg ^ (seg >> 1)) & 1) << 5));
                Piece w;
#pragma unroll
                for (int k = 0; k < kWide; ++k)
                    w[k] = d[r + k];
                *(Piece*)at = w;
            }
        }
}

// Layout B, N stages from bit 5, in place.
template <int N>
__device__ __forceinline__ void layout_b(float* lds, int t)
{
    float v[32];
    // i = bit 5 (e), bits 6-8 (j), bit 9 (h): where bits 2-5 come out
    const int odd = ((t >> 5) ^ (t >> 6)) & 1;
    const int b0 = (t >> 5) * 1024 + ((t & 31) ^ (odd << 5));
    float* at[16];
#pragma unroll
    for (int j = 0; j < 16; ++j)
        at[j] = lds + (b0 ^ ((j >> 1) << 2) ^ ((j & 1) << 5)) + (j >> 1) * 64;
#pragma unroll
    for (int i = 0; i < 32; ++i)
        v[i] = at[i & 15][(i >> 4) * 512];
    stages32<0, N>(v);
#pragma unroll
    for (int i = 0; i < 32; ++i)
        at[i & 15][(i >> 4) * 512] = v[i];
}

// Layout C, from LDS to registers.
__device__ __forceinline__ void layout_c(const float* lds, int t, float (&v)[32])
{
    const int odd = ((t >> 5) ^ (t >> 6)) & 1;
    const float* const c0 = lds + ((t * 32) ^ (odd << 5));
    const int cm = ((t >> 1) & 7) << 2;
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        const v4f c = *(const v4f*)(c0 + (i ^ cm));
        v[i] = c[0];
        v[i + 1] = c[1];
        v[i + 2] = c[2];
        v[i + 3] = c[3];
    }
}

}  // namespace
}  // namespace qse
