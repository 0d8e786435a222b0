// Rotation by I (x) H_b along k and quantisation to e4m3 with a scale for
// each 128 elements (of a row, or of a 128 x 128 tile).
//
// y = x (I (x) H_b) 2^(-b/2): b add/subtract stages in 32 bits.
// s = max(max |y| / 448, 2^-126), q = e4m3(y / s), rounded to nearest even.
// A block with a value that is not finite gets a NaN scale and NaN codes.
//
// Layout: 8 consecutive lanes hold a block of 128, each 16 consecutive
// elements.  So bits 0-3 of a rotation are register stages, bits 4-6 cross
// the 8 lanes, bits 7-9 the 8 blocks of a wave, and bits 10-13 the waves of a
// workgroup (through LDS); the block's maximum is three lane steps, and a
// lane stores its 16 codes at once.
#include <hip/hip_runtime.h>

#include "ffn_device.h"
#include "fwt_device.h"

namespace qse {
namespace {

enum RotateMode : int {
    kRowScales = 0,   // a scale for each block of 128
    kMaxima = 1,      // only the blocks' maxima, to RotateArgs::amax
    kTileGiven = 2,   // codes by the tile scales in RotateArgs::s
};

constexpr float kTop = 448.0f;

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

// The stage on lane bit LB: (a, b) -> (a + b, a - b) over the pairs.
template <int LB>
__device__ __forceinline__ void lane_stage(float (&v)[16], int lane)
{
    if constexpr (LB < 4) {
        const float s = (lane >> LB) & 1 ? -1.0f : 1.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[i] = fma_sign(v[i], s, lane_partner<LB>(v[i]));
    } else {
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            permlane_swap<LB>(v[i], v[i + 1]);
            butterfly(v[i], v[i + 1]);
            permlane_swap<LB>(v[i], v[i + 1]);
        }
    }
}

// Bits 0 .. bits - 1 (at most 10) of a wave's 1024 elements.
__device__ __forceinline__ void wave_stages(float (&v)[16], int bits, int lane)
{
#pragma unroll
    for (int b = 0; b < 4; ++b)
        if (b < bits) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (!(i & (1 << b)))
                    butterfly(v[i], v[i | (1 << b)]);
        }
    if (bits > 4)
        lane_stage<0>(v, lane);
    if (bits > 5)
        lane_stage<1>(v, lane);
    if (bits > 6)
        lane_stage<2>(v, lane);
    if (bits > 7)
        lane_stage<3>(v, lane);
    if (bits > 8)
        lane_stage<4>(v, lane);
    if (bits > 9)
        lane_stage<5>(v, lane);
}

// Largest magnitude of the block's 128 values, as bits: as unsigned numbers
// they order like the magnitudes, with infinity and then NaN on top.
__device__ __forceinline__ unsigned block_max(const float (&v)[16])
{
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const unsigned u = __float_as_uint(v[i]) & 0x7fffffffu;
        m = m > u ? m : u;
    }
    unsigned o = lane_partner_u32<0>(m);
    m = m > o ? m : o;
    o = lane_partner_u32<1>(m);
    m = m > o ? m : o;
    o = lane_partner_u32<2>(m);
    return m > o ? m : o;
}

__device__ __forceinline__ float scale_of(unsigned maxbits)
{
    if (maxbits > 0x7f7fffffu)
        return __uint_as_float(0x7fc00000u);
    const float s = __uint_as_float(maxbits) / kTop;
    return s > 0x1p-126f ? s : 0x1p-126f;
}

// e4m3 codes of v / s: the quotient is refined once, so that it rounds as
// the division does (a code is a few bits; ties between two codes are
// common where the inputs have few bits too).
__device__ __forceinline__ v4i encode(const float (&v)[16], float s)
{
    const float inv = 1.0f / s;
    v4i out;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        float t[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = v[4 * w + i];
            const float q = x * inv;
            t[i] = __builtin_fmaf(__builtin_fmaf(-q, s, x), inv, q);
        }
        int c = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], 0, false);
        out[w] = __builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], c, true);
    }
    return out;
}

// What follows a rotation: maximum, scale and codes of block kb of a row.
template <int MODE>
__device__ __forceinline__ void finish(const RotateArgs& p, float (&v)[16], int64_t row, int64_t kb,
                                       int lane, bool live)
{
    const int l8 = lane & 7;
    float s;
    if constexpr (MODE == kTileGiven) {
        s = live ? p.s[kb * ((p.m + kFfnBlock - 1) / kFfnBlock) + row / kFfnBlock] : 1.0f;
    } else {
        const unsigned top = block_max(v);
        s = scale_of(top);
        if (live && l8 == 0) {
            if constexpr (MODE == kMaxima)
                p.amax[kb * p.m + row] = __uint_as_float(top);
            else
                p.s[kb * p.m + row] = s;
        }
        if constexpr (MODE == kMaxima)
            return;
    }
    const v4i c = encode(v, s);
    if (live && kb * kFfnBlock + l8 * 16 < p.k)
        *(v4i*)(p.q + row * p.ldq + kb * kFfnBlock + l8 * 16) = c;
}

// Rotations of at most 2^10: the blocks of all rows one after another, 8 to a
// wave.  (k is a multiple of 2^b, so a rotation's blocks lie in one wave.)
template <int TYPE, int MODE>
__global__ __launch_bounds__(256) void rows_kernel(const RotateArgs p, float norm)
{
    const int lane = threadIdx.x & 63;
    const int64_t kbs = (p.k + kFfnBlock - 1) / kFfnBlock;
    const int64_t g = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 3;
    const int64_t row = g / kbs, kb = g - row * kbs;
    const bool live = row < p.m;
    const int64_t k0 = kb * kFfnBlock + (lane & 7) * 16;
    const int left = live ? (int)(p.k - k0 < 16 ? p.k - k0 : 16) : 0;
    float v[16];
    load_elements<TYPE>(p.x, row * p.ldx + k0, left, v);
    wave_stages(v, p.bits, lane);
#pragma unroll
    for (int i = 0; i < 16; ++i)
        v[i] *= norm;
    finish<MODE>(p, v, row, kb, lane, live);
}

// Rotations of 2^11 to 2^14: a workgroup of 2^(b - 10) waves for each.  The
// waves' bits are register stages on a second layout, through LDS and back.
template <int TYPE, int MODE, int WB>
__global__ __launch_bounds__(64 << WB) void long_kernel(const RotateArgs p, float norm)
{
    constexpr int kLow = 16 >> WB;      // neighbours a thread takes with the waves' bits
    __shared__ __align__(16) float lds[(1024 << WB) / 16 * 20];
    const int t = threadIdx.x, lane = t & 63;
    const int64_t per = p.k >> (10 + WB);
    const int64_t row = blockIdx.x / per;
    const int64_t k0 = (blockIdx.x - row * per) * (1024 << WB) + t * 16;
    float v[16];
    load_elements<TYPE>(p.x, row * p.ldx + k0, 16, v);
    wave_stages(v, 10, lane);
    // 16 floats and 4 of padding: 16 lanes' 16-byte accesses take all banks
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *(v4f*)(lds + t * 20 + 4 * i) = v4f{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
    __syncthreads();
    float u[1 << WB][kLow];
    const int low = t * kLow;
#pragma unroll
    for (int w = 0; w < (1 << WB); ++w)
#pragma unroll
        for (int i = 0; i < kLow; ++i)
            u[w][i] = lds[(w * 64 + (low + i) / 16) * 20 + (low + i) % 16];
#pragma unroll
    for (int b = 0; b < WB; ++b)
#pragma unroll
        for (int w = 0; w < (1 << WB); ++w)
            if (!(w & (1 << b)))
#pragma unroll
                for (int i = 0; i < kLow; ++i)
                    butterfly(u[w][i], u[w | (1 << b)][i]);
#pragma unroll
    for (int w = 0; w < (1 << WB); ++w)
#pragma unroll
        for (int i = 0; i < kLow; ++i)
            lds[(w * 64 + (low + i) / 16) * 20 + (low + i) % 16] = u[w][i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i)
        v[i] = lds[t * 20 + i] * norm;
    finish<MODE>(p, v, row, k0 / kFfnBlock, lane, true);
}

// Rotations of at most 2^7 on a 128 x 128 tile: tile scales, or a transposed
// input (k x m), which crosses LDS on its way in.
template <int TYPE, bool TILE, bool TRANS>
__global__ __launch_bounds__(1024) void tile_kernel(const RotateArgs p, float norm)
{
    constexpr int kPad = 128 + (TYPE == kTF32 ? 1 : 2);
    using Word = typename std::conditional<TYPE == kTF32, float, unsigned short>::type;
    __shared__ Word in[TRANS ? 128 * kPad : 1];
    __shared__ unsigned top[16];
    const int t = threadIdx.x, lane = t & 63;
    const int64_t kb = blockIdx.x, mb = blockIdx.y;
    const int64_t row = mb * 128 + (t >> 3);
    const int64_t k0 = kb * 128 + (lane & 7) * 16;
    const bool live = row < p.m;
    float v[16];
    if constexpr (TRANS) {
        const int64_t m = mb * 128 + (t & 127);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int64_t k = kb * 128 + i * 8 + (t >> 7);
            in[(i * 8 + (t >> 7)) * kPad + (t & 127)] =
                m < p.m && k < p.k ? ((const Word*)p.x)[k * p.ldx + m] : (Word)0;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[i] = element<TYPE>(in, ((lane & 7) * 16 + i) * kPad + (t >> 3));
    } else {
        const int left = live ? (int)(p.k - k0 < 16 ? p.k - k0 : 16) : 0;
        load_elements<TYPE>(p.x, row * p.ldx + k0, left, v);
    }
    wave_stages(v, p.bits, lane);
#pragma unroll
    for (int i = 0; i < 16; ++i)
        v[i] *= norm;
    if constexpr (!TILE) {
        finish<kRowScales>(p, v, row, kb, lane, live);
    } else {
        unsigned m = block_max(v);
#pragma unroll
        for (int d = 8; d < 64; d *= 2) {
            const unsigned o = (unsigned)__shfl_xor((int)m, d);
            m = m > o ? m : o;
        }
        if (lane == 0)
            top[t >> 6] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 16; ++w)
            m = m > top[w] ? m : top[w];
        const float s = scale_of(m);
        if (t == 0)
            p.s[kb * ((p.m + kFfnBlock - 1) / kFfnBlock) + mb] = s;
        const v4i c = encode(v, s);
        if (live && k0 < p.k)
            *(v4i*)(p.q + row * p.ldq + k0) = c;
    }
}

// Tile scales from the blocks' maxima: a wave for each tile.
__global__ __launch_bounds__(64) void tile_scale_kernel(const float* amax, float* s, int64_t m)
{
    const int64_t kb = blockIdx.x, mb = blockIdx.y;
    unsigned top = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t row = mb * 128 + h * 64 + threadIdx.x;
        const unsigned u = row < m ? __float_as_uint(amax[kb * m + row]) : 0u;
        top = top > u ? top : u;
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const unsigned o = (unsigned)__shfl_xor((int)top, d);
        top = top > o ? top : o;
    }
    if (threadIdx.x == 0)
        s[kb * ((m + kFfnBlock - 1) / kFfnBlock) + mb] = scale_of(top);
}

template <int TYPE, int MODE>
hipError_t rows(const RotateArgs& p, float norm, hipStream_t stream)
{
    const int64_t kbs = (p.k + kFfnBlock - 1) / kFfnBlock;
    if (p.bits <= 10) {
        hipLaunchKernelGGL((rows_kernel<TYPE, MODE>), dim3((unsigned)((p.m * kbs + 31) / 32)),
                           dim3(256), 0, stream, p, norm);
    } else {
        const dim3 grid((unsigned)(p.m * (p.k >> p.bits)));
        const dim3 block(64u << (p.bits - 10));
        switch (p.bits) {
        case 11:
            hipLaunchKernelGGL((long_kernel<TYPE, MODE, 1>), grid, block, 0, stream, p, norm);
            break;
        case 12:
            hipLaunchKernelGGL((long_kernel<TYPE, MODE, 2>), grid, block, 0, stream, p, norm);
            break;
        case 13:
            hipLaunchKernelGGL((long_kernel<TYPE, MODE, 3>), grid, block, 0, stream, p, norm);
            break;
        default:
            hipLaunchKernelGGL((long_kernel<TYPE, MODE, 4>), grid, block, 0, stream, p, norm);
        }
    }
    return hipGetLastError();
}

template <int TYPE>
hipError_t rotate(const RotateArgs& p, bool tile, bool transpose, hipStream_t stream)
{
    const float norm = p.bits & 1 ? (float)(0.70710678118654752440 / (1 << (p.bits / 2)))
                                  : 1.0f / (float)(1 << (p.bits / 2));
    const dim3 tiles((unsigned)((p.k + 127) / 128), (unsigned)((p.m + 127) / 128));
    if (transpose) {
        if (tile)
            hipLaunchKernelGGL((tile_kernel<TYPE, true, true>), tiles, dim3(1024), 0, stream, p, norm);
        else
            hipLaunchKernelGGL((tile_kernel<TYPE, false, true>), tiles, dim3(1024), 0, stream, p, norm);
        return hipGetLastError();
    }
    if (!tile)
        return rows<TYPE, kRowScales>(p, norm, stream);
    if (p.bits <= kFfnMaxBitsT) {
        hipLaunchKernelGGL((tile_kernel<TYPE, true, false>), tiles, dim3(1024), 0, stream, p, norm);
        return hipGetLastError();
    }
    hipError_t e = rows<TYPE, kMaxima>(p, norm, stream);
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(tile_scale_kernel, tiles, dim3(64), 0, stream, p.amax, p.s, p.m);
    e = hipGetLastError();
    return e != hipSuccess ? e : rows<TYPE, kTileGiven>(p, norm, stream);
}

__global__ __launch_bounds__(256) void zero16_kernel(unsigned short* dst, int64_t ld, int64_t rows,
                                                     int64_t cols)
{
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y)
        for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < cols;
             c += (int64_t)gridDim.x * 256)
            dst[r * ld + c] = 0;
}

}  // namespace

hipError_t launch_zero16(void* dst, int64_t ld, int64_t rows, int64_t cols, hipStream_t stream)
{
    const unsigned gx = (unsigned)(cols < 1024 ? (cols + 255) / 256 : 4);
    hipLaunchKernelGGL(zero16_kernel, dim3(gx, (unsigned)(rows < 1024 ? rows : 1024)), dim3(256), 0,
                       stream, (unsigned short*)dst, ld, rows, cols);
    return hipGetLastError();
}

size_t rotate_workspace(int64_t m, int64_t k, int bits, bool tile, bool transpose)
{
    if (!tile || transpose || bits <= kFfnMaxBitsT || m <= 0)
        return 0;
    return (size_t)m * (size_t)((k + kFfnBlock - 1) / kFfnBlock) * sizeof(float);
}

hipError_t launch_rotate(const RotateArgs& p, int type, bool tile, bool transpose,
                         hipStream_t stream)
{
    if (type == kTF32)
        return rotate<kTF32>(p, tile, transpose, stream);
    if (type == kTBf16)
        return rotate<kTBf16>(p, tile, transpose, stream);
    return rotate<kTF16>(p, tile, transpose, stream);
}

}  // namespace qse
