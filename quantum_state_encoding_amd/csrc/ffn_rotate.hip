// Rotation by I (x) H_b along k and quantisation to e4m3 with a scale for
// each 128 elements (of a row, or of a 128 x 128 tile).
//
// y = x (I (x) H_b) 2^(-b/2): b add/subtract stages in 32 bits.
// s = max(max |y| / 448, 2^-126), q = e4m3(y / s), rounded to nearest even.
// A block with a value that is not finite gets a NaN scale and NaN codes.
//
// It is a pass over memory: what is read and written takes 0.2 us a MB at a
// large copy's rate (5.15 TB/s), and the add/subtract stages have to stay
// under that.  A stage on register bits costs a vector instruction an element,
// one across lanes two and more, and the first five of a 16-bit input nothing
// on the matrix cores (H_32, +-1).  So there is a kernel for each way to lay out 2^b:
//   rows_kernel      b <= 7: 16 elements a lane, 8 lanes a block: bits 0-3 in
//                    registers, the others across lanes
//   mid_kernel       b = 8 .. 10: two register layouts with LDS between them
//   long_kernel      b = 11 .. 14: three
//   tile_kernel      b <= 7, tile scales or transposed fp32: a 128 x 128 tile
//   tile_t16_kernel  b <= 7, transposed 16 bits
// Tile scales of longer rotations take two passes, the blocks' maxima first: from
// 2^10 on a 128-row tile of 2^b fp32 columns does not fit a CU.  (At 2^8 and 2^9
// it would, in LDS or in registers; such a kernel is not built.  8192 x 4096 f16
// takes 34 us at both, 22 at 2^7 in one pass.)
#include <hip/hip_runtime.h>

#include "ffn_rotate.h"

namespace qse {
namespace {

enum RotateMode : int {
    kRowScales = 0,   // a scale for each block of 128
    kMaxima = 1,      // only the blocks' maxima, to RotateArgs::amax
    kTileGiven = 2,   // codes by the tile scales in RotateArgs::s
};

constexpr float kTop = 448.0f;

// The stage on lane bit LB: (a, b) -> (a + b, a - b) over the pairs.
template <int LB, int N>
__device__ __forceinline__ void lane_stage(float (&v)[N], int lane)
{
    if constexpr (LB < 4) {
        const float s = (lane >> LB) & 1 ? -1.0f : 1.0f;
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = fma_sign(v[i], s, lane_partner<LB>(v[i]));
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            permlane_swap<LB>(v[i], v[i + 1]);
            butterfly(v[i], v[i + 1]);
            permlane_swap<LB>(v[i], v[i + 1]);
        }
    }
}

// Bits 0 .. bits - 1 (at most 7) of a wave's 1024 elements.
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
}

// Largest magnitude of the block's 128 values (16 on each of 8 lanes, or 32
// on each of 4), as bits: as unsigned numbers they order like the magnitudes,
// with infinity and then NaN on top.
template <int N>
__device__ __forceinline__ unsigned block_max(const float (&v)[N])
{
    float f = 0.0f;      // (the maximum that hands NaN on)
#pragma unroll
    for (int i = 0; i < N; ++i)
        f = __builtin_elementwise_maximum(f, __builtin_fabsf(v[i]));
    unsigned m = __float_as_uint(f) & 0x7fffffffu;
    unsigned o = lane_partner_u32<0>(m);
    m = m > o ? m : o;
    o = lane_partner_u32<1>(m);
    m = m > o ? m : o;
    if constexpr (N == 16) {
        o = lane_partner_u32<2>(m);
        m = m > o ? m : o;
    }
    return m;
}

__device__ __forceinline__ float scale_of(unsigned maxbits)
{
    if (maxbits > 0x7f7fffffu)
        return __uint_as_float(0x7fc00000u);
    const float s = __uint_as_float(maxbits) / kTop;
    return s > 0x1p-126f ? s : 0x1p-126f;
}

// e4m3 codes of v[0 .. 15] / s: the quotient is refined once, so that it
// rounds as the division does (a code is a few bits; ties between two codes
// are common where the inputs have few bits too).
__device__ __forceinline__ v4i encode(const float* v, float s, float inv)
{
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

// Sixteen codes at p, the first `left` of which are the row's: the others are
// its padding, 0 whatever the block's scale (0 / NaN would be NaN).
__device__ __forceinline__ void put_codes(uint8_t* p, v4i c, int64_t left)
{
    if (left < 16) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int b = (int)left - 4 * w;
            c[w] = b >= 4 ? c[w] : b <= 0 ? 0 : c[w] & ((1 << (8 * b)) - 1);
        }
    }
    *(v4i*)p = c;
}

// What follows a rotation, whose factor `norm` (exact: a power of two) is
// still to come: maximum, scale and codes of block kb of a row.  `part` of the
// block's 128 / N lanes has N of its elements.  A power of two moves into the
// scale, where it changes no rounding but that of subnormal results: multiplied
// out they would be rounded to steps of 2^-149, which is 2^-23 of the smallest
// scale, so their codes differ from the other kernels' at most where y / s is
// within 2^-24 of the middle between two codes.
template <int MODE, int N>
__device__ __forceinline__ void finish(const RotateArgs& p, float (&v)[N], float norm, bool exact,
                                       int64_t row, int64_t kb, int part, bool live)
{
    if (!exact) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] *= norm;
        norm = 1.0f;
    }
    float s;
    if constexpr (MODE == kTileGiven) {
        s = live ? p.s[kb * ((p.m + kFfnBlock - 1) / kFfnBlock) + row / kFfnBlock] : 1.0f;
    } else {
        const unsigned top = __float_as_uint(__uint_as_float(block_max(v)) * norm);
        s = scale_of(top);
        if (live && part == 0) {
            if constexpr (MODE == kMaxima)
                p.amax[kb * p.m + row] = __uint_as_float(top);
            else
                p.s[kb * p.m + row] = s;
        }
        if constexpr (MODE == kMaxima)
            return;
    }
    const float sv = s / norm;
    const float inv = 1.0f / sv;
#pragma unroll
    for (int h = 0; h < N; h += 16) {
        const v4i c = encode(v + h, sv, inv);
        const int64_t k = kb * kFfnBlock + part * N + h;
        if (live && k < p.k) {
            // (rotations of more than a block have rows of whole ones)
            put_codes(p.q + row * p.ldq + k, c, N == 16 ? p.k - k : 16);
        }
    }
}

// Rotations of at most 2^7: the blocks of all rows one after another, 8 to a
// wave.  (k is a multiple of 2^b, so a rotation lies in one block.)  Memory
// bounds it, at 2^7 the three lane stages too: 8192 x 4096 fp32 2^5 30.0 us
// (32.6 at a large copy's rate), bf16 2^7 23.0 (19.5).
template <int TYPE>
__global__ __launch_bounds__(256) void rows_kernel(const RotateArgs p, float norm)
{
    const int lane = threadIdx.x & 63;
    const int64_t kbs = (p.k + kFfnBlock - 1) / kFfnBlock;
    const unsigned g = blockIdx.x * 32 + (threadIdx.x >> 3);     // (at most 2^29)
    const unsigned r = g / (unsigned)kbs;
    const int64_t row = r, kb = g - r * (unsigned)kbs;
    const bool live = row < p.m;
    const int64_t k0 = kb * kFfnBlock + (lane & 7) * 16;
    const int left = live ? (int)(p.k - k0 < 16 ? p.k - k0 : 16) : 0;
    float v[16];
    load_elements<TYPE>(p.x, row * p.ldx + k0, left, v);
    wave_stages(v, p.bits, lane);
    finish<kRowScales>(p, v, norm, !(p.bits & 1), row, kb, lane & 7, live);
}

// Rotations of 2^11 to 2^14: a workgroup of 2^b / 32 threads for each, in
// three layouts with LDS between them:
//   A  bits 10 .. b-1 and 0 .. 14-b: 2^(15-b) neighbours of every 1024
//   B  bits 5 .. 9: every 32nd of a 1024, register stages
//   C  bits 15-b .. 4: 32 neighbours, a quarter of a block, register stages
// A is H_32 times 32 inputs: for 16-bit inputs, as they come from memory, on
// the matrix cores (products by +-1 are exact, sums are fp32), for fp32
// register stages.  A lane stage costs two instructions an element, a register
// stage one, and the vector instructions are what comes closest to the
// memory's time: 8192 x 16384 bf16 take 78 us from memory and 95 with A in
// registers (25 instructions an element), 90 with A on the matrix cores (20).
//
// Element i stands in LDS at i ^ (bits 6-8 of i at 2-4) ^ (bits 10 + 11 at 5):
// so the 16-byte accesses of C (16 lanes, 32 elements apart), the 4-byte ones
// of B (two runs of 32) and A's take all banks.  Each layout's addresses are a
// few lane values and constants that are added.
// Rotations of 2^8 to 2^10: a wave takes 2048 elements, 2^(11-b) rotations in
// the order of the rows.  Bits 0-4 are register stages on a lane's 32
// neighbours, for 16-bit inputs the matrix cores' H_32; the others layout B's
// register stages; and layout C hands a lane its quarter of a block.  Against
// stages across lanes (16 elements a lane, no LDS), b = 10: 8192 x 4096 bf16
// 29.4 and 19.5 us (19.7 at a large copy's rate), fp32 34.7 and 32.4 (32.8),
// 4096 x 16384 fp32 with tile scales 109 and 103.
//
// Codes by given scales are taken from the end, which the search for the
// maxima has read last and the last-level cache may hold (4096 x 16384 fp32,
// tile scales: 117 us from the front, 112 from the end).
template <int TYPE, int MODE, int BITS>
__global__ __launch_bounds__(64) void mid_kernel(const RotateArgs p, float norm)
{
    constexpr int kUnits = 2048 >> BITS;
    __shared__ __align__(16) float lds[2048];
    const int t = threadIdx.x, q = t >> 4, l16 = t & 15;
    const unsigned per = (unsigned)(p.k >> BITS);
    const unsigned w = MODE == kTileGiven ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
    const unsigned u0 = w * (unsigned)kUnits;
    const unsigned row0 = u0 / per, rem = u0 - row0 * per;
    // row and first column of rotation u0 + d
    const auto unit = [=](unsigned d, int64_t& row, int64_t& k0) __attribute__((always_inline)) {
        const unsigned v = rem + d;
        const unsigned more = per >= kUnits ? (v >= per ? 1u : 0u) : v / per;
        row = row0 + more;
        k0 = (int64_t)(v - more * per) << BITS;
        return row < p.m;
    };
    struct __attribute__((packed)) Any {
        v4i w;
    };
    if constexpr (TYPE == kTF32) {
        int64_t row, k0;
        unit((unsigned)(t * 32) >> BITS, row, k0);
        row = row < p.m ? row : p.m - 1;     // past the last: any that is there
        const float* x = (const float*)p.x + row * p.ldx + k0 + (t * 32 & ((1 << BITS) - 1));
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            const v4f w = __builtin_bit_cast(v4f, ((const Any*)(x + i))->w);
            v[i] = w[0];
            v[i + 1] = w[1];
            v[i + 2] = w[2];
            v[i + 3] = w[3];
        }
        stages32<0, 5>(v);
        float* const c0 = lds + ((t * 32) ^ (t & 32));
        const int cm = ((t >> 1) & 7) << 2;
#pragma unroll
        for (int i = 0; i < 32; i += 4)
            *(v4f*)(c0 + (i ^ cm)) = v4f{v[i], v[i + 1], v[i + 2], v[i + 3]};
    } else {
        v4i in[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int i = (c * 16 + l16) * 32 + q * 8;
            int64_t row, k0;
            unit((unsigned)i >> BITS, row, k0);
            row = row < p.m ? row : p.m - 1;
            in[c] = ((const Any*)((const unsigned short*)p.x + row * p.ldx + k0 +
                                  (i & ((1 << BITS) - 1))))->w;
        }
        v4i h[2];
        hadamard32<TYPE>(t, h);
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = (c * 16 + l16) * 32 + e * 16 + q * 4;
                *(v4f*)(lds + (i ^ (((i >> 6) & 7) << 2) ^ ((c >> 1) << 5))) = times<TYPE>(h[e], in[c]);
            }
    }
    __syncthreads();
    layout_b<BITS - 5>(lds, t);
    __syncthreads();
    float v[32];
    layout_c(lds, t, v);
    int64_t row, k0;
    const bool live = unit((unsigned)(t * 32) >> BITS, row, k0);
    k0 += t * 32 & ((1 << BITS) - 1);
    finish<MODE>(p, v, norm, !(BITS & 1), row, k0 / kFfnBlock, t & 3, live);
}

template <int TYPE, int MODE, int BITS>
__global__ __launch_bounds__(1 << (BITS - 5)) void long_kernel(const RotateArgs p, float norm)
{
    __shared__ __align__(16) float lds[1 << BITS];
    const int t = threadIdx.x;
    const int64_t per = p.k >> BITS;
    // Rotations of the 32 rows whose scales share a line of memory run on one
    // XCD (workgroup w on XCD w mod 8), whose L2 gathers them.
    // Codes by given scales are taken from the end (see mid_kernel).
    int64_t w = MODE == kTileGiven ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
    const int64_t group = 256 * per;
    if (w < p.m * per / group * group) {
        const int64_t r = w % group;
        w += (r & 7) * (32 * per) + (r >> 3) - r;
    }
    const int64_t row = w / per;
    const int64_t k0 = (w - row * per) << BITS;
    float v[32];
    if constexpr (TYPE != kTF32)
        layout_a16<TYPE, BITS>((const unsigned short*)p.x + row * p.ldx + k0, lds, t);
    else
        layout_a32<BITS>((const float*)p.x + row * p.ldx + k0, lds, t);
    __syncthreads();
    layout_b<5>(lds, t);
    __syncthreads();
    layout_c(lds, t, v);
    stages32<15 - BITS, 5>(v);
    finish<MODE>(p, v, norm, !(BITS & 1), row, k0 / kFfnBlock + (t >> 2), t & 3, true);
}

// Rotations of at most 2^7 on a 128 x 128 tile: tile scales, or a transposed
// fp32 input (k x m), which crosses LDS on its way in, four bytes a lane.  Tile
// scales, 2^7: 4096 x 8192 fp32 29.5 us (32.6 at a large copy's rate), 8192 x
// 4096 bf16 22.3 (19.5).  Transposed, 4096 x 4096 fp32 (16.3): row scales 2^5
// 21.5, tile scales 2^7 23.7.
template <int TYPE, bool TILE, bool TRANS>
__global__ __launch_bounds__(1024) void tile_kernel(const RotateArgs p, float norm)
{
    constexpr int kPad = 129;
    static_assert(!TRANS || TYPE == kTF32, "tile_t16_kernel");
    __shared__ float in[TRANS ? 128 * kPad : 1];
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
                m < p.m && k < p.k ? ((const float*)p.x)[k * p.ldx + m] : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[i] = in[((lane & 7) * 16 + i) * kPad + (t >> 3)];
    } else {
        const int left = live ? (int)(p.k - k0 < 16 ? p.k - k0 : 16) : 0;
        load_elements<TYPE>(p.x, row * p.ldx + k0, left, v);
    }
    wave_stages(v, p.bits, lane);
    if constexpr (!TILE) {
        finish<kRowScales>(p, v, norm, !(p.bits & 1), row, kb, lane & 7, live);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[i] *= norm;
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
        const v4i c = encode(v, s, 1.0f / s);
        if (live && k0 < p.k)
            put_codes(p.q + row * p.ldq + k0, c, p.k - k0);
    }
}

// The same for a transposed input of 16-bit elements: 128 k of 128 rows, in
// 16-byte loads along the rows, stand in LDS as they come, and the transposing
// read gives a lane four k of its row.  16 lanes take a row each, four lanes
// (16 apart) 32 k each: bits 0-4 are register stages, 5 and 6 cross the lanes.
// 8192 x 4000 bf16 2^5, row or tile scales: 20.5 us (19.1 at a copy's rate).
template <int TYPE, bool TILE, int BITS>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(4))) void
tile_t16_kernel(const RotateArgs p, float norm)
{
    typedef short v4s __attribute__((ext_vector_type(4)));
    __shared__ __align__(16) unsigned char in[128 * 256];
    __shared__ unsigned top[4];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6, q = lane >> 4, l16 = lane & 15;
    const int64_t kb = blockIdx.x, mb = blockIdx.y;
    // 32-byte units of a k row are spread over the banks by k: a read takes
    // four k rows at once, and those of k and k + 32
    const auto mask = [](int k) { return (k & 3) | ((k >> 5) & 1) << 2; };
    struct __attribute__((packed)) Any {
        v4i v;
    };
    const unsigned short* src =
        (const unsigned short*)p.x + (kb * 128 + (t >> 4)) * p.ldx + mb * 128 + (t & 15) * 8;
    v4i c[8];
    if (kb * 128 + 128 <= p.k && mb * 128 + 128 <= p.m) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            c[i] = ((const Any*)(src + i * 16 * p.ldx))->v;
    } else {
        const int64_t left = p.m - mb * 128 - (t & 15) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            c[i] = v4i{0, 0, 0, 0};
            if (kb * 128 + i * 16 + (t >> 4) >= p.k)
                continue;
            if (left >= 8) {
                c[i] = ((const Any*)(src + i * 16 * p.ldx))->v;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < left)
                        c[i][e >> 1] |= (int)((unsigned)src[i * 16 * p.ldx + e] << (16 * (e & 1)));
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int kr = i * 16 + (t >> 4), ch = t & 15;
        *(v4i*)(in + kr * 256 + ((ch >> 1) ^ mask(kr)) * 32 + (ch & 1) * 16) = c[i];
    }
    __syncthreads();
    // Sixteen rows: 32 rotated elements a lane, and their largest magnitude
    // over the row's four lanes.
    auto rotated = [&](int h, float (&v)[32]) __attribute__((always_inline)) {
        const unsigned char* at = in + (q * 32 + (l16 >> 2)) * 256 +
                                  ((wave + 4 * h) ^ mask(q * 32 + (l16 >> 2))) * 32 + (l16 & 3) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const v4s r = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) v4s*)(at + e * 4 * 256));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[e * 4 + i] = from16((unsigned short)r[i], TYPE == kTBf16);
        }
        stages32<0, BITS < 5 ? BITS : 5>(v);
        if constexpr (BITS > 5)
            lane_stage<4>(v, lane);
        if constexpr (BITS > 6)
            lane_stage<5>(v, lane);
        float f = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            v[i] *= norm;
            f = __builtin_elementwise_maximum(f, __builtin_fabsf(v[i]));
        }
        unsigned m = __float_as_uint(f) & 0x7fffffffu;
#pragma unroll
        for (int d = 16; d < 64; d *= 2) {
            const unsigned o = (unsigned)__shfl_xor((int)m, d);
            m = m > o ? m : o;
        }
        return m;
    };
    auto write = [&](int h, const float (&v)[32], float s) __attribute__((always_inline)) {
        const int64_t row = mb * 128 + (wave + 4 * h) * 16 + l16;
        const float inv = 1.0f / s;
        if (!TILE && q == 0 && row < p.m)
            p.s[kb * p.m + row] = s;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int64_t k = kb * 128 + q * 32 + e * 16;
            const v4i code = encode(v + e * 16, s, inv);
            if (row < p.m && k < p.k)
                put_codes(p.q + row * p.ldq + k, code, p.k - k);
        }
    };
    if constexpr (!TILE) {
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            float v[32];
            const unsigned m = rotated(h, v);
            write(h, v, scale_of(m));
        }
    } else {
        float v[2][32];
        unsigned m = rotated(0, v[0]);
        const unsigned m1 = rotated(1, v[1]);
        m = m > m1 ? m : m1;
#pragma unroll
        for (int d = 1; d < 16; d *= 2) {
            const unsigned o = (unsigned)__shfl_xor((int)m, d);
            m = m > o ? m : o;
        }
        if (lane == 0)
            top[wave] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 4; ++w)
            m = m > top[w] ? m : top[w];
        const float s = scale_of(m);
        if (t == 0)
            p.s[kb * ((p.m + kFfnBlock - 1) / kFfnBlock) + mb] = s;
        write(0, v[0], s);
        write(1, v[1], s);
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
    if (MODE == kRowScales && p.bits <= 7) {
        hipLaunchKernelGGL((rows_kernel<TYPE>), dim3((unsigned)((p.m * kbs + 31) / 32)), dim3(256),
                           0, stream, p, norm);
    } else if (p.bits <= 10) {
        const int64_t rotations = p.m * (p.k >> p.bits);
        const dim3 grid((unsigned)(((rotations << p.bits) + 2047) / 2048));
        switch (p.bits) {
        case 8:
            hipLaunchKernelGGL((mid_kernel<TYPE, MODE, 8>), grid, dim3(64), 0, stream, p, norm);
            break;
        case 9:
            hipLaunchKernelGGL((mid_kernel<TYPE, MODE, 9>), grid, dim3(64), 0, stream, p, norm);
            break;
        default:
            hipLaunchKernelGGL((mid_kernel<TYPE, MODE, 10>), grid, dim3(64), 0, stream, p, norm);
        }
    } else {
        const dim3 grid((unsigned)(p.m * (p.k >> p.bits)));
        const dim3 block(1u << (p.bits - 5));
        switch (p.bits) {
        case 11:
            hipLaunchKernelGGL((long_kernel<TYPE, MODE, 11>), grid, block, 0, stream, p, norm);
            break;
        case 12:
            hipLaunchKernelGGL((long_kernel<TYPE, MODE, 12>), grid, block, 0, stream, p, norm);
            break;
        case 13:
            hipLaunchKernelGGL((long_kernel<TYPE, MODE, 13>), grid, block, 0, stream, p, norm);
            break;
        default:
            hipLaunchKernelGGL((long_kernel<TYPE, MODE, 14>), grid, block, 0, stream, p, norm);
        }
    }
    return hipGetLastError();
}

template <int TYPE, bool TILE, int BITS = kFfnMaxBitsT>
hipError_t transposed16(const RotateArgs& p, float norm, dim3 tiles, hipStream_t stream)
{
    if constexpr (BITS > 0) {
        if (p.bits != BITS)
            return transposed16<TYPE, TILE, BITS - 1>(p, norm, tiles, stream);
    }
    hipLaunchKernelGGL((tile_t16_kernel<TYPE, TILE, BITS>), tiles, dim3(256), 0, stream, p, norm);
    return hipGetLastError();
}

template <int TYPE>
hipError_t rotate(const RotateArgs& p, bool tile, bool transpose, hipStream_t stream)
{
    const float norm = p.bits & 1 ? (float)(0.70710678118654752440 / (1 << (p.bits / 2)))
                                  : 1.0f / (float)(1 << (p.bits / 2));
    const dim3 tiles((unsigned)((p.k + 127) / 128), (unsigned)((p.m + 127) / 128));
    if constexpr (TYPE != kTF32) {
        if (transpose)
            return tile ? transposed16<TYPE, true>(p, norm, tiles, stream)
                        : transposed16<TYPE, false>(p, norm, tiles, stream);
    } else if (transpose) {
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
