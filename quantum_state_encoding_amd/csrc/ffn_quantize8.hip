// Rotation by I (x) H_b along k and quantisation to 8-bit integers with one
// scale for each row.
//
// y = x (I (x) H_b) 2^(-b/2): b add/subtract stages in 32 bits.
// s = max(max |y| / 127, 2^-126) over the row, q = rint(y / s).
// A row with a value that is not finite gets a NaN scale and zero codes.
//
// The scale needs all of a row before its first code, so a row's rotated values
// stay in registers, 32 a lane, a wave for every 2048, until its waves have
// joined their maxima: one pass over memory, which bounds short rotations; from 2^5 on
// vector instructions do, 18 to 22 an element (2^5, 2^10 and 2^12 of 8192 x 4096: 94 to
// 100 % of the CUs' cycles, 2^14 96 %).  Kernel times, and at a large copy's rate
// (4.95 TB/s): fp32 4100 x 5000, 2^3 17-20 us (20.7); bf16 8192 x 4096, 2^0 18, 2^5 22,
// 2^7 22, 2^10 23, 2^12 23 (20.3), 2048 x 16384, 2^12 26; bf16 8192 x 16384, 2^14 89-95
// (81), fp32 119-139 (136).  Rows above 32768 elements (1024 lanes) are rotated twice,
// for the maximum and for the codes (bf16 1024 x 65536, 2^10: 85-90 us, 41 at that rate).
// The rotations run in ffn_rotate.hip's layouts:
//   b <= 4        twice 16 neighbours of a lane (rows of up to 2048 elements, and
//                 b = 5: 32 neighbours), register stages
//   b = 6 .. 10   H_32 (16-bit inputs: matrix cores), LDS, register stages of
//                 the others
//   b = 11 .. 14  three layouts
#include <hip/hip_runtime.h>

#include <atomic>

#include "ffn_rotate.h"

namespace qse {
namespace {

constexpr float kTop8 = 127.0f;
constexpr int kWaveRow = 2048;         // elements of a wave
constexpr int kRowMax = 32768;         // of a workgroup

__device__ __forceinline__ float scale8_of(unsigned maxbits)
{
    if (maxbits > 0x7f7fffffu)
        return __uint_as_float(0x7fc00000u);
    const float s = __uint_as_float(maxbits) / kTop8;
    return s > 0x1p-126f ? s : 0x1p-126f;
}

// Sixteen codes of v / s: the quotient is refined once, so that it rounds as
// the division does, and adding 3 * 2^22 rounds it to an integer, which the
// sum's lowest byte is.
__device__ __forceinline__ v4i encode8(const float* v, float s, float inv)
{
    v4i out;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        unsigned t[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = v[4 * w + i];
            const float q = x * inv;
            const float r = __builtin_fmaf(__builtin_fmaf(-q, s, x), inv, q);
            t[i] = __float_as_uint(r + 12582912.0f);
        }
        // bytes 0 of two words side by side, twice, and those halves
        const unsigned lo = __builtin_amdgcn_perm(t[1], t[0], 0x0c0c0400u);
        const unsigned hi = __builtin_amdgcn_perm(t[3], t[2], 0x04000c0cu);
        out[w] = (int)(lo | hi);
    }
    return out;
}

// 32 elements of a lane from x[at], the first `left` of which exist.
template <int TYPE>
__device__ __forceinline__ void load32(const void* x, int64_t at, int64_t left, float (&v)[32])
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float u[16];
        const int64_t l = left - 16 * h;
        load_elements<TYPE>(x, at + 16 * h, l > 16 ? 16 : l > 0 ? (int)l : 0, u);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[16 * h + i] = u[i];
    }
}

// The rotated elements of thread t's lane of a workgroup: 32 neighbours from
// element t * 32 of what the workgroup takes at a time.  place(e): whether
// element e of it exists, and the index in x.  lds: 2048 floats for each wave
// (b >= 6).
template <int TYPE, int BITS, class Place>
__device__ __forceinline__ void rotated(const void* x, int bits, float* lds, int t,
                                        const Place& place, float (&v)[32])
{
    if constexpr (BITS <= 5) {
        if constexpr (BITS < 5) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                int64_t at;
                const int64_t left = place((t >> 6) * kWaveRow + h * 1024 + (t & 63) * 16, at);
                float u[16];
                load_elements<TYPE>(x, at, left > 16 ? 16 : (int)left, u);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    v[16 * h + i] = u[i];
            }
        } else {
            int64_t at;
            const int64_t left = place(t * 32, at);
            load32<TYPE>(x, at, left, v);
        }
#pragma unroll
        for (int b = 0; b < BITS; ++b)
            if (b < bits) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (!(i & (1 << b)))
                        butterfly(v[i], v[i | (1 << b)]);
            }
    } else if constexpr (BITS <= 10) {
        const int lane = t & 63, q = lane >> 4, l16 = lane & 15, w0 = t - lane;
        float* const mine = lds + w0 * 32;
        struct __attribute__((packed)) Any {
            v4i w;
        };
        if constexpr (TYPE == kTF32) {
            int64_t at;
            const int64_t left = place(t * 32, at);
            load32<TYPE>(x, at, left, v);
            stages32<0, 5>(v);
            float* const c0 = mine + ((lane * 32) ^ (lane & 32));
            const int cm = ((lane >> 1) & 7) << 2;
#pragma unroll
            for (int i = 0; i < 32; i += 4)
                *(v4f*)(c0 + (i ^ cm)) = v4f{v[i], v[i + 1], v[i + 2], v[i + 3]};
        } else {
            v4i in[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                // (a rotation's elements exist or not together)
                int64_t at;
                const int64_t left = place(w0 * 32 + (c * 16 + l16) * 32 + q * 8, at);
                in[c] = ((const Any*)((const unsigned short*)x + at))->w;
                if (left <= 0)
                    in[c] = v4i{0, 0, 0, 0};
            }
            v4i h[2];
            hadamard32<TYPE>(lane, h);
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = (c * 16 + l16) * 32 + e * 16 + q * 4;
                    *(v4f*)(mine + (i ^ (((i >> 6) & 7) << 2) ^ ((c >> 1) << 5))) =
                        times<TYPE>(h[e], in[c]);
                }
        }
        __syncthreads();
        layout_b<BITS - 5>(mine, lane);
        __syncthreads();
        layout_c(mine, lane, v);
    } else {
        constexpr int kLanes = 1 << (BITS - 5);
        const int u = t & (kLanes - 1);
        float* const mine = lds + (t - u) * 32;
        int64_t at;
        const int64_t left = place((t - u) * 32, at);
        if constexpr (TYPE != kTF32)
            layout_a16<TYPE, BITS>((const unsigned short*)x + at, mine, u);
        else
            layout_a32<BITS>((const float*)x + at, mine, u);
        __syncthreads();
        layout_b<5>(mine, u);
        __syncthreads();
        layout_c(mine, u, v);
        stages32<15 - BITS, 5>(v);
        if (left <= 0) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                v[i] = 0.0f;
        }
    }
}

// The largest magnitude of a lane's 32 elements, as bits: as unsigned numbers
// they order like the magnitudes, with infinity and then NaN on top.
__device__ __forceinline__ unsigned largest(const float (&v)[32])
{
    float f = 0.0f;      // (the maximum that hands NaN on)
#pragma unroll
    for (int i = 0; i < 32; ++i)
        f = __builtin_elementwise_maximum(f, __builtin_fabsf(v[i]));
    return __float_as_uint(f) & 0x7fffffffu;
}

// Codes of a lane's 32 elements, the row's last one `left` from the first; the second
// 16 are NEXT from it.
template <int NEXT>
__device__ __forceinline__ void write32(int8_t* q, int64_t left, const float (&v)[32], float s,
                                        float inv, bool finite)
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (left <= NEXT * h)
            break;
        v4i c = encode8(v + 16 * h, s, inv);
        if (!finite)
            c = v4i{0, 0, 0, 0};
        const int64_t l = left - NEXT * h;
        if (l < 16) {                    // the row's padding is zeros
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int b = (int)l - 4 * w;
                c[w] = b >= 4 ? c[w] : b <= 0 ? 0 : c[w] & ((1 << (8 * b)) - 1);
            }
        }
        *(v4i*)(q + NEXT * h) = c;
    }
}

// ONE: a workgroup of up to 16 waves for each row (TWICE: of 16, for rows above
// kRowMax).  Otherwise a row takes 2^shift lanes, at most a wave.
template <int TYPE, int BITS, bool ONE, bool TWICE>
__global__ __launch_bounds__(ONE ? 1024 : 256) void quantize8_kernel(const Quantize8Args p,
                                                                     float norm, int shift)
{
    static_assert(ONE || (BITS >= 5 && BITS <= 11), "a wave's row, in 32 neighbours of a lane");
    extern __shared__ __align__(16) float lds[];
    __shared__ unsigned tops[16];
    const int t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const bool exact = !(p.bits & 1);    // (norm is a power of two: see finish in ffn_rotate.hip)
    float v[32];
    int64_t row = 0;
    unsigned top = 0;
    const auto place = [&](int64_t begin) __attribute__((always_inline)) {
        return [=](int e, int64_t& at) __attribute__((always_inline)) -> int64_t {
            int64_t r, c;
            if constexpr (ONE) {
                r = blockIdx.x;
                c = begin + e;
            } else {
                r = ((int64_t)blockIdx.x << (8 - shift)) + (e >> (shift + 5));
                c = e & ((32 << shift) - 1);
            }
            const bool live = r < p.m && c < p.k;
            at = live ? r * p.ldx + c : 0;
            return live ? p.k - c : 0;
        };
    };
    const auto normalise = [&]() __attribute__((always_inline)) {
        if (!exact) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                v[i] *= norm;
        }
    };
    for (int64_t begin = 0; begin < (TWICE ? p.k : 1); begin += kRowMax) {
        if (TWICE && begin > 0)
            __syncthreads();             // (the last part's values have been read)
        rotated<TYPE, BITS>(p.x, p.bits, lds, t, place(begin), v);
        normalise();
        const unsigned m = largest(v);
        top = top > m ? top : m;
    }
    if constexpr (ONE) {
        row = blockIdx.x;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const unsigned o = (unsigned)__shfl_xor((int)top, d);
            top = top > o ? top : o;
        }
        if (lane == 0)
            tops[wave] = top;
        __syncthreads();
        const int waves = (int)blockDim.x >> 6;
        for (int w = 0; w < waves; ++w)
            top = top > tops[w] ? top : tops[w];
    } else {
        row = ((int64_t)blockIdx.x << (8 - shift)) + (t >> shift);
        for (int d = 1; d < (1 << shift); d *= 2) {
            const unsigned o = (unsigned)__shfl_xor((int)top, d);
            top = top > o ? top : o;
        }
    }
    const float s = scale8_of(__float_as_uint(__uint_as_float(top) * (exact ? norm : 1.0f)));
    const bool finite = s == s;
    const float sv = exact ? s / norm : s;
    const float inv = 1.0f / sv;
    constexpr bool kTwo = ONE && BITS < 5;      // twice 16 neighbours
    constexpr int kNext = kTwo ? 1024 : 16;
    const int col = kTwo  ? wave * kWaveRow + lane * 16
                    : ONE ? t * 32
                          : (t & ((1 << shift) - 1)) * 32;
    if (row < p.m && col == 0)
        p.s[row] = s;
    if constexpr (TWICE) {
        for (int64_t begin = 0; begin < p.k; begin += kRowMax) {
            __syncthreads();
            rotated<TYPE, BITS>(p.x, p.bits, lds, t, place(begin), v);
            normalise();
            write32<kNext>(p.q + row * p.ldq + begin + col, p.k - begin - col, v, sv, inv, finite);
        }
    } else if (row < p.m) {
        write32<kNext>(p.q + row * p.ldq + col, p.k - col, v, sv, inv, finite);
    }
}

// Lanes of a row (as a shift) up to one wave, or the row's waves.
int shift_of(int64_t k)
{
    int s = 0;
    while ((int64_t)32 << s < k)
        ++s;
    return s;
}

template <int TYPE, int BITS>
hipError_t run(const Quantize8Args& p, float norm, hipStream_t stream)
{
    const dim3 grid((unsigned)quantize8_groups(p.m, p.k));
    constexpr size_t kLds = BITS > 5 ? (size_t)kWaveRow * 4 : 0;    // of a wave
    if constexpr (BITS >= 5 && BITS <= 11) {     // (2^12 and more are longer, BITS 4 is for those)
        if (p.k <= kWaveRow) {
            hipLaunchKernelGGL((quantize8_kernel<TYPE, BITS, false, false>), grid, dim3(256),
                               4 * kLds, stream, p, norm, shift_of(p.k));
            return hipGetLastError();
        }
    }
    const bool twice = p.k > kRowMax;
    const int waves = twice ? 16 : (int)((p.k + kWaveRow - 1) / kWaveRow);
    auto* k = twice ? &quantize8_kernel<TYPE, BITS, true, true>
                    : &quantize8_kernel<TYPE, BITS, true, false>;
    const size_t lds = waves * kLds;
    if (lds > 65536 - 64) {
        // once for each device
        static std::atomic<uint64_t> done[2];
        int dev = 0;
        hipError_t e = hipGetDevice(&dev);
        if (e == hipSuccess && (dev >= 64 || !((done[twice].load() >> dev) & 1))) {
            e = hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)(16 * kLds));
            if (e == hipSuccess && dev < 64)
                done[twice].fetch_or((uint64_t)1 << dev);
        }
        if (e != hipSuccess)
            return e;
    }
    hipLaunchKernelGGL(k, grid, dim3(64 * waves), lds, stream, p, norm, 0);
    return hipGetLastError();
}

template <int TYPE>
hipError_t by_bits(const Quantize8Args& p, hipStream_t stream)
{
    const float norm = p.bits & 1 ? (float)(0.70710678118654752440 / (1 << (p.bits / 2)))
                                  : 1.0f / (float)(1 << (p.bits / 2));
    switch (p.bits) {
    case 6:
        return run<TYPE, 6>(p, norm, stream);
    case 7:
        return run<TYPE, 7>(p, norm, stream);
    case 8:
        return run<TYPE, 8>(p, norm, stream);
    case 9:
        return run<TYPE, 9>(p, norm, stream);
    case 10:
        return run<TYPE, 10>(p, norm, stream);
    case 11:
        return run<TYPE, 11>(p, norm, stream);
    case 12:
        return run<TYPE, 12>(p, norm, stream);
    case 13:
        return run<TYPE, 13>(p, norm, stream);
    case 14:
        return run<TYPE, 14>(p, norm, stream);
    default:
        return p.bits < 5 && p.k > kWaveRow ? run<TYPE, 4>(p, norm, stream)
                                            : run<TYPE, 5>(p, norm, stream);
    }
}

}  // namespace

int64_t quantize8_groups(int64_t m, int64_t k)
{
    if (k > kWaveRow)
        return m;
    const int per = 8 - shift_of(k);     // (four waves' rows)
    return (m + (((int64_t)1 << per) - 1)) >> per;
}

hipError_t launch_quantize8(const Quantize8Args& p, int type, hipStream_t stream)
{
    if (type == kTF32)
        return by_bits<kTF32>(p, stream);
    return type == kTBf16 ? by_bits<kTBf16>(p, stream) : by_bits<kTF16>(p, stream);
}

}  // namespace qse
