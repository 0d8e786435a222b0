// Products A B^T on the matrix cores, with the epilogues of the gated block.
//
// C[m][n] = sum_k A[m][k] B[n][k].  e4m3 operands carry a scale for each
// 128 of k: C = sum over k blocks of sa[kb][m] sb[kb][n] P_kb, with P_kb
// the product of the codes in one matrix instruction of 128 (32-bit sums),
// and the weighted sum over kb in 32 bits in registers.
//
// A workgroup computes a BM x BN tile.  Each step stages 128 bytes of every
// row of A and B (one k block of e4m3, 64 16-bit elements) into one of two
// LDS buffers while the other feeds the matrix instructions.
#include <hip/hip_runtime.h>

#include "ffn_device.h"

namespace qse {
namespace {

constexpr int kStep = 128;   // bytes of k per step

enum ScaleMode : int { kNoScale = 0, kTileScale = 1, kRowScale = 2 };

// Where chunk c (16 bytes) of row r stands in its 128-byte LDS row: the 16
// rows that a matrix operand reads at one c fall on 8 slots of the two
// halves of the 64 banks.
__device__ __forceinline__ int slot(int r, int c) { return c ^ ((r >> 1) & 7); }

// The row of A that stands at LDS row r: the 16-row blocks of a wave's
// `block` rows take every (block / 16)th row, so that a lane's rows (one of
// each) are neighbours.
__device__ __forceinline__ constexpr int row_of(int r, int block)
{
    return r / block * block + r % 16 * (block / 16) + r % block / 16;
}

// The tile of workgroup w.  The dispatcher hands consecutive workgroups to
// the 8 XCDs in turn; each XCD gets a contiguous run of the tile order, and
// the order goes down columns of up to 8 row tiles, so the tiles that an
// XCD has in flight share their rows of A and B in its L2.
__device__ __forceinline__ void tile_of(int w, int tiles_m, int tiles_n, int& tm, int& tn)
{
    const int total = tiles_m * tiles_n;
    const int x = w & 7, per = total >> 3, more = total & 7;
    int t = x * per + (x < more ? x : more) + (w >> 3);
    constexpr int kGroup = 8;
    const int g = t / (kGroup * tiles_n);
    const int first = g * kGroup;
    const int rows = tiles_m - first < kGroup ? tiles_m - first : kGroup;
    t -= first * tiles_n;
    tm = first + t % rows;
    tn = t / rows;
}

// A 16-byte chunk of 16-bit elements at any address, zeros past `left` bytes.
__device__ __forceinline__ v4i chunk_at(const char* p, int left)
{
    struct __attribute__((packed)) Any {
        v4i v;
    };
    if (left >= 16)
        return ((const Any*)p)->v;
    v4i v = v4i{0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (2 * e < left)
            v[e >> 1] |= (int)((unsigned)((const unsigned short*)p)[e] << (16 * (e & 1)));
    return v;
}

// Scales at .. at + 3 of the `left` ones from p.
__device__ __forceinline__ v4f load_row_scales(const float* p, int left, int at)
{
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, left * 4, (int)kRsrcFlags);
    return __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rsrc, at * 4, 0, 0));
}

// REG: the operands' rows need not be 16-byte aligned; they go through
// registers, loaded before a step's products and stored to LDS after them.
template <int TYPE, int BM, int BN, int WM, int WN, int EP, int SM, bool REG>
__global__ __launch_bounds__(64 * WM * WN) void product_kernel(const ProductArgs p)
{
    constexpr int W = WM * WN;                   // waves
    constexpr bool kDual = EP != kEpStore;
    constexpr int TM = BM / WM / 16;             // 16-row blocks of A per wave
    constexpr int TN = BN / WN / 16;             // of B (dual: half gate, half up)
    constexpr int BNO = kDual ? BN / 2 : BN;     // output columns of the tile
    constexpr int GA = BM / 8 / W, GB = BN / 8 / W;
    constexpr int kBuf = (BM + BN) * kStep;
    static_assert(BM % (8 * W) == 0 && BNO % (8 * W) == 0, "whole 8-row groups per wave");
    extern __shared__ __align__(16) unsigned char lds[];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    int tm, tn;
    tile_of((int)blockIdx.x, p.tiles_m, p.tiles_n, tm, tn);
    const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BNO;
    const int mrows = (int)(p.m - m0 < BM ? p.m - m0 : BM);
    const int nrows = (int)(p.n - n0 < BNO ? p.n - n0 : BNO);

    // Descriptors end with the last row's last chunk (a 16-byte aligned
    // chunk that holds a valid byte lies in that byte's page).
    const int64_t kround = (p.kbytes + 15) & ~(int64_t)15;
    const v4i ra = make_rsrc((const char*)p.a + m0 * p.lda, (uint64_t)((mrows - 1) * p.lda + kround));
    const v4i rb =
        make_rsrc((const char*)p.b0 + n0 * p.ldb0, (uint64_t)((nrows - 1) * p.ldb0 + kround));
    const v4i ru = kDual ? make_rsrc((const char*)p.b1 + n0 * p.ldb1,
                                      (uint64_t)((nrows - 1) * p.ldb1 + kround))
                         : rb;
    // A wave stages groups of 8 LDS rows, wave, wave + W, ...; its first row of
    // A and of B is rows(...)(0), and group g lies a constant further on.
    // (Rows past an operand's last are past its descriptor: what stands in
    // LDS for them feeds results that are not stored.)
    constexpr int kRowsB = BNO / WN;                 // rows of one projection per wave
    const int lr = lane >> 3, lc = slot(wave * 8 + (lane >> 3), lane & 7);
    const int ra0 = row_of(wave * 8 + lr, TM * 16);
    const int rb0 = wave * 8 + lr;
    const unsigned va = (unsigned)(ra0 * p.lda) + lc * 16;
    const unsigned vb = (unsigned)(rb0 * p.ldb0) + lc * 16;
    const unsigned vu = kDual ? (unsigned)(rb0 * p.ldb1) + lc * 16 : 0;
    v4i held[REG ? GA + GB : 1];
    auto fetch = [&](int kt) {
#pragma unroll
        for (int g = 0; g < GA + GB; ++g) {
            const bool isb = g >= GA;
            const int gg = isb ? g - GA : g;
            const bool up = isb && kDual && gg >= GB / 2;
            const int ro = isb ? rb0 + (up ? gg - GB / 2 : gg) * 8 * W
                               : ra0 + row_of(gg * 8 * W, TM * 16);
            const int rows = isb ? nrows : mrows;
            const int64_t row = (isb ? n0 : m0) + (ro < rows ? ro : rows - 1);
            const char* base = (const char*)(isb ? (up ? p.b1 : p.b0) : p.a);
            const int64_t ld = isb ? (up ? p.ldb1 : p.ldb0) : p.lda;
            const int64_t at = (int64_t)kt * kStep + lc * 16;
            held[g] = chunk_at(base + row * ld + at, (int)(p.kbytes - at < 16 ? p.kbytes - at : 16));
        }
    };
    auto put = [&](int kt) {
#pragma unroll
        for (int g = 0; g < GA + GB; ++g) {
            const int gg = g >= GA ? g - GA : g;
            *(v4i*)(lds + (kt & 1) * kBuf + (g >= GA ? BM * kStep : 0) + (wave + gg * W) * 1024 +
                    lane * 16) = held[g];
        }
    };
    const unsigned lds0 = (unsigned)(uintptr_t)(__attribute__((address_space(3))) void*)lds;
    auto stage = [&](int kt) {
        const unsigned base = lds0 + (kt & 1) * kBuf + wave * 1024;
        const unsigned so = (unsigned)kt * kStep;
#pragma unroll
        for (int g = 0; g < GA; ++g)
            load_to_lds(ra, base + g * W * 1024, va,
                        so + (unsigned)(row_of(g * 8 * W, TM * 16) * p.lda));
#pragma unroll
        for (int g = 0; g < GB; ++g) {
            const bool up = kDual && g >= GB / 2;
            load_to_lds(up ? ru : rb, base + (BM + g * 8 * W) * kStep, up ? vu : vb,
                        so + (unsigned)((up ? g - GB / 2 : g) * 8 * W * (up ? p.ldb1 : p.ldb0)));
        }
    };

    const int nk = (int)((p.kbytes + kStep - 1) / kStep);
    v4f acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
            acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

    // Scales: rows of A stand on lanes, TM consecutive ones on a lane (that is
    // what row_of is for), rows of B on the four registers of a result.
    const int q = lane >> 4, l16 = lane & 15;
    float sa[TM], sa_next[TM];
    float sb[2], sb_next[2];
    const int nb0 = (int)((n0 + wn * kRowsB) / kFfnBlock);
    const int mleft = mrows > wm * TM * 16 ? mrows - wm * TM * 16 : 0;
    auto load_scales = [&](int kt) {
        if constexpr (SM != kNoScale) {
#pragma unroll
            for (int i = 0; i < TM; i += 4) {
                const v4f v = load_row_scales(p.sa + (int64_t)kt * p.m + m0 + wm * TM * 16, mleft,
                                              l16 * TM + i);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    sa_next[i + r] = v[r];
            }
            if constexpr (SM == kTileScale) {
                sb_next[0] = p.sb0[(int64_t)kt * p.sb_n + nb0];
                if constexpr (kDual)
                    sb_next[1] = p.sb1[(int64_t)kt * p.sb_n + nb0];
            }
        }
    };

    if constexpr (REG) {
        fetch(0);
        put(0);
    } else {
        stage(0);
    }
    load_scales(0);
    const int swz = l16 >> 1;
    const int ao = (wm * TM * 16 + l16) * kStep + ((q ^ swz) * 16);
    // B rows of this wave in LDS: gate rows, then up rows BNO further on.
    const int bo = (BM + wn * kRowsB + l16) * kStep + ((q ^ swz) * 16);
    const int ktail = (int)(p.kbytes % kStep);

    for (int kt = 0; kt < nk; ++kt) {
        if constexpr (!REG)
            wait_vm<0>();
        __syncthreads();
        unsigned char* buf = lds + (kt & 1) * kBuf;
        if (!REG && kt == nk - 1 && ktail) {
            // Past the end of k both operands are 0, whatever was read there.
            for (int r = threadIdx.x; r < BM + BN; r += 64 * W) {
                for (int c = ktail >> 4; c < 8; ++c) {
                    v4i* at = (v4i*)(buf + r * kStep + slot(r, c) * 16);
                    const int keep = ktail - c * 16;   // bytes of this chunk
                    v4i v = v4i{0, 0, 0, 0};
                    if (keep > 0) {
                        v = *at;
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const int b = keep - 4 * w;
                            v[w] = b >= 4 ? v[w] : b <= 0 ? 0 : v[w] & ((1 << (8 * b)) - 1);
                        }
                    }
                    *at = v;
                }
            }
            __syncthreads();
        }
        sb[0] = sb_next[0];
        sb[1] = sb_next[1];
#pragma unroll
        for (int i = 0; i < TM; ++i)
            sa[i] = sa_next[i];
        if (kt + 1 < nk) {
            if constexpr (REG)
                fetch(kt + 1);
            else
                stage(kt + 1);
            load_scales(kt + 1);
        }
        v4i b[TN][2];
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int row = kDual && j >= TN / 2 ? BNO + (j - TN / 2) * 16 : j * 16;
            b[j][0] = *(const v4i*)(buf + bo + row * kStep);
            b[j][1] = *(const v4i*)(buf + (bo ^ 64) + row * kStep);
        }
        v4f sbr[SM == kRowScale ? TN : 1];
        if constexpr (SM == kRowScale) {
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    int n = wn * kRowsB + j * 16 + q * 4 + r;
                    n = n < nrows ? n : nrows - 1;
                    sbr[j][r] = p.sb0[(int64_t)kt * p.sb_n + n0 + n];
                }
        }
        // Rows of A in turn: while the matrix instructions of one run, the
        // next one's operand comes from LDS, and the sums of the last one
        // are scaled and added.
        v4i a[2][2];
        v4f t[2][SM == kNoScale ? 1 : TN];
        a[0][0] = *(const v4i*)(buf + ao);
        a[0][1] = *(const v4i*)(buf + (ao ^ 64));
        auto add = [&](int i) {
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const float s = sa[i] * (kDual && j >= TN / 2 ? sb[1] : sb[0]);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    acc[i][j][r] =
                        __builtin_fmaf(t[i & 1][j][r], SM == kTileScale ? s : sa[i] * sbr[j][r],
                                       acc[i][j][r]);
            }
        };
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            if (i + 1 < TM) {
                a[(i + 1) & 1][0] = *(const v4i*)(buf + ao + (i + 1) * 16 * kStep);
                a[(i + 1) & 1][1] = *(const v4i*)(buf + (ao ^ 64) + (i + 1) * 16 * kStep);
            }
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                if constexpr (SM == kNoScale)
                    acc[i][j] = matrix_step<TYPE>(b[j], a[i & 1], acc[i][j]);
                else
                    t[i & 1][j] = matrix_step<TYPE>(b[j], a[i & 1], v4f{0.f, 0.f, 0.f, 0.f});
            }
            if constexpr (SM != kNoScale)
                if (i > 0)
                    add(i - 1);
            if (i + 1 < TM)
                __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);   // two LDS reads
            if constexpr (SM != kNoScale) {
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // matrix
                    __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);   // vector
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (SM != kNoScale)
            add(TM - 1);
        if constexpr (REG) {
            if (kt + 1 < nk)
                put(kt + 1);
        }
    }

    // Results: lane l holds rows l % 16 * TM .. of A and four consecutive rows
    // of B, stored at once where the output's alignment allows.
    const bool bf = p.ctype == kTBf16;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int r = wm * (TM * 16) + l16 * TM + i;
        if (r >= mrows)
            continue;
        const int64_t m = m0 + r;
#pragma unroll
        for (int j = 0; j < (kDual ? TN / 2 : TN); ++j) {
            const int nc = wn * kRowsB + j * 16 + q * 4;
            if (nc >= nrows)
                continue;
            const int64_t at = m * p.ldc + n0 + nc;
            const int cnt = nrows - nc < 4 ? nrows - nc : 4;
            v4f v = acc[i][j], u;
            if constexpr (EP == kEpGate) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float f, d;
                    activation(p.act, acc[i][j][k], f, d);
                    v[k] = f * acc[i][j + TN / 2][k];
                }
            } else if constexpr (EP == kEpGateGrad) {
                const v4f g = load4(p.dh, m * p.lddh + n0 + nc, bf, cnt, p.wide_dh);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float f, d;
                    activation(p.act, acc[i][j][k], f, d);
                    v[k] = g[k] * acc[i][j + TN / 2][k] * d;
                    u[k] = g[k] * f;
                }
                store4(p.c, at + p.n, u, p.ctype, cnt, p.wide_c);
            }
            store4(p.c, at, v, p.ctype, cnt, p.wide_c);
        }
    }
}

template <int TYPE, int BM, int BN, int WM, int WN, int EP, int SM, bool REG = false>
hipError_t run(ProductArgs p, hipStream_t stream)
{
    constexpr int BNO = EP != kEpStore ? BN / 2 : BN;
    constexpr size_t kLds = 2 * (size_t)(BM + BN) * kStep;
    const int64_t csize = p.ctype == kTF32 ? 4 : 2;
    p.wide_c = (((uintptr_t)p.c | (uintptr_t)(p.ldc * csize)) & (4 * csize - 1)) == 0 &&
               (EP != kEpGateGrad || p.n % 4 == 0);
    p.wide_dh = (((uintptr_t)p.dh | (uintptr_t)(p.lddh * 2)) & 7) == 0;
    p.tiles_m = (int)((p.m + BM - 1) / BM);
    p.tiles_n = (int)((p.n + BNO - 1) / BNO);
    auto* k = &product_kernel<TYPE, BM, BN, WM, WN, EP, SM, REG>;
    if (kLds > 65536) {
        const hipError_t e = hipFuncSetAttribute((const void*)k,
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, (int)kLds);
        if (e != hipSuccess)
            return e;
    }
    hipLaunchKernelGGL(k, dim3((unsigned)(p.tiles_m * p.tiles_n)), dim3(64 * WM * WN), kLds, stream, p);
    return hipGetLastError();
}

template <int TYPE, int EP, int SM>
hipError_t pick(const ProductArgs& p, hipStream_t stream)
{
    if constexpr (EP != kEpStore && SM == kNoScale) {
        const uintptr_t any = (uintptr_t)p.a | (uintptr_t)p.b0 | (uintptr_t)p.b1 |
                              (uintptr_t)p.lda | (uintptr_t)p.ldb0 | (uintptr_t)p.ldb1;
        if (any & 15)
            return run<TYPE, 128, 128, 2, 2, EP, SM, true>(p, stream);
    }
    const int64_t bno = EP != kEpStore ? 128 : 256;
    // The widened operands, or a scale for each row of B, leave no registers
    // for the larger tile.
    if constexpr (TYPE != kTE4m3Exact && SM != kRowScale) {
        const int64_t bno = EP != kEpStore ? 128 : 256;
        if (((p.m + 255) / 256) * ((p.n + bno - 1) / bno) >= 192)
            return run<TYPE, 256, 256, 2, 4, EP, SM>(p, stream);
    }
    return run<TYPE, 128, 128, 2, 2, EP, SM>(p, stream);
}

}  // namespace

hipError_t launch_product(const ProductArgs& p, int type, int ep, bool row_scales,
                          hipStream_t stream)
{
    if (p.m <= kStripRows && ep != kEpGateGrad && (ep == kEpGate || type == kTE4m3))
        return launch_strip(p, type, ep, row_scales, stream);
    if (type == kTE4m3 && p.ctype == kTF32) {
        if (ep == kEpGate)
            return pick<kTE4m3Exact, kEpGate, kTileScale>(p, stream);
        return row_scales ? pick<kTE4m3Exact, kEpStore, kRowScale>(p, stream)
                          : pick<kTE4m3Exact, kEpStore, kTileScale>(p, stream);
    }
    if (type == kTE4m3) {
        if (ep == kEpGate)
            return pick<kTE4m3, kEpGate, kTileScale>(p, stream);
        return row_scales ? pick<kTE4m3, kEpStore, kRowScale>(p, stream)
                          : pick<kTE4m3, kEpStore, kTileScale>(p, stream);
    }
    if (type == kTBf16) {
        if (ep == kEpGate)
            return pick<kTBf16, kEpGate, kNoScale>(p, stream);
        if (ep == kEpGateGrad)
            return pick<kTBf16, kEpGateGrad, kNoScale>(p, stream);
        return pick<kTBf16, kEpStore, kNoScale>(p, stream);
    }
    if (ep == kEpGate)
        return pick<kTF16, kEpGate, kNoScale>(p, stream);
    if (ep == kEpGateGrad)
        return pick<kTF16, kEpGateGrad, kNoScale>(p, stream);
    return pick<kTF16, kEpStore, kNoScale>(p, stream);
}

}  // namespace qse
