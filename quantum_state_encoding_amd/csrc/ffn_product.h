// The body of a product's tile and how it is launched: shared by the products
// of one pair of operands (ffn_matmul.hip), of 8-bit integers (ffn_int8.hip)
// and of rows grouped by expert (ffn_grouped.hip).  Internal.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <type_traits>

#include "ffn_device.h"

namespace qse {
namespace {

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
__device__ __forceinline__ int place_of(int w, int total)
{
    const int x = w & 7, per = total >> 3, more = total & 7;
    return x * per + (x < more ? x : more) + (w >> 3);
}
__device__ __forceinline__ void tile_at(int t, int tiles_m, int tiles_n, int& tm, int& tn)
{
    constexpr int kGroup = 8;
    const int g = t / (kGroup * tiles_n);
    const int first = g * kGroup;
    const int rows = tiles_m - first < kGroup ? tiles_m - first : kGroup;
    t -= first * tiles_n;
    tm = first + t % rows;
    tn = t / rows;
}
__device__ __forceinline__ void tile_of(int w, int tiles_m, int tiles_n, int& tm, int& tn)
{
    tile_at(place_of(w, tiles_m * tiles_n), tiles_m, tiles_n, tm, tn);
}

// An operand that is stored with its rows side by side, [k][rows] (AT, BT;
// 16-bit types): a step stages 64 k of it as they are, and the transposing
// LDS read gives a lane four k of its row.  Its 16 lanes take four k rows of
// 32 bytes each, so those 32-byte units are spread over the banks by k.
__device__ __forceinline__ int unit_mask(int k) { return (k & 3) | ((k >> 3) & 1) << 2; }

// WIDE: the block's rows are every second four of 32 (wide_row).  A lane then takes eight
// bytes of every sixteen of two units, so the masks m and m ^ 1 of two k send them to the
// same banks: two ways, 6 to 7 % of the cycles of grouped gradients (none without WIDE).
template <int BR, bool WIDE = false>
__device__ __forceinline__ v4i read_t_half(const unsigned char* tile, int block, int lane, int h)
{
    typedef short v4s __attribute__((ext_vector_type(4)));
    const int q = lane >> 4, l16 = lane & 15;
    const int unit = WIDE ? (block & ~1) + ((l16 >> 1) & 1) : block;
    const unsigned char* at = tile + (q * 8 + (l16 >> 2)) * (BR * 2) +
                              ((unit ^ unit_mask(q * 8 + (l16 >> 2))) * 32) +
                              (WIDE ? (l16 & 1) * 16 + (block & 1) * 8 : (l16 & 3) * 8);
    v4s r[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
        r[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) v4s*)(at + (h * 32 + e * 4) * (BR * 2)));
    return __builtin_bit_cast(v4i, __builtin_shufflevector(r[0], r[1], 0, 1, 2, 3, 4, 5, 6, 7));
}
template <int BR>
__device__ __forceinline__ void read_t(v4i (&out)[2], const unsigned char* tile, int block, int lane)
{
#pragma unroll
    for (int h = 0; h < 2; ++h)
        out[h] = read_t_half<BR>(tile, block, lane, h);
}

// From a tile's sums to results: lane l holds rows l % 16 * TM .. of A (AT:
// every 16th from l % 16) and four consecutive rows of B, stored at once.
// acc: rows i0, i0 + 1, .. of the wave's BM / WM / 16, and the 16-row blocks
// of B from j0 on (dual: gate's, then up's).
//
// A tile runs this once, as straight code, and its time is mostly that of
// fetching the code: so a whole tile has a path of its own without bounds, and
// each activation too (gated e4m3 m 8192 n 16384 k 4096: 992 us without,
// 970 with them).
//
// WIDE (plain stores): B's rows stand in LDS as wide_row says, so that a lane has
// eight neighbours of each pair of blocks and a row of C gets 64 bytes at once, in
// whole tiles 128 (see below): a round of 256 bf16 tiles of 256 x 256 takes 16 us
// beside its steps with four neighbours in a store, 11 with eight, 9.5 with 128
// bytes.  Stores that pass the caches by take longer (12).
__device__ __forceinline__ constexpr int wide_row(int r)
{
    return (r & ~31) | ((r >> 2) & 3) * 8 | ((r >> 4) & 1) * 4 | (r & 3);
}

template <int TYPE, int BM, int BN, int WM, int WN, int EP, bool AT, int NI, int TN, int ACT,
          bool WHOLE, bool WIDE>
__device__ __forceinline__ void finish_rows_as(const ProductArgs& p, const Sums<TYPE> (&acc)[NI][TN],
                                               int i0, int j0, int tm, int tn, int wave, int lane)
{
    constexpr int TM = BM / WM / 16;
    constexpr bool kDual = EP != kEpStore;
    constexpr int BNO = kDual ? BN / 2 : BN, kRowsB = BNO / WN, TJ = kDual ? TN / 2 : TN;
    // (TN: the blocks that acc has)
    const int wm = wave / WN, wn = wave % WN, q = lane >> 4, l16 = lane & 15;
    const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BNO;
    const int mrows = WHOLE || p.m - m0 > BM ? BM : (int)(p.m - m0);
    const int nrows = WHOLE || p.n - n0 > BNO ? BNO : (int)(p.n - n0);
    const int ctype = TYPE == kTE4m3        ? (int)kTBf16
                      : TYPE == kTI8        ? p.ctype
                      : TYPE != kTE4m3Exact ? TYPE
                      : p.ctype == kTF32    ? (int)kTF32
                                            : (int)kTF16;
    const int act = ACT < 0 ? p.act : ACT;
    const auto row_at = [=](int i) __attribute__((always_inline)) {
        return wm * (TM * 16) + (AT ? (i0 + i) * 16 + l16 : l16 * TM + i0 + i);
    };
    const auto column_at = [=](int j) __attribute__((always_inline)) {
        return WIDE ? wn * kRowsB + ((j0 + j) >> 1) * 32 + q * 8 + ((j0 + j) & 1) * 4
                    : wn * kRowsB + (j0 + j) * 16 + q * 4;
    };
    constexpr bool kPairs = WIDE && TJ > 1;
    constexpr int kSide = kPairs ? 8 : 4;    // neighbours of a store
    const auto count_at = [=](int nc) __attribute__((always_inline)) {
        return WHOLE || nrows - nc > kSide ? kSide : nrows - nc;
    };
    v4f before = v4f{0.f, 0.f, 0.f, 0.f};
    // f16 gradients: the factor that dg and du are stored with, or that the
    // sums of what was stored so are multiplied by
    constexpr bool kGrad16 = EP == kEpGateGrad && TYPE == kTF16;
    float factor = 1.0f;
    if constexpr (TYPE == kTF16 && EP != kEpGate) {
        if (EP == kEpStore)
            factor = p.range ? power_of_two(range_exponent(p.range)) : 1.0f;
        else if (p.again)
            factor = power_of_two(-range_exponent(p.range));
    }
    float top = 0.0f;      // the largest finite magnitude
    // All of dh before the first store (a load behind a store that may be to
    // the same address waits for memory each time).
    v4h dh[EP == kEpGateGrad ? NI : 1][TJ];
    if constexpr (EP == kEpGateGrad) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < TJ; ++j) {
                const int r = WHOLE || row_at(i) < mrows ? row_at(i) : mrows - 1;
                const int nc = column_at(j);
                dh[i][j] = load4(p.dh, (m0 + r) * p.lddh + n0 + nc, count_at(nc));
            }
    }
    // 8-bit integers: the scales of this lane's columns
    v4f sb[TYPE == kTI8 ? TJ : 1];
    if constexpr (TYPE == kTI8) {
#pragma unroll
        for (int j = 0; j < TJ; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int nc = column_at(j) + k;
                sb[j][k] = p.sb0[n0 + (WHOLE || nc < nrows ? nc : nrows - 1)];
            }
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int r = row_at(i);
        if (!WHOLE && r >= mrows)
            continue;
        int64_t m = m0 + r;
        float sa = 1.0f;
        if constexpr (TYPE == kTI8)
            sa = p.sa[m];
        void* c = p.c;
        int64_t ldc = p.ldc;
        if (AT && p.split) {      // rows from split on: another matrix
            if (m >= p.split) {
                m -= p.split;
                c = p.c1;
                ldc = p.ldc1;
            }
            if (m >= p.split_rows)
                continue;
        }
        if constexpr (WIDE && WHOLE && TJ == 4) {
            if (ctype != kTF32) {
                // Two lanes side by side have a row each: they give each other
                // half of them, so that a store has all 128 bytes of a row.
                v4i half[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    v4f v[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if constexpr (TYPE == kTI8)
                                v[j][k] = scaled(acc[i][2 * h + j][k], sa, sb[2 * h + j][k]);
                            else if constexpr (TYPE == kTF16)
                                v[j][k] = acc[i][2 * h + j][k] * factor;
                            else
                                v[j][k] = acc[i][2 * h + j][k];
                        }
                    }
                    half[h] = pack8(v[0], v[1], ctype);
                }
                const bool odd = l16 & 1;
                v4i mine, theirs;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int give = odd ? half[0][w] : half[1][w];
                    const int got = __builtin_amdgcn_mov_dpp(give, 0xb1, 0xf, 0xf, true);
                    mine[w] = odd ? got : half[0][w];
                    theirs[w] = odd ? half[1][w] : got;
                }
                const int64_t step = (AT ? 1 : TM) * ldc;
                unsigned short* at = (unsigned short*)c + (odd ? m * ldc - step : m * ldc) + n0 +
                                     wn * kRowsB + (odd ? 32 : 0) + q * 8;
                put16(at, mine);
                put16(at + step, theirs);
                continue;
            }
        }
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
            const int nc = column_at(kPairs ? j & ~1 : j);
            if (!WHOLE && nc >= nrows)
                continue;
            const int64_t at = m * ldc + n0 + nc;
            v4f v, u;
            if constexpr (TYPE == kTI8) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    v[k] = scaled(acc[i][j][k], sa, sb[j][k]);
            } else {
                v = acc[i][j];
            }
            if constexpr (kDual) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float f, d;
                    if constexpr (TYPE == kTE4m3Exact)
                        f = activation_exact(act, acc[i][j][k]);
                    else
                        activation(act, acc[i][j][k], f, d);
                    if constexpr (EP == kEpGate) {
                        v[k] = f * acc[i][j + TN / 2][k];
                    } else {
                        const float g = from16(dh[i][j][k], ctype == kTBf16);
                        v[k] = g * acc[i][j + TN / 2][k] * d;
                        u[k] = g * f;
                        if constexpr (kGrad16) {
                            // (past the last column g is 0)
                            const float a = __builtin_fabsf(v[k]), b = __builtin_fabsf(u[k]);
                            top = __builtin_fmaxf(top, a < __builtin_inff() ? a : 0.0f);
                            top = __builtin_fmaxf(top, b < __builtin_inff() ? b : 0.0f);
                            v[k] *= factor;
                            u[k] *= factor;
                        }
                    }
                }
            } else if constexpr (TYPE == kTF16) {
                v *= factor;
            }
            if constexpr (EP == kEpGateGrad)
                store4(c, at + p.part_c, u, ctype, count_at(nc));
            if constexpr (!kPairs)
                store4(c, at, v, ctype, count_at(nc));
            else if (j & 1)
                store8(c, at, before, v, ctype, count_at(nc));
            else
                before = v;
        }
        // (rows side by side would need more registers than there are)
        if constexpr (kGrad16)
            __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (kGrad16) {
        if (!p.again && top != 0.0f)
            note_range(p.range, __float_as_uint(top));
    }
}

template <int TYPE, int BM, int BN, int WM, int WN, int EP, bool AT, bool WIDE = false, int NI, int TN>
__device__ __forceinline__ void finish_rows(const ProductArgs& p, const Sums<TYPE> (&acc)[NI][TN], int i0,
                                            int j0, int tm, int tn, int wave, int lane)
{
    constexpr int BNO = EP != kEpStore ? BN / 2 : BN;
    if ((int64_t)(tm + 1) * BM > p.m || (int64_t)(tn + 1) * BNO > p.n)
        finish_rows_as<TYPE, BM, BN, WM, WN, EP, AT, NI, TN, -1, false, WIDE>(
            p, acc, i0, j0, tm, tn, wave, lane);
    else if (EP == kEpStore || p.act == 0)
        finish_rows_as<TYPE, BM, BN, WM, WN, EP, AT, NI, TN, 0, true, WIDE>(
            p, acc, i0, j0, tm, tn, wave, lane);
    else
        finish_rows_as<TYPE, BM, BN, WM, WN, EP, AT, NI, TN, 1, true, WIDE>(
            p, acc, i0, j0, tm, tn, wave, lane);
}

// REG: the operands' rows need not be 16-byte aligned; they go through
// registers, loaded before a step's products and stored to LDS after them.
enum Alignment : int {
    kAligned = 0,
    kAnyAddress = 1,
    kShortRows = 2,    // rows of fewer than 16 bytes, element by element
};
// AT, BT: A or B is stored [k][rows].  With p.parts = 2 the contraction goes
// on in a second B (b1), for columns part_a bytes further on in A's rows.
// WK groups of WM x WN waves compute the tile, each WKth step of k; LDS holds
// NS rounds of them.
// The workgroups' numbers are the tiles'.
struct EveryWorkgroup {
    __device__ __forceinline__ int64_t tile() const { return blockIdx.x; }
    __device__ __forceinline__ int64_t tiles() const { return gridDim.x; }
    __device__ __forceinline__ void place(const ProductArgs& p, int& tm, int& tn) const
    {
        tile_of((int)blockIdx.x, p.tiles_m, p.tiles_n, tm, tn);
    }
};

// (tm, tn): the tile that this workgroup computes, where.tile() of where.tiles()
// (asked for late, not to hold registers); part: its share of the contraction's
// p.splits.
template <int TYPE, int BM, int BN, int WM, int WN, int WK, int NS, int EP, int SM, int REG,
          bool AT, bool BT, bool PIPE = false, bool WIDE = PIPE, class Where>
__device__ __forceinline__ void product_body(const ProductArgs& p, int tm, int tn, int part,
                                             const Where& where)
{
    constexpr int W = WM * WN;                   // waves of a group
    constexpr bool kDual = EP != kEpStore;
    constexpr int TM = BM / WM / 16;             // 16-row blocks of A per wave
    constexpr int TN = BN / WN / 16;             // of B (dual: half gate, half up)
    constexpr int BNO = kDual ? BN / 2 : BN;     // output columns of the tile
    constexpr int GA = BM / 8 / W, GB = BN / 8 / W;
    constexpr int kScaleBytes = SM != kNoScale ? (BM + BN) * 4 : 0;
    constexpr int kBuf = (BM + BN) * kStep + kScaleBytes;   // rows, then their scales
    constexpr int kLoads = GA + GB + (SM != kNoScale ? 1 : 0);   // of a wave and step
    static_assert(SM == kNoScale || (BM % 64 == 0 && BNO % 64 == 0 && BM + BN <= 64 * W),
                  "scales: a wave for 64 rows");
    static_assert(BM % (8 * W) == 0 && BNO % (8 * W) == 0, "whole 8-row groups per wave");
    extern __shared__ __align__(16) unsigned char lds[];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(((int)threadIdx.x >> 6) % W);
    const int kg = __builtin_amdgcn_readfirstlane((int)threadIdx.x / (64 * W));
    const int tid = (int)threadIdx.x - kg * 64 * W;   // in the group
    const int wm = wave / WN, wn = wave % WN;
    const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BNO;
    const int mrows = (int)(p.m - m0 < BM ? p.m - m0 : BM);
    const int nrows = (int)(p.n - n0 < BNO ? p.n - n0 : BNO);

    static_assert(!REG || (WK == 1 && NS == 2), "REG");
    static_assert(!(AT || BT) || (SM == kNoScale && !kDual && (!AT || GA == 4) && GB == 4), "[k][rows]");
    constexpr int kRowsB = BNO / WN;                 // rows of one projection per wave
    const int nks = (int)((p.kbytes + kStep - 1) / kStep);   // steps of a part
    const int all = p.parts > 1 ? 2 * nks : nks;
    // this workgroup's steps: all, or its share of them
    const int share = (all + p.splits - 1) / p.splits;
    const int first = part * share;
    const int nk = first + share < all ? first + share : all;
    // A wave stages 1 KiB at a time, pieces wave, wave + W, ...: 8 LDS rows of
    // an operand, or 64 k / (4 W) rows of k of one that is [k][rows].  Piece g
    // lies a constant number of rows behind the wave's first.  Descriptors
    // end with the last row's last chunk (a 16-byte aligned chunk that holds
    // a valid byte lies in that byte's page).  What lies past the operand's
    // last row is past its descriptor: it reads as 0 and feeds results that
    // are not stored.  The range check of a raw buffer compares the lane's
    // offset with the descriptor's size less the scalar offset; a scalar offset
    // past the size would wrap that difference, so none may be: a piece that
    // begins behind the last row begins at the last row instead (piece_a; a
    // lane then reads that row or is out of range), or, where a step's rows are
    // those of k, its offset is cut to the size (within).
    const int64_t kround = (p.kbytes + 15) & ~(int64_t)15;
    const int lr = lane >> 3, lc = slot(wave * 8 + (lane >> 3), lane & 7);
    const int ra0 = row_of(wave * 8 + lr, TM * 16);
    constexpr bool kWide = WIDE && !kDual;
    static_assert(!kWide || kRowsB % 32 == 0, "pairs of blocks");
    const int rb0 = kWide ? wide_row(wave * 8 + lr) : wave * 8 + lr;
    constexpr int kCa = BM / 8, kCb = BN / 8;        // chunks in a row of k
    const int ka0 = wave * (64 / kCa) + lane / kCa, kb0 = wave * (64 / kCb) + lane / kCb;
    const int ca = (((lane % kCa) >> 1) ^ unit_mask(ka0)) * 2 + (lane & 1);
    const int cb = (((lane % kCb) >> 1) ^ unit_mask(kb0)) * 2 + (lane & 1);
    const unsigned va = AT ? (unsigned)(ka0 * p.lda) + ca * 16 : (unsigned)(ra0 * p.lda) + lc * 16;
    const unsigned vb = BT ? (unsigned)(kb0 * p.ldb0) + cb * 16 : (unsigned)(rb0 * p.ldb0) + lc * 16;
    const unsigned vu = kDual || BT ? (unsigned)((BT ? kb0 : rb0) * p.ldb1) + (BT ? cb : lc) * 16 : 0;
    const v4i ra = make_rsrc((const char*)p.a + m0 * p.lda,
                       (uint64_t)((mrows - 1) * p.lda + (p.parts > 1 ? p.part_a : 0) + kround));
    const v4i rb = make_rsrc((const char*)p.b0 + n0 * p.ldb0, (uint64_t)((nrows - 1) * p.ldb0 + kround));
    const v4i ru = kDual ? make_rsrc((const char*)p.b1 + n0 * p.ldb1,
                                      (uint64_t)((nrows - 1) * p.ldb1 + kround))
                         : rb;
    // k rows of a [k][rows] operand from step ks on
    auto rows_of_k = [=](const void* base, int64_t ld, int64_t r0, int64_t rows,
                         int ks) __attribute__((always_inline)) {
        const int64_t left = p.kbytes / 2 - (int64_t)ks * 64;
        return make_rsrc((const char*)base + (int64_t)ks * 64 * ld + r0 * 2,
                         (uint64_t)((left - 1) * ld + (((rows - r0) * 2 + 15) & ~(int64_t)15)));
    };
    // step kt = first + round * WK + group
    auto buffer_of = [=](int kt) __attribute__((always_inline)) {
        return ((((kt - first) / WK) & (NS - 1)) * WK + kg) * kBuf;
    };
    // A step's chunks into registers: where they lie in their row (bytes), and
    // what of it they miss.  [k][rows]: rows of k past the last are zeros.
    const int64_t lena = AT ? p.m * 2 : p.kbytes, lenb = BT ? p.n * 2 : p.kbytes;
    auto from_row = [&](int64_t at, int64_t len) __attribute__((always_inline)) {
        return at < len - 16 ? at : len >= 16 ? len - 16 : 0;
    };
    unsigned rowa[REG && !AT ? GA : 1], rowb[REG && !BT ? GB : 1];   // the rows' offsets
    if constexpr (REG && !AT) {
#pragma unroll
        for (int g = 0; g < GA; ++g) {
            const int r = ra0 + row_of(g * 8 * W, TM * 16);
            rowa[g] = (unsigned)((r < mrows ? r : mrows - 1) * p.lda);
        }
    }
    if constexpr (REG && !BT) {
#pragma unroll
        for (int g = 0; g < GB; ++g) {
            const bool up = kDual && g >= GB / 2;
            const int r = rb0 + (up ? g - GB / 2 : g) * 8 * W;
            rowb[g] = (unsigned)((r < nrows ? r : nrows - 1) * (up ? p.ldb1 : p.ldb0));
        }
    }
    auto fetch = [&](int kt, v4i (&held)[GA + GB]) __attribute__((always_inline)) {
        const bool second = p.parts > 1 && kt >= nks;
        const int ks = second ? kt - nks : kt;
        const int64_t at = (int64_t)ks * kStep + lc * 16;
        const unsigned oa = (unsigned)from_row(AT ? (m0 + ca * 8) * 2 : at, lena);
        const unsigned ob = (unsigned)from_row(BT ? (n0 + cb * 8) * 2 : at, lenb);
        const int64_t left = p.kbytes / 2 - 1 - (int64_t)ks * 64;
        const int klast = (int)(left < 63 ? left : 63);     // of the step's 64 rows of k
#pragma unroll
        for (int g = 0; g < GA; ++g) {
            const int k = ka0 + g * 16 < klast ? ka0 + g * 16 : klast;
            const char* base = (const char*)p.a + (AT ? (int64_t)ks * 64 * p.lda : m0 * p.lda) +
                               (second ? p.part_a : 0);
            held[g] = load16(base + (uint64_t)((AT ? (unsigned)(k * p.lda) : rowa[g]) + oa));
        }
#pragma unroll
        for (int g = 0; g < GB; ++g) {
            const bool up = kDual ? g >= GB / 2 : second;
            const int64_t ld = up ? p.ldb1 : p.ldb0;
            const int k = kb0 + g * 16 < klast ? kb0 + g * 16 : klast;
            const char* base =
                (const char*)(up ? p.b1 : p.b0) + (BT ? (int64_t)ks * 64 : n0) * ld;
            held[GA + g] = load16(base + (uint64_t)((BT ? (unsigned)(k * ld) : rowb[g]) + ob));
        }
    };
    auto fetch_short = [&](int kt, v4i (&held)[GA + GB]) __attribute__((always_inline)) {
        const bool second = p.parts > 1 && kt >= nks;
        const int ks = second ? kt - nks : kt;
        const int64_t at = (int64_t)ks * kStep + lc * 16;
#pragma unroll
        for (int g = 0; g < GA + GB; ++g) {
            const bool isb = g >= GA;
            const int gg = isb ? g - GA : g;
            const bool up = isb && (kDual ? gg >= GB / 2 : second);
            const bool t = isb ? BT : AT;
            const int64_t k = (int64_t)ks * 64 + (isb ? kb0 : ka0) + gg * 16;
            const int r = isb ? rb0 + (kDual && up ? gg - GB / 2 : gg) * 8 * W
                              : ra0 + row_of(gg * 8 * W, TM * 16);
            const int rows = isb ? nrows : mrows;
            const int64_t row = t ? (k < p.kbytes / 2 ? k : 0)
                                  : (isb ? n0 : m0) + (r < rows ? r : rows - 1);
            const int64_t w = t ? ((isb ? n0 : m0) + (isb ? cb : ca) * 8) * 2 : at;
            held[g] = chunk_of_short_row((const char*)(isb ? (up ? p.b1 : p.b0) : p.a) +
                                             row * (isb ? (up ? p.ldb1 : p.ldb0) : p.lda) +
                                             (!isb && second ? p.part_a : 0) + w,
                                         (int)((isb ? lenb : lena) - w));
        }
    };
    // ... and to LDS, with zeros in the place of what they miss
    auto put = [&](int kt, v4i (&held)[GA + GB]) __attribute__((always_inline)) {
        const bool second = p.parts > 1 && kt >= nks;
        const int ks = second ? kt - nks : kt;
        const int64_t at = (int64_t)ks * kStep + lc * 16;
        if (((int64_t)ks + 1) * kStep > p.kbytes || (AT && mrows < BM) || (BT && nrows < BN)) {
            const int64_t wa = AT ? (m0 + ca * 8) * 2 : at, wb = BT ? (n0 + cb * 8) * 2 : at;
            const int pa = (int)(wa - from_row(wa, lena)), pb = (int)(wb - from_row(wb, lenb));
#pragma unroll
            for (int g = 0; g < GA + GB; ++g) {
                const bool isb = g >= GA;
                const int64_t k = (int64_t)ks * 64 + (isb ? kb0 + (g - GA) * 16 : ka0 + g * 16);
                if (REG == kAnyAddress)
                    held[g] = drop(held[g], isb ? pb : pa);
                if ((isb ? BT : AT) && k >= p.kbytes / 2)
                    held[g] = v4i{0, 0, 0, 0};
            }
        }
#pragma unroll
        for (int g = 0; g < GA + GB; ++g) {
            const int gg = g >= GA ? g - GA : g;
            *(v4i*)(lds + buffer_of(kt) + (g >= GA ? BM * kStep : 0) + (wave + gg * W) * 1024 +
                    lane * 16) = held[g];
        }
    };
    const unsigned lds0 = (unsigned)(uintptr_t)(__attribute__((address_space(3))) void*)lds;
    // Scales of 64 rows of the tile per wave (waves past them repeat the last
    // 64): a lane's row, in rows of A or B; past the last one, the last.
    const int sw = wave < (BM + BN) / 64 ? wave : (BM + BN) / 64 - 1;
    const bool sup = kDual && sw * 64 >= BM + BNO;
    const float* sbase = sw * 64 < BM ? p.sa : sup ? p.sb1 : p.sb0;
    const int64_t sn = sw * 64 < BM ? p.m : p.sb_n;
    int64_t sat = sw * 64 + lane + (sw * 64 < BM ? m0 : n0 - BM - (sup ? BNO : 0));
    if (SM == kTileScale && sw * 64 >= BM)
        sat /= kFfnBlock;
    const unsigned vs = (unsigned)(sat < sn ? sat : sn - 1) * 4;
    const auto within = [](unsigned off, v4i rsrc) __attribute__((always_inline)) {
        return off < (unsigned)rsrc[2] ? off : (unsigned)rsrc[2];
    };
    unsigned piece_a[GA], piece_b[GB];       // where the pieces' rows begin
#pragma unroll
    for (int g = 0; g < GA; ++g) {
        const int row = row_of(g * 8 * W, TM * 16);
        piece_a[g] = AT ? (unsigned)(g * 16 * p.lda)
                        : (unsigned)((row < mrows ? row : mrows - 1) * p.lda);
    }
#pragma unroll
    for (int g = 0; g < GB; ++g) {
        const bool up = kDual && g >= GB / 2;
        const int row = (up ? g - GB / 2 : g) * 8 * W;
        piece_b[g] = (unsigned)((row < nrows ? row : nrows - 1) * (up ? p.ldb1 : p.ldb0));
    }
    auto stage = [=](int kt) __attribute__((always_inline)) {
        const bool second = BT && p.parts > 1 && kt >= nks;
        const int ks = second ? kt - nks : kt;
        const unsigned base = lds0 + buffer_of(kt) + wave * 1024;
        const unsigned so = (unsigned)ks * kStep;
        const v4i da = AT ? rows_of_k(p.a, p.lda, m0, p.m, ks) : ra;
        const v4i db =
            BT ? rows_of_k(second ? p.b1 : p.b0, second ? p.ldb1 : p.ldb0, n0, p.n, ks) : rb;
#pragma unroll
        for (int g = 0; g < GA; ++g)
            load_to_lds(da, base + g * W * 1024, va,
                        AT ? within(piece_a[g], da)
                           : so + (second ? (unsigned)p.part_a : 0u) + piece_a[g]);
#pragma unroll
        for (int g = 0; g < GB; ++g) {
            const bool up = kDual && g >= GB / 2;
            load_to_lds(up ? ru : db, base + (BM + g * 8 * W) * kStep, up || second ? vu : vb,
                        BT ? within((unsigned)(g * 16 * (second ? p.ldb1 : p.ldb0)), db)
                           : so + piece_b[g]);
        }
        if constexpr (SM != kNoScale)
            load4_to_lds(make_rsrc(sbase + (int64_t)ks * sn, (uint64_t)sn * 4),
                         base - wave * 1024 + (BM + BN) * kStep + sw * 256, vs);
    };

    Sums<TYPE> acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
            acc[i][j] = Sums<TYPE>{};

    // Scales: rows of A stand on lanes, TM consecutive ones on a lane (that is
    // what row_of is for), rows of B on the four registers of a result.
    const int q = lane >> 4, l16 = lane & 15;
    // Steps that operands at any address are fetched ahead of: two where a tile's
    // registers hold them, since with one a step lasts as long as its loads (64 x 128
    // tiles, bf16 m 921 e 7 n 1501 k 2047: 33 us with one, 27.6 with two; 128 x 128
    // ones, two on a CU, 39.4 and 39.6).
    constexpr int kAhead = REG == kAnyAddress && WIDE && BM == 64 ? 2 : 1;
    if constexpr (REG) {
        v4i held[GA + GB];
        if constexpr (REG == kAnyAddress)
            fetch(first, held);
        else
            fetch_short(first, held);
        put(first, held);
    } else {
#pragma unroll
        for (int s = 0; s < NS - 1; ++s)
            if (first + s * WK + kg < nk)
                stage(first + s * WK + kg);
    }
    const int swz = l16 >> 1;
    const int ao = (wm * TM * 16 + l16) * kStep + ((q ^ swz) * 16);
    // B rows of this wave in LDS: gate rows, then up rows BNO further on.
    const int bo = (BM + wn * kRowsB + l16) * kStep + ((q ^ swz) * 16);
    const int so = (BM + BN) * kStep + (wm * TM * 16 + l16 * TM) * 4;   // scales of A's rows
    const int sbo = (BM + BN) * kStep + (BM + wn * kRowsB + q * 4) * 4;
    const int ktail = (int)(p.kbytes % kStep);

    auto cut = [&](int kt, unsigned char* buf) __attribute__((always_inline)) {
        // Past the end of k both operands are 0, whatever was read there.
        const bool mine = kt == all - 1 || kt == nks - 1;
        if constexpr (AT)
            for (int c = (ktail / 2) * kCa + tid; mine && c < BM * 8; c += 64 * W)
                *(v4i*)(buf + c * 16) = v4i{0, 0, 0, 0};
        if constexpr (BT)
            for (int c = (ktail / 2) * kCb + tid; mine && c < BN * 8; c += 64 * W)
                *(v4i*)(buf + BM * kStep + c * 16) = v4i{0, 0, 0, 0};
        for (int r = tid + (AT ? BM : 0); mine && r < BM + (BT ? 0 : BN); r += 64 * W) {
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
    };

    // A step; what is fetched comes into one, what has been goes to LDS from the other.
    auto step = [&](int kt, auto& into, auto& from) __attribute__((always_inline)) {
        // The step's own loads have arrived, those of later steps go on.
        if constexpr (!REG) {
            if (NS > 2 && kt + (NS - 2) * WK < nk)
                wait_vm<(NS - 2) * kLoads>();
            else
                wait_vm<0>();
        }
        __syncthreads();
        unsigned char* buf = lds + buffer_of(kt);
        const int k0 = kt - kg;      // the round's first step
        if (!REG && ktail && (k0 + WK >= all || (p.parts > 1 && k0 < nks && k0 + WK >= nks))) {
            cut(kt, buf);
            __syncthreads();
        }
        if constexpr (REG == kAnyAddress)
            fetch(kt + kAhead < nk ? kt + kAhead : nk - 1, into);
        else if constexpr (REG == kShortRows)
            fetch_short(kt + 1 < nk ? kt + 1 : kt, into);
        if (WK > 1 && kt >= nk)
            return false;     // (the last round: no barrier follows in the loop)
        float sa[TM], sb[2];
        v4f sbr[TN];
        if constexpr (SM != kNoScale) {
#pragma unroll
            for (int i = 0; i < TM; ++i)
                sa[i] = ((const float*)(buf + so))[i];
            if constexpr (SM == kRowScale) {
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    sbr[j] = *(const v4f*)(buf + sbo + j * 64);
            } else {
                sb[0] = *(const float*)(buf + sbo);
                if constexpr (kDual)
                    sb[1] = *(const float*)(buf + sbo + BNO * 4);
            }
        }
        v4i b[TN][2];
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int row = kDual && j >= TN / 2 ? BNO + (j - TN / 2) * 16 : j * 16;
            if constexpr (BT) {
                b[j][0] = read_t_half<BN, kWide>(buf + BM * kStep, wn * TN + j, lane, 0);
                b[j][1] = read_t_half<BN, kWide>(buf + BM * kStep, wn * TN + j, lane, 1);
            } else {
                b[j][0] = *(const v4i*)(buf + bo + row * kStep);
                b[j][1] = *(const v4i*)(buf + (bo ^ 64) + row * kStep);
            }
        }
        constexpr int kMfmas = TYPE == kTE4m3Exact ? 4 : 1;
        constexpr int kValus = TYPE == kTE4m3Exact ? 4 : SM == kRowScale ? 8 : 5;
        // Rows of A in turn: while the matrix instructions of one run, the
        // next one's operand comes from LDS, and the sums of the last one
        // are scaled and added.
        v4i a[2][2];
        v4f t[2][SM == kNoScale ? 1 : TN];
        auto read_a = [&](int i) __attribute__((always_inline)) {
            if constexpr (AT) {
                read_t<BM>(a[i & 1], buf, wm * TM + i, lane);
            } else {
                a[i & 1][0] = *(const v4i*)(buf + ao + i * 16 * kStep);
                a[i & 1][1] = *(const v4i*)(buf + (ao ^ 64) + i * 16 * kStep);
            }
        };
        read_a(0);
        auto add = [&](int i) __attribute__((always_inline)) {
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
            if (i + 1 < TM)
                read_a(i + 1);
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                if constexpr (TYPE == kTI8)
                    acc[i][j] = matrix_step_i8(b[j], a[i & 1], acc[i][j]);
                else if constexpr (SM == kNoScale)
                    acc[i][j] = matrix_step<TYPE>(b[j], a[i & 1], acc[i][j]);
                else
                    t[i & 1][j] = matrix_step<TYPE>(b[j], a[i & 1], v4f{0.f, 0.f, 0.f, 0.f});
            }
            if constexpr (SM != kNoScale)
                if (i > 0)
                    add(i - 1);
            // (after the first rows' matrix instructions are on their way)
            if constexpr (!REG)
                if (i == 0 && kt + (NS - 1) * WK < nk)
                    stage(kt + (NS - 1) * WK);
            if (i + 1 < TM)
                __builtin_amdgcn_sched_group_barrier(0x100, AT ? 4 : 2, 0);   // LDS reads
            if constexpr (SM != kNoScale) {
#pragma unroll
                for (int j = 0; j < TN * kMfmas; ++j) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // matrix
                    __builtin_amdgcn_sched_group_barrier(0x002, kValus, 0);   // vector
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (SM != kNoScale)
            add(TM - 1);
        if constexpr (REG) {
            if (kt + 1 < nk)
                put(kt + 1, from);
        }
        return true;
    };

    if constexpr (PIPE) {
        // (for the same tiles without: grouped bf16 m 16384 e 8 n 8192 k 4096 982 us,
        // 964 so; int8 m 8192 n 4096 k 16384 420 and 412)
        // Half a step's operands in registers ahead of its matrix instructions:
        // a row block of A is replaced by the next half's as soon as its four
        // have been issued, so the waves of a SIMD have matrix instructions on both
        // sides of the barrier.  At the barrier, in a step's second half, all of
        // the step has been read, so its buffer takes the step after the next, whose
        // loads have a step's time; the next step's have arrived.
        static_assert(!PIPE || (!REG && SM == kNoScale && WK == 1 && NS == 2 && TM >= TN + 1), "PIPE");
        constexpr int kAt = 1;       // row blocks of the second half before the barrier
        v4i a[TM], b[2][TN];
        const auto read_a = [&](const unsigned char* buf, int h, int i) __attribute__((always_inline)) {
            if constexpr (AT)
                return read_t_half<BM>(buf, wm * TM + i, lane, h);
            else
                return *(const v4i*)(buf + (ao ^ (h * 64)) + i * 16 * kStep);
        };
        const auto read_b = [&](const unsigned char* buf, int h, int j) __attribute__((always_inline)) {
            const int row = kDual && j >= TN / 2 ? BNO + (j - TN / 2) * 16 : j * 16;
            if constexpr (BT)
                return read_t_half<BN, kWide>(buf + BM * kStep, wn * TN + j, lane, h);
            else
                return *(const v4i*)(buf + (bo ^ (h * 64)) + row * kStep);
        };
        const auto ragged = [&](int kt) __attribute__((always_inline)) {
            return ktail && (kt == all - 1 || (p.parts > 1 && kt == nks - 1));
        };
        if (first + 1 < nk) {
            stage(first + 1);
            wait_vm<kLoads>();
        } else {
            wait_vm<0>();
        }
        __syncthreads();
        if (first < nk && ragged(first)) {
            cut(first, lds + buffer_of(first));
            __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < TN; ++j)
            b[0][j] = read_b(lds + buffer_of(first), 0, j);
#pragma unroll
        for (int i = 0; i < TM; ++i)
            a[i] = read_a(lds + buffer_of(first), 0, i);
        // The next step's data have arrived, and all of this one's have been read.
        const auto turn = [&](int kt) __attribute__((always_inline)) {
            wait_vm<0>();
            __syncthreads();
            if (kt + 1 < nk && ragged(kt + 1)) {
                cut(kt + 1, lds + buffer_of(kt + 1));
                __syncthreads();
            }
            if (kt + 2 < nk)
                stage(kt + 2);
        };
        if (wm * TM * 16 >= mrows) {
            // a wave without rows: the others have the matrix units for themselves
            for (int kt = first; kt < nk; ++kt)
                turn(kt);
            return;
        }
        for (int kt = first; kt < nk; ++kt) {
            unsigned char* const cur = lds + buffer_of(kt);
            unsigned char* const next = lds + buffer_of(kt + 1);
#pragma unroll
            for (int i = 0; i < TM; ++i) {
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    acc[i][j] = half_step<TYPE>(b[0][j], a[i], acc[i][j]);
                a[i] = read_a(cur, 1, i);
                if (i < TN)
                    b[1][i] = read_b(cur, 1, i);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int i = 0; i < TM; ++i) {
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    acc[i][j] = half_step<TYPE>(b[1][j], a[i], acc[i][j]);
                if (i == kAt) {
                    turn(kt);
#pragma unroll
                    for (int e = 0; e < kAt; ++e)
                        a[e] = read_a(next, 0, e);
                }
                if (i >= kAt)
                    a[i] = read_a(next, 0, i);
                if (i >= kAt && i - kAt < TN)
                    b[0][i - kAt] = read_b(next, 0, i - kAt);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    } else if constexpr (kAhead > 1) {
        v4i held[2][GA + GB];
        fetch(first + 1 < nk ? first + 1 : first, held[1]);
        for (int kt = first; kt < nk; kt += 2) {
            step(kt, held[0], held[1]);
            if (kt + 1 < nk)
                step(kt + 1, held[1], held[0]);
        }
    } else {
        v4i held[REG ? GA + GB : 1];
        for (int kt = first + kg; kt - kg < nk; kt += WK)
            if (!step(kt, held, held))
                break;
    }

    // The groups' sums join in LDS, in the groups' order.
    if constexpr (WK > 1) {
        Sums<TYPE>* sums = (Sums<TYPE>*)lds;     // [group - 1][i][j][thread]
        __syncthreads();
        if (kg > 0) {
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    sums[(((kg - 1) * TM + i) * TN + j) * 64 * W + tid] = acc[i][j];
        }
        __syncthreads();
        if (kg > 0)
            return;
#pragma unroll
        for (int g = 0; g < WK - 1; ++g)
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    acc[i][j] += sums[((g * TM + i) * TN + j) * 64 * W + tid];
    }

    if (p.splits > 1) {        // the shares' sums join in join_kernel
        Sums<TYPE>* out =
            (Sums<TYPE>*)p.partial + (part * where.tiles() + where.tile()) * (TM * TN * 64 * W) + tid;
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                out[(i * TN + j) * 64 * W] = acc[i][j];
        return;
    }
    finish_rows<TYPE, BM, BN, WM, WN, EP, AT, kWide>(p, acc, 0, 0, tm, tn, wave, lane);
}

template <int TYPE, int BM, int BN, int WM, int WN, int WK, int NS, int EP, int SM, int REG,
          bool AT, bool BT, bool PIPE = false, bool WIDE = PIPE>
__global__ __launch_bounds__(64 * WM * WN * WK) __attribute__((amdgpu_waves_per_eu(2))) void
product_kernel(const ProductArgs p)
{
    if constexpr (TYPE == kTF16 && EP == kEpGateGrad) {
        if (p.again && range_exponent(p.range) == 0)
            return;
    }
    int tm, tn;
    tile_of((int)blockIdx.x, p.tiles_m, p.tiles_n, tm, tn);
    product_body<TYPE, BM, BN, WM, WN, WK, NS, EP, SM, REG, AT, BT, PIPE, WIDE>(
        p, tm, tn, (int)blockIdx.y, EveryWorkgroup{});
}

// The shares of a tile's contraction, added in their order: a workgroup for
// each 16 x 16 block of its waves (gated: gate's and up's), so that few tiles
// still spread over the CUs, and eight shares' loads in flight (f16 m 862 n
// 15195 k 67, gradients: the join of 7 tiles in 16 shares takes 4.9 us, 7.3
// with 16 rows of A and all of B to a workgroup).
template <int TYPE, int BM, int BN, int WM, int WN, int EP, bool AT, bool WIDE, class Where>
__device__ __forceinline__ void join_body(const ProductArgs& p, const Where& where)
{
    constexpr int W = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;
    constexpr int P = EP != kEpStore ? 2 : 1, TJ = TN / P;
    constexpr int kAhead = 8;
    using Four = Sums<TYPE>;
    const int64_t stride = where.tiles() * (TM * TN * 64 * W);
    const int i = (int)blockIdx.y, j = (int)blockIdx.z;
    const Four* in = (const Four*)p.partial + where.tile() * (TM * TN * 64 * W) +
                     (i * TN + j) * 64 * W + threadIdx.x;
    Four acc[1][P];
#pragma unroll
    for (int h = 0; h < P; ++h)
        acc[0][h] = in[h * TJ * 64 * W];
    for (int s = 1; s < p.splits; s += kAhead) {
        Four more[kAhead][P];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int h = 0; h < P; ++h)
                more[u][h] = in[(s + u < p.splits ? s + u : s) * stride + h * TJ * 64 * W];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (s + u < p.splits)
#pragma unroll
                for (int h = 0; h < P; ++h)
                    acc[0][h] += more[u][h];
    }
    int tm, tn;
    where.place(p, tm, tn);
    finish_rows<TYPE, BM, BN, WM, WN, EP, AT, WIDE>(
        p, acc, i, j, tm, tn, __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6),
        threadIdx.x & 63);
}

template <int TYPE, int BM, int BN, int WM, int WN, int EP, bool AT, bool WIDE = false>
__global__ __launch_bounds__(64 * WM * WN) void join_kernel(const ProductArgs p)
{
    if constexpr (TYPE == kTF16 && EP == kEpGateGrad) {
        if (p.again && range_exponent(p.range) == 0)
            return;
    }
    join_body<TYPE, BM, BN, WM, WN, EP, AT, WIDE>(p, EveryWorkgroup{});
}

// Tiles whose steps the choices below share: none of 256, of 8-bit integers the smallest.
template <int TYPE, int BM, int BN>
constexpr bool may_split()
{
    return TYPE == kTI8 ? BM == 64 && BN == 64 : BM <= 128 && BN <= 128;
}

template <int TYPE, int BM, int BN, int WM, int WN, int WK, int NS, int EP, int SM, int REG = kAligned,
          bool AT = false, bool BT = false, bool PIPE = false, bool WIDE = PIPE>
hipError_t run(ProductArgs p, int splits, hipStream_t stream)
{
    p.splits = splits;
    constexpr int BNO = EP != kEpStore ? BN / 2 : BN;
    constexpr size_t kLds = WK * NS * (size_t)(BM + BN) * (kStep + (SM != kNoScale ? 4 : 0));
    static_assert(kLds <= 160 * 1024 && (size_t)(WK - 1) * BM * BN * 4 <= kLds, "LDS of a CU");
    p.tiles_m = (int)((p.m + BM - 1) / BM);
    p.tiles_n = (int)((p.n + BNO - 1) / BNO);
    auto* k = &product_kernel<TYPE, BM, BN, WM, WN, WK, NS, EP, SM, REG, AT, BT, PIPE, WIDE>;
    if (kLds > 65536) {
        // once for each device
        static std::atomic<uint64_t> done{0};
        int dev = 0;
        hipError_t e = hipGetDevice(&dev);
        if (e == hipSuccess && (dev >= 64 || !((done.load() >> dev) & 1))) {
            e = hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)kLds);
            if (e == hipSuccess && dev < 64)
                done.fetch_or((uint64_t)1 << dev);
        }
        if (e != hipSuccess)
            return e;
    }
    const unsigned tiles = (unsigned)(p.tiles_m * p.tiles_n);
    hipError_t e = hipSuccess;
    if (splits == 1 || !p.again) {           // (the shares' sums are still there)
        hipLaunchKernelGGL(k, dim3(tiles, (unsigned)splits), dim3(64 * WM * WN * WK), kLds, stream, p);
        e = hipGetLastError();
    }
    if (splits == 1 || e != hipSuccess)
        return e;
    if constexpr (may_split<TYPE, BM, BN>()) {
        const dim3 grid(tiles, BM / WM / 16, BNO / WN / 16);
        hipLaunchKernelGGL((join_kernel<TYPE, BM, BN, WM, WN, EP, AT, WIDE>), grid, dim3(64 * WM * WN), 0,
                           stream, p);
    }
    return hipGetLastError();
}

struct Tile {
    int bm, bn, slots;   // bn: output columns
    float step;
    int area;            // of the sums, 0: not split
};
struct Choice {
    int tile, splits;
    size_t bytes;        // of ProductArgs::partial
};
template <int N>
Choice cheapest(const Tile (&tiles)[N], const ProductArgs& p)
{
    const int64_t steps = (p.kbytes + kStep - 1) / kStep * (p.parts > 1 ? 2 : 1);
    Choice best{0, 1, 0};
    double least = 0;
    for (int i = 0; i < N; ++i) {
        const Tile& t = tiles[i];
        const int64_t count = ((p.m + t.bm - 1) / t.bm) * ((p.n + t.bn - 1) / t.bn);
        double cost = count >= kFfnMaxTiles
                          ? 1e300
                          : (double)((count + t.slots - 1) / t.slots) * t.step * steps;
        int splits = 1;
        if (t.area && p.may_split && count * 2 <= t.slots) {
            int64_t s = t.slots / count < 32 ? t.slots / count : 32;
            s = s < steps / 4 ? s : steps / 4;
            // every share has steps, the last one fewer
            s = s > 1 ? (steps + (steps + s - 1) / s - 1) / ((steps + s - 1) / s) : 1;
            const double shared = (double)((steps + s - 1) / s) * t.step + 5.0;
            if (s > 1 && shared < cost) {
                cost = shared;
                splits = (int)s;
            }
        }
        if (i == 0 || cost < least) {
            least = cost;
            best = Choice{i, splits, splits > 1 ? (size_t)splits * count * t.area * 4 : 0};
        }
    }
    return best;
}

}  // namespace
}  // namespace qse
