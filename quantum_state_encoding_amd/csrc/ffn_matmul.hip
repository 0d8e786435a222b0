// Products A B^T on the matrix cores, with the epilogues of the gated block.
//
// C[m][n] = sum_k A[m][k] B[n][k].  e4m3 operands carry a scale for each
// 128 of k: C = sum over k blocks of sa[kb][m] sb[kb][n] P_kb, with P_kb
// the product of the codes in one matrix instruction of 128 (32-bit sums),
// and the weighted sum over kb in 32 bits in registers.
//
// A workgroup computes a BM x BN tile.  Each step stages 128 bytes of every
// row of A and B (one k block of e4m3, 64 16-bit elements) into LDS, straight
// from memory, while earlier ones feed the matrix instructions: 256 x 256
// where the tiles fill the CUs, since a step's operands then feed most
// instructions, smaller ones for fewer rows.
//
// What bounds it: large products the matrix units and their clock (about
// 1.9 GHz in such a kernel; busy 54-69 % of the CUs' cycles), then the
// prologue and the stores of each round of tiles (8-14 us a round of 256).
// Measured, with what the library's largest products (8192^3) reach on the
// same card in parentheses: e4m3 m 8192 n 4096 k 16384 458 us, 2400 TFLOP/s
// (2772); gated e4m3 m 8192 n 16384 k 4096 970 us, 2270; fp32 out, row scales
// m 4096 n 4096 k 8192 258 us, 1065 (1459, f16: the instruction it uses);
// gated bf16's gradients m 4096 n 8192 k 4096 1333 us, 1237 (1362).  Small
// ones the launch and the latency of one tile: e4m3 m 333 n 4100 k 2056
// 13.1 us (bf16 out; f16 14.9).
#include <hip/hip_runtime.h>

#include <atomic>
#include <type_traits>

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

// An operand that is stored with its rows side by side, [k][rows] (AT, BT;
// 16-bit types): a step stages 64 k of it as they are, and the transposing
// LDS read gives a lane four k of its row.  Its 16 lanes take four k rows of
// 32 bytes each, so those 32-byte units are spread over the banks by k.
__device__ __forceinline__ int unit_mask(int k) { return (k & 3) | ((k >> 3) & 1) << 2; }

template <int BR>
__device__ __forceinline__ void read_t(v4i (&out)[2], const unsigned char* tile, int block, int lane)
{
    typedef short v4s __attribute__((ext_vector_type(4)));
    const int q = lane >> 4, l16 = lane & 15;
    const unsigned char* at = tile + (q * 8 + (l16 >> 2)) * (BR * 2) +
                              ((block ^ unit_mask(q * 8 + (l16 >> 2))) * 32) + (l16 & 3) * 8;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        v4s r[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
            r[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) v4s*)(at + (h * 32 + e * 4) * (BR * 2)));
        out[h] = __builtin_bit_cast(v4i, __builtin_shufflevector(r[0], r[1], 0, 1, 2, 3, 4, 5, 6, 7));
    }
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
template <int TYPE, int BM, int BN, int WM, int WN, int EP, bool AT, int NI, int TN, int ACT,
          bool WHOLE>
__device__ __forceinline__ void finish_rows_as(const ProductArgs& p, const v4f (&acc)[NI][TN],
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
                      : TYPE != kTE4m3Exact ? TYPE
                      : p.ctype == kTF32    ? (int)kTF32
                                            : (int)kTF16;
    const int act = ACT < 0 ? p.act : ACT;
    const auto row_at = [=](int i) __attribute__((always_inline)) {
        return wm * (TM * 16) + (AT ? (i0 + i) * 16 + l16 : l16 * TM + i0 + i);
    };
    const auto column_at = [=](int j) __attribute__((always_inline)) {
        return wn * kRowsB + (j0 + j) * 16 + q * 4;
    };
    const auto count_at = [=](int nc) __attribute__((always_inline)) {
        return WHOLE || nrows - nc > 4 ? 4 : nrows - nc;
    };
    // f16 gradients: the factor that dg and du are stored with, or that the
    // sums of what was stored so are multiplied by
    constexpr bool kGrad16 = EP == kEpGateGrad && TYPE == kTF16;
    float factor = 1.0f;
    if constexpr (TYPE == kTF16 && EP != kEpGate) {
        if (EP == kEpStore)
            factor = power_of_two(range_exponent(p.range));
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
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int r = row_at(i);
        if (!WHOLE && r >= mrows)
            continue;
        int64_t m = m0 + r;
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
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
            const int nc = column_at(j);
            if (!WHOLE && nc >= nrows)
                continue;
            const int64_t at = m * ldc + n0 + nc;
            v4f v = acc[i][j], u;
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
            store4(c, at, v, ctype, count_at(nc));
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

template <int TYPE, int BM, int BN, int WM, int WN, int EP, bool AT, int NI, int TN>
__device__ __forceinline__ void finish_rows(const ProductArgs& p, const v4f (&acc)[NI][TN], int i0,
                                            int j0, int tm, int tn, int wave, int lane)
{
    constexpr int BNO = EP != kEpStore ? BN / 2 : BN;
    if ((int64_t)(tm + 1) * BM > p.m || (int64_t)(tn + 1) * BNO > p.n)
        finish_rows_as<TYPE, BM, BN, WM, WN, EP, AT, NI, TN, -1, false>(p, acc, i0, j0, tm, tn, wave, lane);
    else if (EP == kEpStore || p.act == 0)
        finish_rows_as<TYPE, BM, BN, WM, WN, EP, AT, NI, TN, 0, true>(p, acc, i0, j0, tm, tn, wave, lane);
    else
        finish_rows_as<TYPE, BM, BN, WM, WN, EP, AT, NI, TN, 1, true>(p, acc, i0, j0, tm, tn, wave, lane);
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
template <int TYPE, int BM, int BN, int WM, int WN, int WK, int NS, int EP, int SM, int REG,
          bool AT, bool BT>
__global__ __launch_bounds__(64 * WM * WN * WK) __attribute__((amdgpu_waves_per_eu(2))) void
product_kernel(const ProductArgs p)
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

    if constexpr (TYPE == kTF16 && EP == kEpGateGrad) {
        if (p.again && range_exponent(p.range) == 0)
            return;
    }
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(((int)threadIdx.x >> 6) % W);
    const int kg = __builtin_amdgcn_readfirstlane((int)threadIdx.x / (64 * W));
    const int tid = (int)threadIdx.x - kg * 64 * W;   // in the group
    const int wm = wave / WN, wn = wave % WN;
    int tm, tn;
    tile_of((int)blockIdx.x, p.tiles_m, p.tiles_n, tm, tn);
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
    const int first = (int)blockIdx.y * share;
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
    const int rb0 = wave * 8 + lr;
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

    v4f acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
            acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

    // Scales: rows of A stand on lanes, TM consecutive ones on a lane (that is
    // what row_of is for), rows of B on the four registers of a result.
    const int q = lane >> 4, l16 = lane & 15;
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

    for (int kt = first + kg; kt - kg < nk; kt += WK) {
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
            __syncthreads();
        }
        v4i held[REG ? GA + GB : 1];
        if constexpr (REG == kAnyAddress)
            fetch(kt + 1 < nk ? kt + 1 : kt, held);
        else if constexpr (REG == kShortRows)
            fetch_short(kt + 1 < nk ? kt + 1 : kt, held);
        if (WK > 1 && kt >= nk)
            break;     // (the last round: no barrier follows in the loop)
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
                read_t<BN>(b[j], buf + BM * kStep, wn * TN + j, lane);
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
                if constexpr (SM == kNoScale)
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
                put(kt + 1, held);
        }
    }

    // The groups' sums join in LDS, in the groups' order.
    if constexpr (WK > 1) {
        v4f* sums = (v4f*)lds;     // [group - 1][i][j][thread]
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
        v4f* out = (v4f*)p.partial +
                   ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (TM * TN * 64 * W) + tid;
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                out[(i * TN + j) * 64 * W] = acc[i][j];
        return;
    }
    finish_rows<TYPE, BM, BN, WM, WN, EP, AT>(p, acc, 0, 0, tm, tn, wave, lane);
}

// The shares of a tile's contraction, added in their order: a workgroup for
// each 16 x 16 block of its waves (gated: gate's and up's), so that few tiles
// still spread over the CUs, and eight shares' loads in flight (f16 m 862 n
// 15195 k 67, gradients: the join of 7 tiles in 16 shares takes 4.9 us, 7.3
// with 16 rows of A and all of B to a workgroup).
template <int TYPE, int BM, int BN, int WM, int WN, int EP, bool AT>
__global__ __launch_bounds__(64 * WM * WN) void join_kernel(const ProductArgs p)
{
    constexpr int W = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;
    constexpr int P = EP != kEpStore ? 2 : 1, TJ = TN / P;
    constexpr int kAhead = 8;
    if constexpr (TYPE == kTF16 && EP == kEpGateGrad) {
        if (p.again && range_exponent(p.range) == 0)
            return;
    }
    const int64_t stride = (int64_t)gridDim.x * (TM * TN * 64 * W);
    const int i = (int)blockIdx.y, j = (int)blockIdx.z;
    const v4f* in = (const v4f*)p.partial + (int64_t)blockIdx.x * (TM * TN * 64 * W) +
                    (i * TN + j) * 64 * W + threadIdx.x;
    v4f acc[1][P];
#pragma unroll
    for (int h = 0; h < P; ++h)
        acc[0][h] = in[h * TJ * 64 * W];
    for (int s = 1; s < p.splits; s += kAhead) {
        v4f more[kAhead][P];
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
    tile_of((int)blockIdx.x, p.tiles_m, p.tiles_n, tm, tn);
    finish_rows<TYPE, BM, BN, WM, WN, EP, AT>(p, acc, i, j, tm, tn,
                                              __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6),
                                              threadIdx.x & 63);
}

template <int TYPE, int BM, int BN, int WM, int WN, int WK, int NS, int EP, int SM, int REG = kAligned,
          bool AT = false, bool BT = false>
hipError_t run(ProductArgs p, int splits, hipStream_t stream)
{
    p.splits = splits;
    constexpr int BNO = EP != kEpStore ? BN / 2 : BN;
    constexpr size_t kLds = WK * NS * (size_t)(BM + BN) * (kStep + (SM != kNoScale ? 4 : 0));
    static_assert(kLds <= 160 * 1024 && (size_t)(WK - 1) * BM * BN * 4 <= kLds, "LDS of a CU");
    p.tiles_m = (int)((p.m + BM - 1) / BM);
    p.tiles_n = (int)((p.n + BNO - 1) / BNO);
    auto* k = &product_kernel<TYPE, BM, BN, WM, WN, WK, NS, EP, SM, REG, AT, BT>;
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
    if constexpr (BM <= 128 && BN <= 128) {      // (larger tiles are never split)
        const dim3 grid(tiles, BM / WM / 16, BNO / WN / 16);
        hipLaunchKernelGGL((join_kernel<TYPE, BM, BN, WM, WN, EP, AT>), grid, dim3(64 * WM * WN), 0,
                           stream, p);
    }
    return hipGetLastError();
}

// Which tile.  A round of workgroups (one on each of 256 CUs, or two where
// two fit) takes about a fixed time for each 128-byte step of k, so a product
// takes ceil(tiles / slots) of those.  Microseconds a step, measured with full
// rounds at k of 16384 bytes and more:
//                                  slots   e4m3   exact(+)   16 bits
//   256 x 256                        256   1.75      -         1.6
//   128 x 128, two on a CU           512   1.05     2.0        1.06
//   128 x 128, deeper (*)            256   0.65     1.1        0.62
//   64 x 64, two on a CU             512   0.40     0.70        -
//   64 x 64 (gated: 64 x 128)        256   0.26     0.36       0.42
// (+) e4m3 with an f16 or fp32 result, through the 16-bit instruction.
// (*) two groups of waves for e4m3, four rounds in LDS for 16 bits.  So m 512
// n 4096 k 16384 (e4m3) takes 49 us with 64 x 64 tiles and 82 with 128 x 128
// ones, m 4096 takes 451 and 260, and 227 with 256 x 256 ones.
//
// With a scale for each row of B the two 128 x 128 tiles of a CU take 1.2 us a step
// instead of 1.05 and the others 2-10 % more; the table is the same.
//
// Where the tiles leave half of their slots empty, the workgroups of a tile
// share its steps and a second kernel adds their sums, for about 5 us: m 300
// n 200 k 16000 (fp32 out) takes 44 us in one share, 16 in twelve.  At most
// 32 shares (gradients of bf16 m 862 n 15195 k 67: 16 115 us, 32 99).
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

// 16-bit operands at any address.  Microseconds a step as above: 256 x 256 1.85
// and two 128 x 128 on a CU 1.2 where addresses are multiples of 4 bytes, 2.3 and
// 2.1 at others, where the same two numbers choose.  query: the bytes of
// ProductArgs::partial instead of a launch.
template <int TYPE, int EP, bool AT, bool BT>
hipError_t pick_any(const ProductArgs& p, size_t* query, hipStream_t stream)
{
    const int64_t lena = AT ? p.m * 2 : p.kbytes, lenb = BT ? p.n * 2 : p.kbytes;
    constexpr bool dual = EP != kEpStore;
    constexpr Tile tiles[] = {{256, dual ? 128 : 256, 256, 1.9f, 0},
                              {128, dual ? 64 : 128, 512, 1.2f, 128 * 128}};
    const Choice c = cheapest(tiles, p);
    if (query) {
        *query = c.bytes;
        return hipSuccess;
    }
    if (lena < 16 || lenb < 16)
        return run<TYPE, 128, 128, 2, 2, 1, 2, EP, kNoScale, kShortRows, AT, BT>(p, 1, stream);
    if (c.tile == 0)
        return run<TYPE, 256, 256, 2, 4, 1, 2, EP, kNoScale, kAnyAddress, AT, BT>(p, 1, stream);
    return run<TYPE, 128, 128, 2, 2, 1, 2, EP, kNoScale, kAnyAddress, AT, BT>(p, c.splits, stream);
}

// 16-bit operands.
template <int TYPE, int EP, bool AT, bool BT>
hipError_t pick16(const ProductArgs& p, size_t* query, hipStream_t stream)
{
    size_t any_bytes = 0;
    if (query) {
        (void)pick_any<TYPE, EP, AT, BT>(p, &any_bytes, stream);
    } else {
        const uintptr_t any = (uintptr_t)p.a | (uintptr_t)p.b0 | (uintptr_t)p.b1 |
                              (uintptr_t)p.lda | (uintptr_t)p.ldb0 | (uintptr_t)p.ldb1;
        if (any & 15)
            return pick_any<TYPE, EP, AT, BT>(p, nullptr, stream);
    }
    constexpr bool dual = EP != kEpStore;
    // (A of 64 rows cannot be [k][rows]: a wave stages whole KiB of it)
    constexpr Tile tiles[] = {{256, dual ? 128 : 256, 256, 1.6f, 0},
                              {128, dual ? 64 : 128, 512, 1.06f, 0},
                              {128, dual ? 64 : 128, 256, .62f, 128 * 128},
                              {64, dual ? 64 : 128, 256, AT ? 1e30f : .42f, 64 * 128}};
    const Choice c = cheapest(tiles, p);
    if (query) {
        *query = any_bytes > c.bytes ? any_bytes : c.bytes;
        return hipSuccess;
    }
    switch (c.tile) {
    case 0:
        return run<TYPE, 256, 256, 2, 4, 1, 2, EP, kNoScale, kAligned, AT, BT>(p, 1, stream);
    case 1:
        return run<TYPE, 128, 128, 2, 2, 1, 2, EP, kNoScale, kAligned, AT, BT>(p, 1, stream);
    case 2:
        return run<TYPE, 128, 128, 2, 2, 1, 4, EP, kNoScale, kAligned, AT, BT>(p, c.splits, stream);
    }
    if constexpr (!AT)
        return run<TYPE, 64, 128, 1, 4, 1, 4, EP, kNoScale, kAligned, AT, BT>(p, c.splits, stream);
    return hipErrorInvalidValue;
}

// e4m3 operands.  The widened operands of an f16 or fp32 result, or a scale for
// each row of B, leave no registers for the largest tile.
template <int TYPE, int EP, int SM>
hipError_t pick8(const ProductArgs& p, size_t* query, hipStream_t stream)
{
    constexpr bool exact = TYPE == kTE4m3Exact, dual = EP != kEpStore;
    constexpr float never = 1e30f;
    constexpr float large = exact || SM == kRowScale ? never : 1.75f;
    constexpr Tile tiles[] = {
        {256, dual ? 128 : 256, 256, large, 0},
        {128, dual ? 64 : 128, 512, exact ? 2.0f : 1.05f, 0},
        {128, dual ? 64 : 128, 256, exact ? 1.1f : .65f, 0},
        {64, 64, dual ? 256 : 512, dual ? (exact ? .60f : .40f) : exact ? .70f : .40f,
         dual ? 64 * 128 : 0},
        {64, 64, 256, dual ? never : exact ? .36f : .26f, 64 * 64}};
    const Choice c = cheapest(tiles, p);
    if (query) {
        *query = c.bytes;
        return hipSuccess;
    }
    switch (c.tile) {
    case 1:
        return run<TYPE, 128, 128, 2, 2, 1, 2, EP, SM>(p, 1, stream);
    case 2:
        return run<TYPE, 128, 128, 2, 2, 2, 2, EP, SM>(p, 1, stream);
    case 3:
        if constexpr (dual)
            return run<TYPE, 64, 128, 1, 4, 3, 2, EP, SM>(p, c.splits, stream);
        else
            return run<TYPE, 64, 64, 2, 2, 2, 2, EP, SM>(p, 1, stream);
    case 4:
        // (f16 and fp32 results: four groups of waves 10-15 % faster than two
        // with four rounds in LDS; bf16 results 5-10 % slower)
        if constexpr (!dual)
            return run<TYPE, 64, 64, 2, 2, exact ? 4 : 2, exact ? 2 : 4, EP, SM>(p, c.splits, stream);
    }
    if constexpr (large != never)
        return run<TYPE, 256, 256, 2, 4, 1, 2, EP, SM>(p, 1, stream);
    return hipErrorInvalidValue;
}

template <int TYPE>
hipError_t launch16(const ProductArgs& p, int ep, size_t* query, hipStream_t stream)
{
    if (ep == kEpGate)
        return pick16<TYPE, kEpGate, false, false>(p, query, stream);
    if (ep == kEpGateGrad)
        return pick16<TYPE, kEpGateGrad, false, false>(p, query, stream);
    return ep == kEpStoreT ? pick16<TYPE, kEpStore, true, true>(p, query, stream)
                           : pick16<TYPE, kEpStore, false, true>(p, query, stream);
}

template <int TYPE>
hipError_t launch8(const ProductArgs& p, int ep, bool row_scales, size_t* query, hipStream_t stream)
{
    if (ep == kEpGate)
        return pick8<TYPE, kEpGate, kTileScale>(p, query, stream);
    return row_scales ? pick8<TYPE, kEpStore, kRowScale>(p, query, stream)
                      : pick8<TYPE, kEpStore, kTileScale>(p, query, stream);
}

hipError_t tiles_for(const ProductArgs& p, int type, int ep, bool row_scales, size_t* query,
                     hipStream_t stream)
{
    if (type == kTE4m3)
        return p.ctype != kTBf16 ? launch8<kTE4m3Exact>(p, ep, row_scales, query, stream)
                                 : launch8<kTE4m3>(p, ep, row_scales, query, stream);
    return type == kTBf16 ? launch16<kTBf16>(p, ep, query, stream)
                          : launch16<kTF16>(p, ep, query, stream);
}

// Few rows: the strip kernel, except where 64-row tiles fill the CUs and their
// shared rows of A pay: e4m3 n 16384 k 4096 takes 13.3 us with tiles and 18.0
// with strips at m = 16 (12.5 and 13.1 at m = 1), n 4096 k 16384 33 and 19;
// gated bf16 n 16384 k 4096 takes 53 and 66 us at m = 32, 52 and 51 at 16.
// A tile widens all its codes for an f16 or fp32 result, used or not, a strip
// those it reads: n 16384 k 4096 takes 17.3 us with tiles and 12.9 with strips
// at m = 1, 17.9 and 15.1 at 8, 17.9 and 18.0 at 16 (tile scales; with row
// scales 18.1, 18.4 and 18.5, and 17.6, 19.8 and 22.4).
bool strips(const ProductArgs& p, int type, int ep, bool row_scales)
{
    if (p.m > kStripRows || ep == kEpGateGrad || (ep != kEpGate && type != kTE4m3))
        return false;
    if ((p.n + 63) / 64 < 256)
        return true;
    const bool few = ep == kEpGate ? p.m <= 16 : p.ctype != kTBf16 && !row_scales && p.m <= 8;
    return few && (p.n + 15) / 16 < kFfnMaxTiles;
}

}  // namespace

hipError_t launch_product(const ProductArgs& p, int type, int ep, bool row_scales,
                          hipStream_t stream)
{
    if (strips(p, type, ep, row_scales))
        return launch_strip(p, type, ep, row_scales, stream);
    return tiles_for(p, type, ep, row_scales, nullptr, stream);
}

size_t product_workspace(ProductArgs p, int type, int ep, bool row_scales)
{
    size_t bytes = 0;
    p.may_split = 1;
    if (!strips(p, type, ep, row_scales))
        (void)tiles_for(p, type, ep, row_scales, &bytes, nullptr);
    return bytes;
}

}  // namespace qse
