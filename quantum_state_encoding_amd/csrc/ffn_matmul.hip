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
// instructions, smaller ones for fewer rows.  The tile itself is in ffn_product.h.
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

#include "ffn_product.h"

namespace qse {
namespace {

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
