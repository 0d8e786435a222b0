// Products of 8-bit integers with a scale for each row of A and of B:
// C[m][n] = sa[m] sb[n] sum_k A[m][k] B[n][k], in ffn_matmul.hip's tiles and
// ffn_strip.hip's strips.  The sums are 32-bit integers, exact, so neither the
// tile nor the number of shares changes a result; the scales are the epilogue.
//
// Measured: m 8192 n 4096 k 16384 401-431 us by the card, 2.55-2.74 P operations/s
// (the library's 8192^3 on one of them: 2.16), the matrix units busy 65 % of the
// cycles; m 333 n 4100 k 2056 11.9 us, one tile's first loads, 17 steps and stores;
// one token, n 16384 k 4096, 12.2 us where the weights are in the caches (5.5 TB/s),
// 18.6 where they are not.
#include <hip/hip_runtime.h>

#include "ffn_product.h"
#include "ffn_strip.h"

namespace qse {
namespace {

template <int BM, int BN, int WM, int WN, int WK, int NS>
hipError_t run_int8(const ProductArgs& p, int splits, hipStream_t stream)
{
    return run<kTI8, BM, BN, WM, WN, WK, NS, kEpStore, kNoScale, kAligned, false, false, BM == 256,
               true>(p, splits, stream);
}

// Microseconds a step of 128, as ffn_matmul.hip's table has them; tiles of 64 x 128
// with four steps in LDS took the place of two 64 x 64 ones on a CU (m 128 n 16384
// k 4096: 22.3 us and 19.5), and four steps for 128 x 128 that of two groups of waves
// (m 5327 n 435 k 2730: 22.9 and 20.1).
hipError_t tiles_int8(const ProductArgs& p, size_t* query, hipStream_t stream)
{
    constexpr Tile tiles[] = {{256, 256, 256, 1.5f, 0},
                              {128, 128, 512, 1.0f, 0},
                              {128, 128, 256, .60f, 0},
                              {64, 128, 256, .42f, 0},
                              {64, 64, 256, .26f, 64 * 64}};
    const Choice c = cheapest(tiles, p);
    if (query) {
        *query = c.bytes;
        return hipSuccess;
    }
    switch (c.tile) {
    case 0:
        return run_int8<256, 256, 2, 4, 1, 2>(p, 1, stream);
    case 1:
        return run_int8<128, 128, 2, 2, 1, 2>(p, 1, stream);
    case 2:
        return run_int8<128, 128, 2, 2, 1, 4>(p, 1, stream);
    case 3:
        return run_int8<64, 128, 1, 4, 1, 4>(p, 1, stream);
    }
    return run_int8<64, 64, 2, 2, 2, 4>(p, c.splits, stream);
}

// Few rows of A, unless the tiles fill the CUs.  Microseconds in strips and in tiles, of 1,
// 16 and 32 rows, weights from memory: n 1024 k 4096 4.9 7.5, 6.4 7.5, 8.3 7.6; n 4096
// k 4096 6.3 10.6, 8.1 10.6, 9.5 10.7; n 8192 k 8192 15.2 22.1, 21.2 22.2, 26.4 22.7; and
// where tiles are taken, n 16384 k 4096 15.5 18.6, 21.1 19.2, 26.0 19.6; n 32768 k 4096
// 27.9 35.1, 36.4 36.5, 47.6 36.8; n 65536 k 2048 32.0 29.3, 38.5 30.7, 47.8 31.6.  (The
// number of rows has a say too, which the rule leaves out: up to a quarter, for one row of
// n 32768.)
bool strips(const ProductArgs& p) { return p.m <= kStripRows && (p.n + 63) / 64 < 256; }

template <int MT, int W, int U>
hipError_t strip(const ProductArgs& p, hipStream_t stream)
{
    hipLaunchKernelGGL((strip_kernel<kTI8, MT, W, U, kEpStore, 0, false>),
                       dim3((unsigned)((p.n + 15) / 16)), dim3(64 * W), W * MT * 4 * 64 * 4, stream,
                       p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_int8(const ProductArgs& p, hipStream_t stream)
{
    if (!strips(p))
        return tiles_int8(p, nullptr, stream);
    if (p.m > 16)
        return strip<2, 8, 2>(p, stream);
    return p.kbytes >= 64 * kStep ? strip<1, 16, 4>(p, stream) : strip<1, 8, 4>(p, stream);
}

size_t int8_workspace(ProductArgs p)
{
    size_t bytes = 0;
    p.may_split = 1;
    if (!strips(p))
        (void)tiles_int8(p, &bytes, nullptr);
    return bytes;
}

}  // namespace qse
