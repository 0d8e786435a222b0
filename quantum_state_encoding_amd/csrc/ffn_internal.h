// Internal interface between the feed-forward entry points (ffn_api.cpp)
// and their gfx950 kernels (ffn_rotate.hip, ffn_matmul.hip,
// ffn_strip.hip).  Not installed; not part of the C ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace qse {

constexpr int kFfnBlock = 128;        // contraction elements that share a scale
constexpr int kFfnMaxBits = 14;       // log2 of the largest rotation
constexpr int kFfnMaxBitsT = 7;       // the same, for a transposed input

// Element types, as fwt_ffn_dtype numbers them.
// kTE4m3Exact: e4m3 operands whose products and sums keep 32 bits, for f16 and
// fp32 results.
// kTI8: 8-bit integers, with 32-bit integer sums.
enum FfnType : int { kTBf16 = 0, kTF16 = 1, kTF32 = 2, kTE4m3 = 3, kTE4m3Exact = 4, kTI8 = 5 };

// Largest row stride of a product's operand, in bytes: 256 rows of a tile
// stay within a 32-bit offset of its first one.
constexpr int64_t kFfnMaxStride = (int64_t)1 << 23;

// Workgroups of a launch stay below this: of at most 1024 threads each,
// they have fewer than 2^32 threads, which is a launch's limit.
constexpr int64_t kFfnMaxTiles = (int64_t)1 << 22;

// What a product's epilogue does with its accumulators.
enum FfnEpilogue : int {
    kEpStore = 0,     // C = A B^T; 16-bit operands: with B stored [k][n]
    kEpGate = 1,      // C = act(A B0^T) * (A B1^T)
    kEpGateGrad = 2,  // the gradients of A B0^T and A B1^T from that of C
    kEpStoreT = 3,    // 16-bit operands: kEpStore with A stored [k][m] too
};

// The largest finite magnitude of dg and du in f16, as far as it matters (the
// factor that they are stored with goes by it): a bit pattern, of values above
// the type's range or below kRangeLow only, and whether there are others.
struct GradRange {
    uint32_t top;
    uint32_t within;
};

// One product A B^T (A: m x k, B: n x k, both with k contiguous), or two
// that share A.  Strides of a and b in bytes, of the others in elements.
struct ProductArgs {
    const void* a;
    const void* b0;
    const void* b1;         // the up projection (kEpGate, kEpGateGrad)
    int64_t lda, ldb0, ldb1;
    int64_t m, n;
    int64_t kbytes;         // bytes of a row that are contracted
    const float* sa;        // e4m3: scales [k block][m]
    const float* sb0;       // scales [k block][sb_n]
    const float* sb1;
    int64_t sb_n;           // n (one for each row of B) or ceil(n / 128)
    int parts;              // 2: the contraction goes on over b1 (kEpStore)
    int64_t part_a;         // for columns of A this many bytes further on
    void* c;                // m x n; kEpGateGrad: dg
    int64_t part_c;         // du this many elements further on
    void* c1;               // kEpStoreT: the results' rows from split on, as
    int64_t split;          // many as of the first, split_rows; 0: none
    int64_t split_rows;
    int64_t ldc, ldc1;
    int ctype;
    const void* dh;         // kEpGateGrad: gradient of C, m x n
    int64_t lddh;
    int act;                // 0 silu, 1 gelu
    GradRange* range;       // f16 gradients: of dg and du (kEpGateGrad sets
                            // it, the products that read them go by it)
    int again;              // kEpGateGrad: only where range asks for a factor
    int may_split;          // partial has product_workspace bytes
    void* partial;
    int tiles_m, tiles_n, splits;   // set by the launcher
};

// Enqueue a product.  type: element type of A and B; row_scales: e4m3 with
// a scale for each row of B.
hipError_t launch_product(const ProductArgs& p, int type, int epilogue, bool row_scales,
                          hipStream_t stream);
// Bytes of ProductArgs::partial for a product of these sizes (0: none).
size_t product_workspace(ProductArgs p, int type, int epilogue, bool row_scales);
// Its form for few rows of A (kEpStore: e4m3 only).
constexpr int kStripRows = 32;
hipError_t launch_strip(const ProductArgs& p, int type, int epilogue, bool row_scales,
                        hipStream_t stream);

// Products of rows grouped by expert.  ends (device): group e has the rows from
// ends[e - 1] up to ends[e] of `rows`.
struct GroupArgs {
    const int32_t* ends;
    int experts;
    int64_t rows;
    int64_t stride_b;       // bytes from an expert's weights to the next one's
    int64_t stride_c;       // elements between the experts' results (gradients of weights)
    int zero_rest;          // rows of no expert become 0
};
// C[i] = A[i] B_e^T for the rows i of group e; p.m, the sizes of all of A.
// bt: 16-bit types, B_e is stored [k][n].
hipError_t launch_grouped(const ProductArgs& p, const GroupArgs& g, int type, bool bt,
                          hipStream_t stream);
// C_e = A^T B over the rows of group e: A is rows x p.m, B rows x p.n, 16 bits.
hipError_t launch_grouped_t(const ProductArgs& p, const GroupArgs& g, int type,
                            hipStream_t stream);
// Bytes of ProductArgs::partial that these would use (p.kbytes of
// launch_grouped_t: of all rows).
size_t grouped_workspace(ProductArgs p, const GroupArgs& g, int type, bool bt);
size_t grouped_t_workspace(ProductArgs p, const GroupArgs& g, int type);

// What these are expected to take, microseconds (16 bits): level 0 for operands whose
// addresses and strides are multiples of 16 bytes, 1 of 4, 2 others.
double grouped_cost(const ProductArgs& p, const GroupArgs& g, bool bt, int level);
double grouped_t_cost(const ProductArgs& p, const GroupArgs& g, int level);

// A copy of an operand of 16 bits in rows of padded_row bytes, zeros behind each.
struct RowCopy {
    const void* src;
    void* dst;              // 16-byte aligned
    int64_t ld, stride;     // bytes between src's rows, and its experts
    int64_t rows, cols;     // rows of all
    int64_t each;           // of an expert, 0: rows that the groups share
};
inline int64_t padded_row(int64_t cols) { return (cols * 2 + 15) & ~(int64_t)15; }
// Experts without rows and rows of no expert are not read.
hipError_t launch_row_copies(const RowCopy* copies, int count, const GroupArgs& g,
                             hipStream_t stream);
double row_copies_cost(int64_t bytes);

// A product of 8-bit integers with a scale for each row of A and of B.
hipError_t launch_int8(const ProductArgs& p, hipStream_t stream);
size_t int8_workspace(ProductArgs p);

// Rotation and quantisation to 8-bit integers with a scale for each row.
struct Quantize8Args {
    const void* x;
    int64_t ldx;            // elements
    int64_t m, k;
    int bits;
    int8_t* q;
    int64_t ldq;            // bytes
    float* s;
};
hipError_t launch_quantize8(const Quantize8Args& p, int type, hipStream_t stream);
// Workgroups of that launch.
int64_t quantize8_groups(int64_t m, int64_t k);

// Zeros to rows x cols 16-bit elements.
hipError_t launch_zero16(void* dst, int64_t ld, int64_t rows, int64_t cols, hipStream_t stream);

struct RotateArgs {
    const void* x;          // m x k, or k x m when transposed
    int64_t ldx;            // elements
    int64_t m, k;
    int bits;
    uint8_t* q;             // m x k codes
    int64_t ldq;            // bytes
    float* s;               // scales
    float* amax;            // tile scales of long rotations: workspace [k block][m]
};
hipError_t launch_rotate(const RotateArgs& p, int type, bool tile, bool transpose,
                         hipStream_t stream);
// Bytes of RotateArgs::amax that the call needs.
size_t rotate_workspace(int64_t m, int64_t k, int bits, bool tile, bool transpose);

}  // namespace qse
