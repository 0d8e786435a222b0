// Products of rows grouped by expert, and the gradients of the weights.
//
// C[i] = A[i] B_e^T for the rows i of group e, in ffn_matmul.hip's tiles and
// ffn_strip.hip's strips: a workgroup finds its group and its tile there from
// the groups' ends, which only the device knows, and goes on as in a product of
// that group alone.  The grid has a workgroup for each tile that there could be
// (a last tile that is not whole for each group); those without one end.
//
// What bounds it.  Large groups: the card's power (bf16 steps of 256 x 256 tiles take
// 1.45 us, 1.12 on operands of zeros) and the groups' last tiles, which are half
// empty in the mean and take 0.7 of a whole one's time when at most half of their rows
// exist; a round of tiles takes about 9 us beside its steps.  Few rows: the weights'
// bytes.  Measured by the card, groups uneven: bf16 m 16384 e 8 n 8192 k 4096 895-960 us,
// 1.15-1.23 PFLOP/s (library product 1.46), int8 e 32 n 4096 330-356; gradients
// e 16 n 4096 k 4096 1069-1145 (dx 528-554, dw 557-587); bf16 one row for each of 32
// experts' places, e 64 n 2048 k 4096, 66-73 us, 5.8 TB/s.
#include <hip/hip_runtime.h>

#include "ffn_product.h"
#include "ffn_strip.h"

namespace qse {
namespace {

// A workgroup's group: its first row and number of rows, and which of its tiles.
struct Group {
    int e;
    int first, rows;
    int tile;
    int half;        // 0 all of it, 1 its first rows, 2 the others
};

// An end, cut to the rows.
__device__ __forceinline__ int cut_end(const GroupArgs& g, int end)
{
    const int m = (int)g.rows;
    return end < 0 ? 0 : end < m ? end : m;
}

// Rows of group e: what its own two ends say (where ends fall, find_group's are some of
// them).
__device__ __forceinline__ int rows_of(const GroupArgs& g, int e, int& first)
{
    first = e > 0 ? cut_end(g, g.ends[e - 1]) : 0;
    const int last = cut_end(g, g.ends[e]);
    return last > first ? last - first : 0;
}

// A lane's number joined with those of the lanes before it: within 16 lanes, then with
// the last of the 16 and of the 32 before (numbers that are not negative).  With shuffles
// through LDS instead, bf16 m 128 e 128 n 512 k 512 takes 15.7 us, 13.8 so.
template <class Join>
__device__ __forceinline__ int joined_up(int v, const Join& join)
{
    v = join(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false));
    v = join(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false));
    v = join(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false));
    v = join(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false));
    v = join(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false));
    return join(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false));
}

// The tile of workgroup w among all groups' tiles of bm rows and tiles_n
// columns: 64 groups at a time, one on each lane, whose tiles are summed across
// the wave (every wave finds the same).  Each XCD gets a contiguous run of them.
// HALVES: where the last round of tiles would leave half of the CUs without one,
// two workgroups (of one XCD) take half of each tile's rows.  Behind them all come
// the tiles of the rows of no expert, which take no time to speak of.
//
// The grid has room for groups that share no row.  So that they share none where ends
// fall either, a group begins at the largest end before its own, and the rows of no
// expert at the largest of all.  A row that one group alone claims by its own two ends
// stays with it: an earlier end behind that row would be one of a group that claims
// the row too.
constexpr int kCus = 256;
template <int BM, bool HALVES = false>
__device__ __forceinline__ bool find_group(const GroupArgs& g, int w, int tiles_n, Group& at)
{
    const int lane = threadIdx.x & 63;
    const int groups = g.experts;
    // behind: the largest end before group `base`, then before the next 64
    const auto sum = [=](int base, int& behind, int& first, int& rows,
                         int& tiles) __attribute__((always_inline)) {
        const int e = base + lane, count = groups - base < 64 ? groups - base : 64;
        const bool live = lane < count;
        // (two loads at once, under no condition)
        const int lo = g.ends[live && e > 0 ? e - 1 : 0], hi = g.ends[live ? e : 0];
        first = live && e > 0 ? cut_end(g, lo) : 0;
        const int last = live ? cut_end(g, hi) : 0;
        const auto larger = [](int a, int b) __attribute__((always_inline)) { return a > b ? a : b; };
        if (__builtin_expect(__ballot(live && (first < behind || last < first)) != 0, 0)) {
            const int top = joined_up(last, larger);     // up to this lane's, the one before's
            first = larger(behind, __builtin_amdgcn_update_dpp(0, top, 0x138, 0xf, 0xf, false));
            behind = larger(behind, __builtin_amdgcn_readlane(top, 63));
        } else {
            behind = __builtin_amdgcn_readlane(last, count - 1);
        }
        rows = live && last > first ? last - first : 0;
        tiles = (rows + BM - 1) / BM * tiles_n;
        const int s = joined_up(tiles, [](int a, int b) __attribute__((always_inline)) { return a + b; });
        return s;                        // up to this lane's
    };
    int first = 0, rows = 0, tiles = 0, behind = 0;
    int upto = sum(0, behind, first, rows, tiles);
    int total = __builtin_amdgcn_readlane(upto, 63);
    int largest = behind;
    for (int base = 64; base < groups; base += 64) {
        int f, r, t;
        total += __builtin_amdgcn_readlane(sum(base, largest, f, r, t), 63);
    }
    at.half = 0;
    int items = total;
    if constexpr (HALVES) {
        const int last = total % kCus, whole = total - last;
        if (last <= kCus / 2) {
            items = whole + ((last + 7) >> 3 << 4);
            if (w >= whole && w < items) {
                const int j = w - whole;
                at.half = 1 + ((j >> 3) & 1);
                w = whole + ((j >> 4) << 3) + (j & 7);
                if (w >= total)
                    return false;
            }
        }
    }
    if (w >= items) {
        at.e = g.experts;
        at.tile = w - items;
        at.first = largest;
        at.rows = g.zero_rest ? (int)g.rows - largest : 0;
        return at.tile < (at.rows + BM - 1) / BM * tiles_n;
    }
    const int t = place_of(w, total);
    int before = 0;
    for (int base = 0; base < groups; base += 64) {
        if (base > 0)
            upto = sum(base, behind, first, rows, tiles);
        const uint64_t past = __ballot(before + upto > t);
        if (past) {
            const int l = __builtin_ctzll(past);
            at.e = base + l;
            at.first = __builtin_amdgcn_readlane(first, l);
            at.rows = __builtin_amdgcn_readlane(rows, l);
            at.tile = t - before - __builtin_amdgcn_readlane(upto - tiles, l);
            return true;
        }
        before += __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
}

// The arguments of group `at` alone.
template <int TYPE>
__device__ __forceinline__ void enter(ProductArgs& p, const GroupArgs& g, const Group& at)
{
    p.a = (const char*)p.a + (int64_t)at.first * p.lda;
    p.b0 = (const char*)p.b0 + at.e * g.stride_b;
    p.c = (char*)p.c + (int64_t)at.first * p.ldc * (TYPE == kTI8 && p.ctype == kTF32 ? 4 : 2);
    p.m = at.rows;
    if constexpr (TYPE == kTI8) {
        p.sa += at.first;
        p.sb0 += at.e * p.n;
    }
}

// Tile t of a group's tiles_m x tiles_n, in columns of about 8 row tiles, evenly:
// a few row tiles over a multiple of 8 by themselves would read all of the expert's
// weights once more.
__device__ __forceinline__ void group_tile_at(int t, int tiles_m, int tiles_n, int& tm, int& tn)
{
    const int columns = tiles_m > 10 ? (tiles_m + 5) >> 3 : 1;
    const int rows = tiles_m / columns, more = tiles_m - rows * columns;
    const int wide = more * (rows + 1);          // row tiles of the columns with one more
    const bool late = t >= wide * tiles_n;
    const int r = rows + (late ? 0 : 1);
    t -= late ? wide * tiles_n : 0;
    const int c = t / (r * tiles_n);
    t -= c * r * tiles_n;
    tm = (late ? wide : 0) + c * r + t % r;
    tn = t / r;
}

// Zeros to rows x cols results at (m0, n0), 16 bytes a lane.
__device__ __forceinline__ void zero_tile(void* c, int64_t ldc, int type, int64_t m0, int64_t n0,
                                          int rows, int cols)
{
    const int size = type == kTF32 ? 4 : 2, each = 16 / size;
    const int chunks = (cols + each - 1) / each;
    for (int i = (int)threadIdx.x; i < rows * chunks; i += (int)blockDim.x) {
        const int r = i / chunks, n = (i - r * chunks) * each;
        char* at = (char*)c + ((m0 + r) * ldc + n0 + n) * size;
        if (cols - n >= each)
            put16(at, v4i{0, 0, 0, 0});
        else
            for (int b = 0; b < (cols - n) * size; b += 2)
                *(unsigned short*)(at + b) = 0;
    }
}
template <int BM, int BN>
__device__ __forceinline__ void zero_rows(const ProductArgs& p, const Group& at, int tiles_n)
{
    const int tm = at.tile / tiles_n, tn = at.tile % tiles_n;
    const int64_t left = p.n - (int64_t)tn * BN;
    zero_tile(p.c, p.ldc, p.ctype, at.first + (int64_t)tm * BM, (int64_t)tn * BN,
              at.rows - tm * BM < BM ? at.rows - tm * BM : BM, left < BN ? (int)left : BN);
}

template <int TYPE, int BM, int BN, int WM, int WN, int WK, int NS, int REG, bool BT>
__global__ __launch_bounds__(64 * WM * WN * WK) __attribute__((amdgpu_waves_per_eu(2))) void
grouped_kernel(ProductArgs p, const GroupArgs g)
{
    constexpr bool kPipe = BM == 256 && !REG;
    Group at;
    if (!find_group<BM, kPipe>(g, (int)blockIdx.x, p.tiles_n, at))
        return;
    if (at.e == g.experts) {
        if (blockIdx.y == 0)
            zero_rows<BM, BN>(p, at, p.tiles_n);
        return;
    }
    int tm, tn;
    group_tile_at(at.tile, (at.rows + BM - 1) / BM, p.tiles_n, tm, tn);
    if (kPipe && at.half) {
        const int skip = tm * BM + (at.half - 1) * (BM / 2);
        if (skip >= at.rows)
            return;
        at.first += skip;
        at.rows = at.rows - skip < BM / 2 ? at.rows - skip : BM / 2;
        tm = 0;
    }
    enter<TYPE>(p, g, at);
    product_body<TYPE, BM, BN, WM, WN, WK, NS, kEpStore, kNoScale, REG, false, BT, kPipe, true>(
        p, tm, tn, (int)blockIdx.y, EveryWorkgroup{});
}

// The shares of a group's tile.
template <int BM>
struct GroupPlace : EveryWorkgroup {
    Group at;
    __device__ __forceinline__ void place(const ProductArgs& p, int& tm, int& tn) const
    {
        group_tile_at(at.tile, (at.rows + BM - 1) / BM, p.tiles_n, tm, tn);
    }
};
template <int TYPE, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void grouped_join_kernel(ProductArgs p, const GroupArgs g)
{
    GroupPlace<BM> where;
    if (!find_group<BM>(g, (int)blockIdx.x, p.tiles_n, where.at) || where.at.e == g.experts)
        return;
    enter<TYPE>(p, g, where.at);
    join_body<TYPE, BM, BN, WM, WN, kEpStore, false, true>(p, where);
}

// Few rows to a group: strips of 16 rows of B, for MT * 16 rows of A.
template <int TYPE, int MT, int W, int U, bool ODD>
__global__ __launch_bounds__(64 * W) void grouped_strip_kernel(ProductArgs p, const GroupArgs g)
{
    constexpr int BM = MT * 16;
    Group at;
    if (!find_group<BM>(g, (int)blockIdx.x, p.tiles_n, at))
        return;
    if (at.e == g.experts) {
        zero_rows<BM, 16>(p, at, p.tiles_n);
        return;
    }
    int tm, tn;
    group_tile_at(at.tile, (at.rows + BM - 1) / BM, p.tiles_n, tm, tn);
    at.first += tm * BM;
    at.rows = at.rows - tm * BM < BM ? at.rows - tm * BM : BM;
    enter<TYPE>(p, g, at);
    strip_body<TYPE, MT, W, U, kEpStore, 0, ODD>(p, tn);
}

// C_e = A^T B over the rows of group e (A and B stored [rows][..]): an expert's
// tiles side by side, each with that group's rows as its contraction.
struct GradPlace : EveryWorkgroup {
    int tm, tn;
    __device__ __forceinline__ void place(const ProductArgs&, int& m, int& n) const
    {
        m = tm;
        n = tn;
    }
};
// One expert's tiles after the other's, each expert's spread over the XCDs, since
// their times differ by the experts' (m 16384 e 16 n 4096 k 4096, unevenly: 848 us
// with a run of experts to each XCD, 565 so; those with the most rows first: 580, as
// finding them takes each workgroup longer than it gains).
__device__ __forceinline__ int enter_grad(ProductArgs& p, const GroupArgs& g, GradPlace& where)
{
    const int per = p.tiles_m * p.tiles_n;
    const int e = (int)blockIdx.x / per;
    const int t = place_of((int)blockIdx.x - e * per, per);
    int first;
    const int rows = __builtin_amdgcn_readfirstlane(rows_of(g, e, first));
    first = __builtin_amdgcn_readfirstlane(first);
    tile_at(t, p.tiles_m, p.tiles_n, where.tm, where.tn);
    p.a = (const char*)p.a + first * p.lda;
    p.b0 = (const char*)p.b0 + first * p.ldb0;
    p.c = (char*)p.c + e * g.stride_c * 2;
    p.kbytes = (int64_t)rows * 2;
    return rows;
}

template <int TYPE, int BM, int BN, int WM, int WN, int WK, int NS, int REG>
__global__ __launch_bounds__(64 * WM * WN * WK) __attribute__((amdgpu_waves_per_eu(2))) void
grouped_grad_kernel(ProductArgs p, const GroupArgs g)
{
    GradPlace where;
    const int rows = enter_grad(p, g, where);
    if (rows == 0) {
        const int64_t m0 = (int64_t)where.tm * BM, n0 = (int64_t)where.tn * BN;
        if (blockIdx.y == 0)
            zero_tile(p.c, p.ldc, TYPE, m0, n0, p.m - m0 < BM ? (int)(p.m - m0) : BM,
                      p.n - n0 < BN ? (int)(p.n - n0) : BN);
        return;
    }
    if (p.splits > 1) {                  // (a share without steps is not joined)
        const int steps = (int)((p.kbytes + kStep - 1) / kStep);
        if ((int)blockIdx.y * ((steps + p.splits - 1) / p.splits) >= steps)
            return;
    }
    constexpr bool kPipe = BM == 256 && !REG;
    product_body<TYPE, BM, BN, WM, WN, WK, NS, kEpStore, kNoScale, REG, true, true, kPipe, true>(
        p, where.tm, where.tn, (int)blockIdx.y, where);
}

template <int TYPE, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void grouped_grad_join_kernel(ProductArgs p,
                                                                         const GroupArgs g)
{
    GradPlace where;
    const int rows = enter_grad(p, g, where);
    if (rows == 0)
        return;
    const int steps = (int)((p.kbytes + kStep - 1) / kStep);
    const int share = (steps + p.splits - 1) / p.splits;
    p.splits = (steps + share - 1) / share;      // those that have steps
    join_body<TYPE, BM, BN, WM, WN, kEpStore, true, true>(p, where);
}

// Row tiles that m rows in up to `groups` groups may have.
int64_t most_tiles(int64_t m, int64_t groups, int64_t bm)
{
    const int64_t r = groups < m ? groups : m;
    return (m + r * (bm - 1)) / bm;
}

// (the rows of no expert count whether they are written or not, so that the choice
// and its scratch do not go by it)
int64_t groups_of(const GroupArgs& g) { return g.experts + 1; }

template <class K>
hipError_t allow_lds(K* k, size_t bytes, std::atomic<uint64_t>& done)
{
    if (bytes <= 65536)
        return hipSuccess;
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e == hipSuccess && (dev >= 64 || !((done.load() >> dev) & 1))) {
        e = hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize,
                                (int)bytes);
        if (e == hipSuccess && dev < 64)
            done.fetch_or((uint64_t)1 << dev);
    }
    return e;
}

template <int BM, int BN, int WK, int NS>
constexpr size_t lds_of()
{
    constexpr size_t n = WK * NS * (size_t)(BM + BN) * kStep;
    static_assert(n <= 160 * 1024 && (size_t)(WK - 1) * BM * BN * 4 <= n, "LDS of a CU");
    return n;
}

template <int TYPE, int BM, int BN, int WM, int WN, int WK, int NS, bool BT, int REG = kAligned>
hipError_t run_grouped(ProductArgs p, const GroupArgs& g, int splits, hipStream_t stream)
{
    constexpr size_t kLds = lds_of<BM, BN, WK, NS>();
    static std::atomic<uint64_t> done{0};
    auto* k = &grouped_kernel<TYPE, BM, BN, WM, WN, WK, NS, REG, BT>;
    hipError_t e = allow_lds(k, kLds, done);
    if (e != hipSuccess)
        return e;
    p.splits = splits;
    p.tiles_n = (int)((p.n + BN - 1) / BN);
    unsigned tiles = (unsigned)(most_tiles(p.m, groups_of(g), BM) * p.tiles_n);
    if (BM == 256 && !REG)
        tiles += kCus / 2 + 8;           // (halves, and eights of them that are not whole)
    hipLaunchKernelGGL(k, dim3(tiles, (unsigned)splits), dim3(64 * WM * WN * WK), kLds, stream, p, g);
    e = hipGetLastError();
    if (splits == 1 || e != hipSuccess)
        return e;
    if constexpr (may_split<TYPE, BM, BN>())
        hipLaunchKernelGGL((grouped_join_kernel<TYPE, BM, BN, WM, WN>),
                           dim3(tiles, BM / WM / 16, BN / WN / 16), dim3(64 * WM * WN), 0, stream, p,
                           g);
    return hipGetLastError();
}

template <int TYPE, int BM, int BN, int WM, int WN, int WK, int NS, int REG = kAligned>
hipError_t run_grad(ProductArgs p, const GroupArgs& g, int splits, hipStream_t stream)
{
    constexpr size_t kLds = lds_of<BM, BN, WK, NS>();
    static std::atomic<uint64_t> done{0};
    auto* k = &grouped_grad_kernel<TYPE, BM, BN, WM, WN, WK, NS, REG>;
    hipError_t e = allow_lds(k, kLds, done);
    if (e != hipSuccess)
        return e;
    p.splits = splits;
    p.tiles_m = (int)((p.m + BM - 1) / BM);
    p.tiles_n = (int)((p.n + BN - 1) / BN);
    const unsigned tiles = (unsigned)((int64_t)p.tiles_m * p.tiles_n * g.experts);
    hipLaunchKernelGGL(k, dim3(tiles, (unsigned)splits), dim3(64 * WM * WN * WK), kLds, stream, p, g);
    e = hipGetLastError();
    if (splits == 1 || e != hipSuccess)
        return e;
    if constexpr (BM <= 128 && BN <= 128)
        hipLaunchKernelGGL((grouped_grad_join_kernel<TYPE, BM, BN, WM, WN>),
                           dim3(tiles, BM / WM / 16, BN / WN / 16), dim3(64 * WM * WN), 0, stream, p,
                           g);
    return hipGetLastError();
}

// Which tile.  A round of workgroups takes its steps' time and that of its first
// loads and its stores, and all rounds at least the time of the operands' and
// results' bytes; 0.3 of the shorter of the two does not overlap the longer.
// Microseconds a step of 128 bytes, and a round beside them, measured:
//                              slots   16 bits   any address   8 bits
//   256 x 256                    256   1.45  9     1.9  11    1.45  9
//   128 x 128, two on a CU       512   1.06  6     1.2   7    1.0   6
//   128 x 128, deeper            256    .62  5       -         .60  5
//   64 x 128                     256    .42  4      .68  6     .42  4
//   64 x 128, three on a CU      768                1.4   6
//   8 bits, 64 x 64, deeper      256                           .26  3
// and the bytes at 6.5 TB/s, at any address 2.5, 2.7 and 3.8 (at multiples of four bytes
// 3.7, 4.6 and 5.0, and steps of 1.85, 1.1, 0.62 and 1.3).
// How the rows are spread is not known: a group is taken to have the average
// number, and half a tile of rows more than it fills.  Over 60 sizes (4 to 64
// experts, half a row to 2048 rows for each, unevenly; forward, gradients and 8 bits) the
// choice takes 4.4 % longer than the best tile in the mean, at most 31 % (dx of rows at
// odd addresses, m 7231 e 23 n 2327 k 3109: 244 us, 186 with 256 x 256).  Where most of
// a round's slots are empty the workgroups of a tile may share its steps, for a second
// launch and their sums' bytes.
struct GroupTile {
    int bm, bn, slots;
    float step, round;
    int area;                // of the sums, 0: not split
    float rate = 6.5e6f;     // bytes a microsecond
};
constexpr double kSumBytes = 4.5e6;
constexpr double kNever = 1e30;

struct GroupCosts {
    int64_t steps;
    double bytes;
    bool may_split;
    bool known;              // the number of tiles is
};
// count(tile, most): the tiles to expect, and those of the grid.
template <int N, class Count>
Choice cheapest_grouped(const GroupTile (&tiles)[N], const GroupCosts& w, const Count& count,
                        double& least)
{
    Choice best{0, 1, 0};
    least = 2 * kNever;
    for (int i = 0; i < N; ++i) {
        const GroupTile& t = tiles[i];
        int64_t most = 0;
        const double expect = count(t, most);
        const auto both = [&](double compute) {
            const double memory = w.bytes / t.rate;
            return compute > memory ? compute + 0.3 * memory : memory + 0.3 * compute;
        };
        // (a number that is not known ends anywhere in its last round)
        const double full = expect / t.slots;
        const double rounds = w.known      ? (double)((int64_t)(full - 1e-9) + 1)
                              : full > 0.6 ? full + 0.4
                                           : 1.0;
        double cost = most >= kFfnMaxTiles ? kNever : both(rounds * (w.steps * t.step + t.round));
        int splits = 1;
        if (t.area && w.may_split && most * 2 <= t.slots) {
            int64_t s = t.slots / most < 32 ? t.slots / most : 32;
            s = s < w.steps / 4 ? s : w.steps / 4;
            // every share has steps, the last one fewer
            s = s > 1 ? (w.steps + (w.steps + s - 1) / s - 1) / ((w.steps + s - 1) / s) : 1;
            const double sums = 2.0 * s * most * t.area * 4;
            const double shared =
                both((double)((w.steps + s - 1) / s) * t.step + t.round) + 6.0 + sums / kSumBytes;
            if (s > 1 && shared < cost) {
                cost = shared;
                splits = (int)s;
            }
        }
        if (cost < least) {
            least = cost;
            best = Choice{i, splits, splits > 1 ? (size_t)splits * most * t.area * 4 : 0};
        }
    }
    return best;
}

double groups_with_rows(const ProductArgs& p, const GroupArgs& g)
{
    return (double)(g.experts < p.m ? g.experts : p.m);
}

// Row tiles of bm that a group is expected to have.
double tiles_of_group(const ProductArgs& p, const GroupArgs& g, int bm)
{
    const double avg = p.m / groups_with_rows(p, g);
    if (g.experts == 1)
        return (double)((p.m + bm - 1) / bm);
    return avg > bm / 2 ? avg / bm + 0.5 : 1.0;
}

template <int N>
Choice choose(const GroupTile (&tiles)[N], const ProductArgs& p, const GroupArgs& g, double& least)
{
    const double groups = groups_with_rows(p, g);
    const double bytes = (groups * p.n + p.m) * p.kbytes + 2.0 * p.m * p.n;
    const GroupCosts w{(p.kbytes + kStep - 1) / kStep, bytes, p.may_split != 0, false};
    return cheapest_grouped(
        tiles, w,
        [&](const GroupTile& t, int64_t& most) {
            const int64_t tn = (p.n + t.bn - 1) / t.bn;
            most = most_tiles(p.m, groups_of(g), t.bm) * tn;
            return groups * tiles_of_group(p, g, t.bm) * tn;
        },
        least);
}

// Strips: the weights' bytes for every 16 rows of a group, and some time to start, or
// rounds of two strips on a CU, each the time to start and the steps that its eight
// waves take in turn (0.85 us each).  Rates in bytes a microsecond, 16-bit rows at
// multiples of 16 and of 4 bytes and at others, and of 8-bit integers.
// Groups of a row or two take them (about 26 experts of 2048 x 4096, bf16: 70 us and
// 75 with 64 x 128 tiles, in two rounds; 18 experts of 496 x 3712: 16.8 and 23.9),
// others are faster in tiles (64 experts of 2048 x 4096, 4 rows each in the mean,
// unevenly: 212 us and 169).
constexpr double kStrip16 = 5.7e6, kStrip4 = 3.7e6, kStripOdd = 3.0e6, kStrip8 = 4.6e6;
double strips_cost(const ProductArgs& p, const GroupArgs& g, double rate)
{
    if (most_tiles(p.m, groups_of(g), 16) * ((p.n + 15) / 16) >= kFfnMaxTiles)
        return kNever;
    const double groups = groups_with_rows(p, g), avg = p.m / groups;
    const double each = groups * (avg > 1 ? 1 + avg / 16 : 1);
    const double bytes = 4.0 + each * p.n * p.kbytes / rate;
    const double full = each * ((p.n + 15) / 16) / (2 * kCus);
    const double steps = 4.0 + 0.85 * (double)p.kbytes / (8 * kStep);
    const double rounds = full > 1 ? full * steps : steps;
    return bytes > rounds ? bytes : rounds;
}

template <int TYPE, int MT, int W, int U, bool ODD>
hipError_t run_strips(ProductArgs p, const GroupArgs& g, hipStream_t stream)
{
    p.tiles_n = (int)((p.n + 15) / 16);
    const unsigned count = (unsigned)(most_tiles(p.m, groups_of(g), MT * 16) * p.tiles_n);
    hipLaunchKernelGGL((grouped_strip_kernel<TYPE, MT, W, U, ODD>), dim3(count), dim3(64 * W),
                       W * MT * 4 * 64 * 4, stream, p, g);
    return hipGetLastError();
}

bool any_address(const ProductArgs& p, const GroupArgs& g, uintptr_t mask)
{
    return (((uintptr_t)p.a | (uintptr_t)p.b0 | (uintptr_t)p.lda | (uintptr_t)p.ldb0 |
             (uintptr_t)g.stride_b) & mask) != 0;
}

constexpr GroupTile kTilesAny[] = {{256, 256, 256, 1.9f, 11.f, 0, 2.5e6f},
                                   {128, 128, 512, 1.2f, 7.f, 0, 2.7e6f},
                                   {64, 128, 768, 1.4f, 6.f, 64 * 128, 3.8e6f},
                                   {64, 128, 256, .68f, 6.f, 0, 3.8e6f}};
constexpr GroupTile kTiles16[] = {{256, 256, 256, 1.45f, 9.f, 0},
                                  {128, 128, 512, 1.06f, 6.f, 0},
                                  {128, 128, 256, .62f, 5.f, 128 * 128},
                                  {64, 128, 256, .42f, 4.f, 64 * 128}};
// (multiples of four bytes)
constexpr GroupTile kTilesFour[] = {{256, 256, 256, 1.85f, 11.f, 0, 3.7e6f},
                                    {128, 128, 512, 1.1f, 7.f, 0, 4.6e6f},
                                    {64, 128, 768, 1.3f, 6.f, 64 * 128, 5.0e6f},
                                    {64, 128, 256, .62f, 6.f, 0, 5.0e6f}};

template <int TYPE, bool BT>
hipError_t grouped16(const ProductArgs& p, const GroupArgs& g, size_t* query, hipStream_t stream)
{
    double cost_odd, cost_four, cost_tile;
    const Choice co = choose(kTilesAny, p, g, cost_odd), cf = choose(kTilesFour, p, g, cost_four),
                 c = choose(kTiles16, p, g, cost_tile);
    if (query) {
        *query = co.bytes > c.bytes ? co.bytes : c.bytes;
        *query = *query > cf.bytes ? *query : cf.bytes;
        return hipSuccess;
    }
    const bool anywhere = any_address(p, g, 15), odd = any_address(p, g, 3);
    const Choice ca = odd ? co : cf;
    const double cost = odd ? cost_odd : anywhere ? cost_four : cost_tile;
    if constexpr (!BT) {
        if (strips_cost(p, g, odd ? kStripOdd : anywhere ? kStrip4 : kStrip16) < cost)
            return odd ? run_strips<TYPE, 1, 8, 4, true>(p, g, stream)
                       : run_strips<TYPE, 1, 8, 4, false>(p, g, stream);
    }
    if (anywhere) {
        if (p.kbytes < 16 || (BT && p.n < 8))
            return run_grouped<TYPE, 128, 128, 2, 2, 1, 2, BT, kShortRows>(p, g, 1, stream);
        if (ca.tile == 0)
            return run_grouped<TYPE, 256, 256, 2, 4, 1, 2, BT, kAnyAddress>(p, g, 1, stream);
        if (ca.tile == 1)
            return run_grouped<TYPE, 128, 128, 2, 2, 1, 2, BT, kAnyAddress>(p, g, 1, stream);
        return run_grouped<TYPE, 64, 128, 1, 4, 1, 2, BT, kAnyAddress>(p, g, ca.splits, stream);
    }
    switch (c.tile) {
    case 0:
        return run_grouped<TYPE, 256, 256, 2, 4, 1, 2, BT>(p, g, 1, stream);
    case 1:
        return run_grouped<TYPE, 128, 128, 2, 2, 1, 2, BT>(p, g, 1, stream);
    case 2:
        return run_grouped<TYPE, 128, 128, 2, 2, 1, 4, BT>(p, g, c.splits, stream);
    }
    return run_grouped<TYPE, 64, 128, 1, 4, 1, 4, BT>(p, g, c.splits, stream);
}

hipError_t grouped8(const ProductArgs& p, const GroupArgs& g, size_t* query, hipStream_t stream)
{
    constexpr GroupTile tiles[] = {{256, 256, 256, 1.45f, 9.f, 0},
                                   {128, 128, 512, 1.0f, 6.f, 0},
                                   {128, 128, 256, .60f, 5.f, 0},
                                   {64, 128, 256, .42f, 4.f, 0},
                                   {64, 64, 256, .26f, 3.f, 64 * 64}};
    double cost;
    const Choice c = choose(tiles, p, g, cost);
    const bool strips = strips_cost(p, g, kStrip8) < cost;
    if (query) {
        *query = strips ? 0 : c.bytes;
        return hipSuccess;
    }
    if (strips)
        return run_strips<kTI8, 1, 8, 4, false>(p, g, stream);
    switch (c.tile) {
    case 0:
        return run_grouped<kTI8, 256, 256, 2, 4, 1, 2, false>(p, g, 1, stream);
    case 1:
        return run_grouped<kTI8, 128, 128, 2, 2, 1, 2, false>(p, g, 1, stream);
    case 2:
        return run_grouped<kTI8, 128, 128, 2, 2, 1, 4, false>(p, g, 1, stream);
    case 3:
        return run_grouped<kTI8, 64, 128, 1, 4, 1, 4, false>(p, g, 1, stream);
    }
    return run_grouped<kTI8, 64, 64, 2, 2, 2, 4, false>(p, g, c.splits, stream);
}

// Gradients of weights: an expert's tiles have its own rows as their steps; the
// average's count, twice as many where they may be shared (the expert with the most
// rows ends last).
constexpr GroupTile kGradAny[] = {{256, 256, 256, 1.9f, 11.f, 0},
                                  {128, 128, 512, 1.2f, 7.f, 128 * 128}};
constexpr GroupTile kGrad16[] = {{256, 256, 256, 1.6f, 9.f, 0},
                                 {128, 128, 512, 1.06f, 6.f, 0},
                                 {128, 128, 256, .62f, 5.f, 128 * 128}};
template <int N>
Choice choose_grad(const GroupTile (&tiles)[N], const ProductArgs& p, const GroupArgs& g,
                   double& least)
{
    const auto count = [&](const GroupTile& t, int64_t& most) {
        most = ((p.m + t.bm - 1) / t.bm) * ((p.n + t.bn - 1) / t.bn) * g.experts;
        return (double)most;
    };
    const int64_t rows = (p.kbytes + 2 * g.experts - 1) / (2 * g.experts);
    const double bytes = 2.0 * p.m * p.n * g.experts + (double)p.kbytes * (p.m + p.n);
    const int64_t few = (rows * 2 + kStep - 1) / kStep;
    const GroupCosts w{g.experts > 1 && p.may_split ? 2 * few : few, bytes,
                       p.may_split != 0, true};
    return cheapest_grouped(tiles, w, count, least);
}

template <int TYPE>
hipError_t grad16(const ProductArgs& p, const GroupArgs& g, size_t* query, hipStream_t stream)
{
    double cost;
    const Choice ca = choose_grad(kGradAny, p, g, cost), c = choose_grad(kGrad16, p, g, cost);
    if (query) {
        *query = ca.bytes > c.bytes ? ca.bytes : c.bytes;
        return hipSuccess;
    }
    if (any_address(p, g, 15)) {
        if (p.m < 8 || p.n < 8)
            return run_grad<TYPE, 128, 128, 2, 2, 1, 2, kShortRows>(p, g, 1, stream);
        if (ca.tile == 0)
            return run_grad<TYPE, 256, 256, 2, 4, 1, 2, kAnyAddress>(p, g, 1, stream);
        return run_grad<TYPE, 128, 128, 2, 2, 1, 2, kAnyAddress>(p, g, ca.splits, stream);
    }
    switch (c.tile) {
    case 0:
        return run_grad<TYPE, 256, 256, 2, 4, 1, 2>(p, g, 1, stream);
    case 1:
        return run_grad<TYPE, 128, 128, 2, 2, 1, 2>(p, g, 1, stream);
    }
    return run_grad<TYPE, 128, 128, 2, 2, 1, 4>(p, g, c.splits, stream);
}

// Copies of operands in rows that are no multiples of 16 bytes (RowCopy): a wave for
// every four rows at a time, short ones side by side, so that four chunks of 16 bytes a
// lane are in flight (bf16 m 16000 e 8 n 4001 k 4095, both operands: 145 us,
// 5.5 TB/s read and written).
struct RowCopies {
    RowCopy at[3];
};
__global__ __launch_bounds__(256) void row_copy_kernel(const RowCopies c, const GroupArgs g)
{
    constexpr int R = 4;
    const RowCopy p = c.at[blockIdx.y];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int64_t len = p.cols * 2, ldd = (len + 15) & ~(int64_t)15;
    const int each = (int)p.each;
    int rows = (int)p.rows;
    if (!each) {                         // up to the largest end
        int most = 0;
        for (int e = lane; e < g.experts; e += 64)
            most = g.ends[e] > most ? g.ends[e] : most;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_xor(most, d);
            most = most > o ? most : o;
        }
        most = __builtin_amdgcn_readfirstlane(most);
        rows = most < rows ? most : rows;
    }
    for (int row = ((int)blockIdx.x * 4 + wave) * R; row < rows; row += (int)gridDim.x * 4 * R) {
        const char* src[R];
        bool live[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = row + i < rows ? row + i : rows - 1;
            live[i] = row + i < rows;
            src[i] = (const char*)p.src + r * p.ld;
            if (each) {
                const int e = r / each;
                int first;
                live[i] = live[i] && rows_of(g, e, first) != 0;
                src[i] = (const char*)p.src + e * p.stride + (r - e * each) * p.ld;
            }
        }
        char* const dst = (char*)p.dst + row * ldd;
        if (ldd < 4096) {
            for (int64_t at = lane * 16; at < ldd; at += 1024) {
                v4i v[R];
#pragma unroll
                for (int i = 0; i < R; ++i)
                    if (live[i])
                        v[i] = load16_tail<kTBf16>(src[i], at, len);
#pragma unroll
                for (int i = 0; i < R; ++i)
                    if (live[i])
                        *(v4i*)(dst + i * ldd + at) = v[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if (!live[i])
                    continue;
                for (int64_t at = lane * 16; at < ldd; at += 1024 * R) {
                    v4i v[R];
#pragma unroll
                    for (int u = 0; u < R; ++u)
                        v[u] = load16_tail<kTBf16>(
                            src[i], at + u * 1024 < ldd ? at + u * 1024 : at, len);
#pragma unroll
                    for (int u = 0; u < R; ++u)
                        if (at + u * 1024 < ldd)
                            *(v4i*)(dst + i * ldd + at + u * 1024) = v[u];
                }
            }
        }
    }
}

}  // namespace

// A launch, and the bytes of the copies' writes, at the rate of both.
constexpr double kCopyBytes = 2.7e6;
double row_copies_cost(int64_t bytes) { return 4.0 + (double)bytes / kCopyBytes; }

hipError_t launch_row_copies(const RowCopy* copies, int count, const GroupArgs& g,
                             hipStream_t stream)
{
    RowCopies c{};
    int64_t most = 0;
    for (int i = 0; i < count; ++i) {
        c.at[i] = copies[i];
        most = copies[i].rows > most ? copies[i].rows : most;
    }
    const int64_t groups = (most + 15) / 16;
    hipLaunchKernelGGL(row_copy_kernel,
                       dim3((unsigned)(groups < 8 * kCus ? groups : 8 * kCus), (unsigned)count),
                       dim3(256), 0, stream, c, g);
    return hipGetLastError();
}

double grouped_cost(const ProductArgs& p, const GroupArgs& g, bool bt, int level)
{
    double cost;
    (void)(level == 0   ? choose(kTiles16, p, g, cost)
           : level == 1 ? choose(kTilesFour, p, g, cost)
                        : choose(kTilesAny, p, g, cost));
    if (bt)
        return cost;
    const double strips =
        strips_cost(p, g, level == 0 ? kStrip16 : level == 1 ? kStrip4 : kStripOdd);
    return strips < cost ? strips : cost;
}

double grouped_t_cost(const ProductArgs& p, const GroupArgs& g, int level)
{
    double cost;
    (void)(level ? choose_grad(kGradAny, p, g, cost) : choose_grad(kGrad16, p, g, cost));
    return cost;
}

hipError_t launch_grouped(const ProductArgs& p, const GroupArgs& g, int type, bool bt,
                          hipStream_t stream)
{
    if (type == kTI8)
        return grouped8(p, g, nullptr, stream);
    if (type == kTBf16)
        return bt ? grouped16<kTBf16, true>(p, g, nullptr, stream)
                  : grouped16<kTBf16, false>(p, g, nullptr, stream);
    return bt ? grouped16<kTF16, true>(p, g, nullptr, stream)
              : grouped16<kTF16, false>(p, g, nullptr, stream);
}

size_t grouped_workspace(ProductArgs p, const GroupArgs& g, int type, bool bt)
{
    size_t bytes = 0;
    p.may_split = 1;
    (void)(type == kTI8 ? grouped8(p, g, &bytes, nullptr)
           : bt         ? grouped16<kTBf16, true>(p, g, &bytes, nullptr)
                        : grouped16<kTBf16, false>(p, g, &bytes, nullptr));
    return bytes;
}

hipError_t launch_grouped_t(const ProductArgs& p, const GroupArgs& g, int type, hipStream_t stream)
{
    return type == kTBf16 ? grad16<kTBf16>(p, g, nullptr, stream)
                          : grad16<kTF16>(p, g, nullptr, stream);
}

size_t grouped_t_workspace(ProductArgs p, const GroupArgs& g, int)
{
    size_t bytes = 0;
    p.may_split = 1;
    (void)grad16<kTBf16>(p, g, &bytes, nullptr);
    return bytes;
}

}  // namespace qse
