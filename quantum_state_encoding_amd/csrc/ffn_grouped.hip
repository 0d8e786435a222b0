// Products of rows grouped by expert, and the gradients of the weights.
//
// C[i] = A[i] B_e^T for the rows i of group e, in ffn_matmul.hip's tiles and
// ffn_strip.hip's strips: a workgroup finds its group and its tile there from
// the groups' ends, which only the device knows, and goes on as in a product of
// that group alone.  The grid has a workgroup for each tile that there could be
// (a last tile that is not whole for each group); those without one end.
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

// Rows of group e (e == experts: of the rows behind the last one).
__device__ __forceinline__ int rows_of(const GroupArgs& g, int e, int& first)
{
    const int m = (int)g.rows;
    const int lo = e > 0 ? g.ends[e - 1] : 0, hi = e < g.experts ? g.ends[e] : m;
    first = lo < 0 ? 0 : lo < m ? lo : m;
    const int last = hi < 0 ? 0 : hi < m ? hi : m;
    return last > first ? last - first : 0;
}

// The tile of workgroup w among all groups' tiles of bm rows and tiles_n
// columns: 64 groups at a time, one on each lane, whose tiles are summed across
// the wave (every wave finds the same).  Each XCD gets a contiguous run of them.
// HALVES: where the last round of tiles would leave half of the CUs without one,
// two workgroups (of one XCD) take half of each tile's rows.
constexpr int kCus = 256;
template <int BM, bool HALVES = false>
__device__ __forceinline__ bool find_group(const GroupArgs& g, int w, int tiles_n, Group& at)
{
    const int lane = threadIdx.x & 63;
    const int groups = g.experts + (g.zero_rest ? 1 : 0);
    const auto sum = [=](int base, int& first, int& rows, int& tiles) __attribute__((always_inline)) {
        const int e = base + lane;
        rows = e < groups ? rows_of(g, e, first) : 0;
        tiles = (rows + BM - 1) / BM * tiles_n;
        int s = tiles;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(s, d);
            s += lane >= d ? o : 0;
        }
        return s;                        // up to this lane's
    };
    int first = 0, rows = 0, tiles = 0;
    int upto = sum(0, first, rows, tiles);
    int total = __builtin_amdgcn_readlane(upto, 63);
    for (int base = 64; base < groups; base += 64) {
        int f, r, t;
        total += __builtin_amdgcn_readlane(sum(base, f, r, t), 63);
    }
    at.half = 0;
    if constexpr (HALVES) {
        const int last = total % kCus, whole = total - last;
        if (last <= kCus / 2 && w >= whole) {
            const int j = w - whole;
            at.half = 1 + ((j >> 3) & 1);
            w = whole + ((j >> 4) << 3) + (j & 7);
        }
    }
    if (w >= total)
        return false;
    const int t = place_of(w, total);
    int before = 0;
    for (int base = 0; base < groups; base += 64) {
        if (base > 0)
            upto = sum(base, first, rows, tiles);
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

// Zeros to rows x cols results at (m0, n0).
__device__ __forceinline__ void zero_tile(void* c, int64_t ldc, int type, int64_t m0, int64_t n0,
                                          int rows, int cols)
{
    for (int r = 0; r < rows; ++r)
        for (int n = (int)threadIdx.x; n < cols; n += (int)blockDim.x) {
            const int64_t at = (m0 + r) * ldc + n0 + n;
            if (type == kTF32)
                ((float*)c)[at] = 0.0f;
            else
                ((unsigned short*)c)[at] = 0;
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
        if (blockIdx.y == 0 && at.half < 2)
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
    product_body<TYPE, BM, BN, WM, WN, WK, NS, kEpStore, kNoScale, REG, false, BT,
                 kPipe, true>(
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
// One expert's tiles after the other's, each expert's spread over the XCDs (their
// times differ by the experts'), and of up to 64 experts those with the most rows
// first, so that the last tiles are short.
__device__ __forceinline__ int enter_grad(ProductArgs& p, const GroupArgs& g, GradPlace& where)
{
    const int per = p.tiles_m * p.tiles_n;
    int e = (int)blockIdx.x / per, first;
    const int t = place_of((int)blockIdx.x - e * per, per);
    if (g.experts > 1 && g.experts <= 64) {
        const int lane = threadIdx.x & 63;
        const int n = lane < g.experts ? rows_of(g, lane, first) : -1;
        int rank = 0;
        for (int o = 0; o < g.experts; ++o) {
            const int other = __builtin_amdgcn_readlane(n, o);
            rank += other > n || (other == n && o < lane) ? 1 : 0;
        }
        e = __builtin_ctzll(__ballot(lane < g.experts && rank == e));
    }
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
    product_body<TYPE, BM, BN, WM, WN, WK, NS, kEpStore, kNoScale, REG, true, true,
                 BM == 256 && !REG, true>(
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

int64_t groups_of(const GroupArgs& g) { return g.experts + (g.zero_rest ? 1 : 0); }

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
        tiles += kCus / 2;               // (halves)
    hipLaunchKernelGGL(k, dim3(tiles, (unsigned)splits), dim3(64 * WM * WN * WK), kLds, stream, p, g);
    e = hipGetLastError();
    if (splits == 1 || e != hipSuccess)
        return e;
    if constexpr (BM <= 128 && BN <= 128)
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

// Which tile, as ffn_matmul.hip chooses: rounds of workgroups times the time of
// a step.  How the rows are spread is not known: a group is taken to have the
// average number, and half a tile of rows more than it fills.
template <int N>
Choice cheapest_grouped(const Tile (&tiles)[N], const ProductArgs& p, const GroupArgs& g)
{
    const int64_t steps = (p.kbytes + kStep - 1) / kStep;
    const double groups = (double)(g.experts < p.m ? g.experts : p.m), avg = p.m / groups;
    Choice best{0, 1, 0};
    double least = 0;
    for (int i = 0; i < N; ++i) {
        const Tile& t = tiles[i];
        const int64_t tn = (p.n + t.bn - 1) / t.bn;
        const int64_t most = most_tiles(p.m, groups_of(g), t.bm) * tn;
        const double each = g.experts == 1 || avg <= t.bm / 2 ? (double)((int64_t)(avg / t.bm) + 1)
                                                              : avg / t.bm + 0.5;
        const double rounds = groups * each * tn / t.slots;
        double cost = most >= kFfnMaxTiles ? 1e300 : (rounds < 1 ? 1 : rounds) * t.step * steps;
        int splits = 1;
        if (t.area && p.may_split && most * 2 <= t.slots) {
            int64_t s = t.slots / most < 32 ? t.slots / most : 32;
            s = s < steps / 4 ? s : steps / 4;
            s = s > 1 ? (steps + (steps + s - 1) / s - 1) / ((steps + s - 1) / s) : 1;
            const double shared = (double)((steps + s - 1) / s) * t.step + 5.0;
            if (s > 1 && shared < cost) {
                cost = shared;
                splits = (int)s;
            }
        }
        if (i == 0 || cost < least) {
            least = cost;
            best = Choice{i, splits, splits > 1 ? (size_t)splits * most * t.area * 4 : 0};
        }
    }
    return best;
}

bool any_address(const ProductArgs& p, const GroupArgs& g, uintptr_t mask)
{
    return (((uintptr_t)p.a | (uintptr_t)p.b0 | (uintptr_t)p.lda | (uintptr_t)p.ldb0 |
             (uintptr_t)g.stride_b) & mask) != 0;
}

template <int TYPE, bool BT>
hipError_t grouped16(const ProductArgs& p, const GroupArgs& g, size_t* query, hipStream_t stream)
{
    constexpr Tile any[] = {{256, 256, 256, 1.9f, 0}, {128, 128, 512, 1.2f, 128 * 128}};
    constexpr Tile tiles[] = {{256, 256, 256, 1.6f, 0},
                              {128, 128, 512, 1.06f, 0},
                              {128, 128, 256, .62f, 128 * 128},
                              {64, 128, 256, .42f, 64 * 128}};
    const Choice ca = cheapest_grouped(any, p, g), c = cheapest_grouped(tiles, p, g);
    if (query) {
        *query = ca.bytes > c.bytes ? ca.bytes : c.bytes;
        return hipSuccess;
    }
    if (any_address(p, g, 15)) {
        if (p.kbytes < 16 || (BT && p.n < 8))
            return run_grouped<TYPE, 128, 128, 2, 2, 1, 2, BT, kShortRows>(p, g, 1, stream);
        if (ca.tile == 0)
            return run_grouped<TYPE, 256, 256, 2, 4, 1, 2, BT, kAnyAddress>(p, g, 1, stream);
        return run_grouped<TYPE, 128, 128, 2, 2, 1, 2, BT, kAnyAddress>(p, g, ca.splits, stream);
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
    constexpr Tile tiles[] = {{256, 256, 256, 1.5f, 0},
                              {128, 128, 512, 1.0f, 0},
                              {128, 128, 256, .60f, 0},
                              {64, 64, 512, .40f, 0},
                              {64, 64, 256, .26f, 64 * 64}};
    const Choice c = cheapest_grouped(tiles, p, g);
    if (query) {
        *query = c.bytes;
        return hipSuccess;
    }
    switch (c.tile) {
    case 0:
        return run_grouped<kTI8, 256, 256, 2, 4, 1, 2, false>(p, g, 1, stream);
    case 1:
        return run_grouped<kTI8, 128, 128, 2, 2, 1, 2, false>(p, g, 1, stream);
    case 2:
        return run_grouped<kTI8, 128, 128, 2, 2, 2, 2, false>(p, g, 1, stream);
    case 3:
        return run_grouped<kTI8, 64, 64, 2, 2, 2, 2, false>(p, g, 1, stream);
    }
    return run_grouped<kTI8, 64, 64, 2, 2, 2, 4, false>(p, g, c.splits, stream);
}

template <int TYPE>
hipError_t grad16(const ProductArgs& p, const GroupArgs& g, size_t* query, hipStream_t stream)
{
    // (an expert's tiles take its own rows: the average's steps)
    ProductArgs q = p;
    q.kbytes = (p.kbytes + g.experts - 1) / g.experts;
    constexpr Tile any[] = {{256, 256, 256, 1.9f, 0}, {128, 128, 512, 1.2f, 128 * 128}};
    constexpr Tile tiles[] = {{256, 256, 256, 1.6f, 0},
                              {128, 128, 512, 1.06f, 0},
                              {128, 128, 256, .62f, 128 * 128}};
    const auto pick = [&](const auto& list) {
        const int64_t steps = (q.kbytes + kStep - 1) / kStep;
        Choice best{0, 1, 0};
        double least = 0;
        int i = 0;
        for (const Tile& t : list) {
            const int64_t count =
                ((p.m + t.bm - 1) / t.bm) * ((p.n + t.bn - 1) / t.bn) * g.experts;
            double cost = count >= kFfnMaxTiles
                              ? 1e300
                              : (double)((count + t.slots - 1) / t.slots) * t.step * steps;
            int splits = 1;
            if (t.area && p.may_split && count * 2 <= t.slots) {
                int64_t s = t.slots / count < 32 ? t.slots / count : 32;
                s = s < steps / 4 ? s : steps / 4;
                const double shared = s > 1 ? (double)((steps + s - 1) / s) * t.step + 5.0 : 1e300;
                if (shared < cost) {
                    cost = shared;
                    splits = (int)s;
                }
            }
            if (i == 0 || cost < least) {
                least = cost;
                best = Choice{i, splits, splits > 1 ? (size_t)splits * count * t.area * 4 : 0};
            }
            ++i;
        }
        return best;
    };
    const Choice ca = pick(any), c = pick(tiles);
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

// Few rows to a group: strips.
bool strips(const ProductArgs& p, const GroupArgs& g, bool bt)
{
    return !bt && p.m <= 16 * (int64_t)g.experts &&
           most_tiles(p.m, groups_of(g), 16) * ((p.n + 15) / 16) < kFfnMaxTiles;
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

template <int TYPE>
hipError_t pick_strips(const ProductArgs& p, const GroupArgs& g, hipStream_t stream)
{
    if constexpr (TYPE != kTI8) {
        if (any_address(p, g, 3))
            return run_strips<TYPE, 1, 8, 4, true>(p, g, stream);
    }
    return run_strips<TYPE, 1, 8, 4, false>(p, g, stream);
}

}  // namespace

hipError_t launch_grouped(const ProductArgs& p, const GroupArgs& g, int type, bool bt,
                          hipStream_t stream)
{
    const bool few = strips(p, g, bt);
    if (type == kTI8)
        return few ? pick_strips<kTI8>(p, g, stream) : grouped8(p, g, nullptr, stream);
    if (type == kTBf16)
        return few  ? pick_strips<kTBf16>(p, g, stream)
               : bt ? grouped16<kTBf16, true>(p, g, nullptr, stream)
                    : grouped16<kTBf16, false>(p, g, nullptr, stream);
    return few  ? pick_strips<kTF16>(p, g, stream)
           : bt ? grouped16<kTF16, true>(p, g, nullptr, stream)
                : grouped16<kTF16, false>(p, g, nullptr, stream);
}

size_t grouped_workspace(ProductArgs p, const GroupArgs& g, int type, bool bt)
{
    size_t bytes = 0;
    p.may_split = 1;
    if (!strips(p, g, bt))
        (void)(type == kTI8 ? grouped8(p, g, &bytes, nullptr)
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
