// Launches of the grouped products (group_kernels.hpp).  Compiled once per role
// (DG_GROUP_ROLE), so that the instances build in parallel; role 0's unit holds
// the entry points.
#if DG_GROUP_ROLE == 0
#include "adapter_kernels.hpp"
#else
#include "group_kernels.hpp"
#endif
#include "internal.hpp"

#include <stdio.h>
#include <string.h>

#include <algorithm>

namespace dg {

// Tile shapes, as those of the losses (loss.hip): large ones for many rows a
// group, tiles that just cover the rows, with deep rings, for few.
using GBig = GroupShape<256, 256, 2, 4, 4, 64, 1>;
using GTall = GroupShape<256, 128, 4, 2, 4, 64, 2>;
using GMid = GroupShape<128, 128, 2, 2, 4, 64, 2>;      // transposed operands
using GLine = GroupShape<128, 128, 2, 2, 2, 128, 2>;    // plain ones
using GDeep = GroupShape<128, 128, 2, 2, 4, 128, 1>;
using GSlim = GroupShape<128, 64, 2, 2, 6, 128, 1>;
using GFew = GroupShape<64, 128, 1, 4, 3, 128, 2>;
using GFewSlim = GroupShape<64, 64, 1, 4, 4, 128, 2>;
using GLow = GroupShape<32, 128, 1, 4, 3, 128, 2>;
using GLowSlim = GroupShape<32, 64, 1, 4, 5, 128, 2>;
using GOne = GroupShape<16, 32, 1, 2, 6, 128, 2>;
enum { G_BIG, G_TALL, G_MID, G_LINE, G_DEEP, G_SLIM, G_FEW, G_FEW_SLIM, G_LOW, G_LOW_SLIM, G_ONE };

hipError_t launch_group_fwd(int shape, const GroupArgs& a, int64_t extra, int cus, hipStream_t s);
hipError_t launch_group_gated(int shape, const GroupArgs& a, int64_t extra, int cus, hipStream_t s);
hipError_t launch_group_dx(int shape, const GroupArgs& a, int64_t extra, int cus, hipStream_t s);
hipError_t launch_group_dw(int shape, const GroupArgs& a, int64_t extra, int cus, hipStream_t s);
hipError_t launch_group_adapt(int shape, const GroupArgs& a, int64_t extra, int cus, hipStream_t s);

namespace {

// `extra`: groups whose last tile of rows may be partly filled
template <class S, int ROLE>
hipError_t go(const GroupArgs& a, int64_t extra, int cus, hipStream_t s)
{
    GroupArgs copy = a;
    copy.tiles_n = (int)cdiv(a.N, S::TN);
    if (ROLE == GROUP_ADAPT) {
        // adapters that share a k-tile are told apart by 32-bit offsets into B; else an
        // adapter's units fill whole k-tiles
        copy.pack = a.groups * a.lb_group < (INT64_C(1) << 31);
        copy.units = (int)(copy.pack ? cdiv(a.R, 16) : cdiv(a.R, S::KT / 2) * (S::KT / 32));
    }
    const int64_t tiles_m = ROLE == GROUP_DW ? a.groups * cdiv(a.M, S::TM)
                                             : ROLE == GROUP_ADAPT ? cdiv(a.S, S::TM) : a.S / S::TM + extra;
    const int64_t items = tiles_m * copy.tiles_n;
    if (items > INT32_MAX)
        return hipErrorInvalidValue;
    const int64_t grid = std::min<int64_t>(items, (int64_t)cus * S::PER_CU);
    void* args[] = {&copy};
    return hipLaunchKernel(reinterpret_cast<const void*>(&group_gemm_kernel<S, ROLE>), dim3((unsigned)grid),
                           dim3(S::THREADS), args, 0, s);
}

template <int ROLE>
hipError_t go_plain(int shape, const GroupArgs& a, int64_t extra, int cus, hipStream_t s)
{
    switch (shape) {
    case G_BIG:
        return go<GBig, ROLE>(a, extra, cus, s);
    case G_TALL:
        return go<GTall, ROLE>(a, extra, cus, s);
    case G_DEEP:
        return go<GDeep, ROLE>(a, extra, cus, s);
    case G_SLIM:
        return go<GSlim, ROLE>(a, extra, cus, s);
    case G_FEW:
        return go<GFew, ROLE>(a, extra, cus, s);
    case G_FEW_SLIM:
        return go<GFewSlim, ROLE>(a, extra, cus, s);
    case G_LOW_SLIM:
        return go<GLowSlim, ROLE>(a, extra, cus, s);
    case G_ONE:
        return go<GOne, ROLE>(a, extra, cus, s);
    }
    return go<GLine, ROLE>(a, extra, cus, s);
}

}  // namespace

#if DG_GROUP_ROLE == 0
hipError_t launch_group_fwd(int shape, const GroupArgs& a, int64_t extra, int cus, hipStream_t s)
{
    return go_plain<GROUP_FWD>(shape, a, extra, cus, s);
}
#elif DG_GROUP_ROLE == 4
hipError_t launch_group_gated(int shape, const GroupArgs& a, int64_t extra, int cus, hipStream_t s)
{
    return go_plain<GROUP_GATED>(shape, a, extra, cus, s);
}
#elif DG_GROUP_ROLE == 3
hipError_t launch_group_adapt(int shape, const GroupArgs& a, int64_t extra, int cus, hipStream_t s)
{
    return go_plain<GROUP_ADAPT>(shape, a, extra, cus, s);
}
#elif DG_GROUP_ROLE == 1
hipError_t launch_group_dx(int shape, const GroupArgs& a, int64_t extra, int cus, hipStream_t s)
{
    switch (shape) {
    case G_BIG:
        return go<GBig, GROUP_DX>(a, extra, cus, s);
    case G_TALL:
        return go<GTall, GROUP_DX>(a, extra, cus, s);
    case G_FEW:
        return go<GFew, GROUP_DX>(a, extra, cus, s);
    case G_LOW:
        return go<GLow, GROUP_DX>(a, extra, cus, s);
    }
    return go<GMid, GROUP_DX>(a, extra, cus, s);
}
#elif DG_GROUP_ROLE == 2
hipError_t launch_group_dw(int shape, const GroupArgs& a, int64_t extra, int cus, hipStream_t s)
{
    // (256 x 256 tiles spill registers into the K loop here, and took 368 us where 256 x
    // 128 ones took 299)
    return shape == G_TALL ? go<GTall, GROUP_DW>(a, extra, cus, s) : go<GMid, GROUP_DW>(a, extra, cus, s);
}
#endif

#if DG_GROUP_ROLE == 0

namespace {

// What one round of tiles (every CU holding its fill of workgroups) takes, in
// microseconds: kt for each 32 values of K, epi for the rest; kt1 where there is at
// most one workgroup a CU; start, once; across: how much longer than the others' the
// k-tiles get where rows of W do not start at whole 64 bytes, so that a piece of a row
// lies in two lines (32 groups, 25940 rows, N 1776, K 4032 and 4040: 256 x 256 tiles 390
// and 576 us, 128 x 128 of two stages 432 and 540).  Fitted to the times of all shapes at 242
// sizes, most drawn at random (1 to 8192 tokens, 1 to 8 choices, 4 to 128 groups, N 256
// to 11008, K 256 to 11008; 2 to 4095 rows with adapters): the shape chosen takes 2 %
// longer than the best on average with groups, 1 % with adapters, and 30 % at most
// (groups of equal size just under a whole tile's rows, which the host cannot see).  Slots
// that take no part it cannot see either: up to 1.75 times the best shape's time where a
// third of those of 54 groups do.
struct Cost {
    int shape, tm, tn, per_cu;
    double kt, kt1, epi, start, across;
};
template <class S>
constexpr Cost cost_of(int shape, double kt, double kt1, double epi, double start = 0.0, double across = 1.0)
{
    return {shape, S::TM, S::TN, S::PER_CU, kt, kt1, epi, start, across};
}
constexpr Cost kPlain[] = {cost_of<GBig>(G_BIG, 0.74, 0.62, 7.5, 0.0, 1.3),
                           cost_of<GTall>(G_TALL, 0.48, 0.42, 3.8, 0.0, 1.3),
                           cost_of<GLine>(G_LINE, 0.54, 0.37, 2.5),
                           cost_of<GDeep>(G_DEEP, 0.27, 0.27, 2.3, 0.0, 1.1),
                           cost_of<GSlim>(G_SLIM, 0.20, 0.11, 2.0, 0.0, 1.1),
                           cost_of<GFew>(G_FEW, 0.41, 0.22, 4.6),
                           cost_of<GFewSlim>(G_FEW_SLIM, 0.21, 0.14, 4.3),
                           cost_of<GLowSlim>(G_LOW_SLIM, 0.17, 0.12, 2.7),
                           cost_of<GOne>(G_ONE, 0.11, 0.08, 1.9)};
constexpr Cost kAdapt[] = {cost_of<GBig>(G_BIG, 0.74, 0.48, 6.6),          cost_of<GTall>(G_TALL, 0.48, 0.42, 4.3),
                           cost_of<GLine>(G_LINE, 0.43, 0.38, 2.5),        cost_of<GDeep>(G_DEEP, 0.28, 0.27, 2.3),
                           cost_of<GSlim>(G_SLIM, 0.20, 0.19, 2.0),        cost_of<GFew>(G_FEW, 0.41, 0.19, 5.9),
                           cost_of<GFewSlim>(G_FEW_SLIM, 0.21, 0.13, 4.0), cost_of<GLowSlim>(G_LOW_SLIM, 0.17, 0.11, 2.9),
                           cost_of<GOne>(G_ONE, 0.12, 0.08, 1.9)};
constexpr Cost kDx[] = {cost_of<GBig>(G_BIG, 0.74, 0.62, 7.5), cost_of<GTall>(G_TALL, 0.48, 0.42, 3.8),
                        cost_of<GMid>(G_MID, 0.56, 0.41, 0.5), cost_of<GFew>(G_FEW, 0.57, 0.15, 4.6),
                        cost_of<GLow>(G_LOW, 0.40, 0.13, 1.3)};
// dW, 1 to 6300 rows a group, N 520 to 11008: the smaller tile takes less for few rows
// (14 a group of 4096 x 4096: 65 us against 72) and few tiles (256 a group, 32 of 1024 x
// 2048: 58 against 60), the larger one else (1024 a group, 8 of 11008 x 4096: 757
// against 862; 252 a group, 16 of them: 617 against 678)
constexpr Cost kDw[] = {cost_of<GTall>(G_TALL, 0.47, 0.47, 3.9, 4.0), cost_of<GMid>(G_MID, 0.57, 0.57, 3.4)};

// Estimated time of `tiles` rows of tiles over `cols` columns and `kts` times 32
// values of K.
double tiles_us(const Cost& c, double tiles, int64_t cols, double kts, int cus, bool across)
{
    if (across)
        kts *= c.across;
    const double items = tiles * (double)cdiv(cols, c.tn), round = (double)cus * c.per_cu;
    const double full = (double)(int64_t)(items / round), left = items - full * round;
    return c.start + full * (kts * c.kt + c.epi) + (left > 0.5 ? kts * (left > cus ? c.kt : c.kt1) + c.epi : 0.0);
}

// Tiles of tm rows that T tokens of k slots are expected to make in `used` of the groups:
// a group's last tile is half empty on average, and groups are uneven.  Where a token
// has as many slots as there are groups, it is in all of them, as a rule, and each has
// T rows (6 groups of 189 rows, 5296 x 2416: 89 us without this, 63 with it).
double row_tiles(int64_t T, int64_t k, int64_t groups, int64_t used, int tm)
{
    if (k == groups)
        return (double)(used * cdiv(T, tm));
    const double rows = (double)(T * k);
    const double mean = rows / (double)used;
    return (double)used * std::max(mean > 1.5 ? 1.07 : 1.0, mean / tm + 0.59);
}

// The shape of the least estimate.  `reads`: microseconds that the groups' weights
// take from memory; a row of tiles past a group's first reads them from the caches, at
// four times the rate.  Where that is longer than the products it counts in
// their place, and these for a little, between shapes that read alike (57 rows a group
// of 64, N 4096, K 11008: 64 x 128 tiles, of which many groups need two, 1347 us, 128 x
// 128 1145).  The smallest tiles only where they make no second round: what bounds such
// a product is reading W, which they do less well (16 x 2 rows of 8 groups of 4096 x
// 4096: 51 us against 44).
struct Picked {
    int shape;
    double us;
};
template <int N, class Tiles>
Picked pick(const Cost (&of)[N], int64_t cols, double kts, int cus, double reads, int64_t used, bool across,
            Tiles&& tiles)
{
    Picked best = {-1, 0.0};
    for (const Cost& c : of) {
        const double t = tiles(c.tm);
        if (c.shape == G_ONE && t * (double)cdiv(cols, c.tn) > (double)cus * c.per_cu)
            continue;
        const double us = tiles_us(c, t, cols, kts, cus, across);
        const double all = std::max(us, reads * (1.0 + (t / (double)used - 1.0) * 0.25)) + 0.05 * us;
        if (best.shape < 0 || all < best.us)
            best = {c.shape, all};
    }
    return best;
}

// Microseconds to read `groups` weights of N x K once, at 5 TB/s.
double weights_us(int64_t groups, int64_t N, int64_t K)
{
    return (double)groups * (double)N * (double)K * 2.0 / 5.0e6;
}

GroupArgs base_args(const ProductCall& c)
{
    GroupArgs a;
    memset(&a, 0, sizeof a);
    a.offsets = c.offsets;
    a.groups = (int)c.groups;
    a.S = (int)(c.T * c.k);
    a.order = c.order;
    a.k_mul = divide_by(c.k);
    return a;
}

int vec_of(const uint16_t* C, int64_t ldc, int64_t N)
{
    return ((uintptr_t)C & 15u) == 0 && ldc % 8 == 0 && N % 8 == 0;
}

}  // namespace

// Adapters in slices of K: rows at most, and what the workspace holds for the
// slices' sums: 8 slices of 16384 columns, 32 MiB at most.
constexpr int64_t kSplitRows = 2048;
// waves of a workgroup of one token's kernel
constexpr int kTokenWaves = 16;
static int64_t split_bytes(int64_t T)
{
    return T <= kSplitRows ? std::min<int64_t>(T << 19, INT64_C(32) << 20) : 0;
}
static int64_t inner_bytes(int64_t T, int64_t R) { return cdiv(T * R * 4, 256) * 256; }

int64_t group_grad_workspace(int64_t T, int64_t k, int64_t K) { return T * k * K * 2; }

int64_t adapters_workspace(int64_t T, int64_t R) { return inner_bytes(T, R) + split_bytes(T); }

// The shapes of a call's products.
static int forward_shape(const ProductCall& c)
{
    const int64_t used = std::min(c.groups, c.T * c.k);
    const bool across = ((uintptr_t)c.W | (uint64_t)c.ldw * 2 | (uint64_t)c.ldw_group * 2) % 64 != 0;
    return pick(kPlain, c.N, (double)cdiv(c.K, 32), c.cus, weights_us(used, c.N, c.K), used, across,
                [&](int tm) { return row_tiles(c.T, c.k, c.groups, used, tm); }).shape;
}
static int dx_shape(const ProductCall& c)
{
    const int64_t used = std::min(c.groups, c.T * c.k);
    return pick(kDx, c.K, (double)cdiv(c.N, 32), c.cus, weights_us(used, c.N, c.K), used, false,
                [&](int tm) { return row_tiles(c.T, c.k, c.groups, used, tm); }).shape;
}
static int dw_shape(const ProductCall& c)
{
    return pick(kDw, c.K, (double)cdiv(cdiv(c.T * c.k, c.groups), 32), c.cus, 0.0, 1, false,
                [&](int tm) { return (double)(c.groups * cdiv(c.N, tm)); }).shape;
}

hipError_t group_forward(const ProductCall& c)
{
    const int64_t S = c.T * c.k, used = std::min(c.groups, S);
    GroupArgs a = base_args(c);
    a.A = reinterpret_cast<const uint8_t*>(c.X);
    a.lda_b = c.ldx * 2;
    a.a_bytes = c.order ? (uint32_t)((c.T - 1) * c.ldx * 2 + c.K * 2) : 0u;
    a.B = reinterpret_cast<const uint8_t*>(c.W);
    a.ldb_b = c.ldw * 2;
    a.b_group = c.ldw_group * 2;
    a.N = (int)c.N;
    a.K = (int)c.K;
    a.C = c.Y;
    a.ldc = c.ldy;
    a.c_vec = vec_of(c.Y, c.ldy, c.N);
    a.act = c.act;
    a.mul = c.mul;
    a.ld_mul = c.ld_mul;
    a.mul_vec = c.mul && ((uintptr_t)c.mul & 7u) == 0 && c.ld_mul % 4 == 0 && c.N % 4 == 0;
    a.b_nt = 1;
    const int shape = forward_shape(c);
    return c.act || c.mul ? launch_group_gated(shape, a, used, c.cus, c.stream)
                          : launch_group_fwd(shape, a, used, c.cus, c.stream);
}

hipError_t group_backward(const ProductCall& c)
{
    const int64_t S = c.T * c.k, used = std::min(c.groups, S);
    if (c.dX) {
        GroupArgs a = base_args(c);
        a.A = reinterpret_cast<const uint8_t*>(c.dY);
        a.lda_b = c.lddy * 2;
        a.B = reinterpret_cast<const uint8_t*>(c.W);
        a.ldb_b = c.ldw * 2;
        a.b_group = c.ldw_group * 2;
        a.N = (int)c.K;
        a.K = (int)c.N;
        a.C = c.dX;
        a.ldc = c.lddx;
        a.c_vec = vec_of(c.dX, c.lddx, c.K);
        a.b_nt = 1;
        const hipError_t e = launch_group_dx(dx_shape(c), a, used, c.cus, c.stream);
        if (e != hipSuccess)
            return e;
    }
    if (!c.dW)
        return hipSuccess;
    const uint16_t* Xs = c.X;
    int64_t ldxs = c.ldx;
    if (c.order) {
        PickCall g;
        g.X = c.X;
        g.ldx = c.ldx;
        g.offsets = c.offsets;
        g.order = c.order;
        g.S = S;
        g.k = c.k;
        g.groups = c.groups;
        g.K = c.K;
        g.Xs = reinterpret_cast<uint16_t*>(c.ws);
        g.stream = c.stream;
        const hipError_t e = group_pick(g);
        if (e != hipSuccess)
            return e;
        Xs = g.Xs;
        ldxs = c.K;
    }
    GroupArgs a = base_args(c);
    a.A = reinterpret_cast<const uint8_t*>(c.dY);
    a.lda_b = c.lddy * 2;
    a.B = reinterpret_cast<const uint8_t*>(Xs);
    a.ldb_b = ldxs * 2;
    a.M = (int)c.N;
    a.N = (int)c.K;
    a.C = c.dW;
    a.ldc = c.lddw;
    a.c_group = c.lddw_group;
    a.c_vec = vec_of(c.dW, c.lddw, c.K) && c.lddw_group % 8 == 0;
    // Stored past the caches: an optimizer reads dW when it is long out of them, and the
    // rows of X and dY stay (32 groups of 1024 x 2048: 256 rows a group 84 -> 57 us, 16
    // rows 42 -> 36).  Y and dX, which the next kernel reads, are not: alone they gain 0 to
    // 2 %, with that kernel they lose up to 5.  Not where rows start inside 64 bytes: the
    // ends of a tile's rows would go to memory as parts of lines (15 rows in 62 groups of
    // 984 x 5528: 357 us, 189 through the caches; of 984 x 5504 159 and 164).
    if (a.c_vec && ((uintptr_t)c.dW | (uint64_t)c.lddw * 2 | (uint64_t)c.lddw_group * 2) % 64 == 0)
        a.c_vec = 2;
    return launch_group_dw(dw_shape(c), a, 0, c.cus, c.stream);
}

template <class Args>
hipError_t launch(const void* kernel, dim3 grid, int block, Args a, hipStream_t s)
{
    void* args[] = {&a};
    return hipLaunchKernel(kernel, grid, dim3((unsigned)block), args, 0, s);
}

// The inner values.  Where a workgroup for each row and 16 ranks makes one round,
// that; else the smallest tile whose workgroups do (a workgroup takes 2.5 us and 1.9
// for each 16 rows of X or A, K 4096: 4095 rows of 64 ranks 19 us as 32 x 64, 34 as
// 16 x 16; 597 of 32 ranks 7.6 as 16 x 16, 13.7 as 64 x 32).
constexpr struct {
    int nr, mb;
} kInner[] = {{1, 1}, {1, 2}, {2, 2}, {1, 4}, {4, 2}, {2, 4}, {4, 4}};
constexpr int kInnerTiles = (int)(sizeof kInner / sizeof kInner[0]);

// The tile, or -1: a workgroup a row.
int inner_tile(int64_t T, int64_t groups, int64_t R, int cus)
{
    const int64_t units = cdiv(R, 16);
    if (T * units <= cus)
        return -1;
    // groups in use are not known here; each has a partly filled tile
    const int64_t some = std::min<int64_t>(std::min<int64_t>(groups, 16), T / 16 + 1);
    int best = 0;
    for (int t = 0; t < kInnerTiles; ++t) {
        if (kInner[t].nr > 1 && kInner[t].nr / 2 >= units)
            continue;
        best = t;
        if ((T / (16 * kInner[t].mb) + some) * cdiv(units, kInner[t].nr) <= cus)
            break;
    }
    return best;
}

hipError_t launch_inner(const InnerArgs& i, int cus, hipStream_t s)
{
    const int64_t T = i.S, units = cdiv(i.R, 16);
    const int t = inner_tile(T, i.groups, i.R, cus);
    if (t < 0)
        return launch(reinterpret_cast<const void*>(&adapter_inner_row_kernel), dim3((unsigned)T, (unsigned)units),
                      1024, i, s);
    const void* const kernels[kInnerTiles] = {reinterpret_cast<const void*>(&adapter_inner_kernel<1, 1>),
                                              reinterpret_cast<const void*>(&adapter_inner_kernel<1, 2>),
                                              reinterpret_cast<const void*>(&adapter_inner_kernel<2, 2>),
                                              reinterpret_cast<const void*>(&adapter_inner_kernel<1, 4>),
                                              reinterpret_cast<const void*>(&adapter_inner_kernel<4, 2>),
                                              reinterpret_cast<const void*>(&adapter_inner_kernel<2, 4>),
                                              reinterpret_cast<const void*>(&adapter_inner_kernel<4, 4>)};
    return launch(kernels[t],
                  dim3((unsigned)(T / (16 * kInner[t].mb) + std::min<int64_t>(i.groups, T)),
                       (unsigned)cdiv(units, kInner[t].nr)),
                  512, i, s);
}

// tiles of the slices
using SLow = GroupShape<32, 128, 1, 4, 3, 128, 2>;
using SFew = GroupShape<64, 128, 1, 4, 3, 128, 2>;
using SMid = GroupShape<128, 128, 2, 2, 4, 128, 2>;

// Few rows: tile rows and slices of the least estimate, in microseconds: a CU's
// k-tiles of 64 values one after the other, W, the slices' sums, what the inner values
// read and what the join reads of B.  Fitted to 356 times (2 to 512 rows, N 512 to
// 11008, K 1024 to 11008, 8 to 64 ranks); the choice takes 4 % longer than the best of
// these on average, 18 % at most.  At 58 sizes of 513 to 2048 rows (N 256 to 11008, K 256 to
// 8192, 8 to 128 ranks) this form or the whole product, as said here, takes 0.7 % longer than
// the better one on average, 12 % at most.
struct AdapterPlan {
    int tm;
    int64_t slices;
    double us;
};
AdapterPlan adapter_plan(int64_t T, int64_t N, int64_t K, int64_t R, int cus)
{
    constexpr struct {
        int tm, start;             // start: in k-tiles
        double kt;                 // for each byte of a k-tile
    } shapes[] = {{SLow::TM, 3, 7.0e-6}, {SFew::TM, 0, 7.0e-6}, {SMid::TM, 0, 8.5e-6}};
    AdapterPlan best = {0, 0, 0.0};
    const int64_t kts = cdiv(K, 64), sums = T * cdiv(N, 4) * 16;
    const double rest = 5.7 + 0.154e-6 * (double)(N * K * 2) + 0.088e-6 * (double)(T * cdiv(R, 16) * 20 * K * 2) +
                        0.33e-6 * (double)(cdiv(T, kJoinRows) * N * R * 2);
    for (const auto& sh : shapes) {
        const int64_t tiles = cdiv(T, sh.tm) * cdiv(N, SLow::TN);
        const double kt = sh.kt * (double)((std::min<int64_t>(T, sh.tm) + SLow::TN) * 128);
        for (int64_t most = 1; most <= 8 && most * sums <= split_bytes(T); ++most) {
            const int64_t each = cdiv(kts, most), slices = cdiv(kts, each);
            const double us = rest + kt * (double)(cdiv(tiles * slices, cus) * (each + sh.start)) + 0.257e-6 * (double)(slices * sums);
            if (!best.tm || us < best.us)
                best = {sh.tm, slices, us};
        }
    }
    return best;
}

template <class S>
hipError_t go_split(const ProductCall& c, int64_t slices)
{
    const int64_t T = c.T, kts = cdiv(c.K * 2, S::KTB);
    SplitArgs a;
    a.X = reinterpret_cast<const uint8_t*>(c.X);
    a.ldx_b = c.ldx * 2;
    a.W = reinterpret_cast<const uint8_t*>(c.W);
    a.ldw_b = c.ldw * 2;
    a.T = (int)T;
    a.N = (int)c.N;
    a.K = (int)c.K;
    a.tiles_m = (int)cdiv(T, S::TM);
    a.kts = (int)cdiv(kts, slices);
    a.slices = (int)cdiv(kts, a.kts);
    a.main = (int)(a.tiles_m * a.slices * cdiv(c.N, S::TN));
    a.nt = a.tiles_m == 1;
    a.planes = reinterpret_cast<float*>(c.ws + inner_bytes(T, c.R));
    a.pitch = (int)cdiv(c.N, 4) * 4;
    a.offsets = c.offsets;
    a.order = c.order;
    a.groups = (int)c.groups;
    a.R = (int)c.R;
    a.A = reinterpret_cast<const uint8_t*>(c.A);
    a.lda_b = c.lda * 2;
    a.a_group = c.lda_group * 2;
    a.scale = c.scale;
    a.U = reinterpret_cast<float*>(c.ws);
    const hipError_t e = launch(reinterpret_cast<const void*>(&adapter_split_kernel<S>),
                                dim3((unsigned)(a.main + T * cdiv(c.R, 16))), S::THREADS, a, c.stream);
    if (e != hipSuccess)
        return e;
    JoinArgs j;
    j.planes = a.planes;
    j.slices = a.slices;
    j.T = a.T;
    j.N = a.N;
    j.pitch = a.pitch;
    j.offsets = c.offsets;
    j.order = c.order;
    j.groups = a.groups;
    j.R = a.R;
    j.U = a.U;
    j.B = c.B;
    j.ldb = c.ldb;
    j.b_group = c.ldb_group;
    j.Y = c.Y;
    j.ldy = c.ldy;
    const void* join = c.R <= 16   ? reinterpret_cast<const void*>(&adapter_join_kernel<2>)
                       : c.R <= 32 ? reinterpret_cast<const void*>(&adapter_join_kernel<4>)
                                   : reinterpret_cast<const void*>(&adapter_join_kernel<8>);
    return launch(join, dim3((unsigned)cdiv(T, kJoinRows), (unsigned)cdiv(c.N, 256)), 256, j, c.stream);
}

// How a call of linear_adapters is done.
struct AdapterChoice {
    int64_t token_rows;            // > 0: one token in one launch, rows of W a wave
    AdapterPlan split;             // tm > 0: slices of K
    int shape;                     // else the whole product's
};
AdapterChoice adapter_choice(const ProductCall& c)
{
    const int64_t T = c.T;
    AdapterChoice a = {0, {0, 0, 0.0}, -1};
    // One token in one launch, where that forms the inner values in every workgroup in
    // little time (4096 x 4096, rank 32: 12 us, in slices 14; rank 64 16 and 14, rank 256 57
    // and 17; 2048 x 2048, rank 64: 11 and 14): one workgroup of 16 waves a CU, with as
    // many rows a wave as that takes, up to 4.
    if (T == 1 && c.R * c.K <= 1 << 17) {
        a.token_rows = std::min<int64_t>(4, cdiv(c.N, (int64_t)c.cus * kTokenWaves));
        return a;
    }
    // every row counts, groups or not; the ranks as k-tiles of about as many adapters
    // as a tile of 64 rows has
    const int64_t near = std::min<int64_t>(std::min(c.groups, T), cdiv(std::min(c.groups, T) * 64, T) + 1);
    const double kts = (double)cdiv(c.K, 32) + (double)(near * cdiv(c.R, 16));
    const Picked whole = pick(kAdapt, c.N, kts, c.cus, 0.0, 1, false,
                              [&](int tm) { return (double)cdiv(T, tm); });
    a.shape = whole.shape;
    // In slices of K where that takes less: the whole product has the inner values in a
    // launch before it, and its ranks.  16 ranks: 48 rows of 11008 x 4096 26.6 us against
    // 35.5, 40 of 4096 x 4096 14.7 against 24.7, 300 of them 26.8 against 32.1; 400 of
    // 11008 x 4096 82 against 77.
    if (T <= kSplitRows) {
        const AdapterPlan s = adapter_plan(T, c.N, c.K, c.R, c.cus);
        if (s.tm && (T == 1 || s.us < 7.3 + 1.05 * whole.us))
            a.split = s;
    }
    return a;
}

hipError_t adapters_forward(const ProductCall& c)
{
    const int64_t T = c.T;
    const AdapterChoice choice = adapter_choice(c);
    if (choice.token_rows > 0) {
        TokenArgs t;
        t.X = c.X;
        t.W = c.W;
        t.ldw = c.ldw;
        t.A = c.A;
        t.lda = c.lda;
        t.a_group = c.lda_group;
        t.B = c.B;
        t.ldb = c.ldb;
        t.b_group = c.ldb_group;
        t.scale = c.scale;
        t.offsets = c.offsets;
        t.groups = (int)c.groups;
        t.N = (int)c.N;
        t.K = (int)c.K;
        t.R = (int)c.R;
        t.Y = c.Y;
        const int64_t rows = choice.token_rows;
        const void* kernel = rows == 1   ? reinterpret_cast<const void*>(&adapter_token_kernel<1, kTokenWaves>)
                             : rows == 2 ? reinterpret_cast<const void*>(&adapter_token_kernel<2, kTokenWaves>)
                             : rows == 3 ? reinterpret_cast<const void*>(&adapter_token_kernel<3, kTokenWaves>)
                                         : reinterpret_cast<const void*>(&adapter_token_kernel<4, kTokenWaves>);
        return launch(kernel, dim3((unsigned)cdiv(c.N, rows * kTokenWaves)), 64 * kTokenWaves, t, c.stream);
    }
    if (choice.split.tm)
        return choice.split.tm == SLow::TM   ? go_split<SLow>(c, choice.split.slices)
               : choice.split.tm == SFew::TM ? go_split<SFew>(c, choice.split.slices)
                                             : go_split<SMid>(c, choice.split.slices);
    const uint32_t x_bytes = (uint32_t)((T - 1) * c.ldx * 2 + c.K * 2);
    InnerArgs i;
    i.X = reinterpret_cast<const uint8_t*>(c.X);
    i.ldx_b = c.ldx * 2;
    i.x_bytes = x_bytes;
    i.offsets = c.offsets;
    i.order = c.order;
    i.groups = (int)c.groups;
    i.S = (int)T;
    i.A = reinterpret_cast<const uint8_t*>(c.A);
    i.lda_b = c.lda * 2;
    i.a_group = c.lda_group * 2;
    i.scale = c.scale;
    i.R = (int)c.R;
    i.K = (int)c.K;
    i.U = reinterpret_cast<uint16_t*>(c.ws);
    const hipError_t e = launch_inner(i, c.cus, c.stream);
    if (e != hipSuccess)
        return e;
    GroupArgs a = base_args(c);
    a.A = reinterpret_cast<const uint8_t*>(c.X);
    a.lda_b = c.ldx * 2;
    a.a_bytes = x_bytes;
    a.B = reinterpret_cast<const uint8_t*>(c.W);
    a.ldb_b = c.ldw * 2;
    a.N = (int)c.N;
    a.K = (int)c.K;
    a.C = c.Y;
    a.ldc = c.ldy;
    a.c_vec = vec_of(c.Y, c.ldy, c.N);
    a.b_nt = T <= 64;
    a.U = c.ws;
    a.LB = reinterpret_cast<const uint8_t*>(c.B);
    a.ldlb_b = c.ldb * 2;
    a.lb_group = c.ldb_group * 2;
    a.R = (int)c.R;
    return launch_group_adapt(choice.shape, a, 0, c.cus, c.stream);
}

// What a call takes, as a text: for the tests, which are to reach every instance.
extern "C" int dg_group_choice(int op, int64_t T, int64_t k, int64_t groups, int64_t N, int64_t K, int64_t R, int cus,
                               char* text, size_t bytes)
{
    static const char* const names[] = {"256x256", "256x128", "128x128 transposed", "128x128", "128x128 deep", "128x64",
                                        "64x128", "64x64", "32x128", "32x64", "16x32"};
    ProductCall c;
    memset(&c, 0, sizeof c);
    c.T = T;
    c.k = k;
    c.groups = groups;
    c.N = N;
    c.K = K;
    c.R = R;
    c.cus = cus;
    c.ldw = K;
    c.ldw_group = N * K;
    if (op < GROUP_ADAPT)
        return snprintf(text, bytes, "%s",
                        names[op == GROUP_FWD ? forward_shape(c) : op == GROUP_DX ? dx_shape(c) : dw_shape(c)]);
    const AdapterChoice a = adapter_choice(c);
    if (a.token_rows > 0)
        return snprintf(text, bytes, "token %d", (int)a.token_rows);
    if (a.split.tm)
        return snprintf(text, bytes, "slices %d", a.split.tm);
    const int t = inner_tile(T, groups, R, cus);
    return t < 0 ? snprintf(text, bytes, "whole %s, inner row", names[a.shape])
                 : snprintf(text, bytes, "whole %s, inner %dx%d", names[a.shape], 16 * kInner[t].mb, 16 * kInner[t].nr);
}

#endif

}  // namespace dg
