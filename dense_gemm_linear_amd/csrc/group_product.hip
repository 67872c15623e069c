// Launches of the grouped products (group_kernels.hpp).  Compiled once per role
// (DG_GROUP_ROLE), so that the instances build in parallel; role 0's unit holds
// the entry points.
#include "group_kernels.hpp"
#include "internal.hpp"

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
    case G_LOW:
        return go<GLow, ROLE>(a, extra, cus, s);
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
    switch (shape) {
    case G_BIG:
        return go<GBig, GROUP_DW>(a, extra, cus, s);
    case G_TALL:
        return go<GTall, GROUP_DW>(a, extra, cus, s);
    }
    return go<GMid, GROUP_DW>(a, extra, cus, s);
}
#endif

#if DG_GROUP_ROLE == 0

namespace {

struct Cost {
    int shape, tm, tn, per_cu;
    double kt, kt1, epi;         // as ShapeCost in loss.hip: us a round for 32 of K, and its rest
};
constexpr Cost kCosts[] = {{G_BIG, GBig::TM, GBig::TN, GBig::PER_CU, 0.72, 0.72, 9.0},
                           {G_TALL, GTall::TM, GTall::TN, GTall::PER_CU, 0.48, 0.48, 4.5},
                           {G_MID, GMid::TM, GMid::TN, GMid::PER_CU, 0.64, 0.50, 0.5},
                           {G_LINE, GLine::TM, GLine::TN, GLine::PER_CU, 0.56, 0.47, 1.0},
                           {G_DEEP, GDeep::TM, GDeep::TN, GDeep::PER_CU, 0.30, 0.29, 2.0}};

// Estimated time of `tiles` rows of tiles over `cols` columns and k values.
double tiles_us(const Cost& c, double tiles, int64_t cols, int64_t k, int cus)
{
    const double items = tiles * (double)cdiv(cols, c.tn), round = (double)cus * c.per_cu;
    const double full = (double)(int64_t)(items / round), left = items - full * round, kts = (double)cdiv(k, 32);
    return full * (kts * c.kt + c.epi) + (left > 0.5 ? kts * (left > cus ? c.kt : c.kt1) + c.epi : 0.0);
}

// Tiles of tm rows that `rows` rows in `used` groups are expected to make: half
// a tile a group is empty on average.
double row_tiles(int64_t rows, int64_t used, int tm)
{
    if (used == 1)
        return (double)cdiv(rows, tm);
    return (double)used * std::max(1.0, (double)rows / (double)used / tm + 0.5);
}

int pick(std::initializer_list<int> of, int64_t rows, int64_t used, int64_t cols, int64_t k, int cus)
{
    int best = -1;
    double us = 0.0;
    for (int i : of) {
        const double t = tiles_us(kCosts[i], row_tiles(rows, used, kCosts[i].tm), cols, k, cus);
        if (best < 0 || t < us) {
            best = kCosts[i].shape;
            us = t;
        }
    }
    return best;
}

// Shape of a product whose W rows are read as they lie.  Few rows a group: the
// tile that covers twice their mean, narrow where wide tiles make no full round.
int plain_shape(int64_t rows, int64_t used, int64_t cols, int64_t k, int cus)
{
    const int64_t mean = cdiv(rows, used);
    if (mean <= 2 && used * cdiv(cols, 32) <= 8 * cus)
        return G_ONE;
    if (mean <= 16)
        return used * cdiv(cols, 128) <= 2 * cus ? G_LOW_SLIM : G_LOW;
    if (mean <= 40)
        return used * cdiv(cols, 128) <= 2 * cus ? G_FEW_SLIM : G_FEW;
    return pick({0, 1, 3, 4}, rows, used, cols, k, cus);
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

int64_t group_grad_workspace(int64_t T, int64_t k, int64_t K) { return T * k * K * 2; }

int64_t adapters_workspace(int64_t T, int64_t R) { return T * R * 4; }

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
    a.mul_vec = ((uintptr_t)c.mul & 7u) == 0 && c.ld_mul % 4 == 0 && c.N % 4 == 0;
    a.b_nt = 1;
    const int shape = plain_shape(S, used, c.N, c.K, c.cus);
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
        const int64_t mean = cdiv(S, used);
        const int shape = mean <= 16 ? G_LOW : mean <= 40 ? G_FEW : pick({0, 1, 2}, S, used, c.K, c.N, c.cus);
        const hipError_t e = launch_group_dx(shape, a, used, c.cus, c.stream);
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
    int shape = G_MID;
    double best = 0.0;
    for (int i : {0, 1, 2}) {
        const double us = tiles_us(kCosts[i], (double)(c.groups * cdiv(c.N, kCosts[i].tm)), c.K, cdiv(S, c.groups),
                                   c.cus);
        if (best == 0.0 || us < best) {
            best = us;
            shape = kCosts[i].shape;
        }
    }
    return launch_group_dw(shape, a, 0, c.cus, c.stream);
}

hipError_t adapters_forward(const ProductCall& c)
{
    const int64_t T = c.T;
    const uint32_t x_bytes = (uint32_t)((T - 1) * c.ldx * 2 + c.K * 2);
    if (c.R > 0 && c.groups > 0) {
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
        // 16 rows a workgroup; 32, which read A half as often, where 16 make more
        // than one round
        const int64_t cols = c.R > 32 ? 64 : c.R > 16 ? 32 : 16, wide = cdiv(c.R, cols);
        const bool two = (T / 16 + std::min(c.groups, T)) * wide > c.cus;
        const int64_t blocks = T / (two ? 32 : 16) + std::min(c.groups, T);
        void* args[] = {&i};
        const void* kernel =
            two ? (cols == 64   ? reinterpret_cast<const void*>(&adapter_inner_kernel<4, 2, 8, 2>)
                   : cols == 32 ? reinterpret_cast<const void*>(&adapter_inner_kernel<2, 2, 8, 4>)
                                : reinterpret_cast<const void*>(&adapter_inner_kernel<1, 2, 8, 4>))
                : (cols == 64   ? reinterpret_cast<const void*>(&adapter_inner_kernel<4, 1, 16, 2>)
                   : cols == 32 ? reinterpret_cast<const void*>(&adapter_inner_kernel<2, 1, 16, 2>)
                                : reinterpret_cast<const void*>(&adapter_inner_kernel<1, 1, 16, 4>));
        const hipError_t e = hipLaunchKernel(kernel, dim3((unsigned)blocks, (unsigned)wide),
                                             dim3(two ? 512 : 1024), args, 0, c.stream);
        if (e != hipSuccess)
            return e;
    }
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
    // one group of T rows: the number is known
    const bool narrow = cdiv(c.N, 128) <= 2 * c.cus;
    const int shape = T <= 16 && cdiv(c.N, 32) <= 8 * c.cus ? G_ONE
                      : T <= 32 ? (narrow ? G_LOW_SLIM : G_LOW)
                      : T <= 64 ? (narrow ? G_FEW_SLIM : G_FEW)
                                : pick({0, 1, 3, 4}, T, 1, c.N, c.K, c.cus);
    return launch_group_adapt(shape, a, 0, c.cus, c.stream);
}

#endif

}  // namespace dg
