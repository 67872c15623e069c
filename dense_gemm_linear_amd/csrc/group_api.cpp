// The C ABI of the grouped rows' operators: argument checks, then the launches.
#include <math.h>
#include <string.h>

#include "group.hpp"
#include "internal.hpp"

namespace dg {
namespace {

constexpr int64_t kMaxPitch = INT64_C(1) << 21;      // elements: a tile's rows stay within 31 bits
constexpr int64_t kMaxAdapterRows = INT64_C(1) << 20; // their table packs a row and a group in 32 bits
constexpr int64_t kMaxWidth = INT64_C(1) << 16;
constexpr int64_t kMaxColumns = INT64_C(1) << 20;

// A single row's pitch, or a single group's distance, says nothing and may be anything:
// what the kernels see is that of a row as long as it must be.
int64_t pitch_of(int64_t rows, int64_t ld, int64_t width) { return rows > 1 ? ld : (width + 7) / 8 * 8; }
int64_t stride_of(int64_t groups, int64_t stride) { return groups > 1 ? stride : 0; }

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// T tokens with k choices among `groups` groups
gemm_status check_slots(int64_t T, int64_t k, int64_t groups)
{
    if (T < 0 || k < 1 || groups < 1)
        return GEMM_ERR_INVALID_VALUE;
    if (T >= kMaxSorted || k > kMaxGroupSlots || T * k >= kMaxSorted || groups > kMaxGroups)
        return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

// rows of `width` elements that the products read 16 bytes at a time
gemm_status check_operand(const uint16_t* p, int64_t ld, int64_t rows, int64_t width)
{
    if (!p || !aligned(p, 16) || (rows > 1 && (ld < width || ld % 8 != 0)))
        return GEMM_ERR_INVALID_VALUE;
    return rows > 1 && ld > kMaxPitch ? GEMM_ERR_UNSUPPORTED : GEMM_OK;
}

gemm_status check_output(const uint16_t* p, int64_t ld, int64_t rows, int64_t width)
{
    if (!p || !aligned(p, 2) || (rows > 1 && ld < width))
        return GEMM_ERR_INVALID_VALUE;
    return rows > 1 && ld > kMaxPitch ? GEMM_ERR_UNSUPPORTED : GEMM_OK;
}

// [groups][rows][ld] with `stride` elements between groups
gemm_status check_stack(int64_t stride, int64_t groups, int64_t rows, int64_t ld, int64_t width, int64_t multiple)
{
    if (groups > 1 && (stride < (rows - 1) * ld + width || stride % multiple != 0))
        return GEMM_ERR_INVALID_VALUE;
    return groups > 1 && stride > INT64_C(1) << 40 ? GEMM_ERR_UNSUPPORTED : GEMM_OK;
}

gemm_status first_of(std::initializer_list<gemm_status> all)
{
    gemm_status bad = GEMM_OK;
    for (gemm_status s : all)
        if (s != GEMM_OK && (bad == GEMM_OK || s == GEMM_ERR_INVALID_VALUE))
            bad = s;
    return bad;
}

gemm_status check_sizes(int64_t N, int64_t K)
{
    if (N < 1 || K < 1)
        return GEMM_ERR_INVALID_VALUE;
    return K % 8 != 0 || K > kMaxWidth || N > kMaxColumns ? GEMM_ERR_UNSUPPORTED : GEMM_OK;
}

// rows of X that the loads pick up by their own 32-bit offsets
gemm_status check_picked(int64_t T, int64_t ldx, int64_t K)
{
    return (T - 1) * ldx * 2 + K * 2 >= INT64_C(1) << 31 ? GEMM_ERR_UNSUPPORTED : GEMM_OK;
}

gemm_status done(hipError_t e) { return e == hipSuccess ? GEMM_OK : GEMM_ERR_HIP; }

}  // namespace
}  // namespace dg

extern "C" {

size_t group_sort_workspace_bytes(int64_t T, int64_t k, int64_t groups)
{
    if (dg::check_slots(T, k, groups) != GEMM_OK)
        return 0;
    return (size_t)dg::sort_plan(T * k, groups).bytes;
}

gemm_status group_sort(const int64_t* ids, int64_t ld_ids, int64_t T, int64_t k, int64_t groups,
                       int32_t* offsets, int32_t* order, int32_t* place, void* workspace,
                       size_t workspace_bytes, void* stream)
{
    gemm_status st = dg::check_slots(T, k, groups);
    if (st != GEMM_OK)
        return st;
    if (!offsets || !dg::aligned(offsets, 4))
        return GEMM_ERR_INVALID_VALUE;
    if (T > 0 && (!ids || !dg::aligned(ids, 8) || (T > 1 && ld_ids < k) || !order || !dg::aligned(order, 4) ||
                  !place || !dg::aligned(place, 4)))
        return GEMM_ERR_INVALID_VALUE;
    const int64_t need = dg::sort_plan(T * k, groups).bytes;
    if (need > 0 && (!workspace || !dg::aligned(workspace, 16) || (int64_t)workspace_bytes < need))
        return GEMM_ERR_INVALID_VALUE;
    int cus;
    st = dg::device_info(&cus);
    if (st != GEMM_OK)
        return st;
    dg::SortCall c = {ids, T > 1 ? ld_ids : k, T, k, groups, offsets, order, place, workspace,
                      reinterpret_cast<hipStream_t>(stream)};
    return dg::done(dg::group_sort(c));
}

gemm_status group_gather(const void* X, int64_t ldx, const int32_t* place, int64_t T, int64_t k,
                         int64_t D, int32_t elem_bytes, void* Xs, int64_t ldxs, void* stream)
{
    gemm_status st = dg::check_slots(T, k, 1);
    if (st != GEMM_OK)
        return st;
    if (D < 1 || (elem_bytes != 1 && elem_bytes != 2 && elem_bytes != 4))
        return GEMM_ERR_INVALID_VALUE;
    if (D > dg::kMaxColumns)
        return GEMM_ERR_UNSUPPORTED;
    if (T == 0)
        return GEMM_OK;
    const uintptr_t e = (uintptr_t)elem_bytes;
    if (!X || !dg::aligned(X, e) || (T > 1 && ldx < D) || !place || !dg::aligned(place, 4) || !Xs ||
        !dg::aligned(Xs, e) || (T * k > 1 && ldxs < D))
        return GEMM_ERR_INVALID_VALUE;
    int cus;
    st = dg::device_info(&cus);
    if (st != GEMM_OK)
        return st;
    dg::GatherCall c = {static_cast<const uint8_t*>(X), ldx * elem_bytes, place, T, k, D * elem_bytes,
                        static_cast<uint8_t*>(Xs), ldxs * elem_bytes, reinterpret_cast<hipStream_t>(stream)};
    return dg::done(dg::group_gather(c));
}

gemm_status group_combine(const uint16_t* Y, int64_t ldy, const int32_t* place, const float* weights,
                          int64_t ld_weights, int64_t T, int64_t k, int64_t D, uint16_t* out, int64_t ldo,
                          void* stream)
{
    gemm_status st = dg::check_slots(T, k, 1);
    if (st != GEMM_OK)
        return st;
    if (D < 1)
        return GEMM_ERR_INVALID_VALUE;
    if (D > dg::kMaxColumns)
        return GEMM_ERR_UNSUPPORTED;
    if (T == 0)
        return GEMM_OK;
    if (!Y || !dg::aligned(Y, 2) || (T * k > 1 && ldy < D) || !place || !dg::aligned(place, 4) ||
        !dg::aligned(weights, 4) || (weights && T > 1 && ld_weights < k) || !out || !dg::aligned(out, 2) ||
        (T > 1 && ldo < D))
        return GEMM_ERR_INVALID_VALUE;
    int cus;
    st = dg::device_info(&cus);
    if (st != GEMM_OK)
        return st;
    dg::CombineCall c;
    memset(&c, 0, sizeof c);
    c.Y = Y;
    c.ldy = ldy;
    c.place = place;
    c.weights = weights;
    c.ld_weights = ld_weights;
    c.T = T;
    c.k = k;
    c.D = D;
    c.out = out;
    c.ldo = ldo;
    c.stream = reinterpret_cast<hipStream_t>(stream);
    return dg::done(dg::group_combine(c));
}

gemm_status group_combine_grad(const uint16_t* dout, int64_t ld_dout, const uint16_t* Y, int64_t ldy,
                               const int32_t* place, const float* weights, int64_t ld_weights, int64_t T,
                               int64_t k, int64_t D, uint16_t* dY, int64_t lddy, float* dweights,
                               void* stream)
{
    gemm_status st = dg::check_slots(T, k, 1);
    if (st != GEMM_OK)
        return st;
    if (D < 1)
        return GEMM_ERR_INVALID_VALUE;
    if (D > dg::kMaxColumns)
        return GEMM_ERR_UNSUPPORTED;
    if (T == 0)
        return GEMM_OK;
    if ((!dY && !dweights) || !dout || !dg::aligned(dout, 2) || (T > 1 && ld_dout < D) || !place ||
        !dg::aligned(place, 4) || !dg::aligned(weights, 4) || (weights && T > 1 && ld_weights < k) ||
        !dg::aligned(dY, 2) || (dY && T * k > 1 && lddy < D) || !dg::aligned(dweights, 4) ||
        (dweights && (!Y || !dg::aligned(Y, 2) || (T * k > 1 && ldy < D))))
        return GEMM_ERR_INVALID_VALUE;
    int cus;
    st = dg::device_info(&cus);
    if (st != GEMM_OK)
        return st;
    dg::CombineCall c;
    memset(&c, 0, sizeof c);
    c.dout = dout;
    c.lddo = ld_dout;
    c.Y = Y;
    c.ldy = ldy;
    c.place = place;
    c.weights = weights;
    c.ld_weights = ld_weights;
    c.T = T;
    c.k = k;
    c.D = D;
    c.dY = dY;
    c.lddy = lddy;
    c.dweights = dweights;
    c.stream = reinterpret_cast<hipStream_t>(stream);
    return dg::done(dg::group_combine_grad(c));
}

gemm_status group_linear(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw, int64_t w_stride,
                         const int32_t* offsets, const int32_t* order, int64_t T, int64_t k, int64_t groups,
                         int64_t N, int64_t K, int32_t activation, const uint16_t* mul, int64_t ld_mul,
                         uint16_t* Y, int64_t ldy, void* stream)
{
    gemm_status st = dg::first_of({dg::check_slots(T, k, groups), dg::check_sizes(N, K)});
    if (st != GEMM_OK)
        return st;
    if (activation < GEMM_ACT_NONE || activation > GEMM_ACT_GELU_TANH)
        return GEMM_ERR_INVALID_VALUE;
    if (T == 0)
        return GEMM_OK;
    const int64_t S = T * k;
    if ((!order && k != 1) || !offsets || !dg::aligned(offsets, 4) || !dg::aligned(order, 4))
        return GEMM_ERR_INVALID_VALUE;
    st = dg::first_of({dg::check_operand(X, ldx, T, K), dg::check_operand(W, ldw, N, K),
                       dg::check_stack(w_stride, groups, N, ldw, K, 8), dg::check_output(Y, ldy, S, N),
                       mul ? dg::check_output(mul, ld_mul, S, N) : GEMM_OK,
                       order ? dg::check_picked(T, ldx, K) : GEMM_OK});
    if (st != GEMM_OK)
        return st;
    dg::ProductCall c;
    memset(&c, 0, sizeof c);
    st = dg::device_info(&c.cus);
    if (st != GEMM_OK)
        return st;
    c.X = X;
    c.ldx = dg::pitch_of(T, ldx, K);
    c.W = W;
    c.ldw = dg::pitch_of(N, ldw, K);
    c.ldw_group = dg::stride_of(groups, w_stride);
    c.offsets = offsets;
    c.order = order;
    c.T = T;
    c.k = k;
    c.groups = groups;
    c.N = N;
    c.K = K;
    c.act = activation;
    c.mul = mul;
    c.ld_mul = dg::pitch_of(S, ld_mul, N);
    c.Y = Y;
    c.ldy = dg::pitch_of(S, ldy, N);
    c.stream = reinterpret_cast<hipStream_t>(stream);
    return dg::done(dg::group_forward(c));
}

size_t group_linear_grad_workspace_bytes(int64_t T, int64_t k, int64_t K)
{
    if (dg::check_slots(T, k, 1) != GEMM_OK || dg::check_sizes(1, K) != GEMM_OK)
        return 0;
    return (size_t)dg::group_grad_workspace(T, k, K);
}

gemm_status group_linear_grad(const uint16_t* dY, int64_t lddy, const uint16_t* X, int64_t ldx,
                              const uint16_t* W, int64_t ldw, int64_t w_stride, const int32_t* offsets,
                              const int32_t* order, int64_t T, int64_t k, int64_t groups, int64_t N, int64_t K,
                              uint16_t* dX, int64_t lddx, uint16_t* dW, int64_t lddw, int64_t dw_stride,
                              void* workspace, size_t workspace_bytes, void* stream)
{
    gemm_status st = dg::first_of({dg::check_slots(T, k, groups), dg::check_sizes(N, K),
                                   N % 8 != 0 || N > dg::kMaxWidth ? GEMM_ERR_UNSUPPORTED : GEMM_OK});
    if (st != GEMM_OK)
        return st;
    if (!dX && !dW)
        return GEMM_ERR_INVALID_VALUE;
    const int64_t S = T * k;
    if (dW) {
        st = dg::first_of({dg::check_output(dW, lddw, N, K), dg::check_stack(dw_stride, groups, N, lddw, K, 1)});
        if (st != GEMM_OK)
            return st;
    }
    if (T > 0) {
        if ((!order && k != 1) || !offsets || !dg::aligned(offsets, 4) || !dg::aligned(order, 4))
            return GEMM_ERR_INVALID_VALUE;
        st = dg::first_of({dg::check_operand(dY, lddy, S, N),
                           dX ? dg::check_operand(W, ldw, N, K) : GEMM_OK,
                           dX ? dg::check_stack(w_stride, groups, N, ldw, K, 8) : GEMM_OK,
                           dX ? dg::check_output(dX, lddx, S, K) : GEMM_OK,
                           dW ? dg::check_operand(X, ldx, T, K) : GEMM_OK});
        if (st != GEMM_OK)
            return st;
        if (dW && order && (!workspace || !dg::aligned(workspace, 256) ||
                            (int64_t)workspace_bytes < dg::group_grad_workspace(T, k, K)))
            return GEMM_ERR_INVALID_VALUE;
    } else if (!dW) {
        return GEMM_OK;
    }
    dg::ProductCall c;
    memset(&c, 0, sizeof c);
    st = dg::device_info(&c.cus);
    if (st != GEMM_OK)
        return st;
    c.stream = reinterpret_cast<hipStream_t>(stream);
    if (T == 0) {
        // no row: the weights' gradients are zero
        dg::Epilogue none;
        memset(&none, 0, sizeof none);
        for (int64_t g = 0; g < groups; ++g) {
            st = dg::done(dg::launch_zero_c(dW + g * dw_stride, lddw, N, K, none, c.stream));
            if (st != GEMM_OK)
                return st;
        }
        return GEMM_OK;
    }
    c.dY = dY;
    c.lddy = dg::pitch_of(S, lddy, N);
    c.X = X;
    c.ldx = dg::pitch_of(T, ldx, K);
    c.W = W;
    c.ldw = dg::pitch_of(N, ldw, K);
    c.ldw_group = dg::stride_of(groups, w_stride);
    c.offsets = offsets;
    c.order = order;
    c.T = T;
    c.k = k;
    c.groups = groups;
    c.N = N;
    c.K = K;
    c.dX = dX;
    c.lddx = dg::pitch_of(S, lddx, K);
    c.dW = dW;
    c.lddw = lddw;
    c.lddw_group = dg::stride_of(groups, dw_stride);
    c.ws = static_cast<uint8_t*>(workspace);
    return dg::done(dg::group_backward(c));
}

size_t linear_adapters_workspace_bytes(int64_t T, int64_t R, int64_t groups)
{
    if (dg::check_slots(T, 1, groups) != GEMM_OK || T > dg::kMaxAdapterRows || R < 1 || R % 8 != 0 || R > dg::kMaxRank)
        return 0;
    return (size_t)dg::adapters_workspace(T, R);
}

gemm_status linear_adapters(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw, const uint16_t* A,
                            int64_t lda, int64_t a_stride, const uint16_t* B, int64_t ldb, int64_t b_stride,
                            const float* scale, const int32_t* offsets, const int32_t* order, int64_t T,
                            int64_t N, int64_t K, int64_t R, int64_t groups, uint16_t* Y, int64_t ldy,
                            void* workspace, size_t workspace_bytes, void* stream)
{
    gemm_status st = dg::first_of({dg::check_slots(T, 1, groups), dg::check_sizes(N, K),
                                   T > dg::kMaxAdapterRows ? GEMM_ERR_UNSUPPORTED : GEMM_OK,
                                   R < 1 ? GEMM_ERR_INVALID_VALUE
                                         : R % 8 != 0 || R > dg::kMaxRank ? GEMM_ERR_UNSUPPORTED : GEMM_OK});
    if (st != GEMM_OK)
        return st;
    if (T == 0)
        return GEMM_OK;
    if (!offsets || !dg::aligned(offsets, 4) || !order || !dg::aligned(order, 4) || !dg::aligned(scale, 4) ||
        !workspace || !dg::aligned(workspace, 256) ||
        (int64_t)workspace_bytes < dg::adapters_workspace(T, R))
        return GEMM_ERR_INVALID_VALUE;
    st = dg::first_of({dg::check_operand(X, ldx, T, K), dg::check_operand(W, ldw, N, K),
                       dg::check_operand(A, lda, R, K), dg::check_stack(a_stride, groups, R, lda, K, 8),
                       dg::check_operand(B, ldb, N, R), dg::check_stack(b_stride, groups, N, ldb, R, 8),
                       dg::check_output(Y, ldy, T, N), dg::check_picked(T, ldx, K)});
    if (st != GEMM_OK)
        return st;
    dg::ProductCall c;
    memset(&c, 0, sizeof c);
    st = dg::device_info(&c.cus);
    if (st != GEMM_OK)
        return st;
    c.X = X;
    c.ldx = dg::pitch_of(T, ldx, K);
    c.W = W;
    c.ldw = dg::pitch_of(N, ldw, K);
    c.A = A;
    c.lda = dg::pitch_of(R, lda, K);
    c.lda_group = dg::stride_of(groups, a_stride);
    c.B = B;
    c.ldb = dg::pitch_of(N, ldb, R);
    c.ldb_group = dg::stride_of(groups, b_stride);
    c.scale = scale;
    c.offsets = offsets;
    c.order = order;
    c.T = T;
    c.k = 1;
    c.groups = groups;
    c.N = N;
    c.K = K;
    c.R = R;
    c.Y = Y;
    c.ldy = dg::pitch_of(T, ldy, N);
    c.ws = static_cast<uint8_t*>(workspace);
    c.stream = reinterpret_cast<hipStream_t>(stream);
    return dg::done(dg::adapters_forward(c));
}

}  // extern "C"
