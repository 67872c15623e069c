// The C ABI of the linear head's losses: argument checks, then the launches.
#include <math.h>
#include <string.h>

#include "internal.hpp"
#include "loss.hpp"

namespace dg {
namespace {

// Row pitches up to 4 MiB: a tile's 256 rows stay within a 31-bit offset.
constexpr int64_t kMaxPitch = INT64_C(1) << 21;      // elements
constexpr int64_t kMaxRows = INT64_C(1) << 20;
constexpr int64_t kMaxVocab = INT64_C(1) << 24;
constexpr int64_t kMaxWidth = INT64_C(1) << 16;

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// What forward and gradient share: sizes, X, W, workspace.
gemm_status check_common(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw, int64_t T,
                         int64_t V, int64_t D, int64_t slots, float scale, void* ws, size_t ws_bytes,
                         bool backward)
{
    if (T < 0 || V < 1 || D < 1 || !(fabsf(scale) < INFINITY) || !W || !aligned(W, 16) || ldw < D ||
        ldw % 8 != 0)
        return GEMM_ERR_INVALID_VALUE;
    if (D % 8 != 0 || T > kMaxRows || V > kMaxVocab || D > kMaxWidth || ldw > kMaxPitch)
        return GEMM_ERR_UNSUPPORTED;
    if (T == 0)
        return GEMM_OK;
    if (!X || !aligned(X, 16) || ldx < D || ldx % 8 != 0)
        return GEMM_ERR_INVALID_VALUE;
    if (ldx > kMaxPitch)
        return GEMM_ERR_UNSUPPORTED;
    if (!ws || !aligned(ws, 256) || (int64_t)ws_bytes < loss_plan(T, V, D, slots, backward).bytes)
        return GEMM_ERR_INVALID_VALUE;
    return GEMM_OK;
}

gemm_status check_slots(const int64_t* index, int64_t ld_index, const float* teacher,
                        int64_t ld_teacher, int64_t T, int64_t slots)
{
    if (slots < 1)
        return GEMM_ERR_INVALID_VALUE;
    if (slots > kMaxLossSlots)
        return GEMM_ERR_UNSUPPORTED;
    if (T > 0 && (!index || !aligned(index, 8) || ld_index < slots || !teacher || !aligned(teacher, 4) ||
                  ld_teacher < slots))
        return GEMM_ERR_INVALID_VALUE;
    return GEMM_OK;
}

gemm_status check_grad(const float* lse, const float* dloss, int64_t dloss_count, int64_t T, int64_t D,
                       const uint16_t* dX, int64_t lddx, const uint16_t* dW, int64_t lddw)
{
    // (without rows dX holds nothing and its pointer says nothing)
    if (!dX && !dW && T > 0)
        return GEMM_ERR_INVALID_VALUE;
    if (dW && (!aligned(dW, 2) || lddw < D))
        return GEMM_ERR_INVALID_VALUE;
    if (dW && lddw > kMaxPitch)
        return GEMM_ERR_UNSUPPORTED;
    if (T == 0)
        return GEMM_OK;
    if (!lse || !aligned(lse, 4) || !dloss || !aligned(dloss, 4) || (dloss_count != 1 && dloss_count != T))
        return GEMM_ERR_INVALID_VALUE;
    if (dX && (!aligned(dX, 2) || lddx < D))
        return GEMM_ERR_INVALID_VALUE;
    return GEMM_OK;
}

LossCall base_call(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw, int64_t T, int64_t V,
                   int64_t D, float scale, void* ws, void* stream)
{
    LossCall c;
    memset(&c, 0, sizeof c);
    c.X = X;
    c.ldx = ldx;
    c.W = W;
    c.ldw = ldw;
    c.T = T;
    c.V = V;
    c.D = D;
    c.scale = scale;
    c.ws = static_cast<uint8_t*>(ws);
    c.stream = reinterpret_cast<hipStream_t>(stream);
    return c;
}

gemm_status run(LossCall& c, bool backward)
{
    gemm_status st = device_info(&c.cus);
    if (st != GEMM_OK)
        return st;
    hipError_t err;
    if (c.T == 0) {
        // no row: nothing to score, the weight's gradient is zero
        Epilogue none;
        memset(&none, 0, sizeof none);
        err = backward && c.dW ? launch_zero_c(c.dW, c.lddw, c.V, c.D, none, c.stream) : hipSuccess;
    } else {
        err = backward ? loss_backward(c) : loss_forward(c);
    }
    return err == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

}  // namespace
}  // namespace dg

extern "C" {

size_t linear_loss_workspace_bytes(int64_t T, int64_t V, int64_t D, int64_t slots, int32_t backward)
{
    if (T < 1 || V < 1 || D < 1 || D % 8 != 0 || slots < 0 || slots > dg::kMaxLossSlots ||
        T > dg::kMaxRows || V > dg::kMaxVocab || D > dg::kMaxWidth)
        return 0;
    return (size_t)dg::loss_plan(T, V, D, slots, backward != 0).bytes;
}

gemm_status linear_cross_entropy(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw,
                                 const int64_t* labels, int64_t T, int64_t V, int64_t D, float scale,
                                 float z_loss, int64_t ignore_index, float* loss, float* lse,
                                 void* workspace, size_t workspace_bytes, void* stream)
{
    gemm_status st = dg::check_common(X, ldx, W, ldw, T, V, D, 0, scale, workspace, workspace_bytes, false);
    if (st != GEMM_OK)
        return st;
    if (!(fabsf(z_loss) < INFINITY) ||
        (T > 0 && (!labels || !dg::aligned(labels, 8) || !loss || !dg::aligned(loss, 4) || !lse ||
                   !dg::aligned(lse, 4))))
        return GEMM_ERR_INVALID_VALUE;
    if (T == 0)
        return GEMM_OK;
    dg::LossCall c = dg::base_call(X, ldx, W, ldw, T, V, D, scale, workspace, stream);
    c.z_loss = z_loss;
    c.labels = labels;
    c.ignore_index = ignore_index;
    c.loss = loss;
    c.lse = lse;
    return dg::run(c, false);
}

gemm_status linear_cross_entropy_grad(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw,
                                      const int64_t* labels, int64_t T, int64_t V, int64_t D,
                                      float scale, float z_loss, int64_t ignore_index,
                                      const float* loss, const float* lse, const float* dloss,
                                      int64_t dloss_count, uint16_t* dX, int64_t lddx, uint16_t* dW,
                                      int64_t lddw, void* workspace, size_t workspace_bytes,
                                      void* stream)
{
    gemm_status st = dg::check_common(X, ldx, W, ldw, T, V, D, 0, scale, workspace, workspace_bytes, true);
    if (st == GEMM_OK)
        st = dg::check_grad(lse, dloss, dloss_count, T, D, dX, lddx, dW, lddw);
    if (st != GEMM_OK)
        return st;
    if (!(fabsf(z_loss) < INFINITY) ||
        (T > 0 && (!labels || !dg::aligned(labels, 8) || !loss || !dg::aligned(loss, 4))))
        return GEMM_ERR_INVALID_VALUE;
    if (T == 0 && !dW)
        return GEMM_OK;
    dg::LossCall c = dg::base_call(X, ldx, W, ldw, T, V, D, scale, workspace, stream);
    c.z_loss = z_loss;
    c.labels = labels;
    c.ignore_index = ignore_index;
    c.loss_in = loss;
    c.lse_in = lse;
    c.dloss = dloss;
    c.dloss_stride = dloss_count == T ? 1 : 0;
    c.dX = dX;
    c.lddx = lddx;
    c.dW = dW;
    c.lddw = lddw;
    return dg::run(c, true);
}

gemm_status linear_distillation(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw,
                                const int64_t* index, int64_t ld_index, const float* teacher,
                                int64_t ld_teacher, int64_t T, int64_t V, int64_t D, int64_t slots,
                                float scale, float* loss, float* lse, float* logp, void* workspace,
                                size_t workspace_bytes, void* stream)
{
    gemm_status st = dg::check_slots(index, ld_index, teacher, ld_teacher, T, slots);
    if (st == GEMM_OK)
        st = dg::check_common(X, ldx, W, ldw, T, V, D, slots, scale, workspace, workspace_bytes, false);
    if (st != GEMM_OK)
        return st;
    if (T == 0)
        return GEMM_OK;
    if (!loss || !dg::aligned(loss, 4) || !lse || !dg::aligned(lse, 4) || !logp || !dg::aligned(logp, 4))
        return GEMM_ERR_INVALID_VALUE;
    dg::LossCall c = dg::base_call(X, ldx, W, ldw, T, V, D, scale, workspace, stream);
    c.index = index;
    c.ld_index = ld_index;
    c.teacher = teacher;
    c.ld_teacher = ld_teacher;
    c.slots = slots;
    c.loss = loss;
    c.lse = lse;
    c.logp = logp;
    return dg::run(c, false);
}

gemm_status linear_distillation_grad(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw,
                                     const int64_t* index, int64_t ld_index, const float* teacher,
                                     int64_t ld_teacher, int64_t T, int64_t V, int64_t D, int64_t slots,
                                     float scale, const float* lse, const float* logp,
                                     const float* dloss, int64_t dloss_count, uint16_t* dX,
                                     int64_t lddx, uint16_t* dW, int64_t lddw, void* workspace,
                                     size_t workspace_bytes, void* stream)
{
    gemm_status st = dg::check_slots(index, ld_index, teacher, ld_teacher, T, slots);
    if (st == GEMM_OK)
        st = dg::check_common(X, ldx, W, ldw, T, V, D, slots, scale, workspace, workspace_bytes, true);
    if (st == GEMM_OK)
        st = dg::check_grad(lse, dloss, dloss_count, T, D, dX, lddx, dW, lddw);
    if (st != GEMM_OK)
        return st;
    if (T == 0 && !dW)
        return GEMM_OK;
    if (T > 0 && (!logp || !dg::aligned(logp, 4)))
        return GEMM_ERR_INVALID_VALUE;
    dg::LossCall c = dg::base_call(X, ldx, W, ldw, T, V, D, scale, workspace, stream);
    c.index = index;
    c.ld_index = ld_index;
    c.teacher = teacher;
    c.ld_teacher = ld_teacher;
    c.slots = slots;
    c.lse_in = lse;
    c.logp_in = logp;
    c.dloss = dloss;
    c.dloss_stride = dloss_count == T ? 1 : 0;
    c.dX = dX;
    c.lddx = lddx;
    c.dW = dW;
    c.lddw = lddw;
    return dg::run(c, true);
}

}  // extern "C"
