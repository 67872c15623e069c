// Host-side declarations of the grouped rows' operators: sorting and joining
// (group.hip), products (group_product.hip), their C ABI (group_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/densegemm.h"

namespace dg {

constexpr int64_t kMaxGroups = 512;
constexpr int64_t kMaxGroupSlots = 64;               // choices a token
// slots in all, less than: their rows at 256 threads each make a grid below 2^32 threads
constexpr int64_t kMaxSorted = INT64_C(1) << 24;
constexpr int64_t kMaxRank = 256;

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
// x / k as the high half of x times this: exact while x * k < 2^32 (2^24 * 64
// at most).  0 stands for k = 1.
inline uint32_t divide_by(int64_t k)
{
    return k == 1 ? 0u : (uint32_t)(((UINT64_C(1) << 32) + (uint64_t)k - 1) / (uint64_t)k);
}

// group_sort of more slots than one workgroup takes: chunks of slots with a
// workgroup each, whose counts lie in the workspace.
struct SortPlan {
    int64_t chunk, chunks;       // slots a workgroup, workgroups
    int64_t bytes;               // workspace: 0 for one chunk
};
SortPlan sort_plan(int64_t S, int64_t groups);

struct SortCall {
    const int64_t* ids;
    int64_t ld_ids;
    int64_t T, k, groups;
    int* offsets;
    int* order;
    int* place;
    void* ws;
    hipStream_t stream;
};
hipError_t group_sort(const SortCall& c);

struct GatherCall {
    const uint8_t* X;
    int64_t ldx_b;
    const int* place;
    int64_t T, k, row_b;         // row_b: bytes of a row
    uint8_t* Xs;
    int64_t ldxs_b;
    hipStream_t stream;
};
hipError_t group_gather(const GatherCall& c);

struct CombineCall {
    const uint16_t* Y;
    int64_t ldy;
    const int* place;
    const float* weights;        // null: 1
    int64_t ld_weights;
    int64_t T, k, D;
    uint16_t* out;               // combine
    int64_t ldo;
    const uint16_t* dout;        // gradient
    int64_t lddo;
    uint16_t* dY;
    int64_t lddy;
    float* dweights;
    hipStream_t stream;
};
hipError_t group_combine(const CombineCall& c);
hipError_t group_combine_grad(const CombineCall& c);

// One grouped product, or a linear layer with adapters.  Arguments checked.
struct ProductCall {
    const uint16_t* X;           // rows by token (order given) or sorted
    int64_t ldx;
    const uint16_t* W;           // [groups][N][ldw]
    int64_t ldw, ldw_group;
    const int* offsets;
    const int* order;
    int64_t T, k, groups, N, K;  // S = T k sorted rows
    // forward
    uint16_t* Y;
    int64_t ldy;
    int act;
    const uint16_t* mul;
    int64_t ld_mul;
    // gradient
    const uint16_t* dY;
    int64_t lddy;
    uint16_t* dX;
    int64_t lddx;
    uint16_t* dW;
    int64_t lddw, lddw_group;
    // adapters
    const uint16_t* A;           // [groups][R][lda]
    int64_t lda, lda_group;
    const uint16_t* B;           // [groups][N][ldb]
    int64_t ldb, ldb_group;
    const float* scale;          // [groups] or null
    int64_t R;
    uint8_t* ws;
    int cus;
    hipStream_t stream;
};
hipError_t group_forward(const ProductCall& c);
hipError_t group_backward(const ProductCall& c);
hipError_t adapters_forward(const ProductCall& c);
// workspaces: the sorted rows of X for dW, the adapters' inner values
int64_t group_grad_workspace(int64_t T, int64_t k, int64_t K);
int64_t adapters_workspace(int64_t T, int64_t R);

// a row of X by sorted position, for dW (group.hip)
struct PickCall {
    const uint16_t* X;
    int64_t ldx;
    const int* offsets;
    const int* order;
    int64_t S, k, groups, K;
    uint16_t* Xs;                // [S][K]
    hipStream_t stream;
};
hipError_t group_pick(const PickCall& c);

}  // namespace dg
