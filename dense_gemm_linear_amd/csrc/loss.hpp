// Host-side declarations of the linear head's losses (loss.hip, loss_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/densegemm.h"

namespace dg {

constexpr int kMaxLossSlots = 256;

// Workspace of one call: byte offsets from its start, and the sizes that fix
// them.  Everything follows from (T, V, D, slots, backward).
struct LossPlan {
    int64_t rows_pad;            // T rounded up to 256
    int64_t rows;                // rows of the large tables: T of few rows, else rows_pad
    int64_t tiles_n_max;         // forward: tile columns of the narrowest tile
    int64_t piece;               // backward: columns of the vocabulary at a time
    int64_t ldg;                 // backward: pitch of G
    int dx_shape, splits;        // backward: tile shape and K slices of the dX product
    int pair;                    // backward: K slices of dX where it shares a launch with dW, 0: never
    bool few;                    // at most one tile of rows; backward: G in two halves
    int64_t off_count, off_chunks, off_map, off_pos, off_rows, off_x;
    int64_t off_part, off_zlabel;                       // forward
    int64_t off_q, off_qsum, off_rest, off_lead, off_flag;        // distillation targets
    int64_t off_g, off_planes;                          // backward
    int64_t groups;              // backward of more rows: the vocabulary's groups of columns
    int64_t off_group, off_place;
    int64_t bytes;
};
LossPlan loss_plan(int64_t T, int64_t V, int64_t D, int64_t slots, bool backward);

// One call, arguments checked.
struct LossCall {
    const uint16_t* X;
    int64_t ldx;
    const uint16_t* W;
    int64_t ldw;
    int64_t T, V, D;
    float scale, z_loss;
    // cross entropy
    const int64_t* labels;
    int64_t ignore_index;
    // distillation
    const int64_t* index;
    const float* teacher;
    int64_t ld_index, ld_teacher;
    int64_t slots;               // 0: cross entropy
    // forward
    float* loss;
    float* lse;
    float* logp;
    // gradient
    const float* loss_in;
    const float* lse_in;
    const float* logp_in;
    const float* dloss;
    int64_t dloss_stride;        // 0: one value for every row
    uint16_t* dX;
    int64_t lddx;
    uint16_t* dW;
    int64_t lddw;
    uint8_t* ws;
    int cus;
    hipStream_t stream;
};
hipError_t loss_forward(const LossCall& c);
hipError_t loss_backward(const LossCall& c);

}  // namespace dg
