// The loss over a large vocabulary: launches and workspace, shared by head_loss.hip and api.hip.
#pragma once
#include <hip/hip_runtime.h>

#include "internal.h"

namespace qn {

// A head of V rows: bf16 [V, d] at row stride ldw, or (codes not null) an NF4 weight.
struct HeadCall {
    const uint16_t* W; int64_t ldw;
    const uint8_t* codes; BlockConsts bc;
    int64_t V, d;
    const uint16_t* X; int64_t ldx;
    const int64_t* target;                    // [T]; outside [0, V): not counted
    int64_t T;
    const float* scale;                       // [T] or null (1)
    float* loss;                              // [T]
    uint16_t* dX; int64_t lddx;               // or null: the loss alone
};

// Pieces of the vocabulary and the workspace's parts (byte offsets; parts a call does not use
// have size 0). false: a size that the kernels do not take (an operand of 4 GiB or more). ldw: the head's
// row stride (d of an NF4 head); the workspace for ldw = d is enough for any.
struct HeadPlan {
    int64_t piece;                            // rows per piece, a multiple of 256
    int pieces, lt, slots;                    // tiles of 1 << lt; tiles of sums of the gradient's product
    int64_t ints, part, E, rows, wt, acc, bytes;
};
bool head_plan(int64_t V, int64_t d, int64_t ldw, int64_t T, bool nf4, bool grad, HeadPlan* p);

hipError_t launch_head_loss(const HeadCall& c, const HeadPlan& p, char* ws, hipStream_t st);

}  // namespace qn
