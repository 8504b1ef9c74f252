// Internal declarations of the operators for many adapters on one layer (plan, forward,
// gradients) and of the AdamW step over their tensors.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.h"

namespace qn {

// ---- adamw.hip ----
constexpr int kAdamBlock = 256;             // elements per state block (one wave, 4 per lane)
constexpr int kAdamChunkBlocks = 8;         // blocks per workgroup
constexpr int kAdamChunk = kAdamBlock * kAdamChunkBlocks;

// One tensor of a step's table; the table is an array of these, then one AdamChunk per
// workgroup.
struct AdamTensor {
    void* p;                                // float32 or bf16 parameters [n]
    const void* g;                          // float32 or bf16 gradient [n]
    uint16_t* copy;                         // bf16 copy of p [n], or null
    int64_t n;
    int64_t first_block;                    // its first block in the state arrays
    int64_t vec;                            // 1: p, g, copy take 4 elements per access
};
struct AdamChunk {
    int32_t tensor;
    int32_t chunk;                          // chunk of the tensor
};

struct AdamArgs {
    const AdamTensor* tensors;
    const AdamChunk* chunks;
    void* m; void* v;                       // float32, or uint8 codes [blocks * 256]
    float* m_scale; float* v_scale;         // 8-bit states: largest magnitude per block
    const float* grad_scale;                // device scalar or null
    const float* lr_dev;                    // device learning rate or null (then lr)
    const int64_t* step_dev;                // device step number or null (then step)
    double lr, beta1, beta2, weight_decay;
    int64_t step;
    float eps;
    uint32_t seed;
};

hipError_t launch_adamw(const AdamArgs& a, int64_t n_chunks, bool states8, bool grad_bf16, bool param_bf16,
                        hipStream_t st);
// float32 values of the 8-bit states of `blocks` blocks
hipError_t launch_adamw_moments(const uint8_t* m, const float* m_scale, const uint8_t* v, const float* v_scale,
                                int64_t blocks, float* m_out, float* v_out, hipStream_t st);

}  // namespace qn
