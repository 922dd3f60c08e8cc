// Argument block and launcher of route_scored.cu.
#pragma once

#include "kernels.cuh"

namespace moe {

struct RouteScoredArgs {
    const void* logits;   // [R] rows of E, ld elements apart
    int64_t ld;
    int R, E, k;
    const float* bias;    // [E] or NULL
    moe_route_rule rule;
    int gs;               // experts per group
    uint32_t ginv;        // ceil(2^20 / gs): e / gs = (e * ginv) >> 20 for e < 1024
    int32_t* topk_idx;
    float* topk_w;
    float* topk_score;    // or NULL
};
cudaError_t launch_route_scored(const RouteScoredArgs&, int dtype, int num_sms, cudaStream_t);

}  // namespace moe
