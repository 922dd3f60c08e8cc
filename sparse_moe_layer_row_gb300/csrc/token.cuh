// Argument block and launcher of token.cu (the whole layer for a few rows).
#pragma once

#include "fp8.cuh"

namespace moe {

constexpr int kTokenRows = 8;      // the N of one mma.sync tile
constexpr int kTokenMaxH = 8192;   // x lies in shared memory
constexpr int kTokenMaxI = 16384;  // I and Is (a division by multiplication)

struct TokenArgs {
    const __nv_bfloat16* x;       // [R, H]
    int R, H, E, k, I, Is;
    int given;                    // topk_idx and topk_w are inputs
    const __nv_bfloat16* wr;      // router [E, H]
    const float* bias;            // [E] or NULL
    // weights, bf16 or e4m3: gate, up, down; the shared expert's
    const void *wg, *wu, *wd, *sg, *su, *sd;
    // e4m3: their scales per 128 x 128 block
    const float *cg, *cu, *cd, *csg, *csu, *csd;
    float* logits;                // [R, E], for rows of many equal ones
    int32_t* topk_idx;            // [R, k]
    float* topk_w;
    void* h;                      // 4 bytes for each of R (k I + Is) values
    uint64_t* counters;           // of the grid barrier: given routing, whole pass
    uint64_t* tagged;             // [8, kMaxExperts] logits with the number of their call
    uint32_t* status;
    __nv_bfloat16* y;             // [R, H]
    float* y_f32;                 // or NULL
    uint32_t inv_utiles;          // set by the launcher, as are the next two
    int arena, depth;             // shared memory of x and h; tiles in flight
    uint64_t wait_ns;             // limit of a grid barrier's wait (0: the built-in limit)
};
cudaError_t token_set_attributes();
cudaError_t launch_token(bool fp8, TokenArgs, int num_sms, cudaStream_t);

}  // namespace moe
