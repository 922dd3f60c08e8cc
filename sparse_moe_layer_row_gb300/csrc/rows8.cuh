// Argument blocks and launchers of rows8.cu (norm of rows, int8 codes of rows)
// and i8_gemm.cu (the product on int8 codes).
#pragma once

#include "fp8.cuh"

namespace moe {

struct RmsNormArgs {
    const void* x;            // [R] rows of H values, ldx elements apart
    int64_t ldx;
    const void* residual;     // likewise, or NULL
    int64_t ldr;
    void* total;              // x + residual in the residual's type, or NULL
    int64_t ldt;
    const void* w;            // [H], or NULL: ones
    int res_f32, w_f32;       // residual and total, w: fp32 instead of the type of x
    int R, H;
    float eps, inv_h;         // inv_h: 1 / H
    void* y;                  // the type of x, or NULL
    int64_t ldy;
    uint8_t* codes;           // [R, H], or NULL
    float* scales;            // e4m3: [ceil(H / 128), R]; int8: [R]
};
// What a call makes of its rows.
enum { kNormOnly = 0, kNormE4m3 = 1, kNormI8 = 2, kQuantI8 = 3 };
cudaError_t launch_rows8(int what, const RmsNormArgs&, int dtype, int num_sms, cudaStream_t);

struct I8GemmArgs {
    const int8_t* xq;         // [R, K]
    const float* xs;          // [R]
    const int8_t* wq;         // [N, K]
    const float* ws;          // [N]
    int R, N, K;
    void* y;                  // [R] rows of N, ldy elements apart
    int64_t ldy;
    int ydtype;
    uint32_t* status;
    int y_vec;                // rows of y begin on 32 bytes
    int width;                // rows of B in a tile: 256, 128 or 64
    uint64_t wait_ns;         // limit of a wait of the tiles (0: the built-in limit)
};
// Few rows or little work: k_i8_rows, which needs no workspace.
bool i8_rows_applies(int R, int N, int K);
cudaError_t launch_i8_rows(const I8GemmArgs&, cudaStream_t);
// Else k_i8_widen and k_i8_tiles.  The operand with fewer rows (B) is widened to fp16 ahead, in
// `wide`, the other one (A) as it is read.
inline bool i8_swapped(int R, int N) { return N < R; }   // A: x, B: W; else A: W, B: x
int i8_width(int R, int N, int K);   // rows of B in a tile
// a: codes of A in boxes of 128 x 128, b: `wide` in 64 x width / 2, both with the 128-byte swizzle;
// clusters: CTA pairs resident at once.
cudaError_t i8_tiles_set_attributes(int num_sms, int* clusters);
cudaError_t launch_i8_tiles(const I8GemmArgs&, const CUtensorMap& a, const CUtensorMap& b, void* wide, int num_sms,
                            int clusters, cudaStream_t);
// The maps of A [M, K] and B [C, K] (implemented in api.cu).
bool encode_i8_tiles(CUtensorMap* a, CUtensorMap* b, const void* codes, const void* wide, int M, int C, int K, int width);

// An int32 sum of K products of codes stays in range (128 * 128 * K < 2^31).
constexpr int kI8MaxK = (1 << 17) - 16;

}  // namespace moe
