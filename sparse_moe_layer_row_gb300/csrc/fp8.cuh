// 8-bit floating point (e4m3) with one fp32 scale per block of 128: the value
// rule shared by the quantising kernel (fp8_quant.cu) and the gate/up GEMM's
// epilogue (fp8_gemm.cu), and the argument blocks and launchers of both.
//
// A block of 128 values v with largest magnitude a = max(|v|, 2^-100) has the
// scale s = a / 448 (448: the largest e4m3 value), rounded once to fp32, and
// the codes q = e4m3(448 v / a), halves to the even code; it stands for q * s.
// 448 v / a is formed as (7/8 v) / (a / 512): both operands are exact (7/8 v
// for inputs of up to 21 significant bits, a / 512 always) and neither
// overflows, so a quotient that is exactly between two codes is seen as such.
// For 16-bit values the fp32 quotient changes no code: |448 v - m a| for a middle m is 0
// or at least 2^-16 of m a (11, 11 and 5 significant bits).  fp32 values (and h) have
// their two roundings, 2^-23 of the quotient.
// Every |v| <= a, so no code exceeds 448.  The floor 2^-100 keeps a / 512 and s
// normal numbers; a block of zeros has codes 0 and the scale 2^-100 / 448.
// Infinities and NaN: the largest magnitude is taken over the bits of |v|, in
// which infinity follows every number and NaN follows infinity.  A block with
// a NaN has a NaN scale and NaN codes; one with an infinity has an infinite
// scale, NaN codes at its infinities and 0 elsewhere.  Either way every sum
// that the block enters is NaN: a poisoned row stays visible.
#pragma once

#include <cuda_fp16.h>

#include "kernels.cuh"

namespace moe {

constexpr int kFp8Block = 128;
constexpr uint32_t kFp8AmaxMinBits = 27u << 23;   // 2^-100

// Bits of the block's a from the largest |v| bits found.
__device__ __forceinline__ uint32_t fp8_amax_bits(uint32_t m) {
    return m > kFp8AmaxMinBits ? m : kFp8AmaxMinBits;
}

// Two values already divided by the scale -> two codes (v0 in the low byte).
__device__ __forceinline__ uint32_t fp8_pair(float v0, float v1) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(v1), "f"(v0));
    return r;
}

__host__ __device__ inline int fp8_blocks(int n) { return (n + kFp8Block - 1) / kFp8Block; }

struct Fp8QuantArgs {
    const void* x;        // [R] rows of K values, ld elements apart
    int64_t ld;
    int R, K;
    uint8_t* codes;       // [R, K]
    float* scales;        // [ceil(K / 128), R]
};
cudaError_t launch_fp8_quantize(const Fp8QuantArgs&, int dtype, int num_sms, cudaStream_t);
// The scatter and the quantising of bf16 x (rows 16-byte aligned, K a multiple of 8).
cudaError_t launch_fp8_front(const ScatterArgs&, const Fp8QuantArgs&, bool small, int num_sms, cudaStream_t);

// GEMM modes (kGateUp and kDown as in kernels.cuh).
constexpr int kDense = 2;
constexpr int kFp8Rows = 128;     // rows of x (pairs) per unit: the MMA's M
constexpr int kFp8GuRows = 128;   // intermediate indices per gate/up unit
constexpr int kFp8DnCols = 256;   // hidden outputs per down unit

struct Fp8GemmArgs {
    GemmArgs g;           // units, sizes, pair lists, staging, status (kGateUp, kDown)
    // gate/up: codes and scales of x; its output, the codes and scales of h
    const uint8_t* xq;    // [R, H]
    const float* xs;      // [H / 128, R]
    uint8_t* hq;          // [max_pairs, I] routed, in pair order
    float* hs;            // [ceil(I / 128), max_pairs]
    uint8_t* shq;         // [max_rows, Is] shared expert
    float* shs;           // [ceil(Is / 128), max_rows]
    int max_pairs, max_rows;
    // weight scales, per 128 x 128 block: [E][row blocks][K blocks]; shared without [E]
    const float *sc_a, *sc_b;           // gate, up / down, down / dense, dense
    const float *sc_sa, *sc_sb;         // the shared expert's
    // dense: y [R, N] = x W^T
    int R, N, K;
    void* y;
    int64_t ldy;
    int ydtype;
    int y_vec;            // y rows may be stored 16 bytes at a time
};
struct Fp8Maps {
    CUtensorMap w0, w1;   // routed (or dense) weights: gate, up / down, down
    CUtensorMap s0, s1;   // the shared expert's
    CUtensorMap a0, a1;   // rows: h codes of routed pairs / shared rows; dense: x codes
};
// Calls with at most kFp8StreamPairs pairs per expert on average take units of up
// to kFp8StreamRows pairs and the streaming kernels (fp8_stream.cu).  At H = 2048, I =
// 512, 8 of 256 experts, streaming against the 128-row tiles: 256 rows (8 pairs) 158
// against 181 us, 384 rows 187 against 183, 512 rows (16 pairs) 221 against 185.
// The average knows neither the shared expert's rows (1 of 256 experts: 1024 rows 175
// against 182, 2048 rows 221 against 200, 3072 rows 273 against 210; 2 of 256: 1536 rows 219
// against 199) nor how many experts a coreset leaves (8 of 256, all pairs on 32 of
// them: 128 rows 87 against 47, 384 rows 161 against 58): there the tiles would be faster.
constexpr int kFp8StreamRows = 32;
constexpr int kFp8StreamPairs = 12;
inline bool fp8_streams(int64_t rows, int E, int k) { return rows * k <= (int64_t)kFp8StreamPairs * E; }
cudaError_t fp8_stream_set_attributes();
cudaError_t launch_fp8_stream(int mode, const Fp8Maps&, const Fp8GemmArgs&, int num_sms, cudaStream_t);
cudaError_t fp8_gemm_set_attributes();
cudaError_t launch_fp8_gemm(int mode, const Fp8Maps&, const Fp8GemmArgs&, int num_sms, cudaStream_t);

// The dense product for few rows or little work (fp8_rows.cu).
struct Fp8RowsArgs {
    const uint8_t* xq;
    const float* xs;
    const uint8_t* wq;
    const float* ws;
    int R, N, K;
    void* y;
    int64_t ldy;
    int ydtype;
};
bool fp8_rows_applies(int R, int N, int K, int num_sms);
cudaError_t launch_fp8_rows(const Fp8RowsArgs&, cudaStream_t);

// The expert FFN of up to kFp8DecodeRows rows (fp8_decode.cu), for calls whose gate/up
// CTAs (kFp8DecodeSub per unit) are resident at once, two per SM: at the sizes above, 1 row
// (288 CTAs) takes 16.0 us against 20.1 streaming, 2 rows (544) 21.5 against 21.1, 4 rows
// 32 against 24.
constexpr int kFp8DecodeRows = 8, kFp8DecodeSub = 8;
inline bool fp8_decodes(int rows, int gu_units, int num_sms) {
    return rows <= kFp8DecodeRows && gu_units * kFp8DecodeSub <= 2 * num_sms;
}
struct Fp8DecodeArgs {
    Fp8GemmArgs f;        // units, sizes, pair lists, x codes, scales, staging
    // weights: gate, up / down, down; the shared expert's
    const uint8_t *w_a, *w_b, *w_sa, *w_sb;
    float* h32;           // [pairs, I] h before it is quantised
    float* sh32;          // [rows, Is]
};
// units: a bound on the number in the unit list
cudaError_t launch_fp8_decode(int mode, const Fp8DecodeArgs&, int units, cudaStream_t);

// Tensor map of e4m3 codes, row-major [d2][d1][d0] (rank 2 if d2 == 0), box of
// 128 x 128 codes in the 128-byte swizzle, zeros outside (implemented in api.cu).
bool encode_fp8(CUtensorMap* m, const void* ptr, uint64_t d0, uint64_t d1, uint64_t d2);

}  // namespace moe
