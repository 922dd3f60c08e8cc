// moe_fp8_gemm for few rows or little work: y = x W^T on e4m3 codes where the
// 128 x 256 tiles of fp8_gemm.cu would leave most SMs without a unit.
//
// A CTA takes 16 outputs and 32 rows, and its eight warps share K: warp w takes
// the blocks of 128 w, w + 8, ...  The weights are the M of mma.sync m16n8k32, the rows
// its N; operands go from global memory to registers, two blocks at a time,
// since nothing is used twice within a warp.  K is permuted inside a block as in
// fp8_stream.cu, so that a lane's operands are 16-byte loads.  A block's sum is
// promoted by its two scales into fp32 registers, and the warps' sums are added
// in warp order through shared memory: the same bits on every run.
// One round of loads, one round of MMAs, one exchange: the kernel is bound by
// latency up to a few MB of weights.  1 x 2048 x 2048 takes 2.2 us (0.6 at the measured
// copy rate), against 12.4 as one row of a 128-row tile.
#include "fp8.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8;
constexpr int kCols = 16, kRowsPerCta = 32;

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void store_one(void* y, int64_t i, int dtype, float v) {
    if (dtype == MOE_F32) static_cast<float*>(y)[i] = v;
    else if (dtype == MOE_BF16) static_cast<__nv_bfloat16*>(y)[i] = __float2bfloat16_rn(v);
    else static_cast<__half*>(y)[i] = __float2half_rn(v);
}

}  // namespace

// NT tiles of 8 rows per CTA
template <int NT>
__global__ void __launch_bounds__(32 * kWarps) k_fp8_rows(Fp8RowsArgs a) {
    pdl_wait();  // see common.cuh: nothing global is touched before
    pdl_trigger();
    __shared__ float part[kWarps][NT * 8][kCols + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gi = lane >> 2, c = lane & 3;
    const int n0 = blockIdx.x * kCols, r0 = blockIdx.y * kRowsPerCta;
    const int kb_n = fp8_blocks(a.K);
    // rows of W and of x past the end repeat the last: they feed outputs that are not stored
    const uint8_t* wa = a.wq + (int64_t)min(n0 + gi, a.N - 1) * a.K + 32 * c;
    const uint8_t* wb = a.wq + (int64_t)min(n0 + gi + 8, a.N - 1) * a.K + 32 * c;
    const uint8_t* xr[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) xr[t] = a.xq + (int64_t)min(r0 + 8 * t + gi, a.R - 1) * a.K + 32 * c;
    const float* sw = a.ws + (int64_t)(n0 / kFp8Block) * kb_n;   // 16 outputs lie in one block
    float acc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[t][j] = 0.0f;
    auto load = [&](const uint8_t* p, int kb, int half) {   // zeros past the row's end (K % 16 == 0)
        const int at = kb * kFp8Block + 16 * half;
        return at + 32 * c < a.K ? __ldg(reinterpret_cast<const uint4*>(p + at)) : make_uint4(0, 0, 0, 0);
    };
    for (int kb = warp; kb < kb_n; kb += 2 * kWarps) {
        // this block and the warp's next: every load first
        uint4 va[2][2], vb[2][2], vx[2][NT][2];
        float s0[2][NT], s1[2][NT], w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = kb + h * kWarps;
            const bool on = k < kb_n;
            const int kk = on ? k : kb;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                va[h][i] = on ? load(wa, kk, i) : make_uint4(0, 0, 0, 0);
                vb[h][i] = on ? load(wb, kk, i) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int t = 0; t < NT; ++t) vx[h][t][i] = on ? load(xr[t], kk, i) : make_uint4(0, 0, 0, 0);
            }
            w[h] = on ? __ldg(sw + kk) : 0.0f;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const float* sx = a.xs + (int64_t)kk * a.R + r0 + 8 * t + 2 * c;
                s0[h][t] = on && r0 + 8 * t + 2 * c < a.R ? __ldg(sx) : 0.0f;
                s1[h][t] = on && r0 + 8 * t + 2 * c + 1 < a.R ? __ldg(sx + 1) : 0.0f;
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                mma_e4m3(d, va[h][0].x, vb[h][0].x, va[h][0].y, vb[h][0].y, vx[h][t][0].x, vx[h][t][0].y);
                mma_e4m3(d, va[h][0].z, vb[h][0].z, va[h][0].w, vb[h][0].w, vx[h][t][0].z, vx[h][t][0].w);
                mma_e4m3(d, va[h][1].x, vb[h][1].x, va[h][1].y, vb[h][1].y, vx[h][t][1].x, vx[h][t][1].y);
                mma_e4m3(d, va[h][1].z, vb[h][1].z, va[h][1].w, vb[h][1].w, vx[h][t][1].z, vx[h][t][1].w);
                const float f0 = s0[h][t] * w[h], f1 = s1[h][t] * w[h];
                acc[t][0] = fmaf(f0, d[0], acc[t][0]);
                acc[t][1] = fmaf(f1, d[1], acc[t][1]);
                acc[t][2] = fmaf(f0, d[2], acc[t][2]);
                acc[t][3] = fmaf(f1, d[3], acc[t][3]);
            }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {   // D: outputs gi and gi + 8 of rows 2c and 2c + 1
        part[warp][8 * t + 2 * c][gi] = acc[t][0];
        part[warp][8 * t + 2 * c + 1][gi] = acc[t][1];
        part[warp][8 * t + 2 * c][gi + 8] = acc[t][2];
        part[warp][8 * t + 2 * c + 1][gi + 8] = acc[t][3];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < NT * 8 * kCols; i += 32 * kWarps) {
        const int r = i / kCols, n = i % kCols;
        if (r0 + r >= a.R || n0 + n >= a.N) continue;
        float v = part[0][r][n];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) v += part[w][r][n];
        store_one(a.y, (int64_t)(r0 + r) * a.ldy + n0 + n, a.ydtype, v);
    }
}

// By what the two kernels were measured to take (ns): this one 2300 + CTAs (7 + 0.006 K)
// with 17 to 32 rows per CTA, the 128 x 256 tiles 4750 + 4 K per round of one tile per
// SM.  For example (us, this kernel first) 64 x 4096 x 2048: 10.5 and 12.2; 128 x
// 4096 x 2048: 18.6 and 13.3; 256 x 1024 x 2048: 10.8 and 13.0; 512 x 2048 x 512: 23.7 and
// 6.8; 77 x 1000 x 1104: 5.5 and 9.1; 32 x 8192 x 8192: 29 and 34; 8 x 8192 x 8192: 11 and 33.
// Up to 32 rows the rows alone decide, which is right for up to 8 rows (8 x 151,936 x
// 2048: 54 and 60; x 7168: 168 and 206) and, with 9 to 32, up to some 8192 outputs (16 x
// 8192 x 2048: 7.8 and 10.5; 32 x 8192 x 2048: 11.1 and 10.6).  Beyond them the tiles
// would be faster: 16 x 32,768 x 2048: 24 and 16; 32 x 32,768 x 2048: 35 and 16; 32 x
// 151,936 x 2048: 166 and 64; 32 x 16,384 x 7168: 60 and 32.
bool fp8_rows_applies(int R, int N, int K, int num_sms) {
    if (R <= kRowsPerCta) return true;
    if (R > 65535 * kRowsPerCta) return false;   // the grid's y: row tiles
    const int64_t ctas = (int64_t)((N + kCols - 1) / kCols) * ((R + kRowsPerCta - 1) / kRowsPerCta);
    const int64_t tiles = (int64_t)((R + 127) / 128) * ((N + 255) / 256);
    const int64_t rounds = (tiles + num_sms - 1) / num_sms;
    return 2300 + ctas * (7000 + 6 * (int64_t)K) / 1000 <= rounds * (4750 + 4 * (int64_t)K);
}

cudaError_t launch_fp8_rows(const Fp8RowsArgs& a, cudaStream_t st) {
    const dim3 grid((unsigned)((a.N + kCols - 1) / kCols), (unsigned)((a.R + kRowsPerCta - 1) / kRowsPerCta));
    auto k = a.R <= 8 ? k_fp8_rows<1> : a.R <= 16 ? k_fp8_rows<2> : k_fp8_rows<4>;
    return launch_kernel(k, grid, dim3(32 * kWarps), 0, st, a);
}

}  // namespace moe
