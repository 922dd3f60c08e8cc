// moe_i8_gemm: y[r, n] = xs[r] ws[n] sum_k xq[r, k] wq[n, k] on int8 codes.
//
// k_i8_rows: a CTA takes 16 outputs and 32 rows, and its eight warps share K: warp w
// takes the blocks of 128 w, w + 8, ...  The weights are the M of mma.sync m16n8k32, the
// rows its N, the sums int32 and exact.  Operands go from global memory to registers, two
// blocks at a time; K is permuted inside a block, alike in both operands, so that a lane's
// are 16-byte loads.  The warps' sums are added through shared memory.
#include "rows8.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8;
constexpr int kCols = 16, kRowsPerCta = 32;

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                       uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
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
__global__ void __launch_bounds__(32 * kWarps) k_i8_rows(I8GemmArgs a) {
    pdl_wait();  // see common.cuh: nothing global is touched before
    pdl_trigger();
    __shared__ int part[kWarps][NT * 8][kCols + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gi = lane >> 2, c = lane & 3;
    const int r0 = blockIdx.y * kRowsPerCta;
    const int64_t n0 = (int64_t)blockIdx.x * kCols;
    const int kb_n = fp8_blocks(a.K);
    // rows of W and of x past the end repeat the last: they feed outputs that are not stored
    const int8_t* wa = a.wq + min(n0 + gi, (int64_t)a.N - 1) * a.K + 32 * c;
    const int8_t* wb = a.wq + min(n0 + gi + 8, (int64_t)a.N - 1) * a.K + 32 * c;
    const int8_t* xr[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) xr[t] = a.xq + (int64_t)min(r0 + 8 * t + gi, a.R - 1) * a.K + 32 * c;
    int acc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[t][j] = 0;
    auto load = [&](const int8_t* p, int kb, int half) {   // zeros past the row's end (K % 16 == 0)
        const int at = kb * kFp8Block + 16 * half;
        return at + 32 * c < a.K ? __ldg(reinterpret_cast<const uint4*>(p + at)) : make_uint4(0, 0, 0, 0);
    };
    for (int kb = warp; kb < kb_n; kb += 2 * kWarps) {
        // this block and the warp's next: every load first; none past the last block
        uint4 va[2][2], vb[2][2], vx[2][NT][2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int k = kb + h * kWarps;
                va[h][i] = load(wa, k, i);
                vb[h][i] = load(wb, k, i);
#pragma unroll
                for (int t = 0; t < NT; ++t) vx[h][t][i] = load(xr[t], k, i);
            }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mma_s8(acc[t], va[h][i].x, vb[h][i].x, va[h][i].y, vb[h][i].y, vx[h][t][i].x, vx[h][t][i].y);
                    mma_s8(acc[t], va[h][i].z, vb[h][i].z, va[h][i].w, vb[h][i].w, vx[h][t][i].z, vx[h][t][i].w);
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
        int v = part[0][r][n];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) v += part[w][r][n];
        store_one(a.y, (int64_t)(r0 + r) * a.ldy + n0 + n, a.ydtype,
                  (float)v * (__ldg(a.xs + r0 + r) * __ldg(a.ws + n0 + n)));
    }
}

cudaError_t launch_i8_rows(const I8GemmArgs& a, cudaStream_t st) {
    const dim3 grid((unsigned)((a.N + kCols - 1) / kCols), (unsigned)((a.R + kRowsPerCta - 1) / kRowsPerCta));
    auto k = a.R <= 8 ? k_i8_rows<1> : a.R <= 16 ? k_i8_rows<2> : k_i8_rows<4>;
    return launch_kernel(k, grid, dim3(32 * kWarps), 0, st, a);
}

}  // namespace moe
