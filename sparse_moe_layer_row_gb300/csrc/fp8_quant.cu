// moe_fp8_quantize: rows -> e4m3 codes and one fp32 scale per block of 128
// along the row (the value rule is in fp8.cuh).
//
// Reads each input once and writes each code and scale once; bound by HBM.  A
// half-warp takes one (row, block of 128): eight values per lane, the largest
// magnitude by four xor steps, eight codes per lane as one 8-byte store; four
// blocks are loaded before the first is used.
#include "fp8.cuh"
#include "scatter_dev.cuh"

namespace moe {

namespace {

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }

// Eight values of a block of 128 that 16 lanes hold: codes (two per word) and the
// block's a.  The quotient (7/8 v) / (a / 512) by Markstein's method (IBM J. Res. Dev. 34,
// 1990): with r the correctly rounded reciprocal of d, q0 = n r and q0 + (n - q0 d) r is
// the correctly rounded n / d (where it is no subnormal, and those have the code 0).
// Infinities and NaN, where n - q0 d is NaN, take the division itself.
__device__ __forceinline__ float block_codes(const float (&v)[8], uint32_t (&q)[4]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float am = __uint_as_float(fp8_amax_bits(m));
    const float d = am * (1.0f / 512.0f);
    float w[8];
    if (m < 0x7F800000u) {
        const float r = __frcp_rn(d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float n = 0.875f * v[i], q0 = n * r;
            w[i] = __fmaf_rn(__fmaf_rn(-q0, d, n), r, q0);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __fdiv_rn(0.875f * v[i], d);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = fp8_pair(w[2 * i], w[2 * i + 1]);
    return am;
}

// The (row, block) tasks first, first + step, ... of this half-warp.  VEC: x rows are
// 16-byte aligned and K is a multiple of 8.
template <typename T, bool VEC>
__device__ __forceinline__ void quantize_tasks(const Fp8QuantArgs& a, int64_t first, int64_t step) {
    constexpr int kFlight = VEC && sizeof(T) == 2 ? 4 : 2;   // blocks loaded before the first is used
    const int kb = fp8_blocks(a.K);
    const int hl = threadIdx.x & 15;   // lane of the half-warp
    const int64_t ntasks = (int64_t)a.R * kb;
    // both half-warps of a warp run the same number of rounds (the shuffles are warp-wide)
    for (int64_t t0 = first & ~(int64_t)1; t0 < ntasks; t0 += kFlight * step) {
        float v[kFlight][8];
        int row[kFlight], col[kFlight];
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            const int64_t t = t0 + f * step + (first & 1);
            const bool on = t < ntasks;
            row[f] = on ? (int)((uint64_t)t < 0x80000000u ? (uint32_t)t / (uint32_t)kb : t / kb) : -1;
            const int c0 = on ? (int)(t - (int64_t)row[f] * kb) * kFp8Block + hl * 8 : 0;
            col[f] = c0;
            const T* src = static_cast<const T*>(a.x) + (int64_t)max(row[f], 0) * a.ld + c0;
            if (VEC) {
                constexpr int kWords = (int)sizeof(T) * 8 / 16;   // 16-byte loads of eight values
                uint4 w[kWords];
                const bool in = on && c0 < a.K;   // K is a multiple of 8: all eight or none
#pragma unroll
                for (int i = 0; i < kWords; ++i)
                    w[i] = in ? __ldg(reinterpret_cast<const uint4*>(src) + i) : make_uint4(0, 0, 0, 0);
                const T* e = reinterpret_cast<const T*>(w);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[f][i] = to_f32(e[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[f][i] = on && c0 + i < a.K ? to_f32(src[i]) : 0.0f;
            }
        }
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            uint32_t q[4];
            const float am = block_codes(v[f], q);
            if (row[f] < 0) continue;
            const int c0 = col[f];
            uint8_t* dst = a.codes + (int64_t)row[f] * a.K + c0;
            if (VEC) {
                if (c0 < a.K)
                    *reinterpret_cast<uint2*>(dst) = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c0 + i < a.K) dst[i] = (uint8_t)(q[i >> 1] >> (8 * (i & 1)));
            }
            if (hl == 0) a.scales[(int64_t)(c0 / kFp8Block) * a.R + row[f]] = __fdiv_rn(am, 448.0f);
        }
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) k_fp8_quantize(Fp8QuantArgs a) {
    pdl_wait();  // see common.cuh: nothing global is touched before
    pdl_trigger();
    quantize_tasks<T, VEC>(a, (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4), (int64_t)gridDim.x * 16);
}

// The front of an e4m3 plan's forward: the first step of the scatter (all of it for few
// rows) in the first CTAs, the quantising of x in the others, so that neither waits
// for the other.
__global__ void __launch_bounds__(kSmallThreads) k_fp8_front_small(ScatterArgs s, Fp8QuantArgs a) {
    pdl_wait();
    pdl_trigger();
    __shared__ ScatterSmallSmem sm;
    if (blockIdx.x == 0) {
        scatter_small(s, sm);
    } else {
        constexpr int kHalves = kSmallThreads / 16;
        quantize_tasks<__nv_bfloat16, true>(a, (int64_t)(blockIdx.x - 1) * kHalves + (threadIdx.x >> 4),
                                            (int64_t)(gridDim.x - 1) * kHalves);
    }
}
__global__ void __launch_bounds__(kScatThreads) k_fp8_front_hist(ScatterArgs s, Fp8QuantArgs a) {
    pdl_wait();
    pdl_trigger();
    if ((int)blockIdx.x < s.nb) {
        scatter_hist(s, blockIdx.x);
    } else {
        constexpr int kHalves = kScatThreads / 16;
        quantize_tasks<__nv_bfloat16, true>(a, (int64_t)((int)blockIdx.x - s.nb) * kHalves + (threadIdx.x >> 4),
                                            (int64_t)((int)gridDim.x - s.nb) * kHalves);
    }
}

template <typename T>
cudaError_t launch(const Fp8QuantArgs& a, int num_sms, cudaStream_t st) {
    const bool vec = a.K % 8 == 0 && a.ld * (int64_t)sizeof(T) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(a.x) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(a.codes) % 8 == 0;
    // few tasks: one per half-warp; many: the SMs' share, several in flight each
    int64_t blocks = ((int64_t)a.R * fp8_blocks(a.K) + 15) / 16;
    if (blocks > (int64_t)num_sms * 8) blocks = (int64_t)num_sms * 8;
    return vec ? launch_kernel(k_fp8_quantize<T, true>, dim3((unsigned)blocks), dim3(256), 0, st, a)
               : launch_kernel(k_fp8_quantize<T, false>, dim3((unsigned)blocks), dim3(256), 0, st, a);
}

}  // namespace

cudaError_t launch_fp8_front(const ScatterArgs& s, const Fp8QuantArgs& a, bool small, int num_sms,
                             cudaStream_t st) {
    const int64_t halves = (int64_t)a.R * fp8_blocks(a.K);
    if (small) {
        int64_t blocks = (halves + kSmallThreads / 16 - 1) / (kSmallThreads / 16);
        if (blocks > num_sms) blocks = num_sms;
        return launch_kernel(k_fp8_front_small, dim3((unsigned)(1 + blocks)), dim3(kSmallThreads), 0, st, s, a);
    }
    int64_t blocks = (halves + kScatThreads / 16 - 1) / (kScatThreads / 16);
    if (blocks > (int64_t)num_sms * 6) blocks = (int64_t)num_sms * 6;
    cudaError_t e = launch_kernel(k_fp8_front_hist, dim3((unsigned)(s.nb + blocks)), dim3(kScatThreads), 0, st, s, a);
    return e == cudaSuccess ? launch_scatter_rest(s, st) : e;
}

cudaError_t launch_fp8_quantize(const Fp8QuantArgs& a, int dtype, int num_sms, cudaStream_t st) {
    if (dtype == MOE_BF16) return launch<__nv_bfloat16>(a, num_sms, st);
    if (dtype == MOE_F16) return launch<__half>(a, num_sms, st);
    return launch<float>(a, num_sms, st);
}

}  // namespace moe
