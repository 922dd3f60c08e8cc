// moe_fp8_quantize: rows -> e4m3 codes and one fp32 scale per block of 128
// along the row (the value rule is in fp8.cuh).
//
// Reads each input once and writes each code and scale once; bound by HBM.  A
// half-warp takes one (row, block of 128): eight values per lane, the largest
// magnitude by four xor steps, eight codes per lane as one 8-byte store.
#include "fp8.cuh"

namespace moe {

namespace {

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }

// VEC: x rows are 16-byte aligned and K is a multiple of 8.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) k_fp8_quantize(Fp8QuantArgs a) {
    pdl_wait();  // see common.cuh: nothing global is touched before
    pdl_trigger();
    const int kb = fp8_blocks(a.K);
    const int hl = threadIdx.x & 15;   // lane of the half-warp
    const int64_t ntasks = (int64_t)a.R * kb;
    const int64_t step = (int64_t)gridDim.x * (blockDim.x / 16);
    // both half-warps of a warp run the same number of rounds (the shuffles are warp-wide)
    const int64_t first = (int64_t)blockIdx.x * (blockDim.x / 16) + (threadIdx.x >> 4);
    const int64_t warp_first = first & ~(int64_t)1;
    for (int64_t t0 = warp_first; t0 < ntasks; t0 += step) {
        const int64_t t = t0 + (first & 1);
        const bool on = t < ntasks;
        const int r = on ? (int)(t / kb) : 0;
        const int b = on ? (int)(t - (int64_t)r * kb) : 0;
        const int c0 = b * kFp8Block + hl * 8;
        const T* src = static_cast<const T*>(a.x) + (int64_t)r * a.ld + c0;
        float v[8];
        if (VEC) {
            constexpr int kWords = (int)sizeof(T) * 8 / 16;   // 16-byte loads of eight values
            uint4 w[kWords];
            const bool in = on && c0 < a.K;   // K is a multiple of 8: all eight or none
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                w[i] = in ? __ldg(reinterpret_cast<const uint4*>(src) + i) : make_uint4(0, 0, 0, 0);
            const T* e = reinterpret_cast<const T*>(w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = to_f32(e[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = on && c0 + i < a.K ? to_f32(src[i]) : 0.0f;
        }
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float am = __uint_as_float(fp8_amax_bits(m));
        const float d = am * (1.0f / 512.0f);
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            q[i] = fp8_pair(__fdiv_rn(0.875f * v[2 * i], d), __fdiv_rn(0.875f * v[2 * i + 1], d));
        if (!on) continue;
        uint8_t* dst = a.codes + (int64_t)r * a.K + c0;
        if (VEC) {
            if (c0 < a.K)
                *reinterpret_cast<uint2*>(dst) = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c0 + i < a.K) dst[i] = (uint8_t)(q[i >> 1] >> (8 * (i & 1)));
        }
        if (hl == 0) a.scales[(int64_t)b * a.R + r] = __fdiv_rn(am, 448.0f);
    }
}

template <typename T>
cudaError_t launch(const Fp8QuantArgs& a, int num_sms, cudaStream_t st) {
    const bool vec = a.K % 8 == 0 && a.ld * (int64_t)sizeof(T) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(a.x) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(a.codes) % 8 == 0;
    int64_t blocks = ((int64_t)a.R * fp8_blocks(a.K) + 15) / 16;
    if (blocks > (int64_t)num_sms * 32) blocks = (int64_t)num_sms * 32;
    return vec ? launch_kernel(k_fp8_quantize<T, true>, dim3((unsigned)blocks), dim3(256), 0, st, a)
               : launch_kernel(k_fp8_quantize<T, false>, dim3((unsigned)blocks), dim3(256), 0, st, a);
}

}  // namespace

cudaError_t launch_fp8_quantize(const Fp8QuantArgs& a, int dtype, int num_sms, cudaStream_t st) {
    if (dtype == MOE_BF16) return launch<__nv_bfloat16>(a, num_sms, st);
    if (dtype == MOE_F16) return launch<__half>(a, num_sms, st);
    return launch<float>(a, num_sms, st);
}

}  // namespace moe
