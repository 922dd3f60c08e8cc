// moe_fp8_quantize: rows -> e4m3 codes and one fp32 scale per block of 128
// along the row (the value rule is in fp8.cuh).
//
// Reads each input once and writes each code and scale once.  8192 x 2048 bf16 takes
// 12.2 us (4.2 TB/s; 7.6 us at the measured copy rate).  No unit is at its limit (0.67
// issues per clock, 41% of the warps, 26% of HBM): each warp waits for its loads, and
// 65,536 tasks over 9728 warps are 6.7 each, taken four at a time, so that the second
// round is partly empty.  A warp takes two blocks of 128 of a row, one per half-warp:
// eight values per lane, the largest magnitude by four xor steps, eight codes per lane
// as one 8-byte store.
// Four such tasks are loaded before the first is used, and the arithmetic is kept
// small (16-bit maxima of the raw words, packed fp32, no index division): at 207
// instructions per task the same rows took 17.3 us.
#include "fp8.cuh"
#include "scatter_dev.cuh"

namespace moe {

namespace {

// The largest magnitude of a lane's eight values, as fp32 bits (NaN above infinity above
// every number): for 16-bit types by 16-bit integer maxima of the raw words.
__device__ __forceinline__ uint32_t amax_words(const uint4& w) {
    const uint32_t k = 0x7FFF7FFFu;
    const uint32_t m = __vmaxu2(__vmaxu2(w.x & k, w.y & k), __vmaxu2(w.z & k, w.w & k));
    return max(m & 0xFFFFu, m >> 16);
}
__device__ __forceinline__ uint32_t f32_bits(uint32_t b, __nv_bfloat16) { return b << 16; }
__device__ __forceinline__ uint32_t f32_bits(uint32_t b, __half) {
    const __half h = __ushort_as_half((unsigned short)b);
    return __float_as_uint(__half2float(h)) & 0x7FFFFFFFu;   // a NaN stays one
}

// Codes of a lane's eight values of a block (two words) and the block's scale; m: the
// lane's largest magnitude as fp32 bits.  16 lanes hold the block.
__device__ __forceinline__ float block_codes(const float2 (&v)[4], uint32_t m, uint32_t (&q)[2]) {
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float am = __uint_as_float(fp8_amax_bits(m));
    const float d = am * (1.0f / 512.0f);
    float2 w[4];
    float scale;
    if (m < 0x7F800000u) {
        const float r = __frcp_rn(d), r448 = 1.0f / 448.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = quotient2(mul2(v[i], 0.875f), d, r);
        scale = am * r448;
        scale = __fmaf_rn(__fmaf_rn(-scale, 448.0f, am), r448, scale);
    } else {   // an infinity or a NaN, for which n - q0 d is NaN
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = make_float2(__fdiv_rn(0.875f * v[i].x, d), __fdiv_rn(0.875f * v[i].y, d));
        scale = __fdiv_rn(am, 448.0f);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
        q[i] = fp8_pair(w[2 * i].x, w[2 * i].y) | fp8_pair(w[2 * i + 1].x, w[2 * i + 1].y) << 16;
    return scale;
}

// The warp's tasks first, first + step, ...: a row's blocks 2 p and 2 p + 1, a block per
// half-warp.  VEC: x rows are 16-byte aligned and K is a multiple of 8.
template <typename T, bool VEC>
__device__ __forceinline__ void quantize_tasks(const Fp8QuantArgs& a, int first, int step) {
    constexpr bool kWords = VEC && sizeof(T) == 2;
    constexpr int kFlight = kWords ? 4 : 2;   // tasks loaded before the first is used
    const int kb = fp8_blocks(a.K), kp = (kb + 1) >> 1;
    const int hl = threadIdx.x & 15, half = (threadIdx.x >> 4) & 1;
    // (row, p) of a task, advanced without division
    int row = first / kp, p = first - row * kp;
    const int drow = step / kp, dp = step - drow * kp;
    while (row < a.R) {
        uint4 raw[kFlight];
        float2 v[kFlight][4];
        int rows[kFlight], ps[kFlight];
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            rows[f] = row;
            ps[f] = p;
            const int c0 = (2 * p + half) * kFp8Block + hl * 8;
            const bool on = row < a.R && c0 < a.K;
            const T* src = static_cast<const T*>(a.x) + (int64_t)row * a.ld + c0;
            if (kWords) {
                raw[f] = on ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
            } else {
                float e[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) e[i] = 0.0f;
                if (VEC) {   // fp32
                    if (on) {
                        const float4 lo = __ldg(reinterpret_cast<const float4*>(src));
                        const float4 hi = __ldg(reinterpret_cast<const float4*>(src) + 1);
                        e[0] = lo.x; e[1] = lo.y; e[2] = lo.z; e[3] = lo.w;
                        e[4] = hi.x; e[5] = hi.y; e[6] = hi.z; e[7] = hi.w;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (row < a.R && c0 + i < a.K) e[i] = to_f32(src[i]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) v[f][i] = make_float2(e[2 * i], e[2 * i + 1]);
            }
            row += drow;
            p += dp;
            if (p >= kp) { p -= kp; ++row; }
        }
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            uint32_t m = 0, q[2];
            if constexpr (kWords) {
                m = f32_bits(amax_words(raw[f]), T());
                const T* e = reinterpret_cast<const T*>(&raw[f]);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[f][i] = make_float2(to_f32(e[2 * i]), to_f32(e[2 * i + 1]));
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    m = max(m, max(__float_as_uint(v[f][i].x) & 0x7FFFFFFFu, __float_as_uint(v[f][i].y) & 0x7FFFFFFFu));
            }
            const float scale = block_codes(v[f], m, q);
            const int b = 2 * ps[f] + half, c0 = b * kFp8Block + hl * 8;
            if (rows[f] >= a.R || b >= kb) continue;
            uint8_t* dst = a.codes + (int64_t)rows[f] * a.K + c0;
            if (VEC) {
                if (c0 < a.K) *reinterpret_cast<uint2*>(dst) = make_uint2(q[0], q[1]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c0 + i < a.K) dst[i] = (uint8_t)(q[i >> 2] >> (8 * (i & 3)));
            }
            if (hl == 0) a.scales[(int64_t)b * a.R + rows[f]] = scale;
        }
        __syncwarp();
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) k_fp8_quantize(Fp8QuantArgs a) {
    pdl_wait();  // see common.cuh: nothing global is touched before
    pdl_trigger();
    quantize_tasks<T, VEC>(a, blockIdx.x * 8 + (threadIdx.x >> 5), gridDim.x * 8);
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
        constexpr int kWarps = kSmallThreads / 32;
        quantize_tasks<__nv_bfloat16, true>(a, (blockIdx.x - 1) * kWarps + (threadIdx.x >> 5), (gridDim.x - 1) * kWarps);
    }
}
__global__ void __launch_bounds__(kScatThreads) k_fp8_front_hist(ScatterArgs s, Fp8QuantArgs a) {
    pdl_wait();
    pdl_trigger();
    if ((int)blockIdx.x < s.nb) {
        scatter_hist(s, blockIdx.x);
    } else {
        constexpr int kWarps = kScatThreads / 32;
        quantize_tasks<__nv_bfloat16, true>(a, (blockIdx.x - s.nb) * kWarps + (threadIdx.x >> 5),
                                            (gridDim.x - s.nb) * kWarps);
    }
}

template <typename T>
cudaError_t launch(const Fp8QuantArgs& a, int num_sms, cudaStream_t st) {
    const bool vec = a.K % 8 == 0 && a.ld * (int64_t)sizeof(T) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(a.x) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(a.codes) % 8 == 0;
    // few tasks: one per warp; many: the SMs' share, several in flight each
    int64_t blocks = ((int64_t)a.R * ((fp8_blocks(a.K) + 1) / 2) + 7) / 8;
    if (blocks > (int64_t)num_sms * 8) blocks = (int64_t)num_sms * 8;
    return vec ? launch_kernel(k_fp8_quantize<T, true>, dim3((unsigned)blocks), dim3(256), 0, st, a)
               : launch_kernel(k_fp8_quantize<T, false>, dim3((unsigned)blocks), dim3(256), 0, st, a);
}

}  // namespace

cudaError_t launch_fp8_front(const ScatterArgs& s, const Fp8QuantArgs& a, bool small, int num_sms,
                             cudaStream_t st) {
    const int64_t tasks = (int64_t)a.R * ((fp8_blocks(a.K) + 1) / 2);
    if (small) {
        int64_t blocks = (tasks + kSmallThreads / 32 - 1) / (kSmallThreads / 32);
        if (blocks > num_sms) blocks = num_sms;
        return launch_kernel(k_fp8_front_small, dim3((unsigned)(1 + blocks)), dim3(kSmallThreads), 0, st, s, a);
    }
    int64_t blocks = (tasks + kScatThreads / 32 - 1) / (kScatThreads / 32);
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
