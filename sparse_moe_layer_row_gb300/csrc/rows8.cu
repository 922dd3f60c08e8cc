// moe_add_rmsnorm and moe_i8_quantize: what is done to each row of activations
// before a product.
//
//   norm      r = x + residual, rounded to the residual's type and stored;
//             p = r w;  rstd = 1 / sqrt(sum r^2 / H + eps);  y = p rstd
//   e4m3      per block of 128: a = max |p|, code of 448 p / a, scale a rstd / 448
//   int8      per row: a = max |p|, code of 127 p / a, scale a rstd / 127
//   quantise  int8 without the norm: p = x, rstd = 1
//
// rstd cancels in the quotients, so codes do not depend on the sum of squares: they
// are those of the stored r, formed as fp8.cuh says (int8: (127/128 p) / (a / 128),
// which neither overflows nor, for 16-bit p, rounds across a middle).
//
// Each value is read once and each result written once.  A row lies in the registers
// of one CTA (one warp for short rows), eight consecutive values per thread and
// vector, so that a block of 128 is a half-warp's vector; the sum of squares and the
// row's largest |p| are combined in one exchange.  Rows beyond 32,768 values are read twice.
// Sums are fp32: 8 NV squares per thread, then a tree.  A row whose sum of squares
// overflows is scaled by 2^-80 and summed again.
#include "rows8.cuh"

namespace moe {

namespace {

constexpr float kTiny = 1.0f / (1 << 20) / (1 << 20) / (1 << 20) / (1 << 20);   // 2^-80

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Eight consecutive values: 16-byte accesses, or one at a time up to `n`.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, int n, float (&v)[8]) {
    if (VEC) {
        if (sizeof(T) == 4) {
            const float4 lo = *reinterpret_cast<const float4*>(p), hi = *(reinterpret_cast<const float4*>(p) + 1);
            v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
            v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
        } else {
            const uint4 w = *reinterpret_cast<const uint4*>(p);
            const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = to_f32(e[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f32(p[i]) : 0.0f;
    }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, int n, const float (&v)[8]) {
    if (VEC) {
        if (sizeof(T) == 4) {
            *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
            *(reinterpret_cast<float4*>(p) + 1) = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            uint4 w;
            T* e = reinterpret_cast<T*>(&w);
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = from_f32<T>(v[i]);
            *reinterpret_cast<uint4*>(p) = w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = from_f32<T>(v[i]);
    }
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// int8 codes of eight values whose row's largest magnitude has the bits m.
__device__ __forceinline__ uint2 i8_codes(const float (&p)[8], uint32_t m) {
    const float d = __uint_as_float(m) * (1.0f / 128.0f);
    int q[8];
    if (m < 0x7F800000u) {
        const float r = __frcp_rn(d);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 w = quotient2(mul2(make_float2(p[2 * i], p[2 * i + 1]), 127.0f / 128.0f), d, r);
            // |w| <= 127 and 1.5 * 2^23: the sum is rounded to an integer, which is its low byte
            q[2 * i] = __float_as_int(w.x + 12582912.0f);
            q[2 * i + 1] = __float_as_int(w.y + 12582912.0f);
        }
    } else {   // an infinity or a NaN: codes 0, so that code times scale is NaN
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = 0;
    }
    uint2 o;
    o.x = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
    o.y = __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410);
    return o;
}
// e4m3 codes of eight values whose block's largest magnitude has the bits m.
__device__ __forceinline__ uint2 e4m3_codes(const float (&p)[8], uint32_t m) {
    const float d = __uint_as_float(m) * (1.0f / 512.0f);
    float2 w[4];
    if (m < 0x7F800000u) {
        const float r = __frcp_rn(d);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = quotient2(mul2(make_float2(p[2 * i], p[2 * i + 1]), 0.875f), d, r);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = make_float2(__fdiv_rn(0.875f * p[2 * i], d), __fdiv_rn(0.875f * p[2 * i + 1], d));
    }
    return make_uint2(fp8_pair(w[0].x, w[0].y) | fp8_pair(w[1].x, w[1].y) << 16,
                      fp8_pair(w[2].x, w[2].y) | fp8_pair(w[3].x, w[3].y) << 16);
}

// The row's sum of squares and largest magnitude over the threads that hold it (`warps`
// warps: the whole CTA, or one warp of several rows'), the same in each of them.
__device__ __forceinline__ void combine_row(float& ss, uint32_t& m, int warps) {
    __shared__ float s_ss[32];
    __shared__ uint32_t s_m[32];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    if (warps == 1) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();   // an earlier exchange has been read
    if (lane == 0) { s_ss[warp] = ss; s_m[warp] = m; }
    __syncthreads();
    ss = lane < warps ? s_ss[lane] : 0.0f;
    m = lane < warps ? s_m[lane] : 0u;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
}

}  // namespace

// A row per `warps` warps; a CTA has several rows only where that is one.  NV vectors of
// eight values per thread; ONE: they hold the row, else it is gone through twice.
template <int WHAT, typename T, bool VEC, int NV, bool ONE>
__global__ void __launch_bounds__(1024) k_rows8(RmsNormArgs a, int warps) {
    pdl_wait();  // see common.cuh: nothing global is touched before
    pdl_trigger();
    constexpr bool kNorm = WHAT != kQuantI8, kRowMax = WHAT == kNormI8 || WHAT == kQuantI8;
    const int lane = threadIdx.x & 31;
    const int t = warps == 1 ? lane : threadIdx.x;
    const int step = 256 * warps;   // values per vector of the row's threads
    const int64_t row = warps == 1 ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= a.R) return;   // whole warps, and no CTA-wide barrier where warps == 1
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;

    // r of the eight values from c on; `stored`: the sum has been written
    auto load_r = [&](int c, bool stored, float (&r)[8]) {
        const int n = a.H - c;
        if (n <= 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) r[i] = 0.0f;
            return;
        }
        if (kNorm && stored && a.residual && a.total) {
            if (a.res_f32) load8<float, VEC>(static_cast<const float*>(a.total) + row * a.ldt + c, n, r);
            else load8<T, VEC>(static_cast<const T*>(a.total) + row * a.ldt + c, n, r);
            return;
        }
        load8<T, VEC>(x + c, n, r);
        if (!kNorm || !a.residual) return;
        float b[8];
        if (a.res_f32) load8<float, VEC>(static_cast<const float*>(a.residual) + row * a.ldr + c, n, b);
        else load8<T, VEC>(static_cast<const T*>(a.residual) + row * a.ldr + c, n, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            r[i] += b[i];
            if (!a.res_f32) r[i] = to_f32(from_f32<T>(r[i]));
        }
    };
    auto store_total = [&](int c, const float (&r)[8]) {
        const int n = a.H - c;
        if (!kNorm || !a.total || n <= 0) return;
        if (a.res_f32) store8<float, VEC>(static_cast<float*>(a.total) + row * a.ldt + c, n, r);
        else store8<T, VEC>(static_cast<T*>(a.total) + row * a.ldt + c, n, r);
    };
    auto times_w = [&](int c, float (&p)[8]) {
        const int n = a.H - c;
        if (!kNorm || !a.w || n <= 0) return;
        float w[8];
        if (a.w_f32) load8<float, VEC>(static_cast<const float*>(a.w) + c, n, w);
        else load8<T, VEC>(static_cast<const T*>(a.w) + c, n, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] *= w[i];
    };
    auto add_in = [&](int c, const float (&r)[8], float f, float& ss, uint32_t& m) {
        float p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            p[i] = r[i] * f;
            if (kNorm) ss = fmaf(p[i], p[i], ss);
        }
        if (kRowMax) {
            times_w(c, p);
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, magnitude(p[i]));
        }
    };

    float r[NV][8], ss = 0.0f;
    uint32_t m = 0;
    for (int c0 = 0; c0 < a.H; c0 += NV * step) {
#pragma unroll
        for (int v = 0; v < NV; ++v) load_r(c0 + v * step + 8 * t, false, r[v]);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = c0 + v * step + 8 * t;
            store_total(c, r[v]);
            add_in(c, r[v], 1.0f, ss, m);
        }
        if (ONE) break;
    }
    combine_row(ss, m, warps);
    float f = 1.0f;
    if (kNorm && !(ss < INFINITY)) {   // beyond fp32's range, or not finite at all; the same in each thread
        f = kTiny;
        ss = 0.0f;
        m = 0;
        for (int c0 = 0; c0 < a.H; c0 += NV * step)
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = c0 + v * step + 8 * t;
                if (!ONE) load_r(c, true, r[v]);
                add_in(c, r[v], f, ss, m);
            }
        combine_row(ss, m, warps);
    }
    const float rstd = kNorm ? __frcp_rn(__fsqrt_rn(__fdiv_rn(ss, (float)a.H) + (f == 1.0f ? a.eps : 0.0f))) : 1.0f;
    if (kRowMax) {
        m = fp8_amax_bits(m);
        if (t == 0) a.scales[row] = __fdiv_rn(kNorm ? __uint_as_float(m) * rstd : __uint_as_float(m), 127.0f);
    }
    for (int c0 = 0; c0 < a.H; c0 += NV * step) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = c0 + v * step + 8 * t, n = a.H - c;
            if (!ONE) load_r(c, true, r[v]);
            float p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = kNorm ? r[v][i] * f : r[v][i];
            times_w(c, p);
            uint2 q = make_uint2(0, 0);
            if (WHAT == kNormE4m3) {   // every lane takes part in the block's maximum
                uint32_t bm = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) bm = max(bm, magnitude(p[i]));
#pragma unroll
                for (int o = 8; o >= 1; o >>= 1) bm = max(bm, __shfl_xor_sync(0xffffffffu, bm, o));
                bm = fp8_amax_bits(bm);
                q = e4m3_codes(p, bm);
                if ((lane & 15) == 0 && n > 0)
                    a.scales[(int64_t)(c / kFp8Block) * a.R + row] = __fdiv_rn(__uint_as_float(bm) * rstd, 448.0f);
            }
            if (kRowMax) q = i8_codes(p, m);
            if (n <= 0) continue;
            if (WHAT != kNormOnly) {
                uint8_t* dst = a.codes + row * a.H + c;
                if (VEC) {
                    *reinterpret_cast<uint2*>(dst) = q;
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (i < n) dst[i] = (uint8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
                }
            }
            if (kNorm && (WHAT == kNormOnly || a.y)) {
#pragma unroll
                for (int i = 0; i < 8; ++i) p[i] *= rstd;
                store8<T, VEC>(static_cast<T*>(a.y) + row * a.ldy + c, n, p);
            }
        }
        if (ONE) break;
    }
}

namespace {

bool rows_aligned(const void* p, int64_t ld, size_t size, int64_t R) {
    return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (R <= 1 || ld * (int64_t)size % 16 == 0));
}

template <int WHAT, typename T, bool VEC, int NV, bool ONE>
cudaError_t launch_as(const RmsNormArgs& a, int warps, cudaStream_t st) {
    const int rows = warps == 1 ? 4 : 1;   // per CTA
    return launch_kernel(k_rows8<WHAT, T, VEC, NV, ONE>, dim3((unsigned)(((int64_t)a.R + rows - 1) / rows)),
                         dim3(32 * warps * rows), 0, st, a, warps);
}

template <int WHAT, typename T>
cudaError_t launch_t(const RmsNormArgs& a, int num_sms, cudaStream_t st) {
    const size_t rs = a.res_f32 ? 4 : sizeof(T), es = sizeof(T);
    const bool vec = a.H % 8 == 0 && rows_aligned(a.x, a.ldx, es, a.R) && rows_aligned(a.residual, a.ldr, rs, a.R) &&
                     rows_aligned(a.total, a.ldt, rs, a.R) && rows_aligned(a.y, a.ldy, es, a.R) &&
                     reinterpret_cast<uintptr_t>(a.w) % 16 == 0 && reinterpret_cast<uintptr_t>(a.codes) % 8 == 0;
    const int per_warp = (a.H + 255) / 256;   // vectors that one warp would hold
    auto warps = [&](int nv) { return (per_warp + nv - 1) / nv; };
    if (warps(4) > 32) return vec ? launch_as<WHAT, T, true, 4, false>(a, 32, st) : launch_as<WHAT, T, false, 4, false>(a, 32, st);
    if (!vec) return launch_as<WHAT, T, false, 4, true>(a, warps(4), st);
    // few rows: a row over many threads, for the latency
    if (a.R <= 4 * num_sms && warps(1) <= 32) return launch_as<WHAT, T, true, 1, true>(a, warps(1), st);
    if (warps(2) <= 32) return launch_as<WHAT, T, true, 2, true>(a, warps(2), st);
    return launch_as<WHAT, T, true, 4, true>(a, warps(4), st);
}

template <typename T>
cudaError_t launch_what(int what, const RmsNormArgs& a, int num_sms, cudaStream_t st) {
    switch (what) {
        case kNormOnly: return launch_t<kNormOnly, T>(a, num_sms, st);
        case kNormE4m3: return launch_t<kNormE4m3, T>(a, num_sms, st);
        case kNormI8: return launch_t<kNormI8, T>(a, num_sms, st);
        default: return launch_t<kQuantI8, T>(a, num_sms, st);
    }
}

}  // namespace

cudaError_t launch_rows8(int what, const RmsNormArgs& a, int dtype, int num_sms, cudaStream_t st) {
    if (dtype == MOE_BF16) return launch_what<__nv_bfloat16>(what, a, num_sms, st);
    if (dtype == MOE_F16) return launch_what<__half>(what, a, num_sms, st);
    return launch_what<float>(what, a, num_sms, st);
}

}  // namespace moe
