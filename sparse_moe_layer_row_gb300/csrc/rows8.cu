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
// Between a row's loads and its stores lie the exchange and two passes of arithmetic, some
// 2 us in which a CTA that comes and goes with its row asks memory for nothing: CTAs stay, and
// load their next row before the exchange of this one.
// 8192 x 2048, bf16 with a residual: y 22.5 us (6.0 TB/s, floor 20.2), e4m3 20.9 (5.7, 17.7), int8
// 20.6; int8 quantising 10.0 (5.0 TB/s, floor 7.6); with an fp32 residual 31.0 (6.5 TB/s, floor 30.2);
// e4m3 without a residual 14.8 (floor 7.6).  CTAs that come and go: 29.7 (e4m3), 12.3 (quantising).
// What binds codes is latency: 24 instructions a value (quantising: 11), issued in 57% (61%) of a
// scheduler's cycles by a third of the warps that an SM holds, whose registers a row takes; HBM is
// at 43% (34%) there.  One row takes 1.7 us; 777 x 1000, fp16 with an fp32 residual and int8 codes,
// 3.3 (floor 1.3).  Rows off 16 bytes go value by value: 8192 x 1001 19 us (e4m3, floor 3.7) and 42
// (y with a residual, floor 9.9).
// Sums are fp32: 8 NV squares per thread, then a tree; rows read twice add up such pieces and keep
// what each addition drops (without, constant rows of 2^22 values were off by 1.2e-5, of 2^28 by
// 4e-4).  A row whose sum of squares overflows is read again and the squares of 2^-80 r are summed
// (huge_row); its codes are those of p all the same.
#include <type_traits>

#include "rows8.cuh"

namespace moe {

namespace {

constexpr float kTiny = 1.0f / (1 << 20) / (1 << 20) / (1 << 20) / (1 << 20);   // 2^-80
constexpr float kRoot = 1.0f / (1 << 20) / (1 << 20);                           // 2^-40

// Two values in 16 bits each.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<float>(float, float) { return 0; }   // never called

// Eight consecutive values as they lie in memory (16-bit types: lo alone).
struct Raw8 {
    uint4 lo, hi;
};
template <typename T>
__device__ __forceinline__ Raw8 load_raw(const T* p) {
    Raw8 r;
    r.lo = *reinterpret_cast<const uint4*>(p);
    r.hi = sizeof(T) == 4 ? *(reinterpret_cast<const uint4*>(p) + 1) : make_uint4(0, 0, 0, 0);
    return r;
}
template <typename T>
__device__ __forceinline__ void values(const Raw8& r, float (&v)[8]) {
    if (sizeof(T) == 4) {
        v[0] = __uint_as_float(r.lo.x); v[1] = __uint_as_float(r.lo.y);
        v[2] = __uint_as_float(r.lo.z); v[3] = __uint_as_float(r.lo.w);
        v[4] = __uint_as_float(r.hi.x); v[5] = __uint_as_float(r.hi.y);
        v[6] = __uint_as_float(r.hi.z); v[7] = __uint_as_float(r.hi.w);
    } else {
        const T* e = reinterpret_cast<const T*>(&r.lo);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f32(e[i]);
    }
}
template <typename T>
__device__ __forceinline__ Raw8 raw_of(const float (&v)[8]) {   // rounded
    Raw8 r;
    if (sizeof(T) == 4) {
        r.lo = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        r.hi = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
    } else {
        r.lo = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
        r.hi = make_uint4(0, 0, 0, 0);
    }
    return r;
}
template <typename T>
__device__ __forceinline__ void store_raw(T* p, const Raw8& r) {
    *reinterpret_cast<uint4*>(p) = r.lo;
    if (sizeof(T) == 4) *(reinterpret_cast<uint4*>(p) + 1) = r.hi;
}

// The same, one value at a time up to `n`, where addresses or H do not allow 16 bytes.
template <typename T, bool VEC>
__device__ __forceinline__ Raw8 load8(const T* p, int n) {
    if (VEC) return load_raw(p);
    Raw8 r{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    T* e = reinterpret_cast<T*>(&r);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) e[i] = p[i];
    return r;
}
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, int n, const Raw8& r) {
    if (VEC) {
        store_raw(p, r);
        return;
    }
    const T* e = reinterpret_cast<const T*>(&r);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = e[i];
}

// The largest of |a|, |b| and c >= 0 (a NaN if there is one, whose bits follow infinity's).
__device__ __forceinline__ float max_magnitude(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(c));
    return d;
}
__device__ __forceinline__ float largest(const float (&p)[8], float m) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) m = max_magnitude(p[i], p[i + 1], m);
    return m;
}

// a / m, rounded once, by Markstein's correction (fp8.cuh); r: 1 / m rounded
__device__ __forceinline__ float over(float a, float m, float r) {
    const float q = a * r;
    return a < INFINITY ? __fmaf_rn(__fmaf_rn(-q, m, a), r, q) : a;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 c, a, b;\n\tmov.b64 {%0, %1}, c;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
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
            const float2 s = add2(w, make_float2(12582912.0f, 12582912.0f));
            q[2 * i] = __float_as_int(s.x);
            q[2 * i + 1] = __float_as_int(s.y);
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

// A sum of many parts: sum + low, where low collects what each addition drops (Knuth's two-sum).
struct LongSum {
    float sum = 0.0f, low = 0.0f;
    __device__ __forceinline__ void add(float v) {
        const float s = __fadd_rn(sum, v), b = __fsub_rn(s, sum);
        low += __fadd_rn(__fsub_rn(sum, __fsub_rn(s, b)), __fsub_rn(v, b));
        sum = s;
    }
    __device__ __forceinline__ float value() const { return sum < INFINITY ? sum + low : sum; }
};

// The row's sum of squares and largest magnitude over the threads that hold it (`warps`
// warps: the whole CTA, or one warp of several rows'), the same in each of them.  Two buffers,
// taken in turn: one is written again behind the barrier of the other.
struct Exchange {
    float ss[2][32];
    uint32_t m[2][32];
};
template <bool SS, bool M>
__device__ __forceinline__ void combine_row(Exchange& x, int& buf, float& ss, uint32_t& m, int warps) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        if (SS) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (M) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    if (warps == 1) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) {
        if (SS) x.ss[buf][warp] = ss;
        if (M) x.m[buf][warp] = m;
    }
    __syncthreads();
    if (SS) ss = lane < warps ? x.ss[buf][lane] : 0.0f;
    if (M) m = lane < warps ? x.m[buf][lane] : 0u;
    buf ^= 1;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        if (SS) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (M) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
}

// x and the residual of eight values from c on; `stored`: their sum, which has been written
struct In { Raw8 x, res; };
template <int WHAT, typename T, bool VEC>
__device__ __forceinline__ In load_in(const RmsNormArgs& a, int64_t row, int c, bool stored) {
    constexpr bool kNorm = WHAT != kQuantI8;
    In in{};
    const int n = a.H - c;
    if (n <= 0 || row >= a.R) return in;
    if (kNorm && stored && a.residual && a.total) {
        if (a.res_f32) in.res = load8<float, VEC>(static_cast<const float*>(a.total) + row * a.ldt + c, n);
        else in.x = load8<T, VEC>(static_cast<const T*>(a.total) + row * a.ldt + c, n);
        return in;
    }
    in.x = load8<T, VEC>(static_cast<const T*>(a.x) + row * a.ldx + c, n);
    if (kNorm && a.residual) {
        if (a.res_f32) in.res = load8<float, VEC>(static_cast<const float*>(a.residual) + row * a.ldr + c, n);
        else in.res = load8<T, VEC>(static_cast<const T*>(a.residual) + row * a.ldr + c, n);
    }
    return in;
}
// r, and its store
template <int WHAT, typename T, bool VEC>
__device__ __forceinline__ void sum_in(const RmsNormArgs& a, int64_t row, const In& in, int c, bool stored, float (&r)[8]) {
    values<T>(in.x, r);
    if (WHAT == kQuantI8 || !a.residual) return;
    const int n = a.H - c;
    if (stored && a.total) {
        if (a.res_f32) values<float>(in.res, r);
        return;
    }
    float b[8];
    if (a.res_f32) {
        values<float>(in.res, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] += b[i];
        if (!stored && a.total && n > 0)
            store8<float, VEC>(static_cast<float*>(a.total) + row * a.ldt + c, n, raw_of<float>(r));
    } else {
        values<T>(in.res, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] += b[i];
        const Raw8 sum = raw_of<T>(r);
        values<T>(sum, r);
        if (!stored && a.total && n > 0) store8<T, VEC>(static_cast<T*>(a.total) + row * a.ldt + c, n, sum);
    }
}
template <int WHAT, typename T, bool VEC>
__device__ __forceinline__ void times_w(const RmsNormArgs& a, int c, float (&p)[8]) {
    const int n = a.H - c;
    if (WHAT == kQuantI8 || !a.w || n <= 0) return;
    float w[8];
    if (a.w_f32) values<float>(load8<float, VEC>(static_cast<const float*>(a.w) + c, n), w);
    else values<T>(load8<T, VEC>(static_cast<const T*>(a.w) + c, n), w);
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] *= w[i];
}
template <bool VEC>
__device__ __forceinline__ void store_codes(const RmsNormArgs& a, int64_t row, int c, uint2 q) {
    uint8_t* dst = a.codes + row * a.H + c;
    if (VEC) {
        *reinterpret_cast<uint2*>(dst) = q;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < a.H - c) dst[i] = (uint8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
    }
}

// A row whose sum of squares passes fp32, or with an infinity or a NaN: read again, with the squares
// of 2^-80 r.  The codes are those of p as everywhere; where a block's largest |p| (int8: the row's, m)
// passes fp32 itself they are those of 2^-80 r times w.  All threads of the row call it (buf: as
// combine_row's, which is called once).
template <int WHAT, typename T, bool VEC>
__device__ __noinline__ void huge_row(const RmsNormArgs& a, int64_t row, int warps, int t, uint32_t m, Exchange& x, int buf) {
    constexpr bool kRowMax = WHAT == kNormI8;
    const int step = 256 * warps;
    LongSum all;
    float mf = 0.0f;
#pragma unroll 1
    for (int c0 = 0; c0 < a.H; c0 += step) {
        const int c = c0 + 8 * t;
        float r[8], ss = 0.0f;
        sum_in<WHAT, T, VEC>(a, row, load_in<WHAT, T, VEC>(a, row, c, true), c, true, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            r[i] *= kTiny;
            ss = fmaf(r[i], r[i], ss);
        }
        all.add(ss);
        if (kRowMax) {
            times_w<WHAT, T, VEC>(a, c, r);
            mf = largest(r, mf);
        }
    }
    float ss = all.value();
    uint32_t small = __float_as_uint(mf);
    combine_row<true, kRowMax>(x, buf, ss, small, warps);
    const float rstd = rsqrtf(fmaf(ss, a.inv_h, a.eps * kTiny * kTiny));   // that of 2^-80 r
    // 2^-80 v rstd, in two steps that neither overflow nor lose a result's bits
    auto normed = [&](float v) { return (v * kRoot) * (rstd * kRoot); };
    constexpr uint32_t kInf = 0x7F800000u;
    const bool row_over = kRowMax && m == kInf;
    if (kRowMax) {
        m = fp8_amax_bits(row_over ? small : m);
        const float v = __uint_as_float(m);
        if (t == 0) a.scales[row] = over(row_over ? v * rstd : normed(v), 127.0f, 1.0f / 127.0f);
    }
#pragma unroll 1
    for (int c0 = 0; c0 < a.H; c0 += step) {
        const int c = c0 + 8 * t, n = a.H - c;
        float p[8], s[8];
        sum_in<WHAT, T, VEC>(a, row, load_in<WHAT, T, VEC>(a, row, c, true), c, true, p);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = p[i] * kTiny;
        times_w<WHAT, T, VEC>(a, c, p);
        times_w<WHAT, T, VEC>(a, c, s);
        uint2 q = make_uint2(0, 0);
        if (WHAT == kNormE4m3) {   // every lane takes part in the block's maxima
            uint32_t bm = __float_as_uint(largest(p, 0.0f)), bs = __float_as_uint(largest(s, 0.0f));
#pragma unroll
            for (int o = 8; o >= 1; o >>= 1) {
                bm = max(bm, __shfl_xor_sync(0xffffffffu, bm, o));
                bs = max(bs, __shfl_xor_sync(0xffffffffu, bs, o));
            }
            const bool block_over = bm == kInf;
            bm = fp8_amax_bits(block_over ? bs : bm);
            const float v = __uint_as_float(bm);
            q = block_over ? e4m3_codes(s, bm) : e4m3_codes(p, bm);
            if ((t & 15) == 0 && n > 0)
                a.scales[(int64_t)(c / kFp8Block) * a.R + row] = over(block_over ? v * rstd : normed(v), 448.0f, 1.0f / 448.0f);
        }
        if (kRowMax) q = row_over ? i8_codes(s, m) : i8_codes(p, m);
        if (n <= 0) continue;
        if (WHAT != kNormOnly) store_codes<VEC>(a, row, c, q);
        if (WHAT == kNormOnly || a.y) {
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = fabsf(p[i]) < INFINITY ? normed(p[i]) : s[i] * rstd;
            store8<T, VEC>(static_cast<T*>(a.y) + row * a.ldy + c, n, raw_of<T>(p));
        }
    }
}

}  // namespace

namespace {

__device__ __forceinline__ float2 mul22(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 c, a, b;\n\tmov.b64 {%0, %1}, c;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma22(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 c, a, b, c;\n\tmov.b64 {%0, %1}, c;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

// Many rows of at most 8192 values on 16-byte addresses.  RES: no residual, one of x's type, an
// fp32 one; FULL: the threads' vectors end with the row.  w lies in shared memory, in fp32.
template <int WHAT, typename T, int RES, bool FULL, int NV>
__device__ __forceinline__ void rows_many(const RmsNormArgs& a, int warps, const float* s_w, Exchange& s_x) {
    constexpr bool kNorm = WHAT != kQuantI8, kRowMax = WHAT == kNormI8 || WHAT == kQuantI8;
    using RT = std::conditional_t<RES == 2, float, T>;
    int buf = 0;
    const int lane = threadIdx.x & 31;
    const int t = warps == 1 ? lane : threadIdx.x;
    const int step = 256 * warps;
    const int per_cta = warps == 1 ? blockDim.x >> 5 : 1;
    const int stride = (int)gridDim.x * per_cta;
    int row = (int)blockIdx.x * per_cta + (warps == 1 ? threadIdx.x >> 5 : 0);
    const int c0 = 8 * t;
    auto inside = [&](int v) { return FULL || c0 + v * step < a.H; };
    Raw8 nx[NV], nr[RES ? NV : 1];
    auto load_row = [&](int row) {
        const T* x = static_cast<const T*>(a.x) + (int64_t)row * a.ldx + c0;
        const RT* res = static_cast<const RT*>(a.residual) + (int64_t)row * a.ldr + c0;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            nx[v].lo = nx[v].hi = make_uint4(0, 0, 0, 0);
            if (inside(v)) nx[v] = load_raw(x + v * step);
            if (RES) {
                nr[v].lo = nr[v].hi = make_uint4(0, 0, 0, 0);
                if (inside(v)) nr[v] = load_raw(res + v * step);
            }
        }
    };
    auto pairs = [](const float (&f)[8], float2 (&p)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = make_float2(f[2 * i], f[2 * i + 1]);
    };
    auto singles = [](const float2 (&p)[4], float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = p[i].x;
            f[2 * i + 1] = p[i].y;
        }
    };
    auto times_w = [&](int v, float2 (&p)[4]) {
        if (!kNorm) return;
        const float4 w0 = *reinterpret_cast<const float4*>(s_w + c0 + v * step);
        const float4 w1 = *reinterpret_cast<const float4*>(s_w + c0 + v * step + 4);
        p[0] = mul22(p[0], make_float2(w0.x, w0.y));
        p[1] = mul22(p[1], make_float2(w0.z, w0.w));
        p[2] = mul22(p[2], make_float2(w1.x, w1.y));
        p[3] = mul22(p[3], make_float2(w1.z, w1.w));
    };
    auto largest4 = [](const float2 (&p)[4], float m) {
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max_magnitude(p[i].x, p[i].y, m);
        return m;
    };
    // to the end, or to a row for huge_row, whose m it returns
    auto run = [&]() {
        for (; row < a.R; row += stride) {   // the same rows in every thread of a barrier
            float2 r[NV][4], s2 = make_float2(0.0f, 0.0f);
            float ss = 0.0f, mf = 0.0f;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float f[8];
                values<T>(nx[v], f);
                pairs(f, r[v]);
                if (RES) {
                    values<RT>(nr[v], f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) r[v][i] = add2(r[v][i], make_float2(f[2 * i], f[2 * i + 1]));
                    singles(r[v], f);
                    const Raw8 sum = raw_of<RT>(f);
                    if (sizeof(RT) == 2) {
                        values<RT>(sum, f);
                        pairs(f, r[v]);
                    }
                    if (a.total && inside(v)) store_raw(static_cast<RT*>(a.total) + (int64_t)row * a.ldt + c0 + v * step, sum);
                }
            }
            if (row + stride < a.R) load_row(row + stride);   // before the exchange
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (kNorm)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s2 = fma22(r[v][i], r[v][i], s2);
                if (kRowMax) {
                    float2 p[4] = {r[v][0], r[v][1], r[v][2], r[v][3]};
                    if (inside(v)) times_w(v, p);
                    mf = largest4(p, mf);
                }
            }
            ss = s2.x + s2.y;
            uint32_t m = __float_as_uint(mf);
            combine_row<kNorm, kRowMax>(s_x, buf, ss, m, warps);
            if (kNorm && !(ss < INFINITY)) return m;   // the same in each thread
            const float rstd = kNorm ? rsqrtf(fmaf(ss, a.inv_h, a.eps)) : 1.0f;
            if (kRowMax) {
                m = fp8_amax_bits(m);
                if (t == 0) a.scales[row] = over(kNorm ? __uint_as_float(m) * rstd : __uint_as_float(m), 127.0f, 1.0f / 127.0f);
            }
            uint32_t bm[NV];   // e4m3: the blocks' largest magnitudes, their exchanges side by side
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (inside(v)) times_w(v, r[v]);
                if (WHAT == kNormE4m3) bm[v] = __float_as_uint(largest4(r[v], 0.0f));
            }
            if (WHAT == kNormE4m3)
#pragma unroll
                for (int o = 8; o >= 1; o >>= 1)
#pragma unroll
                    for (int v = 0; v < NV; ++v) bm[v] = max(bm[v], __shfl_xor_sync(0xffffffffu, bm[v], o));
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float p[8];
                singles(r[v], p);
                if (WHAT == kNormE4m3) {
                    const uint32_t b = fp8_amax_bits(bm[v]);
                    const uint2 q = e4m3_codes(p, b);
                    if (inside(v)) {
                        *reinterpret_cast<uint2*>(a.codes + (int64_t)row * a.H + c0 + v * step) = q;
                        if ((lane & 15) == 0)
                            a.scales[(int64_t)((c0 + v * step) / kFp8Block) * a.R + row] =
                                over(__uint_as_float(b) * rstd, 448.0f, 1.0f / 448.0f);
                    }
                }
                if (kRowMax) {
                    const uint2 q = i8_codes(p, m);
                    if (inside(v)) *reinterpret_cast<uint2*>(a.codes + (int64_t)row * a.H + c0 + v * step) = q;
                }
                if (kNorm && (WHAT == kNormOnly || a.y) && inside(v)) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) r[v][i] = mul2(r[v][i], rstd);
                    singles(r[v], p);
                    store_raw(static_cast<T*>(a.y) + (int64_t)row * a.ldy + c0 + v * step, raw_of<T>(p));
                }
            }
        }
        return 0u;
    };
    if (!kNorm) {
        if (row < a.R) load_row(row);
        run();
        return;
    }
    while (row < a.R) {
        load_row(row);
        const uint32_t m = run();
        if (row >= a.R) break;
        // out of the loop, whose registers need not outlast the call
        huge_row<WHAT, T, true>(a, row, warps, t, m, s_x, buf);
        if (warps != 1) buf ^= 1;
        row += stride;
    }
}

}  // namespace

template <int WHAT, typename T, int NV, int MINB>
__global__ void __launch_bounds__(256, MINB) k_rows8_many(const __grid_constant__ RmsNormArgs a, int warps) {
    pdl_wait();  // see common.cuh: nothing global is touched before
    pdl_trigger();
    extern __shared__ __align__(16) float s_w[];
    __shared__ Exchange s_x;
    if (WHAT != kQuantI8) {
        for (int c = 8 * threadIdx.x; c < a.H; c += 8 * blockDim.x) {
            float f[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
            if (a.w) {
                if (a.w_f32) values<float>(load_raw(static_cast<const float*>(a.w) + c), f);
                else values<T>(load_raw(static_cast<const T*>(a.w) + c), f);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) s_w[c + i] = f[i];
        }
        __syncthreads();
    }
    const bool full = a.H == 256 * NV * warps;
    if (WHAT == kQuantI8 || !a.residual) {
        if (full) rows_many<WHAT, T, 0, true, NV>(a, warps, s_w, s_x);
        else rows_many<WHAT, T, 0, false, NV>(a, warps, s_w, s_x);
    } else if (!a.res_f32 || sizeof(T) == 4) {
        if (full) rows_many<WHAT, T, 1, true, NV>(a, warps, s_w, s_x);
        else rows_many<WHAT, T, 1, false, NV>(a, warps, s_w, s_x);
    } else if constexpr (NV < 4) {   // (launch_t has no such call for four)
        if (full) rows_many<WHAT, T, 2, true, NV>(a, warps, s_w, s_x);
        else rows_many<WHAT, T, 2, false, NV>(a, warps, s_w, s_x);
    }
}

// A row per `warps` warps; a CTA has several only where that is one.  NV vectors of eight values per
// thread; ONE: they hold the row, else it is gone through twice.  MAXT, MINB: threads of a CTA at
// most, CTAs per SM at least.
template <int WHAT, typename T, bool VEC, int NV, bool ONE, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) k_rows8(const __grid_constant__ RmsNormArgs a, int warps) {
    pdl_wait();  // see common.cuh: nothing global is touched before
    pdl_trigger();
    constexpr bool kNorm = WHAT != kQuantI8, kRowMax = WHAT == kNormI8 || WHAT == kQuantI8;
    __shared__ Exchange s_x;
    int buf = 0;
    const int lane = threadIdx.x & 31;
    const int t = warps == 1 ? lane : threadIdx.x;
    const int step = 256 * warps;   // values per vector of the row's threads
    const int per_cta = warps == 1 ? blockDim.x >> 5 : 1;
    const int64_t row = (int64_t)blockIdx.x * per_cta + (warps == 1 ? threadIdx.x >> 5 : 0);
    if (row >= a.R) return;   // whole warps, and no barrier follows where a CTA has several rows

    auto add_in = [&](int c, const float (&r)[8], float& ss, float& m) {
        if (kNorm)
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(r[i], r[i], ss);
        if (kRowMax) {
            float p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = r[i];
            times_w<WHAT, T, VEC>(a, c, p);
            m = largest(p, m);
        }
    };
    float r[NV][8], ss = 0.0f, mf = 0.0f;
    LongSum all;
    for (int c0 = 0; c0 < a.H; c0 += NV * step) {
        In in[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) in[v] = load_in<WHAT, T, VEC>(a, row, c0 + v * step + 8 * t, false);
#pragma unroll
        for (int v = 0; v < NV; ++v) sum_in<WHAT, T, VEC>(a, row, in[v], c0 + v * step + 8 * t, false, r[v]);
#pragma unroll
        for (int v = 0; v < NV; ++v) add_in(c0 + v * step + 8 * t, r[v], ss, mf);
        if (ONE) break;
        if (kNorm) {
            all.add(ss);
            ss = 0.0f;
        }
    }
    if (!ONE && kNorm) ss = all.value();
    uint32_t m = __float_as_uint(mf);
    combine_row<kNorm, kRowMax>(s_x, buf, ss, m, warps);
    if constexpr (kNorm) {
        if (!(ss < INFINITY)) {   // the same in each thread
            huge_row<WHAT, T, VEC>(a, row, warps, t, m, s_x, buf);
            return;
        }
    }
    const float rstd = kNorm ? rsqrtf(fmaf(ss, a.inv_h, a.eps)) : 1.0f;
    if (kRowMax) {
        m = fp8_amax_bits(m);
        if (t == 0) a.scales[row] = over(kNorm ? __uint_as_float(m) * rstd : __uint_as_float(m), 127.0f, 1.0f / 127.0f);
    }
    for (int c0 = 0; c0 < a.H; c0 += NV * step) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = c0 + v * step + 8 * t, n = a.H - c;
            if (!ONE) sum_in<WHAT, T, VEC>(a, row, load_in<WHAT, T, VEC>(a, row, c, true), c, true, r[v]);
            float p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = r[v][i];
            times_w<WHAT, T, VEC>(a, c, p);
            uint2 q = make_uint2(0, 0);
            if (WHAT == kNormE4m3) {   // every lane takes part in the block's maximum
                uint32_t bm = __float_as_uint(largest(p, 0.0f));
#pragma unroll
                for (int o = 8; o >= 1; o >>= 1) bm = max(bm, __shfl_xor_sync(0xffffffffu, bm, o));
                bm = fp8_amax_bits(bm);
                q = e4m3_codes(p, bm);
                if ((lane & 15) == 0 && n > 0)
                    a.scales[(int64_t)(c / kFp8Block) * a.R + row] = over(__uint_as_float(bm) * rstd, 448.0f, 1.0f / 448.0f);
            }
            if (kRowMax) q = i8_codes(p, m);
            if (n <= 0) continue;
            if (WHAT != kNormOnly) store_codes<VEC>(a, row, c, q);
            if (kNorm && (WHAT == kNormOnly || a.y)) {
#pragma unroll
                for (int i = 0; i < 8; ++i) p[i] *= rstd;
                store8<T, VEC>(static_cast<T*>(a.y) + row * a.ldy + c, n, raw_of<T>(p));
            }
        }
        if (ONE) break;
    }
}

namespace {

bool rows_aligned(const void* p, int64_t ld, size_t size, int64_t R) {
    return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (R <= 1 || ld * (int64_t)size % 16 == 0));
}

template <int WHAT, typename T, bool VEC, int NV, bool ONE, int MAXT, int MINB>
cudaError_t launch_as(const RmsNormArgs& a, int warps, cudaStream_t st) {
    const int per_cta = warps == 1 ? 4 : 1, threads = 32 * warps * per_cta;
    const int64_t grid = ((int64_t)a.R + per_cta - 1) / per_cta;
    return launch_kernel(k_rows8<WHAT, T, VEC, NV, ONE, MAXT, MINB>, dim3((unsigned)grid), dim3(threads), 0, st, a, warps);
}

template <int WHAT, typename T, int NV, int MINB>
cudaError_t launch_many(const RmsNormArgs& a, int warps, int num_sms, cudaStream_t st) {
    const int per_cta = warps == 1 ? 4 : 1, threads = 32 * warps * per_cta;
    int64_t grid = ((int64_t)a.R + per_cta - 1) / per_cta;
    const int64_t resident = (int64_t)num_sms * (256 * MINB / threads);
    if (grid > resident) grid = resident;
    return launch_kernel(k_rows8_many<WHAT, T, NV, MINB>, dim3((unsigned)grid), dim3(threads),
                         WHAT == kQuantI8 ? 0 : (size_t)a.H * 4, st, a, warps);
}

template <int WHAT, typename T>
cudaError_t launch_t(const RmsNormArgs& a, int num_sms, cudaStream_t st) {
    const size_t rs = a.res_f32 ? 4 : sizeof(T), es = sizeof(T);
    const bool vec = a.H % 8 == 0 && rows_aligned(a.x, a.ldx, es, a.R) && rows_aligned(a.residual, a.ldr, rs, a.R) &&
                     rows_aligned(a.total, a.ldt, rs, a.R) && rows_aligned(a.y, a.ldy, es, a.R) &&
                     reinterpret_cast<uintptr_t>(a.w) % 16 == 0 && reinterpret_cast<uintptr_t>(a.codes) % 8 == 0;
    const int per_warp = (a.H + 255) / 256;   // vectors that one warp would hold
    auto warps = [&](int nv) { return (per_warp + nv - 1) / nv; };
    if (warps(4) > 32)
        return vec ? launch_as<WHAT, T, true, 4, false, 1024, 1>(a, 32, st)
                   : launch_as<WHAT, T, false, 4, false, 1024, 1>(a, 32, st);
    if (!vec) return warps(4) <= 8 ? launch_as<WHAT, T, false, 4, true, 256, 3>(a, warps(4), st)
                                   : launch_as<WHAT, T, false, 4, true, 1024, 1>(a, warps(4), st);
    // few rows: a row over many threads, for the latency
    if (a.R <= 2 * num_sms && warps(1) <= 32) return launch_as<WHAT, T, true, 1, true, 1024, 1>(a, warps(1), st);
    // many: much of a row per thread, since the exchange costs each warp as much as eight values a lane
    if (per_warp == 1) return launch_many<WHAT, T, 1, 4>(a, 1, num_sms, st);
    if (per_warp == 2) return launch_many<WHAT, T, 2, 3>(a, 1, num_sms, st);
    // (an fp32 residual of 16-bit rows takes HBM longer than the arithmetic anyway, and CTAs that
    // stay were slower there: 8192 x 4096 73.6 us against 63.7, which are 58.8 by now)
    if (WHAT != kQuantI8 && a.res_f32 && warps(2) <= 32) return launch_as<WHAT, T, true, 2, true, 1024, 1>(a, warps(2), st);
    // (8192 x 2048 with e4m3 codes: two vectors 20.8 us, four 22.4; int8 quantising 13.1 and 11.1)
    if (WHAT != kQuantI8 && warps(2) <= 8) return launch_many<WHAT, T, 2, 3>(a, warps(2), num_sms, st);
    if (warps(4) <= 8) return launch_many<WHAT, T, 4, WHAT == kQuantI8 ? 3 : 2>(a, warps(4), num_sms, st);
    return launch_as<WHAT, T, true, 4, true, 1024, 1>(a, warps(4), st);
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
