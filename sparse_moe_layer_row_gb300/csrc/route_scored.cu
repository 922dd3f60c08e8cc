// moe_route_scored: rows of router logits -> the k experts of each row and
// their weights, under a routing rule (include/moe_block.h): softmax or sigmoid
// scores, a bias that only steers the choice, expert groups, renormalisation.
//
// One warp per row, the experts in its lanes' registers.  The order of the
// experts is that of real numbers, not of 32-bit roundings:
//   * without a bias a score rises strictly with its logit, so the logits
//     themselves are compared, exactly;
//   * sums (score + bias, a group's two largest) are formed in fp32 with a known
//     error bound; where two neighbours of the resulting order, or the last
//     group taken and the first one left, are closer than their bounds, the
//     candidates are ordered again in two-part fp32 (2^-40; a 64-bit instruction
//     takes this GPU 62 clocks), and what is closer still with 64-bit scores.
//     With bounds near 1e-6 and neighbouring keys some 1e-2 apart the first
//     happens to about one row in a thousand.
//
// 8192 rows of 256 experts in 8 groups take 14.0 us (1.3 by their bytes).  No unit is at
// its limit (0.59 issues per clock, 42% of the warps, 6% of HBM): a row is a chain of
// dependent warp reductions (sort, group and rank loops), 2048 CTAs over some 1216
// resident ones leave a last round, and the rows that 32 bits leave open end last.
// Taking the k best one by one, with 64-bit scores for every unsure row, took 42.
#include <cfloat>

#include "route_common.cuh"
#include "route_scored.cuh"

namespace moe {

namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kRouteThreads = 128;   // at most; four rows per CTA
constexpr uint32_t kMaskKey = 0x007FFFFFu;   // order_key(-inf); a NaN's key is 0

__device__ __forceinline__ float ld_logit(const float* p) { return __ldg(p); }
__device__ __forceinline__ float ld_logit(const __nv_bfloat16* p) {
    return __bfloat162float(__ldg(p));
}
__device__ __forceinline__ float ld_logit(const __half* p) { return __half2float(__ldg(p)); }

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// The warp's values in descending order of the lanes (bitonic).
__device__ __forceinline__ uint32_t warp_sort_desc(uint32_t v, int lane) {
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int stride = size >> 1; stride > 0; stride >>= 1) {
            const uint32_t o = __shfl_xor_sync(kAll, v, stride);
            const bool larger = ((lane & size) == 0) == ((lane & stride) == 0);
            v = larger ? max(v, o) : min(v, o);
        }
    return v;
}

// Two-part fp32 arithmetic (Dekker 1971, Knuth's two-sum): h + l, |l| <= half a step of h.
struct Two {
    float h, l;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two norm(float h, float l) {
    const float s = __fadd_rn(h, l);
    return {s, __fsub_rn(l, __fsub_rn(s, h))};
}
__device__ __forceinline__ Two add(Two a, Two b) {
    const Two s = two_sum(a.h, b.h);
    return norm(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ Two mul(Two a, Two b) {
    const float p = __fmul_rn(a.h, b.h);
    return norm(p, __fmaf_rn(a.l, b.h, __fmaf_rn(a.h, b.l, __fmaf_rn(a.h, b.h, -p))));
}

__device__ __forceinline__ Two div(Two a, Two b) {
    const float q = __fdiv_rn(a.h, b.h);
    const float rest = __fadd_rn(__fmaf_rn(-q, b.h, a.h), __fmaf_rn(-q, b.l, a.l));
    return norm(q, __fdiv_rn(rest, b.h));
}
__device__ __forceinline__ bool less(Two a, Two b) { return a.h < b.h || (a.h == b.h && a.l < b.l); }

// e^t for |t| <= 80 (clamped).  Cody-Waite reduction with ln 2 in three parts (12 bits,
// so that n times it is exact; two fp32), the Taylor polynomial of e^r to degree 13, its
// terms from r^7 on in fp32, the others in two parts.  A sigmoid by it is within 2^-46
// (3000 random arguments against 60 digits); callers count on 2^-40.
__device__ __forceinline__ Two exp_two(Two t) {
    if (!(fabsf(t.h) <= 80.0f)) t = {t.h > 0.0f ? 80.0f : -80.0f, 0.0f};
    const float n = rintf(__fmul_rn(t.h, 1.44269504088896341f));
    const float kHi = 0.693115234375f;              // 2839 / 4096
    const float kMid = 0x1.0bfbe8p-15f, kLo = 0x1.cf79acp-40f;
    const float p = __fmul_rn(n, kMid);
    Two r = two_sum(t.h, -__fmul_rn(n, kHi));
    r = add(r, {-p, __fsub_rn(t.l, __fadd_rn(__fmaf_rn(n, kMid, -p), __fmul_rn(n, kLo)))});
    float q = (float)(1.0 / 6227020800.0);          // 1 / 13!
    q = __fmaf_rn(q, r.h, (float)(1.0 / 479001600.0));
    q = __fmaf_rn(q, r.h, (float)(1.0 / 39916800.0));
    q = __fmaf_rn(q, r.h, (float)(1.0 / 3628800.0));
    q = __fmaf_rn(q, r.h, (float)(1.0 / 362880.0));
    q = __fmaf_rn(q, r.h, (float)(1.0 / 40320.0));
    q = __fmaf_rn(q, r.h, (float)(1.0 / 5040.0));
    Two e = add({0x1.6c16c2p-10f, -0x1.27d27ep-35f}, mul({q, 0.0f}, r));   // 1 / 6!
    e = add({0x1.111112p-7f, -0x1.ddddde0p-32f}, mul(e, r));               // 1 / 5!
    e = add({0x1.555556p-5f, -0x1.555556p-30f}, mul(e, r));                // 1 / 4!
    e = add({0x1.555556p-3f, -0x1.555556p-28f}, mul(e, r));                // 1 / 3!
    e = add({0.5f, 0.0f}, mul(e, r));
    e = add({1.0f, 0.0f}, mul(e, r));
    e = add({1.0f, 0.0f}, mul(e, r));
    const float scale = __uint_as_float((uint32_t)((int)n + 127) << 23);
    return {__fmul_rn(e.h, scale), __fmul_rn(e.l, scale)};
}

// A softmax numerator, e^(z - zmax).
__device__ __forceinline__ Two numerator_two(float z, float zmax) {
    if (z == zmax) return {1.0f, 0.0f};
    if (zmax == INFINITY) return {0.0f, 0.0f};
    return exp_two(two_sum(z, -zmax));
}

// Score + b of an expert that is not masked (softmax: over `total`).
__device__ __forceinline__ Two score_two(bool sig, float z, float zmax, Two total, float b) {
    Two s;
    if (sig) {   // inf: the clamp gives 0 or 1 to 2^-115
        const Two e = exp_two({-z, 0.0f});
        s = div({1.0f, 0.0f}, add({1.0f, 0.0f}, e));
    } else {
        s = div(numerator_two(z, zmax), total);
    }
    return add(s, {b, 0.0f});
}

// How far apart two-part keys have to be for their order to be settled.
__device__ __forceinline__ bool settled(float diff, float of) {
    return fabsf(diff) > 4e-12f * fmaxf(1.0f, fabsf(of));
}

// Order-preserving 64-bit key; NaN -> 0, below -inf.
__device__ __forceinline__ unsigned long long order_key64(double d) {
    if (d != d) return 0ull;
    const unsigned long long u = (unsigned long long)__double_as_longlong(d);
    return u >> 63 ? ~u : u | 1ull << 63;
}
__device__ __forceinline__ double key_value64(unsigned long long k) {
    return __longlong_as_double((long long)(k >> 63 ? k & ~(1ull << 63) : ~k));
}
constexpr unsigned long long kMaskKey64 = 0x000FFFFFFFFFFFFFull;   // order_key64(-inf)

// The softmax's sum over the row (one where only numerators are compared: no bias).
template <typename T>
__device__ __forceinline__ Two total_two(const RouteScoredArgs& a, const T* zr, int lane, float zmax) {
    if (a.rule.score == MOE_SCORE_SIGMOID || !a.bias) return {1.0f, 0.0f};
    Two t = {0.0f, 0.0f};
    for (int e = lane; e < a.E; e += 32) {
        const float z = ld_logit(zr + e);
        if (z != -INFINITY && z == z) t = add(t, numerator_two(z, zmax));
    }
    for (int o = 16; o >= 1; o >>= 1)
        t = add(t, {__shfl_xor_sync(kAll, t.h, o), __shfl_xor_sync(kAll, t.l, o)});
    return t;
}

// The groups taken (bit h), where the last one in (score x) and the first one out (y)
// are closer than gt.  Lane h holds group h's 32-bit score.  Groups more than gt above x
// are in; those from y - gt to x + gt are ranked by two-part scores.  False: those
// do not settle it either.
template <typename T>
__device__ __forceinline__ bool near_groups(const RouteScoredArgs& a, const T* zr, int lane, float mine,
                                            float x, float y, float gt, float zmax, uint32_t& taken) {
    const int G = a.rule.n_groups;
    const uint32_t sure = __ballot_sync(kAll, lane < G && mine > x + gt);
    const uint32_t near = __ballot_sync(kAll, lane < G && mine <= x + gt && mine >= y - gt);
    const Two total = total_two<T>(a, zr, lane, zmax);
    const Two none = {-FLT_MAX, 0.0f};
    Two key = none;
    for (uint32_t left = near; left; left &= left - 1) {
        const int h = __ffs(left) - 1;
        Two t1 = none, t2 = none;
        for (int r = lane; r < a.gs; r += 32) {
            const int e = h * a.gs + r;
            const float z = ld_logit(zr + e);
            if (z == -INFINITY || z != z) continue;
            const Two v = score_two(a.rule.score == MOE_SCORE_SIGMOID, z, zmax, total,
                                    a.bias ? __ldg(a.bias + e) : 0.0f);
            if (less(t1, v)) { t2 = t1; t1 = v; }
            else if (less(t2, v)) t2 = v;
        }
        __syncwarp();
        for (int o = 16; o >= 1; o >>= 1) {
            const Two u1 = {__shfl_xor_sync(kAll, t1.h, o), __shfl_xor_sync(kAll, t1.l, o)};
            const Two u2 = {__shfl_xor_sync(kAll, t2.h, o), __shfl_xor_sync(kAll, t2.l, o)};
            if (less(t1, u1)) { t2 = less(t1, u2) ? u2 : t1; t1 = u1; }
            else if (less(t2, u1)) t2 = u1;
        }
        if (a.rule.group_score == MOE_GROUP_TOP2 && t2.h > -FLT_MAX) t1 = add(t1, t2);
        if (lane == h) key = t1;
    }
    int rank = __popc(sure);
    bool close = false;
    for (uint32_t left = near; left; left &= left - 1) {
        const int h = __ffs(left) - 1;
        const Two k = {__shfl_sync(kAll, key.h, h), __shfl_sync(kAll, key.l, h)};
        const float diff = __fadd_rn(__fsub_rn(k.h, key.h), __fsub_rn(k.l, key.l));
        rank += diff > 0.0f;
        close |= h != lane && !settled(diff, key.h);
    }
    const bool is_near = (near >> lane) & 1u;
    if (__any_sync(kAll, is_near && close)) return false;
    taken = sure | __ballot_sync(kAll, is_near && rank < a.rule.top_groups);
    return true;
}

// Renormalised weights of a row that takes scores near or below fp32's least: numerators
// e^(z - m) over the largest chosen logit m, and for the sigmoid s e^-p = e^(z - p) / (1 + e^z)
// with p = min(m, 0), both at most 1.  The low part of z - p counts too (e^l = 1 + l), as the
// difference may be near 100.  Scores below e^-700 are 0 as they are in 64 bits (`off`: masked).
__device__ __noinline__ float ratio_weight(bool sig, float z, bool off, float zmax) {
    off |= z < (sig ? -700.0f : zmax - 700.0f);
    const float m = warp_max(off ? -INFINITY : z), p = sig ? fminf(m, 0.0f) : m;
    float t = 0.0f;
    if (!off) {
        if (sig && z > 0.0f) {
            t = __fdiv_rn(1.0f, 1.0f + expf(-z));
        } else {
            t = 1.0f;
            if (z != p) {
                const Two d = two_sum(z, -p);
                t = expf(d.h);
                t = __fmaf_rn(t, d.l, t);
            }
            if (sig) t = __fdiv_rn(t, 1.0f + expf(z));
        }
    }
    const float sum = warp_sum(t);
    return sum > 0.0f ? __fdiv_rn(t, sum) : 0.0f;
}

// The weights of the chosen experts (lane j: the j-th, my_id), from their unbiased scores.
template <typename T>
__device__ __forceinline__ void write_row(const RouteScoredArgs& a, const T* zr, int row, int lane,
                                          int my_id, float zmax, float inv) {
    const bool sig = a.rule.score == MOE_SCORE_SIGMOID;
    const float zj = lane < a.k ? ld_logit(zr + my_id) : -INFINITY;
    const bool off = zj == -INFINITY || zj != zj;
    float s = 0.0f;
    if (!off) {
        if (!sig) s = zj == zmax ? inv : expf(zj - zmax) * inv;
        else if (zj < -87.0f) s = expf(zj);   // 1 + e^z is 1, and e^-z may be infinite
        else s = __fdiv_rn(1.0f, 1.0f + expf(-zj));
    }
    float w = s;
    if (a.rule.renormalize) {
        if (__any_sync(kAll, !off && s < 0x1p-100f)) {
            w = ratio_weight(sig, zj, off, zmax);
        } else {
            const float sum = warp_sum(s);
            w = sum > 0.0f ? __fdiv_rn(s, sum) : 0.0f;
        }
    }
    if (lane < a.k) {
        const int64_t o = (int64_t)row * a.k + lane;
        a.topk_idx[o] = my_id;
        a.topk_w[o] = w * a.rule.scale;
        if (a.topk_score) a.topk_score[o] = s;
    }
}

// A row with 64-bit scores throughout: for rows that two-part keys do not settle (keys
// within 4e-12, or more than 32 candidates); written for size, not speed.
template <typename T>
__device__ __noinline__ void route_exact(const RouteScoredArgs& a, int row, int lane, float inv) {
    const T* zr = static_cast<const T*>(a.logits) + (int64_t)row * a.ld;
    const int ne = (a.E + 31) >> 5;
    unsigned long long ek[32], gk[32];   // element order, and the value a group ranks by
    float zmax = -INFINITY;
    for (int i = 0; i < ne; ++i) {
        const int e = lane + 32 * i;
        if (e < a.E) zmax = fmaxf(zmax, ld_logit(zr + e));   // fmaxf skips NaN
    }
    zmax = warp_max(zmax);
    auto part = [&](float z) {   // the score, or its softmax numerator
        if (a.rule.score == MOE_SCORE_SIGMOID) return 1.0 / (1.0 + exp(-(double)z));
        if (z == -INFINITY || z != z) return 0.0;
        return z == zmax ? 1.0 : exp((double)z - (double)zmax);
    };
    double total = 1.0;
    if (a.rule.score == MOE_SCORE_SOFTMAX) {
        total = 0.0;
        for (int i = 0; i < ne; ++i) {
            const int e = lane + 32 * i;
            if (e < a.E) total += part(ld_logit(zr + e));
        }
        for (int o = 16; o >= 1; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
    }
    for (int i = 0; i < ne; ++i) {
        const int e = lane + 32 * i;
        ek[i] = gk[i] = 0ull;
        if (e >= a.E) continue;
        const float z = ld_logit(zr + e) + 0.0f;
        if (z == -INFINITY || z != z) {
            ek[i] = z != z ? 0ull : kMaskKey64;
            gk[i] = kMaskKey64;
            continue;
        }
        const double v = part(z) / total + (a.bias ? (double)__ldg(a.bias + e) : 0.0);
        gk[i] = order_key64(v);
        ek[i] = a.bias ? gk[i] : order_key64((double)z);
    }
    uint32_t groups = kAll;
    if (a.rule.n_groups > 1) {
        unsigned long long mine = 0ull;   // lane g: group g's key
        for (int g = 0; g < a.rule.n_groups; ++g) {
            unsigned long long t1 = 0ull, t2 = 0ull;
            for (int i = 0; i < ne; ++i) {
                const int e = lane + 32 * i;
                if (e < g * a.gs || e >= (g + 1) * a.gs) continue;
                // largest element: without a bias the logits decide, as for the choice
                const unsigned long long v = a.rule.group_score == MOE_GROUP_MAX ? max(ek[i], kMaskKey64) : gk[i];
                t2 = max(t2, min(t1, v));
                t1 = max(t1, v);
            }
            for (int o = 16; o >= 1; o >>= 1) {
                const unsigned long long u1 = __shfl_xor_sync(kAll, t1, o), u2 = __shfl_xor_sync(kAll, t2, o);
                t2 = max(max(t2, u2), min(t1, u1));
                t1 = max(t1, u1);
            }
            if (a.rule.group_score == MOE_GROUP_TOP2 && t1 > kMaskKey64 && t2 > kMaskKey64)
                t1 = order_key64(key_value64(t1) + key_value64(t2));
            if (lane == g) mine = t1;
        }
        int rank = 0;
        for (int g = 0; g < a.rule.n_groups; ++g) {
            const unsigned long long k = __shfl_sync(kAll, mine, g);
            rank += k > mine || (k == mine && g < lane);
        }
        groups = __ballot_sync(kAll, lane < a.rule.n_groups && rank < a.rule.top_groups);
    }
    uint32_t left = 0;
    for (int i = 0; i < ne; ++i) {
        const int e = lane + 32 * i;
        if (e < a.E && ((groups >> (e / a.gs)) & 1u)) left |= 1u << i;
    }
    int my_id = 0;
    for (int j = 0; j < a.k; ++j) {
        unsigned long long bk = 0ull;
        int be = 0x7FFFFFFF;
        for (int i = 0; i < ne; ++i)
            if (((left >> i) & 1u) && (be == 0x7FFFFFFF || ek[i] > bk)) { bk = ek[i]; be = lane + 32 * i; }
        unsigned long long wk = bk;
        int we = be;
        for (int o = 16; o >= 1; o >>= 1) {
            const unsigned long long ok = __shfl_xor_sync(kAll, wk, o);
            const int oe = __shfl_xor_sync(kAll, we, o);
            // a lane with nothing left (id 0x7FFFFFFF) loses to any other
            if (we == 0x7FFFFFFF || (oe != 0x7FFFFFFF && (ok > wk || (ok == wk && oe < we)))) { wk = ok; we = oe; }
        }
        if (we == be) left &= ~(1u << ((we - lane) >> 5));
        if (lane == j) my_id = we;
    }
    write_row<T>(a, zr, row, lane, my_id, zmax, inv);   // inv: as for every other row
}

}  // namespace

// NE consecutive logits (or biases) of a lane, as 16-byte loads.
template <int NE>
__device__ __forceinline__ void load_consecutive(const float* p, float (&v)[NE]) {
#pragma unroll
    for (int i = 0; i < NE; i += 4) {
        const float4 w = __ldg(reinterpret_cast<const float4*>(p + i));
        v[i] = w.x; v[i + 1] = w.y; v[i + 2] = w.z; v[i + 3] = w.w;
    }
}
template <int NE, typename T>
__device__ __forceinline__ void load_consecutive(const T* p, float (&v)[NE]) {
#pragma unroll
    for (int i = 0; i < NE; i += 8) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(p + i));
        const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i + j] = (float)e[j];
    }
}

// CONTIG: E = 32 NE, 16-byte aligned rows and bias, and groups of whole lanes (a power
// of two of them): lane p holds the experts p NE .. p NE + NE - 1.  Otherwise
// p, p + 32, ..., and group scores go through shared memory.
// Routes one row.  True: two-part keys do not settle it, and nothing is written.
template <typename T, int NE, bool CONTIG>
__device__ __forceinline__ bool route_row(const RouteScoredArgs& a, int row, int lane,
                                          const float (&bias)[NE], uint2* slots, uint32_t* keys,
                                          float& inv) {
    const int G = a.rule.n_groups;
    // lanes that share a group: those that hold it, or 32 / (G rounded up to a power of two)
    const int L = CONTIG ? a.gs / NE : G > 1 ? 32 >> (32 - __clz(G - 1)) : 32;
    const bool sig = a.rule.score == MOE_SCORE_SIGMOID;
    const bool top2 = a.rule.group_score == MOE_GROUP_TOP2 && G > 1;
    auto id_of = [&](int i) { return CONTIG ? lane * NE + i : lane + 32 * i; };
    const T* zr = static_cast<const T*>(a.logits) + (int64_t)row * a.ld;
    float z[NE];
    if (CONTIG) {
        load_consecutive<NE>(zr + lane * NE, z);
    } else {
#pragma unroll
        for (int i = 0; i < NE; ++i) {   // every load first
            const int e = lane + 32 * i;
            z[i] = e < a.E ? ld_logit(zr + e) : -INFINITY;
        }
    }
    // scores (fast exponential and quotient: the error bounds below)
    float zmax = -INFINITY;
    inv = 0.0f;   // softmax: one over the sum
    float v[NE];
    // |error| of score + bias: a sigmoid's is s(1 - s) times the relative error of
    // e^-z (2^-22 + |z| 2^-23.4) plus the quotient's 2^-23, under 3e-7; a softmax
    // score's is its own size times the errors of its exponential, of the sum of E and
    // of the quotient, under 2e-6 of the row's largest score.  tol: two of them.
    float tol = 0.0f;
    if (!sig) {
#pragma unroll
        for (int i = 0; i < NE; ++i) zmax = fmaxf(zmax, z[i]);
        zmax = warp_max(zmax);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            v[i] = z[i] == -INFINITY || z[i] != z[i] ? 0.0f : z[i] == zmax ? 1.0f : __expf(z[i] - zmax);
            sum += v[i];
        }
        sum = warp_sum(sum);
        inv = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
#pragma unroll
        for (int i = 0; i < NE; ++i) v[i] *= inv;
        tol = 4e-6f * inv;
    } else if (a.bias || top2) {
#pragma unroll
        for (int i = 0; i < NE; ++i) v[i] = __fdividef(1.0f, 1.0f + __expf(-z[i]));
        tol = 6e-7f;
    }
    // v: what groups rank by; key: what the choice ranks by (without a bias, the logits)
    uint32_t key[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const float zi = z[i] + 0.0f;   // -0 -> +0
        const bool nan = zi != zi, masked = nan || zi == -INFINITY;
        if (a.bias) v[i] += bias[i];
        key[i] = order_key(a.bias ? v[i] : zi);
        if (masked) key[i] = nan ? 0u : kMaskKey;
        if (masked) v[i] = -INFINITY;
    }
    uint32_t valid = 0;
    if (G > 1) {
        uint32_t t1 = 0, t2 = 0;   // the two largest of the lane's part of its group
        const int g = lane / L, l = lane - g * L;
        if (CONTIG) {
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const uint32_t x = max(top2 ? order_key(v[i]) : key[i], kMaskKey);
                t2 = max(t2, min(t1, x));
                t1 = max(t1, x);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int e = lane + 32 * i;
                if (e < a.E) {
                    const int h = (int)(((uint32_t)e * a.ginv) >> 20);
                    keys[e + h * L] = max(top2 ? order_key(v[i]) : key[i], kMaskKey);
                }
            }
            __syncwarp();
            if (g < G)
                for (int r = l; r < a.gs; r += L) {
                    const uint32_t x = keys[g * (a.gs + L) + r];
                    t2 = max(t2, min(t1, x));
                    t1 = max(t1, x);
                }
            __syncwarp();
        }
        for (int o = L >> 1; o >= 1; o >>= 1) {
            const uint32_t u1 = __shfl_xor_sync(kAll, t1, o), u2 = __shfl_xor_sync(kAll, t2, o);
            t2 = max(max(t2, u2), min(t1, u1));
            t1 = max(t1, u1);
        }
        // a sum beyond fp32 stays in its range: no infinity, which is the masked groups' value
        if (top2 && t2 > kMaskKey)
            t1 = order_key(fmaxf(fminf(key_value(t1) + key_value(t2), FLT_MAX), -FLT_MAX));
        int rank = 0;
        for (int h = 0; h < G; ++h) {
            const uint32_t x = __shfl_sync(kAll, t1, h * L);
            rank += x > t1 || (x == t1 && h < g);
        }
        const bool lead = g < G && l == 0;
        uint32_t taken = __ballot_sync(kAll, lead && rank < a.rule.top_groups);
        if ((top2 || a.bias) && a.rule.top_groups < G) {
            const int in = __ffs(__ballot_sync(kAll, lead && rank == a.rule.top_groups - 1)) - 1;
            const int out = __ffs(__ballot_sync(kAll, lead && rank == a.rule.top_groups)) - 1;
            const float x = key_value(__shfl_sync(kAll, t1, in)), y = key_value(__shfl_sync(kAll, t1, out));
            // a sum of two keys: twice the error, and its own rounding
            const float gt = 2.0f * tol + 4e-7f * (fabsf(x) + fabsf(y));
            if (y > -INFINITY && !(x - y > gt)) {
                if (!(gt < INFINITY)) return true;   // 32 bits say nothing about keys this large
                // lane h: group h's score
                const float mine = key_value(__shfl_sync(kAll, t1, min(lane, G - 1) * L));
                uint32_t m = 0;
                if (!near_groups<T>(a, zr, lane, mine, x, y, gt, zmax, m)) return true;
                taken = 0;
                for (int h = 0; h < G; ++h) taken |= ((m >> h) & 1u) << (h * L);
            }
        }
        if (CONTIG) {
            valid = (taken >> (g * L)) & 1u ? kAll >> (32 - NE) : 0u;
        } else {
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int e = lane + 32 * i;
                const int h = (int)(((uint32_t)e * a.ginv) >> 20);
                if (e < a.E && ((taken >> (h * L)) & 1u)) valid |= 1u << i;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (id_of(i) < a.E) valid |= 1u << i;
    }
    // The k largest, and with a bias every key not certainly below the k-th: lane j
    // gets the j-th of these `count` candidates.
    int my_id = 0, count = 0;
    bool unsure = false, many = false;
    // Candidates: the k-th largest of the lanes' own largest keys is a lower bound of
    // the k-th largest key, and few keys reach it
    uint32_t bound = 0;
#pragma unroll
    for (int i = 0; i < NE; ++i)
        if ((valid >> i) & 1u) bound = max(bound, key[i]);
    bound = __shfl_sync(kAll, warp_sort_desc(bound, lane), a.k - 1);
    if (a.bias && bound > kMaskKey) {
        const float x = key_value(bound);
        bound = order_key(x - (tol + 5e-7f * fabsf(x)));
    }
    uint32_t cand = 0;
#pragma unroll
    for (int i = 0; i < NE; ++i)
        if (((valid >> i) & 1u) && key[i] >= bound) cand |= 1u << i;
    const int nc = __popc(cand);
    count = __reduce_add_sync(kAll, nc);
    if (count <= 32) {
        int at = nc;   // slots before this lane's
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(kAll, at, o);
            if (lane >= o) at += t;
        }
        at -= nc;
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if ((cand >> i) & 1u) slots[at++] = make_uint2(key[i], (uint32_t)id_of(i));
        __syncwarp();
        const uint2 mine = slots[lane < count ? lane : 0];
        int rank = 0;
        for (int h = 0; h < count; ++h) {
            const uint2 o = slots[h];
            rank += o.x > mine.x || (o.x == mine.x && o.y < mine.y);
        }
        __syncwarp();
        if (lane < count) slots[rank] = mine;
        __syncwarp();
        const uint2 sorted = slots[lane < count ? lane : 0];
        __syncwarp();   // the next row writes here
        my_id = (int)sorted.y;
        if (a.bias) {   // the order of neighbours up to the k-th and the one after it
            const uint32_t nk = __shfl_down_sync(kAll, sorted.x, 1);
            const float x = key_value(sorted.x), y = key_value(nk);
            const bool near = lane < a.k && lane + 1 < count && nk > kMaskKey &&
                              !(x - y > tol + 2e-7f * (fabsf(x) + fabsf(y)));
            unsure = __any_sync(kAll, near);
        }
    } else {
        // many equal or nearly equal keys: one at a time.  Each lane offers its largest
        // (equal keys: the lower id) and the warp takes the largest offer.
        count = 0;
        float prev = 0.0f, kth = 0.0f;
        while (true) {
            uint32_t bk = 0;
            int bi = -1;
#pragma unroll
            for (int i = NE - 1; i >= 0; --i)
                if (((valid >> i) & 1u) && key[i] >= bk) { bk = key[i]; bi = i; }
            const uint32_t mk = __reduce_max_sync(kAll, bk);
            const bool top = bi >= 0 && bk == mk;
            uint32_t who = __ballot_sync(kAll, top);
            if (!who) break;   // nothing left
            if (a.bias) {
                const float x = key_value(mk);
                const bool near = count > 0 && mk > kMaskKey && !(prev - x > tol + 2e-7f * (fabsf(prev) + fabsf(x)));
                if (count >= a.k && (mk <= kMaskKey || kth - x > tol + 2e-7f * (fabsf(kth) + fabsf(x)))) break;
                unsure |= near;
                prev = x;
                if (count == a.k - 1) kth = x;
                many = count == 32;
            }
            if (count == (a.bias ? 32 : a.k)) break;
            const int id = id_of(bi);
            int win = id;
            if (who & (who - 1)) {   // equal keys: the lowest id
                win = (int)__reduce_min_sync(kAll, top ? (uint32_t)id : 0xFFFFFFFFu);
                who = __ballot_sync(kAll, top && id == win);
            }
            win = __shfl_sync(kAll, win, __ffs(who) - 1);
            if (top && id == win) valid &= ~(1u << bi);
            if (lane == count) my_id = win;
            ++count;
        }
    }
    if (unsure) {   // the same in every lane
        if (many) return true;
        // the candidates again, one per lane, with two-part keys
        const Two total = total_two<T>(a, zr, lane, zmax);
        const float zc = ld_logit(zr + my_id), bc = __ldg(a.bias + my_id);
        const bool off = zc == -INFINITY || zc != zc;
        const Two k = off ? Two{zc != zc ? -FLT_MAX : -0.5f * FLT_MAX, 0.0f} : score_two(sig, zc, zmax, total, bc);
        int rank = 0;
        bool close = false;
        for (int h = 0; h < count; ++h) {
            const Two o = {__shfl_sync(kAll, k.h, h), __shfl_sync(kAll, k.l, h)};
            const float oz = __shfl_sync(kAll, zc, h), ob = __shfl_sync(kAll, bc, h);
            const int oid = __shfl_sync(kAll, my_id, h);
            const float diff = __fadd_rn(__fsub_rn(o.h, k.h), __fsub_rn(o.l, k.l));
            // equal logits and biases: equal keys
            const bool same = off ? diff == 0.0f : oz == zc && ob == bc;
            rank += same ? oid < my_id : diff > 0.0f;
            close |= !same && !settled(diff, k.h);
        }
        if (__any_sync(kAll, lane < count && close)) return true;
        if (lane < count) slots[rank].y = (uint32_t)my_id;
        __syncwarp();
        my_id = (int)slots[lane < count ? lane : 0].y;
        __syncwarp();   // the next row writes here
    }
    write_row<T>(a, zr, row, lane, my_id, zmax, inv);
    return false;
}

template <typename T, int NE, bool CONTIG>
__global__ void __launch_bounds__(kRouteThreads, NE <= 8 ? 1024 / kRouteThreads : 1)
k_route_scored(RouteScoredArgs a) {
    pdl_wait();  // see common.cuh: nothing global is touched before
    pdl_trigger();
    extern __shared__ __align__(8) uint32_t s_keys[];   // candidates; !CONTIG, n_groups > 1: group keys
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, wpc = blockDim.x >> 5;
    uint2* slots = reinterpret_cast<uint2*>(s_keys) + wid * 32;   // candidates (key, id), per warp
    float* invs = reinterpret_cast<float*>(s_keys + wpc * 64) + wid * 32;   // of rows left to 64 bits
    uint32_t* keys = s_keys + wpc * 96 + wid * (a.E + 32);
    float bias[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) bias[i] = 0.0f;
    if (a.bias) {
        if (CONTIG) {
            load_consecutive<NE>(a.bias + lane * NE, bias);
        } else {
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (lane + 32 * i < a.E) bias[i] = __ldg(a.bias + lane + 32 * i);
        }
    }
    // 32 rows of the warp at a time, then those of them that are left to 64 bits
    const int step = gridDim.x * wpc;
    for (int64_t first = blockIdx.x * wpc + wid; first < a.R; first += (int64_t)32 * step) {
        uint32_t left = 0;
        for (int i = 0; i < 32; ++i) {
            const int64_t row = first + (int64_t)i * step;
            if (row >= a.R) break;
            float inv;
            if (route_row<T, NE, CONTIG>(a, (int)row, lane, bias, slots, keys, inv)) {
                left |= 1u << i;
                invs[i] = inv;   // the same in every lane
            }
        }
        __syncwarp();
        for (; left; left &= left - 1) {
            const int i = __ffs(left) - 1;
            route_exact<T>(a, (int)(first + (int64_t)i * step), lane, invs[i]);
        }
        __syncwarp();
    }
}

template <typename T>
static cudaError_t launch_t(const RouteScoredArgs& a, int num_sms, cudaStream_t st) {
    // one warp per CTA until every SM has some, then up to four
    int wpc = a.R / num_sms;
    wpc = wpc < 1 ? 1 : wpc > kRouteThreads / 32 ? kRouteThreads / 32 : wpc;
    int64_t grid = ((int64_t)a.R + wpc - 1) / wpc;
    if (grid > (int64_t)num_sms * (64 / wpc)) grid = (int64_t)num_sms * (64 / wpc);
    const size_t smem = sizeof(uint32_t) * wpc * (96 + (a.rule.n_groups > 1 ? a.E + 32 : 0));
    const int ne = (a.E + 31) / 32;
    // consecutive experts per lane where every lane holds 8, 16 or 32 and the addresses allow
    const int lanes = a.gs / (ne > 0 ? ne : 1);   // per group
    const bool contig = a.E == 32 * ne && (ne == 8 || ne == 16 || ne == 32) && a.gs % ne == 0 &&
                        (lanes & (lanes - 1)) == 0 && a.ld * (int64_t)sizeof(T) % 16 == 0 &&
                        reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 &&
                        reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
    auto k = contig ? (ne == 8 ? k_route_scored<T, 8, true> : ne == 16 ? k_route_scored<T, 16, true>
                                                            : k_route_scored<T, 32, true>)
           : ne <= 1 ? k_route_scored<T, 1, false> : ne <= 2 ? k_route_scored<T, 2, false>
           : ne <= 4 ? k_route_scored<T, 4, false> : ne <= 8 ? k_route_scored<T, 8, false>
           : ne <= 16 ? k_route_scored<T, 16, false> : k_route_scored<T, 32, false>;
    return launch_kernel(k, dim3((unsigned)grid), dim3(32 * wpc), smem, st, a);
}

cudaError_t launch_route_scored(const RouteScoredArgs& a, int dtype, int num_sms, cudaStream_t st) {
    if (dtype == MOE_BF16) return launch_t<__nv_bfloat16>(a, num_sms, st);
    if (dtype == MOE_F16) return launch_t<__half>(a, num_sms, st);
    return launch_t<float>(a, num_sms, st);
}

}  // namespace moe
