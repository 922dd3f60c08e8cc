// moe_route_scored: rows of router logits -> the k experts of each row and
// their weights, under a routing rule (include/moe_block.h): softmax or sigmoid
// scores, a bias that only steers the choice, expert groups, renormalisation.
//
// One warp per row; lane p holds the experts p, p + 32, ...  The order of the
// experts is that of real numbers, not of 32-bit roundings:
//   * without a bias a score rises strictly with its logit, so the logits
//     themselves are compared, exactly;
//   * sums (score + bias, a group's two largest) are formed in fp32 with a known
//     error bound; where two neighbours of the resulting order, or the last
//     group taken and the first one left, are closer than their bounds, the row
//     is ordered again with 64-bit scores (route_exact).  With bounds near 1e-6
//     and neighbouring keys some 1e-2 apart that is about one row in a thousand.
#include "route_common.cuh"
#include "route_scored.cuh"

namespace moe {

namespace {

constexpr uint32_t kAll = 0xffffffffu;
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

// The row's choice with 64-bit scores: lane j < k gets the j-th expert.  Rare:
// written for size, not speed.
template <typename T>
__device__ __noinline__ int route_exact(const RouteScoredArgs& a, int row, int lane) {
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
    return my_id;
}

}  // namespace

template <typename T, int NE>
__global__ void __launch_bounds__(256) k_route_scored(RouteScoredArgs a) {
    pdl_wait();  // see common.cuh: nothing global is touched before
    pdl_trigger();
    extern __shared__ uint32_t s_keys[];   // per warp: group keys of the row (n_groups > 1)
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, wpc = blockDim.x >> 5;
    const int G = a.rule.n_groups;
    // lanes that share a group's scan: 32 / (G rounded up to a power of two)
    const int L = G > 1 ? 32 >> (32 - __clz(G - 1)) : 32;
    uint32_t* keys = s_keys + wid * (a.E + G * L);
    const bool sig = a.rule.score == MOE_SCORE_SIGMOID;
    const bool top2 = a.rule.group_score == MOE_GROUP_TOP2 && G > 1;
    for (int row = blockIdx.x * wpc + wid; row < a.R; row += gridDim.x * wpc) {
        const T* zr = static_cast<const T*>(a.logits) + (int64_t)row * a.ld;
        float z[NE], b[NE];
#pragma unroll
        for (int i = 0; i < NE; ++i) {   // every load first
            const int e = lane + 32 * i;
            z[i] = e < a.E ? ld_logit(zr + e) : -INFINITY;
            b[i] = a.bias && e < a.E ? __ldg(a.bias + e) : 0.0f;
        }
        // scores (fast exponential and quotient: the error bounds below)
        float zmax = -INFINITY, inv = 0.0f;
        float v[NE];
        // |error| of score + bias: a sigmoid's is s(1 - s) times the relative error of
        // e^-z (2^-22 + |z| 2^-23.4) plus the quotient's 2^-23, under 3e-7; a softmax
        // score's is its own size times the errors of its exponential, of the sum of E and
        // of the quotient, under 2e-6 of the row's largest score
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
        } else {
#pragma unroll
            for (int i = 0; i < NE; ++i) v[i] = 0.0f;   // the logits decide
        }
        uint32_t key[NE];
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            z[i] += 0.0f;   // -0 -> +0
            const bool masked = z[i] == -INFINITY || z[i] != z[i];
            v[i] = masked ? -INFINITY : v[i] + b[i];
            key[i] = masked ? (z[i] != z[i] ? 0u : kMaskKey) : order_key(a.bias ? v[i] : z[i]);
        }
        bool unsure = false;
        uint32_t valid = 0;
        if (G > 1) {
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int e = lane + 32 * i;
                if (e < a.E) {
                    const int g = (int)(((uint32_t)e * a.ginv) >> 20);
                    keys[e + g * L] = top2 ? max(order_key(v[i]), kMaskKey) : max(key[i], kMaskKey);
                }
            }
            __syncwarp();
            const int g = lane / L, l = lane - g * L;
            uint32_t t1 = 0, t2 = 0;
            if (g < G)
                for (int r = l; r < a.gs; r += L) {
                    const uint32_t x = keys[g * (a.gs + L) + r];
                    t2 = max(t2, min(t1, x));
                    t1 = max(t1, x);
                }
            __syncwarp();
            for (int o = L >> 1; o >= 1; o >>= 1) {
                const uint32_t u1 = __shfl_xor_sync(kAll, t1, o), u2 = __shfl_xor_sync(kAll, t2, o);
                t2 = max(max(t2, u2), min(t1, u1));
                t1 = max(t1, u1);
            }
            if (top2 && t2 > kMaskKey) t1 = order_key(key_value(t1) + key_value(t2));
            int rank = 0;
            for (int h = 0; h < G; ++h) {
                const uint32_t x = __shfl_sync(kAll, t1, h * L);
                rank += x > t1 || (x == t1 && h < g);
            }
            const bool lead = g < G && l == 0;
            const uint32_t taken = __ballot_sync(kAll, lead && rank < a.rule.top_groups);
            if ((top2 || a.bias) && a.rule.top_groups < G) {
                const int in = __ffs(__ballot_sync(kAll, lead && rank == a.rule.top_groups - 1)) - 1;
                const int out = __ffs(__ballot_sync(kAll, lead && rank == a.rule.top_groups)) - 1;
                const float x = key_value(__shfl_sync(kAll, t1, in)), y = key_value(__shfl_sync(kAll, t1, out));
                // a sum of two keys: twice the error, and its own rounding
                if (y > -INFINITY) unsure = !(x - y > 2.0f * tol + 4e-7f * (fabsf(x) + fabsf(y)));
            }
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int e = lane + 32 * i;
                const int h = (int)(((uint32_t)e * a.ginv) >> 20);
                if (e < a.E && ((taken >> (h * L)) & 1u)) valid |= 1u << i;
            }
        } else {
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (lane + 32 * i < a.E) valid |= 1u << i;
        }
        // the k largest, as warp_topk takes them; with a bias one more, and neighbours compared
        unsigned long long c[NE];
#pragma unroll
        for (int i = 0; i < NE; ++i)
            c[i] = ((valid >> i) & 1u) ? (unsigned long long)key[i] << 32 | (uint32_t)~(lane + 32 * i) : 0ull;
        lane_sort_desc<NE>(c);
        int my_id = 0;
        float prev = 0.0f;
        for (int j = 0; j < a.k + (a.bias ? 1 : 0); ++j) {
            const uint32_t hk = (uint32_t)(c[0] >> 32), hl = (uint32_t)c[0];
            const uint32_t mk = __reduce_max_sync(kAll, hk);
            if (a.bias) {
                const float x = key_value(mk);
                if (j > 0 && mk > kMaskKey && !(prev - x > tol + 2e-7f * (fabsf(prev) + fabsf(x))))
                    unsure = true;
                prev = x;
            }
            if (j == a.k) break;
            const uint32_t ml = __reduce_max_sync(kAll, hk == mk ? hl : 0u);
            const bool win = c[0] != 0ull && hk == mk && hl == ml;
#pragma unroll
            for (int i = 0; i + 1 < NE; ++i) c[i] = win ? c[i + 1] : c[i];
            c[NE - 1] = win ? 0ull : c[NE - 1];
            if (lane == j) my_id = (int)~ml;
        }
        if (unsure) my_id = route_exact<T>(a, row, lane);   // the same in every lane
        // weights from the unbiased scores of the chosen
        float s = 0.0f;
        if (lane < a.k) {
            const float zj = ld_logit(zr + my_id);
            if (zj == -INFINITY || zj != zj) s = 0.0f;
            else if (sig) s = __fdiv_rn(1.0f, 1.0f + expf(-zj));
            else s = zj == zmax ? inv : expf(zj - zmax) * inv;
        }
        float w = s;
        if (a.rule.renormalize) {
            const float sum = warp_sum(s);
            w = sum > 0.0f ? __fdiv_rn(s, sum) : 0.0f;
        }
        if (lane < a.k) {
            const int64_t o = (int64_t)row * a.k + lane;
            a.topk_idx[o] = my_id;
            a.topk_w[o] = w * a.rule.scale;
            if (a.topk_score) a.topk_score[o] = s;
        }
    }
}

template <typename T>
static cudaError_t launch_t(const RouteScoredArgs& a, int num_sms, cudaStream_t st) {
    // one warp per CTA until every SM has some, then up to eight
    int wpc = a.R / num_sms;
    wpc = wpc < 1 ? 1 : wpc > 8 ? 8 : wpc;
    int64_t grid = ((int64_t)a.R + wpc - 1) / wpc;
    if (grid > (int64_t)num_sms * (64 / wpc)) grid = (int64_t)num_sms * (64 / wpc);
    const size_t smem = a.rule.n_groups > 1 ? sizeof(uint32_t) * wpc * (a.E + 32) : 0;
    const int ne = (a.E + 31) / 32;
    auto k = ne <= 1 ? k_route_scored<T, 1> : ne <= 2 ? k_route_scored<T, 2>
           : ne <= 4 ? k_route_scored<T, 4> : ne <= 8 ? k_route_scored<T, 8>
           : ne <= 16 ? k_route_scored<T, 16> : k_route_scored<T, 32>;
    return launch_kernel(k, dim3((unsigned)grid), dim3(32 * wpc), smem, st, a);
}

cudaError_t launch_route_scored(const RouteScoredArgs& a, int dtype, int num_sms, cudaStream_t st) {
    if (dtype == MOE_BF16) return launch_t<__nv_bfloat16>(a, num_sms, st);
    if (dtype == MOE_F16) return launch_t<__half>(a, num_sms, st);
    return launch_t<float>(a, num_sms, st);
}

}  // namespace moe
