// Host side of the calls that need no plan: moe_route_scored, the e4m3 and int8
// quantising and products, and moe_add_rmsnorm.  Arguments are checked here, before
// anything is launched.
#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <cmath>

#include "fp8.cuh"
#include "route_scored.cuh"
#include "rows8.cuh"

using namespace moe;

namespace {

moe_status fail(moe_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
moe_status fail(moe_status s, const char* fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return set_error(s, buf);
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

size_t dtype_size(int dt) { return dt == MOE_F32 ? 4 : 2; }

moe_status check_dtype(int dt) {
    if (dt != MOE_BF16 && dt != MOE_F16 && dt != MOE_F32)
        return fail(MOE_ERR_UNSUPPORTED, "dtype=%d: bf16, fp16 or fp32", dt);
    return MOE_OK;
}

// SMs of the current device, looked up once per device; with `gemm` the GEMM
// kernels' attributes are set there too.  A device's entry holds what is done:
// 0 nothing, else the SM count, plus kAttr once the attributes are set.
constexpr int kMaxDevices = 64, kAttr = 1 << 20;
std::atomic<int> g_device[kMaxDevices];

moe_status device_ready(bool gemm, int* sms) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev < 0 || dev >= kMaxDevices)) e = cudaErrorInvalidDevice;
    int have = e == cudaSuccess ? g_device[dev].load(std::memory_order_acquire) : 0;
    if (e == cudaSuccess && !(have & (kAttr - 1))) {
        int n = 0;
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        have |= n;
        if (e == cudaSuccess) g_device[dev].fetch_or(n, std::memory_order_release);
    }
    if (e == cudaSuccess && gemm && !(have & kAttr)) {
        e = fp8_gemm_set_attributes();
        if (e == cudaSuccess) g_device[dev].fetch_or(kAttr, std::memory_order_release);
    }
    *sms = have & (kAttr - 1);
    return e == cudaSuccess ? MOE_OK : fail(MOE_ERR_CUDA, "device query: %s", cudaGetErrorString(e));
}

// CTA pairs of k_i8_tiles that are resident at once on the current device, looked up once per
// device, with the kernel's attributes.
std::atomic<int> g_pairs[kMaxDevices];

moe_status pairs_ready(int sms, int* clusters) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);   // device_ready has checked its range
    if (e == cudaSuccess && !(*clusters = g_pairs[dev].load(std::memory_order_acquire))) {
        e = i8_tiles_set_attributes(sms, clusters);
        if (e == cudaSuccess) g_pairs[dev].store(*clusters, std::memory_order_release);
    }
    return e == cudaSuccess ? MOE_OK : fail(MOE_ERR_CUDA, "device query: %s", cudaGetErrorString(e));
}

std::atomic<uint64_t> g_i8_wait_ns{0};   // moe_i8_gemm_set_wait_limit

moe_status launched(cudaError_t e, const char* what) {
    if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    return set_error(MOE_OK, "");
}

constexpr int64_t kMaxRows = (int64_t)1 << 30;

// Workspace of moe_fp8_gemm: the status counters.
constexpr size_t kGemmWorkspace = 1024;

}  // namespace

extern "C" {

moe_status moe_route_scored(const moe_route_rule* rule, const void* logits, moe_dtype dtype,
                            int64_t row_stride, int32_t R, int32_t E, int32_t k,
                            const float* select_bias, int32_t* topk_idx, float* topk_w,
                            float* topk_score, moe_stream_t stream) {
    if (!rule) return fail(MOE_ERR_INVALID_ARG, "rule is NULL");
    moe_status s = check_dtype(dtype);
    if (s != MOE_OK) return s;
    if (R < 0 || R > kMaxRows) return fail(MOE_ERR_INVALID_ARG, "R=%d outside [0, 2^30]", R);
    if (E < 1 || E > kMaxExperts) return fail(MOE_ERR_UNSUPPORTED, "E=%d must be in [1, %d]", E, kMaxExperts);
    if (k < 1 || k > 32) return fail(MOE_ERR_UNSUPPORTED, "k=%d must be in [1, 32]", k);
    if (rule->score != MOE_SCORE_SOFTMAX && rule->score != MOE_SCORE_SIGMOID)
        return fail(MOE_ERR_INVALID_ARG, "score=%d: softmax or sigmoid", rule->score);
    if (rule->group_score != MOE_GROUP_MAX && rule->group_score != MOE_GROUP_TOP2)
        return fail(MOE_ERR_INVALID_ARG, "group_score=%d: max or top2", rule->group_score);
    if (rule->n_groups < 1 || rule->n_groups > 32 || E % rule->n_groups)
        return fail(MOE_ERR_UNSUPPORTED, "n_groups=%d must be in [1, 32] and divide E=%d", rule->n_groups, E);
    if (rule->top_groups < 1 || rule->top_groups > rule->n_groups)
        return fail(MOE_ERR_INVALID_ARG, "top_groups=%d outside [1, n_groups=%d]", rule->top_groups, rule->n_groups);
    const int gs = E / rule->n_groups;
    if (k > rule->top_groups * gs)
        return fail(MOE_ERR_INVALID_ARG, "k=%d exceeds the %d experts of top_groups groups", k, rule->top_groups * gs);
    if (!std::isfinite(rule->scale)) return fail(MOE_ERR_INVALID_ARG, "scale is not finite");
    if (row_stride < E) return fail(MOE_ERR_INVALID_ARG, "row_stride=%lld is below E=%d", (long long)row_stride, E);
    if (R == 0) return set_error(MOE_OK, "");
    if (!logits || !aligned(logits, dtype_size(dtype)))
        return fail(MOE_ERR_INVALID_ARG, "logits NULL or misaligned");
    if (select_bias && !aligned(select_bias, 4)) return fail(MOE_ERR_INVALID_ARG, "select_bias misaligned");
    if (!topk_idx || !topk_w || !aligned(topk_idx, 4) || !aligned(topk_w, 4) ||
        (topk_score && !aligned(topk_score, 4)))
        return fail(MOE_ERR_INVALID_ARG, "topk_idx/topk_w NULL, or an output misaligned");
    int sms = 0;
    if ((s = device_ready(false, &sms)) != MOE_OK) return s;
    RouteScoredArgs a{logits, row_stride, R, E, k, select_bias, *rule, gs,
                      (uint32_t)(((1u << 20) + gs - 1) / gs), topk_idx, topk_w, topk_score};
    return launched(launch_route_scored(a, dtype, sms, reinterpret_cast<cudaStream_t>(stream)),
                    "route_scored launch");
}

moe_status moe_fp8_quantize(const void* x, moe_dtype dtype, int64_t row_stride, int32_t R,
                            int32_t K, void* codes, float* scales, moe_stream_t stream) {
    moe_status s = check_dtype(dtype);
    if (s != MOE_OK) return s;
    if (R < 0 || R > kMaxRows) return fail(MOE_ERR_INVALID_ARG, "R=%d outside [0, 2^30]", R);
    if (K < 1 || K > kMaxRows) return fail(MOE_ERR_INVALID_ARG, "K=%d outside [1, 2^30]", K);
    if (row_stride < K) return fail(MOE_ERR_INVALID_ARG, "row_stride=%lld is below K=%d", (long long)row_stride, K);
    if (R == 0) return set_error(MOE_OK, "");
    if (!x || !aligned(x, dtype_size(dtype))) return fail(MOE_ERR_INVALID_ARG, "x NULL or misaligned");
    if (!codes || !scales || !aligned(scales, 4))
        return fail(MOE_ERR_INVALID_ARG, "codes/scales NULL or misaligned");
    int sms = 0;
    if ((s = device_ready(false, &sms)) != MOE_OK) return s;
    Fp8QuantArgs a{x, row_stride, R, K, static_cast<uint8_t*>(codes), scales};
    return launched(launch_fp8_quantize(a, dtype, sms, reinterpret_cast<cudaStream_t>(stream)),
                    "quantise launch");
}

size_t moe_fp8_gemm_workspace_bytes(int32_t R, int32_t N, int32_t K) {
    if (R < 0 || R > kMaxRows || N < 1 || N > kMaxRows || K < 16 || K % 16 || K > kMaxRows) {
        fail(MOE_ERR_INVALID_ARG, "R=%d, N=%d, K=%d: R >= 0, N >= 1, K a positive multiple of 16", R, N, K);
        return 0;
    }
    return kGemmWorkspace;
}

moe_status moe_fp8_gemm(const void* xq, const float* xs, int32_t R, const void* wq,
                        const float* ws, int32_t N, int32_t K, void* y, moe_dtype dtype,
                        int64_t row_stride, void* workspace, size_t workspace_bytes,
                        moe_stream_t stream) {
    moe_status s = check_dtype(dtype);
    if (s != MOE_OK) return s;
    const size_t need = moe_fp8_gemm_workspace_bytes(R, N, K);
    if (!need) return K >= 16 && K % 16 ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARG;
    if (row_stride < N) return fail(MOE_ERR_INVALID_ARG, "row_stride=%lld is below N=%d", (long long)row_stride, N);
    if (R == 0) return set_error(MOE_OK, "");
    if (!xq || !wq || !aligned(xq, 16) || !aligned(wq, 16))
        return fail(MOE_ERR_INVALID_ARG, "xq/wq NULL or not 16-byte aligned");
    if (!xs || !ws || !aligned(xs, 4) || !aligned(ws, 4))
        return fail(MOE_ERR_INVALID_ARG, "xs/ws NULL or misaligned");
    const size_t es = dtype_size(dtype);
    if (!y || !aligned(y, es)) return fail(MOE_ERR_INVALID_ARG, "y NULL or misaligned");
    if (!workspace || !aligned(workspace, 256))
        return fail(MOE_ERR_WORKSPACE, "workspace NULL or not 256-byte aligned");
    if (workspace_bytes < need)
        return fail(MOE_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
    int sms = 0;
    if ((s = device_ready(true, &sms)) != MOE_OK) return s;
    if (fp8_rows_applies(R, N, K, sms)) {
        Fp8RowsArgs ra{static_cast<const uint8_t*>(xq), xs, static_cast<const uint8_t*>(wq), ws, R, N, K, y,
                       row_stride, dtype};
        return launched(launch_fp8_rows(ra, reinterpret_cast<cudaStream_t>(stream)), "gemm launch");
    }
    Fp8Maps m{};
    if (!encode_fp8(&m.w0, wq, (uint64_t)K, (uint64_t)N, 0) || !encode_fp8(&m.a0, xq, (uint64_t)K, (uint64_t)R, 0))
        return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed");
    m.w1 = m.s0 = m.s1 = m.w0;
    m.a1 = m.a0;
    Fp8GemmArgs a{};
    a.g.status = static_cast<uint32_t*>(workspace);
    a.xs = xs;
    a.sc_a = ws;
    a.R = R;
    a.N = N;
    a.K = K;
    a.y = y;
    a.ldy = row_stride;
    a.ydtype = dtype;
    a.y_vec = aligned(y, 16) && row_stride * (int64_t)es % 16 == 0;
    return launched(launch_fp8_gemm(kDense, m, a, sms, reinterpret_cast<cudaStream_t>(stream)),
                    "gemm launch");
}

moe_status moe_i8_quantize(const void* x, moe_dtype dtype, int64_t row_stride, int32_t R,
                           int32_t K, int8_t* codes, float* scales, moe_stream_t stream) {
    moe_status s = check_dtype(dtype);
    if (s != MOE_OK) return s;
    if (R < 0 || R > kMaxRows) return fail(MOE_ERR_INVALID_ARG, "R=%d outside [0, 2^30]", R);
    if (K < 1 || K > kMaxRows) return fail(MOE_ERR_INVALID_ARG, "K=%d outside [1, 2^30]", K);
    if (row_stride < K) return fail(MOE_ERR_INVALID_ARG, "row_stride=%lld is below K=%d", (long long)row_stride, K);
    if (R == 0) return set_error(MOE_OK, "");
    if (!x || !aligned(x, dtype_size(dtype))) return fail(MOE_ERR_INVALID_ARG, "x NULL or misaligned");
    if (!codes || !scales || !aligned(scales, 4))
        return fail(MOE_ERR_INVALID_ARG, "codes/scales NULL or misaligned");
    int sms = 0;
    if ((s = device_ready(false, &sms)) != MOE_OK) return s;
    RmsNormArgs a{};
    a.x = x;
    a.ldx = row_stride;
    a.R = R;
    a.H = K;
    a.codes = reinterpret_cast<uint8_t*>(codes);
    a.scales = scales;
    return launched(launch_rows8(kQuantI8, a, dtype, sms, reinterpret_cast<cudaStream_t>(stream)),
                    "quantise launch");
}

// The operand that is widened lies behind what a plan's workspace keeps between calls: a workspace
// may serve both.
constexpr size_t kWideOffset = kTokenEnd;

size_t moe_i8_gemm_workspace_bytes(int32_t R, int32_t N, int32_t K) {
    if (R < 0 || R > kMaxRows || N < 1 || N > kMaxRows || K < 16 || K % 16 || K > kI8MaxK) {
        fail(MOE_ERR_INVALID_ARG, "R=%d, N=%d, K=%d: R >= 0, N >= 1, K a positive multiple of 16 below 2^17", R, N, K);
        return 0;
    }
    return i8_rows_applies(R, N, K) ? kGemmWorkspace : kWideOffset + 2 * (size_t)(R < N ? R : N) * (size_t)K;
}

moe_status moe_i8_gemm_set_wait_limit(uint64_t limit_ns) {
    g_i8_wait_ns.store(limit_ns, std::memory_order_relaxed);
    return set_error(MOE_OK, "");
}

moe_status moe_i8_gemm(const int8_t* xq, const float* xs, int32_t R, const int8_t* wq,
                       const float* ws, int32_t N, int32_t K, void* y, moe_dtype dtype,
                       int64_t row_stride, void* workspace, size_t workspace_bytes,
                       moe_stream_t stream) {
    moe_status s = check_dtype(dtype);
    if (s != MOE_OK) return s;
    const size_t need = moe_i8_gemm_workspace_bytes(R, N, K);
    if (!need) return K >= 16 && (K % 16 || K > kI8MaxK) ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARG;
    if (row_stride < N) return fail(MOE_ERR_INVALID_ARG, "row_stride=%lld is below N=%d", (long long)row_stride, N);
    if (R == 0) return set_error(MOE_OK, "");
    if (!xq || !wq || !aligned(xq, 16) || !aligned(wq, 16))
        return fail(MOE_ERR_INVALID_ARG, "xq/wq NULL or not 16-byte aligned");
    if (!xs || !ws || !aligned(xs, 4) || !aligned(ws, 4))
        return fail(MOE_ERR_INVALID_ARG, "xs/ws NULL or misaligned");
    if (!y || !aligned(y, dtype_size(dtype))) return fail(MOE_ERR_INVALID_ARG, "y NULL or misaligned");
    if (!workspace || !aligned(workspace, 256))
        return fail(MOE_ERR_WORKSPACE, "workspace NULL or not 256-byte aligned");
    if (workspace_bytes < need)
        return fail(MOE_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
    I8GemmArgs a{xq, xs, wq, ws, R, N, K, y, row_stride, dtype, static_cast<uint32_t*>(workspace),
                 aligned(y, 32) && row_stride * (int64_t)dtype_size(dtype) % 32 == 0, i8_width(R, N, K),
                 g_i8_wait_ns.load(std::memory_order_relaxed)};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (i8_rows_applies(R, N, K)) return launched(launch_i8_rows(a, st), "gemm launch");
    int sms = 0, clusters = 0;
    if ((s = device_ready(false, &sms)) != MOE_OK || (s = pairs_ready(sms, &clusters)) != MOE_OK) return s;
    const bool swap = i8_swapped(R, N);
    void* wide = static_cast<uint8_t*>(workspace) + kWideOffset;
    CUtensorMap ma, mb;
    if (!encode_i8_tiles(&ma, &mb, swap ? xq : wq, wide, swap ? R : N, swap ? N : R, K, a.width))
        return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed");
    return launched(launch_i8_tiles(a, ma, mb, wide, sms, clusters, st), "gemm launch");
}

moe_status moe_add_rmsnorm(const void* x, moe_dtype dtype, int64_t x_stride, int32_t R,
                           int32_t H, const void* residual, moe_dtype residual_dtype,
                           int64_t residual_stride, void* total, int64_t total_stride,
                           const void* weight, moe_dtype weight_dtype, float eps, void* y,
                           int64_t y_stride, int32_t code_type, void* codes, float* scales,
                           moe_stream_t stream) {
    moe_status s = check_dtype(dtype);
    if (s != MOE_OK) return s;
    if (R < 0 || R > kMaxRows) return fail(MOE_ERR_INVALID_ARG, "R=%d outside [0, 2^30]", R);
    if (H < 1 || H > kMaxRows) return fail(MOE_ERR_INVALID_ARG, "H=%d outside [1, 2^30]", H);
    if (residual && residual_dtype != dtype && residual_dtype != MOE_F32)
        return fail(MOE_ERR_UNSUPPORTED, "residual_dtype=%d: that of x, or fp32", residual_dtype);
    if (weight && weight_dtype != dtype && weight_dtype != MOE_F32)
        return fail(MOE_ERR_UNSUPPORTED, "weight_dtype=%d: that of x, or fp32", weight_dtype);
    if (code_type != MOE_CODES_NONE && code_type != MOE_CODES_E4M3 && code_type != MOE_CODES_I8)
        return fail(MOE_ERR_UNSUPPORTED, "code_type=%d: none, e4m3 or int8", code_type);
    if (!(eps >= 0x1p-100f && eps <= 0x1p100f))
        return fail(MOE_ERR_INVALID_ARG, "eps=%g outside [2^-100, 2^100]", (double)eps);
    if (x_stride < H) return fail(MOE_ERR_INVALID_ARG, "x_stride=%lld is below H=%d", (long long)x_stride, H);
    if (residual && residual_stride < H)
        return fail(MOE_ERR_INVALID_ARG, "residual_stride=%lld is below H=%d", (long long)residual_stride, H);
    if (total && total_stride < H)
        return fail(MOE_ERR_INVALID_ARG, "total_stride=%lld is below H=%d", (long long)total_stride, H);
    if (y && y_stride < H) return fail(MOE_ERR_INVALID_ARG, "y_stride=%lld is below H=%d", (long long)y_stride, H);
    if (total && !residual) return fail(MOE_ERR_INVALID_ARG, "total without a residual");
    if (R == 0) return set_error(MOE_OK, "");   // a buffer of no rows may be NULL
    if ((code_type == MOE_CODES_NONE) != !codes || !codes != !scales)
        return fail(MOE_ERR_INVALID_ARG, "codes and scales go with a code_type, and it with them");
    if (!y && !codes) return fail(MOE_ERR_INVALID_ARG, "neither y nor codes");
    const size_t es = dtype_size(dtype), rs = dtype_size(residual_dtype);
    if (!x || !aligned(x, es)) return fail(MOE_ERR_INVALID_ARG, "x NULL or misaligned");
    if ((residual && !aligned(residual, rs)) || (total && !aligned(total, rs)))
        return fail(MOE_ERR_INVALID_ARG, "residual or total misaligned");
    if (weight && !aligned(weight, dtype_size(weight_dtype))) return fail(MOE_ERR_INVALID_ARG, "weight misaligned");
    if ((y && !aligned(y, es)) || (scales && !aligned(scales, 4)))
        return fail(MOE_ERR_INVALID_ARG, "y or scales misaligned");
    if (total && total == y) return fail(MOE_ERR_INVALID_ARG, "total and y are the same");
    if (total == residual && total && R > 1 && total_stride != residual_stride)
        return fail(MOE_ERR_INVALID_ARG, "total in the residual's place with another stride");
    if (total == x && total && (residual_dtype != dtype || (R > 1 && total_stride != x_stride)))
        return fail(MOE_ERR_INVALID_ARG, "total in x's place with another type or stride");
    if (y == x && y && R > 1 && y_stride != x_stride)
        return fail(MOE_ERR_INVALID_ARG, "y in x's place with another stride");
    int sms = 0;
    if ((s = device_ready(false, &sms)) != MOE_OK) return s;
    const bool f32 = dtype == MOE_F32;
    RmsNormArgs a{x, x_stride, residual, residual_stride, total, total_stride, weight,
                  !f32 && residual && residual_dtype == MOE_F32, !f32 && weight && weight_dtype == MOE_F32, R, H, eps,
                  1.0f / (float)H, y, y_stride, static_cast<uint8_t*>(codes), scales};
    const int what = code_type == MOE_CODES_E4M3 ? kNormE4m3 : code_type == MOE_CODES_I8 ? kNormI8 : kNormOnly;
    return launched(launch_rows8(what, a, dtype, sms, reinterpret_cast<cudaStream_t>(stream)), "rmsnorm launch");
}

}  // extern "C"
