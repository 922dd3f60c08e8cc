// The whole layer for a few rows (up to 8) in one kernel: router, top-k, gate/up,
// SwiGLU, down, weighted sum and shared expert (moe_token_pass); or all but the router
// (moe_token_forward).
//
//   z = x W_r^T + bias;  top-k, w = softmax over the chosen
//   y = S(x) + sum_j w_j E_j(x),   E(x) = W_down (silu(W_gate x) * (W_up x))
//
// A few rows touch a few experts, whose weights take HBM some microseconds: what a row
// of kernels costs between them is what there is to save.  One CTA per SM, launched
// cooperatively, goes through three steps with a grid barrier between them:
//   1  a warp per expert: its logits for all rows, in the order of route_common.cuh
//   2  every CTA: top-k of all rows (the same code as moe_block_route's, so the same
//      ids and weights), the list of the experts touched, and its share of gate/up
//   3  16 hidden outputs per CTA and turn: down, summed over all experts in registers, so
//      that nothing is staged or combined
// The weights are the M of mma.sync (16 rows), the rows of x its N: column r is row r in
// all of them, whoever it is routed to; what a column holds for an expert that its row
// did not choose is not read.  A gate/up unit is 8 gate and the 8 up rows of the same
// intermediate indices, so that one lane holds g and u of an index.  Four warps share a
// unit's K; all sixteen share the down step's experts and K.  K is permuted alike in both
// operands, so that a lane's are 16-byte loads.
//
// h lies in global memory between the steps: with bf16 weights as two bf16 parts
// (16 significant bits), with e4m3 ones in fp32, quantised by every reader with
// the formula of the other paths.
//
// Barriers: an array of one flag per CTA each, polled by a warp.  A CTA clears its flag
// of the second before it arrives at the first, and that of the first when it has
// passed the second, which every CTA then has reached; so the flags need no clearing by
// the host.  With the routing given there is one barrier: CTAs that have passed it set
// their second flag, and one CTA, beside its work, waits for all of those and clears the first
// array.  Every wait is bounded; a CTA that gives up counts MOE_STATUS_WAIT_TIMEOUT, clears its
// flags and leaves.
#include "route_common.cuh"
#include "token.cuh"

namespace moe {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kGroup = 4;                       // warps that share a gate/up unit
constexpr int kGroups = kWarps / kGroup;
constexpr uint32_t kArrived = 0x5EEDF1A6u;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr int kMaxPairs = kTokenRows * 32;      // k <= 32
constexpr int64_t kPrefetchBytes = 32 << 20;    // of the down weights, a quarter of L2

struct Smem {
    float part[2][kWarps][kTokenRows][17];      // partial sums (token, weight row)
    float wt[kMaxPairs][kTokenRows];            // weight of (listed expert, row)
    float w[kMaxPairs];                         // [R, k]
    int32_t idx[kMaxPairs];
    uint32_t mask[kMaxExperts];                 // rows of an expert
    int32_t list[kMaxPairs];                    // experts touched, ascending
    uint32_t lmask[kMaxPairs];                  // their rows
    int32_t first[kMaxPairs];                   // pairs before them
    uint32_t count[kWarps];
    uint32_t scratch[MOE_STATUS_WORDS];         // for status counts that another CTA makes
    uint32_t bad;                               // rows with a non-finite output
    int nl, ok;
};

// x in shared memory: rows far enough apart that a quarter-warp's 16-byte reads share no bank
template <bool FP8>
__host__ __device__ constexpr int x_stride(int H) { return FP8 ? H + 16 : 2 * H + 64; }
template <bool FP8>
__host__ __device__ constexpr int x_bytes(int H) {
    return kTokenRows * x_stride<FP8>(H) + (FP8 ? (H / kFp8Block) * kTokenRows * 4 : 0);
}

__device__ __forceinline__ uint4 ld_weights(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// What a lane holds of 16 weight rows and 128 of K: rows gi and gi + 8.  bf16: 16 bytes of
// each 32 of K (8 elements); e4m3: 32 bytes in a row.
template <bool FP8>
struct Tile {
    static constexpr int kN = FP8 ? 2 : 4;
    uint4 a[kN], b[kN];
};
// pa, pb: the rows' first element of these 128 of K for lane c; `left`: elements of K from
// there on to the end (zeros past it)
template <bool FP8>
__device__ __forceinline__ void load_tile(Tile<FP8>& t, const uint8_t* pa, const uint8_t* pb, int c, int left) {
#pragma unroll
    for (int i = 0; i < Tile<FP8>::kN; ++i) {
        const int at = FP8 ? 32 * c + 16 * i : 64 * i + 16 * c;   // bytes
        const bool in = FP8 ? at < left : at < 2 * left;
        t.a[i] = in ? ld_weights(pa + at) : make_uint4(0, 0, 0, 0);
        t.b[i] = in ? ld_weights(pb + at) : make_uint4(0, 0, 0, 0);
    }
}
template <bool FP8>
__device__ __forceinline__ void tile_mma(float (&d)[4], const Tile<FP8>& t, const uint4 (&x)[Tile<FP8>::kN]) {
#pragma unroll
    for (int i = 0; i < Tile<FP8>::kN; ++i) {
        if (FP8) {
            mma_e4m3(d, t.a[i].x, t.b[i].x, t.a[i].y, t.b[i].y, x[i].x, x[i].y);
            mma_e4m3(d, t.a[i].z, t.b[i].z, t.a[i].w, t.b[i].w, x[i].z, x[i].w);
        } else {
            mma_bf16(d, t.a[i].x, t.b[i].x, t.a[i].y, t.b[i].y, x[i].x, x[i].y);
            mma_bf16(d, t.a[i].z, t.b[i].z, t.a[i].w, t.b[i].w, x[i].z, x[i].w);
        }
    }
}

__device__ __forceinline__ uint32_t ld_flag(const uint32_t* p) {
    uint32_t v;
    asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void st_flag(uint32_t* p, uint32_t v) {
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// Wait, as one warp, until every CTA's flag is set; false: gave up.
__device__ __forceinline__ bool wait_flags(const uint32_t* flags, int n, uint64_t limit_ns, int lane) {
    const uint64_t t0 = globaltimer_ns();
    for (int i = lane;; ) {
        while (i < n && ld_flag(flags + i) == kArrived) i += 32;
        if (__all_sync(0xffffffffu, i >= n)) break;
        if (__any_sync(0xffffffffu, globaltimer_ns() - t0 > limit_ns)) return false;
    }
    __threadfence();
    return true;
}

// A grid barrier on `flags`; the whole CTA calls it.  False: gave up, the same in every thread.
__device__ __forceinline__ bool grid_barrier(uint32_t* flags, const TokenArgs& a, Smem& s) {
    __syncthreads();
    if (threadIdx.x < 32) {
        if (threadIdx.x == 0) {
            __threadfence();
            st_flag(flags + blockIdx.x, kArrived);
        }
        __syncwarp();
        const bool ok = wait_flags(flags, gridDim.x, a.wait_ns ? a.wait_ns : kWaitLimitNs, threadIdx.x);
        if (threadIdx.x == 0) s.ok = ok;
    }
    __syncthreads();
    return s.ok;
}

__device__ __forceinline__ float warp_sum(float v) {   // the xor butterfly of route_common.cuh
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Logits of one expert for all rows, one warp.
__device__ __forceinline__ void expert_logits(const TokenArgs& a, int e, int lane) {
    constexpr int kS = 4;   // stripes of 256 at a time
    float acc[kTokenRows];
#pragma unroll
    for (int r = 0; r < kTokenRows; ++r) acc[r] = 0.0f;
    const __nv_bfloat16* w = a.wr + (int64_t)e * a.H + lane * 8;
    for (int s0 = 0; s0 < a.H; s0 += 256 * kS) {
        uint4 wv[kS];
#pragma unroll
        for (int i = 0; i < kS; ++i)
            wv[i] = s0 + 256 * i < a.H ? ld_weights(w + s0 + 256 * i) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < kTokenRows; ++r) {
            if (r >= a.R) break;
            const __nv_bfloat16* xr = a.x + (int64_t)r * a.H + lane * 8 + s0;
#pragma unroll
            for (int i = 0; i < kS; ++i)
                if (s0 + 256 * i < a.H) acc[r] = dot8_bf16(__ldg(reinterpret_cast<const uint4*>(xr + 256 * i)), wv[i], acc[r]);
        }
    }
#pragma unroll
    for (int r = 0; r < kTokenRows; ++r) {
        if (r >= a.R) break;
        const float z = warp_sum(acc[r]);
        if (lane == 0) a.logits[(int64_t)r * a.E + e] = z;
    }
}

// x into shared memory: as it is, or as e4m3 codes and scales per block of 128 (fp8.cuh).
template <bool FP8>
__device__ __forceinline__ void stage_x(const TokenArgs& a, uint8_t* sx) {
    const int per_row = a.H / 8;
    float* xs = reinterpret_cast<float*>(sx + kTokenRows * x_stride<FP8>(a.H));   // [H / 128][8]
    for (int i = threadIdx.x; i < a.R * per_row; i += kThreads) {   // H % 256 == 0: whole warps
        const int r = i / per_row, c = i - r * per_row;
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(a.x + (int64_t)r * a.H) + c);
        if (!FP8) {
            *reinterpret_cast<uint4*>(sx + r * x_stride<FP8>(a.H) + 16 * c) = v;
            continue;
        }
        float f[8];
        bf16x8(v, f);
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(f[j]) & 0x7FFFFFFFu);
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        m = fp8_amax_bits(m);
        const float am = __uint_as_float(m), d = am * (1.0f / 512.0f);
        uint32_t q[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
            q[j] = fp8_pair(__fdiv_rn(0.875f * f[4 * j], d), __fdiv_rn(0.875f * f[4 * j + 1], d)) |
                   fp8_pair(__fdiv_rn(0.875f * f[4 * j + 2], d), __fdiv_rn(0.875f * f[4 * j + 3], d)) << 16;
        *reinterpret_cast<uint2*>(sx + r * x_stride<FP8>(a.H) + 8 * c) = make_uint2(q[0], q[1]);
        if ((c & 15) == 0) xs[(c >> 4) * kTokenRows + r] = __fdiv_rn(am, 448.0f);
    }
}

}  // namespace

template <bool FP8>
__global__ void __launch_bounds__(kThreads, 1) k_token(TokenArgs a) {
    extern __shared__ __align__(128) uint8_t base[];
    Smem& s = *reinterpret_cast<Smem*>(base);
    uint8_t* sx = base + (sizeof(Smem) + 127) / 128 * 128;
    const float* xs = reinterpret_cast<const float*>(sx + kTokenRows * x_stride<FP8>(a.H));
    constexpr int kES = FP8 ? 1 : 2;   // bytes per weight
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gi = lane >> 2, c = lane & 3;
    const int G = gridDim.x, cta = blockIdx.x;
    uint32_t* flags1 = a.flags;
    uint32_t* flags2 = a.flags + kTokenMaxCtas;
    if (tid == 0) st_flag(flags2 + cta, 0);   // released before this CTA's arrival below
    const uint8_t *wg = static_cast<const uint8_t*>(a.wg), *wu = static_cast<const uint8_t*>(a.wu),
                  *wd = static_cast<const uint8_t*>(a.wd), *sg = static_cast<const uint8_t*>(a.sg),
                  *su = static_cast<const uint8_t*>(a.su), *sd = static_cast<const uint8_t*>(a.sd);
    const int utiles = a.I / 8, stiles = a.Is / 8, dtiles = a.H / 16;
    auto give_up = [&]() {   // the whole CTA
        if (tid == 0) {
            status_add(a.status, MOE_STATUS_WAIT_TIMEOUT, 1);
            st_flag(flags1 + cta, 0);
        }
    };

    // ---- step 1: logits; the shared expert's weights, which do not depend on them, to L2
    if (tid == kThreads - 1) {
        const uint32_t gb = 8u * a.H * kES, db = 16u * a.Is * kES;
        for (int t = cta; t < stiles; t += G) {
            prefetch_l2(sg + (int64_t)t * gb, gb);
            prefetch_l2(su + (int64_t)t * gb, gb);
        }
        for (int t = cta; t < dtiles; t += G) prefetch_l2(sd + (int64_t)t * db, db);
    }
    if (!a.given)
        for (int e = cta + G * warp; e < a.E; e += G * kWarps) expert_logits(a, e, lane);
    stage_x<FP8>(a, sx);
    for (int i = tid; i < a.E; i += kThreads) s.mask[i] = 0;
    if (tid < MOE_STATUS_WORDS) s.scratch[tid] = 0;
    if (tid == 0) s.bad = 0;
    if (!a.given && !grid_barrier(flags1, a, s)) {
        give_up();
        return;
    }

    // ---- step 2: the experts of each row and the list of all of them
    const int np = a.R * a.k;
    if (!a.given) {
        if (warp < a.R) {
            RouteArgs ra{};
            ra.bias = a.bias;
            ra.R = a.R;
            ra.E = a.E;
            ra.k = a.k;
            ra.nb = 1;
            ra.logits = a.logits;
            ra.topk_idx = s.idx;
            ra.topk_w = s.w;
            ra.status = cta == 0 ? a.status : s.scratch;
            route_topk(ra, warp, warp + 1, lane);
        }
        __syncthreads();
        if (cta == 0)
            for (int i = tid; i < np; i += kThreads) {
                a.topk_idx[i] = s.idx[i];
                a.topk_w[i] = s.w[i];
            }
    } else {
        for (int i = tid; i < np; i += kThreads) {
            s.idx[i] = __ldg(a.topk_idx + i);
            s.w[i] = __ldg(a.topk_w + i);
        }
        __syncthreads();
    }
    for (int i = tid; i < np; i += kThreads) {
        const int e = s.idx[i];
        if (e >= 0 && e < a.E) atomicOr(&s.mask[e], 1u << (i / a.k));
        else if (cta == 0) status_add(a.status, MOE_STATUS_BAD_EXPERT_ID, 1);
    }
    __syncthreads();
    // experts in ascending order: two per thread (E <= 1024)
    {
        const uint32_t m0 = 2 * tid < a.E ? s.mask[2 * tid] : 0u, m1 = 2 * tid + 1 < a.E ? s.mask[2 * tid + 1] : 0u;
        // low half: experts, high half: pairs
        const uint32_t mine = (m0 != 0) + (m1 != 0) + ((__popc(m0) + __popc(m1)) << 16);
        uint32_t at = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t t = __shfl_up_sync(0xffffffffu, at, o);
            if (lane >= o) at += t;
        }
        if (lane == 31) s.count[warp] = at;
        __syncthreads();
        uint32_t total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) at += s.count[w];
            total += s.count[w];
        }
        at -= mine;
        if (tid == 0) s.nl = total & 0xFFFF;
        if (m0) {
            const int l = at & 0xFFFF;
            s.list[l] = 2 * tid;
            s.lmask[l] = m0;
            s.first[l] = at >> 16;
            at += 1 + (__popc(m0) << 16);
        }
        if (m1) {
            const int l = at & 0xFFFF;
            s.list[l] = 2 * tid + 1;
            s.lmask[l] = m1;
            s.first[l] = at >> 16;
        }
    }
    __syncthreads();
    const int nl = s.nl;
    for (int i = tid; i < nl * kTokenRows; i += kThreads) {   // weights in slot order
        const int l = i / kTokenRows, r = i % kTokenRows;
        float w = 0.0f;
        if (r < a.R)
            for (int j = 0; j < a.k; ++j)
                if (s.idx[r * a.k + j] == s.list[l]) w += s.w[r * a.k + j];
        s.wt[l][r] = w;
    }
    if (tid < a.R && cta == 0) {   // rows left with the shared expert alone
        bool any = false;
        for (int j = 0; j < a.k; ++j) any |= s.idx[tid * a.k + j] >= 0 && s.idx[tid * a.k + j] < a.E;
        if (!any) status_add(a.status, MOE_STATUS_EMPTY_ROWS, 1);
    }
    // this CTA's part of the down weights, to L2 while gate/up runs
    if (tid == kThreads - 1) {
        const uint32_t db = 16u * a.I * kES;
        int64_t left = kPrefetchBytes / G;
        for (int t = cta; t < dtiles; t += G)
            for (int l = 0; l < nl && (left -= db) >= 0; ++l)
                prefetch_l2(wd + ((int64_t)s.list[l] * a.H + 16 * t) * a.I * kES, db);
    }

    // ---- gate/up
    __nv_bfloat16* hb = static_cast<__nv_bfloat16*>(a.h);   // bf16: hi | lo, then the shared expert's
    float* hf = static_cast<float*>(a.h);                   // e4m3: fp32
    const int64_t hpart = (int64_t)np * a.I, spart = (int64_t)a.R * a.Is;
    {
        const int group = warp / kGroup, gw = warp % kGroup;
        const int nunits = stiles + nl * utiles;
        const int kblocks = a.H / 128;   // of which this warp takes gw, gw + 4, ...
        const int steps = (kblocks - gw + kGroup - 1) / kGroup;
        const int ustep = G * kGroups;
        // the unit's rows for this lane; a unit past the last has none
        struct Rows { const uint8_t *g, *u; const float *cg, *cu; };
        auto rows_of = [&](int u) {
            Rows q{};
            const bool sh = u < stiles;
            const int l = sh ? 0 : (u - stiles) / utiles;
            const int t = sh ? u : (u - stiles) - l * utiles;
            const int64_t e = sh ? 0 : s.list[l];
            const int ld = sh ? a.Is : a.I;
            const int64_t o = ((e * ld + 8 * t + gi) * a.H + gw * 128) * kES;
            q.g = (sh ? sg : wg) + o;
            q.u = (sh ? su : wu) + o;
            if (FP8) {
                const int64_t so = (e * fp8_blocks(ld) + t / 16) * kblocks + gw;
                q.cg = (sh ? a.csg : a.cg) + so;
                q.cu = (sh ? a.csu : a.cu) + so;
            }
            return q;
        };
        // the tiles of all units of this warp, one ahead
        int u = cta + G * group;
        Tile<FP8> t[2];
        float fg[2] = {0.0f, 0.0f}, fu[2] = {0.0f, 0.0f};
        Rows q{};
        auto load = [&](const Rows& p, int step, int b) {
            load_tile<FP8>(t[b], p.g + (int64_t)step * kGroup * 128 * kES, p.u + (int64_t)step * kGroup * 128 * kES, c, 128);
            if (FP8) {
                fg[b] = __ldg(p.cg + step * kGroup);
                fu[b] = __ldg(p.cu + step * kGroup);
            }
        };
        if (u < nunits) q = rows_of(u);
        bool have = u < nunits && steps > 0;
        if (have) load(q, 0, 0);
        int pb = 0;
        while (u < nunits) {
            float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            Rows qn{};
            const int un = u + ustep;
            if (un < nunits) qn = rows_of(un);
            for (int st = 0; st < steps; st += 2) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    if (st + b < steps) {
                        // the next tile: of this unit, or the first of the next
                        if (st + b + 1 < steps) load(q, st + b + 1, b ^ 1);
                        else if (un < nunits && b == 1) load(qn, 0, 0);
                        const int kb = gw + (st + b) * kGroup;
                        uint4 x[Tile<FP8>::kN];
                        const uint8_t* xr = sx + gi * x_stride<FP8>(a.H) + kb * 128 * kES;
#pragma unroll
                        for (int i = 0; i < Tile<FP8>::kN; ++i)
                            x[i] = gi < a.R ? *reinterpret_cast<const uint4*>(xr + (FP8 ? 32 * c + 16 * i : 64 * i + 16 * c))
                                            : make_uint4(0, 0, 0, 0);
                        if (FP8) {
                            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                            tile_mma<FP8>(d, t[b], x);
                            const float x0 = xs[kb * kTokenRows + 2 * c], x1 = xs[kb * kTokenRows + 2 * c + 1];
                            acc[0] = fmaf(x0 * fg[b], d[0], acc[0]);
                            acc[1] = fmaf(x1 * fg[b], d[1], acc[1]);
                            acc[2] = fmaf(x0 * fu[b], d[2], acc[2]);
                            acc[3] = fmaf(x1 * fu[b], d[3], acc[3]);
                        } else {
                            tile_mma<FP8>(acc, t[b], x);
                        }
                    }
                }
            }
            // an odd number of steps leaves the next unit's first tile to load here
            if (un < nunits && (steps & 1)) load(qn, 0, 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) s.part[pb][warp][2 * c + (j & 1)][gi + 8 * (j >> 1)] = acc[j];
            asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(32 * kGroup) : "memory");
            const int t8 = (tid & (32 * kGroup - 1)) >> 3, i = tid & 7;   // row, index
            const bool sh = u < stiles;
            const int l = sh ? 0 : (u - stiles) / utiles, tt = sh ? u : (u - stiles) - l * utiles;
            const uint32_t m = sh ? (1u << a.R) - 1 : s.lmask[l];
            if (t8 < kTokenRows && ((m >> t8) & 1u)) {
                float g = 0.0f, v = 0.0f;
#pragma unroll
                for (int w = 0; w < kGroup; ++w) {
                    g += s.part[pb][group * kGroup + w][t8][i];
                    v += s.part[pb][group * kGroup + w][t8][8 + i];
                }
                const float h = silu_fast(g) * v;
                const int p = sh ? t8 : s.first[l] + __popc(m & ((1u << t8) - 1));
                const int64_t at = (int64_t)p * (sh ? a.Is : a.I) + 8 * tt + i;
                if (FP8) {
                    hf[(sh ? hpart : 0) + at] = h;
                } else {
                    const __nv_bfloat16 hi = __float2bfloat16_rn(h);
                    __nv_bfloat16* o = hb + (sh ? 2 * hpart : 0) + at;
                    o[0] = hi;
                    o[sh ? spart : hpart] = __float2bfloat16_rn(h - __bfloat162float(hi));
                }
            }
            pb ^= 1;   // read before the barrier of the unit after the next, written after that of the next
            u = un;
            q = qn;
        }
    }

    if (!grid_barrier(a.given ? flags1 : flags2, a, s)) {
        give_up();
        return;
    }
    if (tid == 0) {
        if (a.given) st_flag(flags2 + cta, kArrived);   // passed
        else st_flag(flags1 + cta, 0);
    }

    // ---- step 3: down
    const int kb_r = fp8_blocks(a.I), kb_s = fp8_blocks(a.Is);   // blocks of 128 of an expert's K
    const int items = kb_s + nl * kb_r;
    for (int t = cta; t < dtiles; t += G) {
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int it = warp; it < items; it += kWarps) {
            const bool sh = it < kb_s;
            const int l = sh ? 0 : (it - kb_s) / kb_r;
            const int kb = sh ? it : (it - kb_s) - l * kb_r;
            const int K = sh ? a.Is : a.I;
            const int64_t e = sh ? 0 : s.list[l];
            const uint8_t* w = (sh ? sd : wd) + ((e * a.H + 16 * t + gi) * K + kb * 128) * kES;
            Tile<FP8> tl;
            load_tile<FP8>(tl, w, w + (int64_t)8 * K * kES, c, K - kb * 128);
            const uint32_t m = sh ? (1u << a.R) - 1 : s.lmask[l];
            const bool on = (m >> gi) & 1u;
            const int p = sh ? gi : s.first[l] + __popc(m & ((1u << gi) - 1));
            const int64_t at = (int64_t)p * K + kb * 128;
            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            float f0 = sh ? 1.0f : s.wt[l][2 * c], f1 = sh ? 1.0f : s.wt[l][2 * c + 1];
            if constexpr (FP8) {
                const float sw = __ldg((sh ? a.csd : a.cd) + (e * (a.H / kFp8Block) + t / 8) * (sh ? kb_s : kb_r) + kb);
                const float* ph = hf + (sh ? hpart : 0) + at + 32 * c;
                const bool in = on && kb * 128 + 32 * c < K;   // K % 64 == 0: all 32 values or none
                float4 v[8];
                uint32_t mx = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[i] = in ? __ldcg(reinterpret_cast<const float4*>(ph) + i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    mx = max(mx, max(max(__float_as_uint(v[i].x) & 0x7FFFFFFFu, __float_as_uint(v[i].y) & 0x7FFFFFFFu),
                                     max(__float_as_uint(v[i].z) & 0x7FFFFFFFu, __float_as_uint(v[i].w) & 0x7FFFFFFFu)));
                }
                mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float bm = __uint_as_float(fp8_amax_bits(mx));
                const float inv = __fdiv_rn(448.0f, bm), scale = __fdiv_rn(bm, 448.0f);
                uint32_t q[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    q[i] = fp8_pair(v[i].x * inv, v[i].y * inv) | fp8_pair(v[i].z * inv, v[i].w * inv) << 16;
                const uint4 x[2] = {make_uint4(q[0], q[1], q[2], q[3]), make_uint4(q[4], q[5], q[6], q[7])};
                tile_mma<FP8>(d, tl, x);
                f0 *= __shfl_sync(0xffffffffu, scale, 8 * c) * sw;   // row r's scale is in lanes 4 r ..
                f1 *= __shfl_sync(0xffffffffu, scale, 8 * c + 4) * sw;
            } else {
                const __nv_bfloat16* ph = hb + (sh ? 2 * hpart : 0) + at;
                const int64_t lo = sh ? spart : hpart;
                uint4 x[2][Tile<FP8>::kN];
#pragma unroll
                for (int i = 0; i < Tile<FP8>::kN; ++i) {
                    const int k = 32 * i + 8 * c;
                    const bool in = on && kb * 128 + k < K;
                    x[0][i] = in ? __ldcg(reinterpret_cast<const uint4*>(ph + k)) : make_uint4(0, 0, 0, 0);
                    x[1][i] = in ? __ldcg(reinterpret_cast<const uint4*>(ph + lo + k)) : make_uint4(0, 0, 0, 0);
                }
                tile_mma<FP8>(d, tl, x[0]);
                tile_mma<FP8>(d, tl, x[1]);
            }
            // columns of rows that did not choose the expert stay out (its weights may not be finite)
            if ((m >> (2 * c)) & 1u) { acc[0] = fmaf(f0, d[0], acc[0]); acc[2] = fmaf(f0, d[2], acc[2]); }
            if ((m >> (2 * c + 1)) & 1u) { acc[1] = fmaf(f1, d[1], acc[1]); acc[3] = fmaf(f1, d[3], acc[3]); }
        }
        __syncthreads();   // an earlier turn's sums have been read
#pragma unroll
        for (int j = 0; j < 4; ++j) s.part[0][warp][2 * c + (j & 1)][gi + 8 * (j >> 1)] = acc[j];
        __syncthreads();
        if (tid < kTokenRows * 16 && (tid >> 4) < a.R) {
            const int r = tid >> 4, n = tid & 15;
            float v = s.part[0][0][r][n];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) v += s.part[0][w][r][n];
            const int64_t at = (int64_t)r * a.H + 16 * t + n;
            a.y[at] = __float2bfloat16_rn(v);
            if (a.y_f32) a.y_f32[at] = v;
            if (!(fabsf(v) < INFINITY)) atomicOr(&s.bad, 1u << r);
        }
        __syncthreads();
        if (tid == 0) {
            status_add(a.status, MOE_STATUS_NONFINITE_OUTPUT, __popc(s.bad));
            s.bad = 0;
        }
    }
    // clear the barrier's flags once every CTA has passed it
    if (a.given && cta == G - 1 && warp == kWarps - 1) {
        const bool ok = wait_flags(flags2, G, a.wait_ns ? a.wait_ns : kWaitLimitNs, lane);
        if (!ok && lane == 0) status_add(a.status, MOE_STATUS_WAIT_TIMEOUT, 1);
        for (int i = lane; i < G; i += 32) st_flag(flags1 + i, 0);
    }
}

namespace {
template <bool FP8>
int smem_bytes(int H) { return (int)(sizeof(Smem) + 127) / 128 * 128 + x_bytes<FP8>(H); }
}  // namespace

cudaError_t token_set_attributes() {
    cudaError_t e = cudaFuncSetAttribute(k_token<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         smem_bytes<false>(kTokenMaxH));
    return e == cudaSuccess ? cudaFuncSetAttribute(k_token<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   smem_bytes<true>(kTokenMaxH)) : e;
}

cudaError_t launch_token(bool fp8, const TokenArgs& a, int num_sms, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(num_sms < kTokenMaxCtas ? num_sms : kTokenMaxCtas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = fp8 ? smem_bytes<true>(a.H) : smem_bytes<false>(a.H);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;   // every CTA is resident: they wait for one another
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return fp8 ? cudaLaunchKernelEx(&cfg, k_token<true>, a) : cudaLaunchKernelEx(&cfg, k_token<false>, a);
}

}  // namespace moe
