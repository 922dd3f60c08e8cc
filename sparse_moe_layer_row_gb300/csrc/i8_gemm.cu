// moe_i8_gemm: y[r, n] = xs[r] ws[n] sum_k xq[r, k] wq[n, k] on int8 codes.
//
// sm_103a has no fast path for int8 products: mma.sync on int8 takes an SM some 20 clocks for 16 x
// 8 x 32, which up to 8 rows hide behind the weights' loads.  With more, codes become fp16 in
// registers (exact, as their products and sums below 2^24 are in fp32), and the sum of whole
// numbers is the fp16 tensor core's.  Past 2^24 the tensor core drops what lies below its
// accumulator's last bit, at every addition of 16 products and always towards zero:
//   k_i8_rows   a warp's share of K is summed in pieces of 1024, none of which passes 2^24, and the
//               pieces and shares in int32 (shares whose fp32 sum cannot pass 2^24: in fp32): the whole
//               number for any K.  Costs 0.1 us of 4.7 (32 x 4096 x 2048).
//   k_i8_tiles  parts of 8192 of K, added in fp32: off by (512 + parts) 2^-23 of the addends' magnitudes
//               at most.  Codes of 100 to 127 at K = 7168: 1.2e-5; in one part K = 131056 had 7.6e-4.
//               Parts of 1024, exact up to K = 2048, were 3 to 8% slower for every K above 1024
//               (2048 x 4096 x 7168: 83.7 against 77.1 us; the accumulators' way out is not overlapped).
//
// k_i8_rows: a CTA takes 16 outputs and 32 rows, and its eight warps share K: warp w
// takes the blocks of 128 w, w + 8, ...  The weights are the M of mma.sync m16n8k16 (up to 8
// rows: m16n8k32 on int8), the rows its N.  Operands go from global memory to registers, two blocks at a time; K is
// permuted inside a block, alike in both operands, so that a lane's are 16-byte loads and
// four codes of a row make one MMA's operand.  The warps' sums are added through shared memory.
// Bound by the round trip to memory (1 x 2048 x 2048 2.1 us, floor 0.6; 8 x 32768 x 2048 13.7 us,
// 4.9 TB/s of W), with more rows by the conversions and mma.sync (32 x 4096 x 2048 4.7 us,
// 77 x 1000 x 1104 4.7); mma.sync on int8 there took 911 us for 8192 x 4096 x 2048.
//
// k_i8_tiles: tcgen05 kind::f16 (the bf16 rate).  A CTA pair (cta_group::2) takes 256 rows of A by up
// to 256 of B, where B is the operand with fewer rows:
//   A (M = 256)  128 rows per CTA: raw codes by TMA (16 KB per 128 of K), which the converter warps
//                turn into fp16 in tensor memory, from where the MMA reads A
//   B (N <= 256) fp16, half of the rows per CTA, by TMA.  k_i8_widen writes it to the workspace
//                first: every tile of A needs it, and converting it there would double the
//                shared-memory traffic of the loop
// so that A is read as bytes and never written, and an SM's shared memory carries 96 KB per 128 of
// K (1024 clocks of the tensor core).  Tensor memory holds the accumulators (256 columns) and four A
// slots of 64, one per stage (narrow tiles leave room for more).  Roles, 512 threads per CTA:
//   warps 0, 3      lane 0: TMA producers of A (`afull`) and of B (`bfull`), ring of 4 stages of 128
//                   of K (6 or 7 with tiles of 128 or 64 rows of B)
//   warp 1          tensor memory; in rank 0, issues the MMAs and commits (`empty` of both ranks:
//                   the stage and its A slot; `tfull`)
//   warp 2 lane 0   forwarder: the CTA's B of a stage has landed -> rank 0's `ready`
//   warps 4..7      converters: 128 codes of a row per thread -> rank 0's `ready`
//   warps 8..15     epilogue: 32 rows of A (a lane each) by 128 of B per warp.  They take the
//                   accumulators into registers at once (`tempty` of rank 0), so that the next
//                   tile's MMAs run while they scale and store.
// Every wait is bounded, and drains follow an abort, as in gemm_pair.cu.
//
// 8192 x 4096 x 2048: 78 us, 1.75 PFLOP/s (floor 73 at the measured burst rate; called back to back
// for long, at the power limit's clock, 88: 81 there).  Of it some 3 us are k_i8_widen's, which reads
// 8 MB and writes 17 (x, the larger operand, took 6; to start on what is widened already, the tiles
// would need flags that a call clears first), 512 clocks per 64 of K the tensor core's, and the last
// tile's epilogue.  Issued by one lane in a branch of its own the 64 of K took 560: the whole warp
// runs the loop.  Stages of 64 of K cost 230 ns each whatever the tile's width (rows of 64 bytes are
// slow to copy); a narrow tile's stages of 128 cost 250, with other pairs at work 340.  Two converter
// warpgroups gained nothing with either; nor did the wait for the tensor memory stores deferred by a
// stage, four conversions in flight and prefetches of A to L2.  Rings of 6 and 7 stages instead of
// 4: 256 x 4096 x 2048 14.4 to 13.1 us.  2048 x 2048 x 2048: 20 us, one round of 64 units.
#include <cstring>
#include <type_traits>

#include "pair.cuh"
#include "rows8.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8;
constexpr int kCols = 16, kRowsPerCta = 32;
constexpr int kExactK = 1024;   // a sum of as many products of codes is at most 2^24: exact in fp32

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                       uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four codes (two's complement, in byte order) -> two words of two fp16: the byte q + 128 is the
// low byte of fp16 1024 + q + 128, exact; minus 1152 gives q.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 k = __half2half2(__ushort_as_half(0x6480));
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), k);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), k);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ void store_one(void* y, int64_t i, int dtype, float v) {
    if (dtype == MOE_F32) static_cast<float*>(y)[i] = v;
    else if (dtype == MOE_BF16) static_cast<__nv_bfloat16*>(y)[i] = __float2bfloat16_rn(v);
    else static_cast<__half*>(y)[i] = __float2half_rn(v);
}

}  // namespace

// NT tiles of 8 rows per CTA
template <int NT, bool LONG>
__global__ void __launch_bounds__(32 * kWarps) k_i8_rows(I8GemmArgs a) {
    using Acc = std::conditional_t<NT == 1, int, float>;
    using Part = std::conditional_t<LONG, int, Acc>;
    pdl_wait();  // see common.cuh: nothing global is touched before
    pdl_trigger();
    __shared__ Part part[kWarps][NT * 8][kCols + 1];
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
    Acc acc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[t][j] = 0;
    int whole[LONG ? NT : 1][4] = {}, held = 0;   // LONG: what acc held before; of the warp's K in acc
    auto fold = [&]() {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                whole[t][j] += (int)acc[t][j];
                acc[t][j] = 0;
            }
        held = 0;
    };
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
            for (int i = 0; i < 2; ++i) {
                if constexpr (NT == 1) {
                    const uint4 x = vx[h][0][i];
                    mma_s8(acc[0], va[h][i].x, vb[h][i].x, va[h][i].y, vb[h][i].y, x.x, x.y);
                    mma_s8(acc[0], va[h][i].z, vb[h][i].z, va[h][i].w, vb[h][i].w, x.z, x.w);
                } else {
                    const uint32_t wa4[4] = {va[h][i].x, va[h][i].y, va[h][i].z, va[h][i].w};
                    const uint32_t wb4[4] = {vb[h][i].x, vb[h][i].y, vb[h][i].z, vb[h][i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t a0, a1, a2, a3;
                        widen4(wa4[j], a0, a2);
                        widen4(wb4[j], a1, a3);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const uint4 x = vx[h][t][i];
                            uint32_t b0, b1;
                            widen4(j == 0 ? x.x : j == 1 ? x.y : j == 2 ? x.z : x.w, b0, b1);
                            mma_f16(acc[t], a0, a1, a2, a3, b0, b1);
                        }
                    }
                }
            }
        if constexpr (LONG) {
            if ((held += 2 * kFp8Block) == kExactK) fold();
        }
    }
    if constexpr (LONG) fold();
#pragma unroll
    for (int t = 0; t < NT; ++t) {   // D: outputs gi and gi + 8 of rows 2c and 2c + 1
        auto value = [&](int j) -> Part {
            if constexpr (LONG) return whole[t][j];
            else return acc[t][j];
        };
        part[warp][8 * t + 2 * c][gi] = value(0);
        part[warp][8 * t + 2 * c + 1][gi] = value(1);
        part[warp][8 * t + 2 * c][gi + 8] = value(2);
        part[warp][8 * t + 2 * c + 1][gi + 8] = value(3);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < NT * 8 * kCols; i += 32 * kWarps) {
        const int r = i / kCols, n = i % kCols;
        if (r0 + r >= a.R || n0 + n >= a.N) continue;
        Part v = part[0][r][n];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) v += part[w][r][n];
        float sum = (float)v;
        if constexpr (std::is_same_v<Part, float>) {
            float most = 0.0f;   // no sum on the way exceeds it (2^24 may have been rounded to)
#pragma unroll
            for (int w = 0; w < kWarps; ++w) most += fabsf(part[w][r][n]);
            if (most >= (float)(1 << 24)) {
                int whole = 0;
                for (int w = 0; w < kWarps; ++w) whole += (int)part[w][r][n];
                sum = (float)whole;
            }
        }
        store_one(a.y, (int64_t)(r0 + r) * a.ldy + n0 + n, a.ydtype,
                  sum * (__ldg(a.xs + r0 + r) * __ldg(a.ws + n0 + n)));
    }
}

// ------------------------------------------------------------------------ tiles

namespace {

constexpr uint64_t kWaitLimitNs = 2000000000ull;   // 2 s: far beyond any legal wait (0 in the arguments)
constexpr uint64_t kDrainLimitNs = 200000000ull;   // 0.2 s when draining after an abort
constexpr int kThreads = 512, kMaxStages = 7;
constexpr int kStepK = 128, kRaw = 128 * 128;        // K and bytes of A per stage
constexpr int kPartK = 8192, kPart = kPartK / kStepK;   // K (and stages) between two reads of the accumulators
// Stages of a tile's ring, by its width: what shared memory (16 KB of A, 128 `width` bytes of B) and
// tensor memory (64 columns of A beside `width` of accumulators) hold.
__host__ __device__ constexpr int stages_of(int width) { return width > 128 ? 4 : width > 64 ? 6 : 7; }
constexpr int kScaleOff = 192 * 1024;                // float [8][128]: sb of an epilogue warp's rows
constexpr int kBarOff = kScaleOff + 8 * 128 * 4;
constexpr int kSmem = kBarOff + 512 + 1024;
constexpr int kTmemCols = 512;
constexpr bool fits(int width) {
    return stages_of(width) * (kRaw + 128 * width) <= kScaleOff && width + 64 * stages_of(width) <= kTmemCols &&
           stages_of(width) <= kMaxStages;
}
static_assert(fits(256) && fits(128) && fits(64), "shared memory and TMEM columns");
static_assert(kSmem <= 227 * 1024, "shared memory budget");
static_assert(8 * (4 * kMaxStages + 3) + 12 <= 512, "barrier region");
// registers per thread after the split; the pool is what the CTA was launched with (checked on
// the host)
constexpr int kLaunchRegs = 128, kFewRegs = 56, kManyRegs = 200;
static_assert(256 * kFewRegs + 256 * kManyRegs <= kThreads * kLaunchRegs, "register split");

// kind::f16 with fp16 A (in tensor memory) and B, fp32 accumulator, both K-major.
__device__ __forceinline__ void mma_f16_pair_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                                uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

}  // namespace

namespace {

template <typename T>
__device__ __forceinline__ T rounded(float v);
template <>
__device__ __forceinline__ float rounded<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half rounded<__half>(float v) { return __float2half_rn(v); }

// What a lane holds of y: v[c] (xs[c] ws), c < n.  Along the rows (one output of n rows from p on): a
// warp stores 32 outputs of a row at a time.
template <typename T>
__device__ __forceinline__ void store_rows(T* p, int64_t ld, const float (&v)[128], const float* xs, float ws, int n) {
#pragma unroll
    for (int c = 0; c < 128; ++c) {
        if (c < n) *p = rounded<T>(v[c] * (xs[c] * ws));
        p += ld;
    }
}
// Along a row (n outputs of one row from p on): 32 bytes a lane and store, where rows lie on them.
template <typename T>
__device__ __forceinline__ void store_along(T* p, bool vec, const float (&v)[128], const float* xs, float ws, int n) {
    constexpr int kN = 32 / (int)sizeof(T);
#pragma unroll
    for (int c = 0; c < 128; c += kN) {
        T o[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) o[i] = rounded<T>(v[c + i] * (xs[c + i] * ws));
        if (vec && c + kN <= n) {
            uint32_t w[8];
            memcpy(w, o, 32);
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + c), "r"(w[0]), "r"(w[1]),
                         "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                         : "memory");
        } else {
#pragma unroll
            for (int i = 0; i < kN; ++i)
                if (c + i < n) p[c + i] = o[i];
        }
    }
}

}  // namespace

// Codes to fp16, 16 per thread and turn.
__global__ void __launch_bounds__(256) k_i8_widen(const int8_t* q, __half* x, int64_t n16) {
    pdl_wait();  // see common.cuh: nothing global is touched before
    pdl_trigger();
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n16; i += gridDim.x * 256ll) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(q) + i);
        uint4 a, b;
        widen4(v.x, a.x, a.y);
        widen4(v.y, a.z, a.w);
        widen4(v.z, b.x, b.y);
        widen4(v.w, b.z, b.w);
        reinterpret_cast<uint4*>(x)[2 * i] = a;
        reinterpret_cast<uint4*>(x)[2 * i + 1] = b;
    }
}

template <bool SWAP, bool LONG>
__global__ void __launch_bounds__(kThreads, 1)
k_i8_tiles(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, I8GemmArgs a) {
    const int M = SWAP ? a.R : a.N, C = SWAP ? a.N : a.R;   // rows of A and of B
    const float *sa = SWAP ? a.xs : a.ws, *sb = SWAP ? a.ws : a.xs;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;   // same offset in both CTAs
    uint8_t* base = smem_raw + (sbase - raw);
    uint64_t* afull = reinterpret_cast<uint64_t*>(base + kBarOff);   // [S] codes landed
    uint64_t* bfull = afull + kMaxStages;                                // [S] x landed
    uint64_t* ready = bfull + kMaxStages;                                // [S] both ranks' x and A (rank 0)
    uint64_t* empty = ready + kMaxStages;                                // [S] stage and A slot free (both)
    uint64_t* tfull = empty + kMaxStages;                                // accumulators ready (both)
    uint64_t* tempty = tfull + 1;                                     // accumulators free (rank 0)
    uint64_t* dbar = tempty + 1;                                      // MMA drain (rank 0)
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(dbar + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* never = abort_flag + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const uint64_t limit = a.wait_ns ? a.wait_ns : kWaitLimitNs;
    const int stages = stages_of(a.width);
    const uint32_t b_tile = 128 * a.width, b_off = sbase + stages * kRaw;   // tiles of B behind the codes (1 KB boundaries)
    const uint32_t a_col = kTmemCols - 64 * stages;                         // A's slots behind the accumulators
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(afull + s, 1);
            mbar_init(bfull + s, 1);
            mbar_init(ready + s, 2 * (1 + 4));   // of each rank: the forwarder, four converter warps
            mbar_init(empty + s, 1);
        }
        mbar_init(tfull, 1);
        mbar_init(tempty, 2 * (a.width > 128 ? 8 : 4));   // the epilogue warps of both ranks
        mbar_init(dbar, 1);
        *abort_flag = 0;
        *never = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc_pair(tmem_slot, kTmemCols);
    tc_fence_before();
    cluster_sync();   // barriers of both CTAs initialised, TMEM allocated
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // The kernel before this one is k_i8_widen, which let it start after its own wait: all but the
    // widened operand was complete by then, so that only B's producer waits (common.cuh).

    // unit u: rows 256 m .. of A, `width` c .. of B (neighbouring units share rows of B)
    const int mt = (M + 255) / 256, nunits = mt * ((C + a.width - 1) / a.width);
    const int nact = active_workers(nunits, (int)cluster_count());   // balanced rounds
    const int ufirst = (int)cluster_id() < nact ? (int)cluster_id() : nunits;
    const int nkb = (a.K + kStepK - 1) / kStepK, parts = (nkb + kPart - 1) / kPart;
    auto rows_of = [&](int u, int& m, int& r0) {   // the MMA's N: rows of B of the unit, in 32s
        const int c = u / mt;
        m = u - c * mt;
        r0 = c * a.width;
        return (min(a.width, C - r0) + 31) / 32 * 32;
    };
    auto give_up = [&]() {   // one lane of a warp
        if (!*abort_flag) { *abort_flag = 1; status_add(a.status, MOE_STATUS_WAIT_TIMEOUT, 1); }
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
        if ((warp == 0 || warp == 3) && lane == 0) {
            // ----------------------------------------------------------- TMA producers
            const bool b = warp == 3;
            if (b) {
                pdl_wait();
                pdl_trigger();
            }
            uint64_t* full = b ? bfull : afull;
            int stage = 0, nfills = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int u = ufirst; ok && u < nunits; u += nact) {
                int m, r0;
                const int n = rows_of(u, m, r0);
                for (int kb = 0; kb < nkb; ++kb) {
                    if (!mbar_wait_bounded(empty + stage, phase ^ 1u, abort_flag, limit)) {
                        give_up();
                        ok = false;
                        break;
                    }
                    mbar_expect_tx(full + stage, b ? b_tile : kRaw);
                    if (b) {
                        const uint32_t to = b_off + stage * b_tile;
                        tma_load_2d(to, &tmB, kb * kStepK, r0 + n / 2 * rank, full + stage);
                        tma_load_2d(to + b_tile / 2, &tmB, kb * kStepK + 64, r0 + n / 2 * rank, full + stage);
                    } else {
                        tma_load_2d(sbase + stage * kRaw, &tmA, kb * kStepK, m * 256 + 128 * rank, full + stage);
                    }
                    ++nfills;
                    if (++stage == stages) { stage = 0; phase ^= 1u; }
                }
            }
            // drain: the last fill of every stage has landed (consumed or not)
            for (int s = 0; s < stages; ++s) {
                if (nfills < stages && s >= nfills) break;
                const uint32_t par = s < stage ? phase : (phase ^ 1u);
                if (!mbar_wait_bounded(full + s, par, never, kDrainLimitNs)) give_up();
            }
        } else if (warp == 1 && rank == 0) {
            // -------------------------------------------------------------- MMA issuer
            // The whole warp runs the loop, so that its values are uniform, and one elected lane
            // issues.
            const bool leader = elect_one();
            int stage = 0;
            uint32_t phase = 0, tphase = 0;
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                if (__all_sync(0xffffffffu, mbar_test_wait_cluster(smem_u32(bar), parity))) return true;
                const bool got = mbar_wait_cluster_bounded(bar, parity, abort_flag, limit);
                if (!__any_sync(0xffffffffu, !got)) return true;
                if (lane == 0) give_up();
                return false;
            };
            for (int u = ufirst; ok && u < nunits; u += nact) {
                int m, r0;
                const int n = rows_of(u, m, r0);
                const uint32_t idesc = 1u << 4 | (uint32_t)(n >> 3) << 17 | (uint32_t)(256 >> 4) << 24;   // fp16 A and B
                for (int kb = 0; kb < nkb; ++kb) {
                    const int at_part = LONG ? kb % kPart : kb;
                    if (at_part == 0) {
                        if (!wait(tempty, tphase ^ 1u)) {
                            ok = false;
                            break;
                        }
                        tphase ^= 1u;
                    }
                    if (!wait(ready + stage, phase)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t bd = smem_desc_sw128(b_off + stage * b_tile);
                    const uint32_t at = tmem + a_col + (uint32_t)(64 * stage);
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)   // 32 bytes along K are 2 in the descriptor's address field
                            mma_f16_pair_ta(tmem, at + 8 * kk, bd + (kk >> 2) * (b_tile >> 5) + 2 * (kk & 3), idesc, (at_part | kk) != 0);
                        tc_commit_pair(empty + stage);
                        if ((LONG && at_part == kPart - 1) || kb == nkb - 1) tc_commit_pair(tfull);
                    }
                    __syncwarp();
                    if (++stage == stages) { stage = 0; phase ^= 1u; }
                }
            }
            // drain: arrives once every MMA issued above has completed
            if (leader) tc_commit_pair_local(dbar);
            __syncwarp();
            if (!mbar_wait_bounded(dbar, 0, never, kDrainLimitNs) && lane == 0) give_up();
        } else if (warp == 2 && lane == 0) {
            // --------------------------------------------------------------- forwarder
            const uint32_t ready0 = mapa_shared(smem_u32(ready), 0);
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int u = ufirst; ok && u < nunits; u += nact)
                for (int kb = 0; kb < nkb; ++kb) {
                    if (!mbar_wait_bounded(bfull + stage, phase, abort_flag, limit)) {
                        give_up();
                        ok = false;
                        break;
                    }
                    mbar_arrive_cluster(ready0 + stage * 8);
                    if (++stage == stages) { stage = 0; phase ^= 1u; }
                }
        }
    } else if (warp < 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
        // -------------------------------------------------------------- converters
        // Row r of the CTA's 128 of A per thread: 128 codes (chunk c of 16 at c ^ (r & 7), the copy's
        // 128-byte swizzle) into lane r of the stage's A slot.
        const uint32_t ready0 = mapa_shared(smem_u32(ready), 0);
        const int r = 32 * (warp & 3) + lane, sw = r & 7;
        const uint32_t tq = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + a_col;
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int u = ufirst; ok && u < nunits; u += nact)
            for (int kb = 0; kb < nkb; ++kb) {
                // codes landed; they were only asked for once the MMA had read the slot
                const bool got = mbar_wait_bounded(afull + stage, phase, abort_flag, limit);
                if (__any_sync(0xffffffffu, !got)) {
                    if (lane == 0) give_up();
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint8_t* row = base + stage * kRaw + r * 128;
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint32_t o[16];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint4 w = *reinterpret_cast<const uint4*>(row + (((2 * h + i) ^ sw) << 4));
                        widen4(w.x, o[8 * i], o[8 * i + 1]);
                        widen4(w.y, o[8 * i + 2], o[8 * i + 3]);
                        widen4(w.z, o[8 * i + 4], o[8 * i + 5]);
                        widen4(w.w, o[8 * i + 6], o[8 * i + 7]);
                    }
                    tmem_st16(tq + (uint32_t)(64 * stage + 16 * h), o);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(ready0 + stage * 8);
                if (++stage == stages) { stage = 0; phase ^= 1u; }
            }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
        // ---------------------------------------------------------------- epilogue
        const int q = warp & 3, half = (warp - 8) >> 2;   // lane quadrant; rows 128 half ..
        const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(128 * half);
        const uint32_t tempty0 = mapa_shared(smem_u32(tempty), 0);
        float* xs = reinterpret_cast<float*>(base + kScaleOff) + 128 * (warp - 8);
        uint32_t tphase = 0;
        auto accumulators_ready = [&]() {
            const bool got = mbar_wait_bounded(tfull, tphase, abort_flag, limit);
            if (__any_sync(0xffffffffu, !got)) {
                if (lane == 0) give_up();
                return false;
            }
            tphase ^= 1u;
            tc_fence_after();
            return true;
        };
        auto release = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(tempty0);
        };
        for (int u = half && a.width <= 128 ? nunits : ufirst; u < nunits; u += nact) {
            int m, r0;
            rows_of(u, m, r0);
            const int ra = m * 256 + 128 * rank + 32 * q + lane, rb = r0 + 128 * half;   // this lane's of A; B's first
            const int n = min(min(a.width - 128 * half, 128), C - rb);   // rows of B of this warp
            const float ls = ra < M ? __ldg(sa + ra) : 0.0f;
            __syncwarp();   // the last tile's scales have been read
#pragma unroll
            for (int i = lane; i < 128; i += 32) xs[i] = i < n ? __ldg(sb + rb + i) : 0.0f;
            __syncwarp();
            float v[128];
            if constexpr (LONG) {   // all parts but the last
#pragma unroll
                for (int c = 0; c < 128; ++c) v[c] = 0.0f;
                bool ok = true;
                for (int part = 1; ok && part < parts; ++part) {
                    ok = accumulators_ready();
                    if (ok) {
#pragma unroll
                        for (int c = 0; c < 128; c += 32) {
                            float lo[16], hi[16];
                            tmem_ld16x2(tq + c, tq + c + 16, lo, hi);
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                v[c + i] += lo[i];
                                v[c + 16 + i] += hi[i];
                            }
                        }
                        release();
                    }
                }
                if (!ok) break;
            }
            if (!accumulators_ready()) break;
#pragma unroll
            for (int c = 0; c < 128; c += 32) {
                float lo[16], hi[16];
                tmem_ld16x2(tq + c, tq + c + 16, lo, hi);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    v[c + i] = LONG ? v[c + i] + lo[i] : lo[i];
                    v[c + 16 + i] = LONG ? v[c + 16 + i] + hi[i] : hi[i];
                }
            }
            release();
            if (ra < M) {
                auto store = [&](auto* y) {
                    if (SWAP) store_along(y + (int64_t)ra * a.ldy + rb, a.y_vec, v, xs, ls, n);
                    else store_rows(y + (int64_t)rb * a.ldy + ra, a.ldy, v, xs, ls, n);
                };
                if (a.ydtype == MOE_F32) store(static_cast<float*>(a.y));
                else if (a.ydtype == MOE_BF16) store(static_cast<__nv_bfloat16*>(a.y));
                else store(static_cast<__half*>(a.y));
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // no CTA leaves while its peer may still signal or read it
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
}

namespace {
cudaLaunchConfig_t tiles_config(cudaLaunchAttribute (&attr)[2], int clusters, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * clusters));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cfg;
}
}  // namespace

// Also the clusters that are resident at once on the current device.
cudaError_t i8_tiles_set_attributes(int num_sms, int* clusters) {
    *clusters = num_sms / 2;
    auto set = [&](auto k) {
        cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        // the register split draws on what the CTA is launched with
        cudaFuncAttributes fa;
        if ((e = cudaFuncGetAttributes(&fa, k)) != cudaSuccess) return e;
        if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidDeviceFunction;
        cudaLaunchAttribute attr[2];
        cudaLaunchConfig_t cfg = tiles_config(attr, num_sms / 2, nullptr);
        cfg.numAttrs = 1;
        int n = 0;
        if ((e = cudaOccupancyMaxActiveClusters(&n, k, &cfg)) != cudaSuccess) return e;
        if (n <= 0) return cudaErrorInvalidConfiguration;
        *clusters = n < *clusters ? n : *clusters;
        return cudaSuccess;
    };
    cudaError_t e = set(k_i8_tiles<false, false>);
    if (e == cudaSuccess) e = set(k_i8_tiles<true, false>);
    if (e == cudaSuccess) e = set(k_i8_tiles<false, true>);
    return e == cudaSuccess ? set(k_i8_tiles<true, true>) : e;
}

cudaError_t launch_i8_tiles(const I8GemmArgs& a, const CUtensorMap& ma, const CUtensorMap& mb, void* wide, int num_sms,
                            int clusters, cudaStream_t st) {
    // a.width: set by the caller, which encoded the maps for it
    const bool swap = i8_swapped(a.R, a.N);
    const int64_t n16 = (int64_t)(swap ? a.N : a.R) * a.K / 16;
    int64_t blocks = (n16 + 255) / 256;
    if (blocks > (int64_t)num_sms * 32) blocks = (int64_t)num_sms * 32;
    cudaError_t e = launch_kernel(k_i8_widen, dim3((unsigned)blocks), dim3(256), 0, st, swap ? a.wq : a.xq,
                                  static_cast<__half*>(wide), n16);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = tiles_config(attr, clusters, st);
    const bool longer = a.K > kPartK;
    auto k = swap ? (longer ? k_i8_tiles<true, true> : k_i8_tiles<true, false>)
                  : (longer ? k_i8_tiles<false, true> : k_i8_tiles<false, false>);
    return cudaLaunchKernelEx(&cfg, k, ma, mb, a);
}

// By what the kernels were measured to take (ns): the rows kernel 1800 + CTAs (5.9 + 0.0031 K) with 17
// to 32 rows per CTA; the tiles 7800 (6500 where a lane holds a row of y) + kStep per 64 of K and round
// of units.  Narrow tiles leave the tensor core waiting for the converters, but give few rows more
// pairs.  Measured, us, rows kernel / tiles of 256, 128, 64:
//    256 x 2048 x 2048   13.5 / 16.7 12.3 11.8       512 x 2048 x 2048   25.2 / 17.4 13.1 13.3
//    128 x 4096 x 2048   14.6 / 14.1 12.5 12.1      1024 x 4096 x 4096      - / 28.1 29.1 45.9
//   1000 x 1000 x  992   24.7 / 12.6 10.2 11.1 (the rule's 64 is not the best)
//   1000 x  512 x  512    9.5 /  9.1  7.1  6.9       128 x 8192 x 4096   43.3 / 22.8 18.9 17.9
namespace {
int64_t tiles_ns(int R, int N, int K, int* width) {
    constexpr int kStep[3] = {265, 200, 170};   // widths 256, 128, 64
    const int64_t M = R > N ? R : N, C = R > N ? N : R, steps = (K + 63) / 64;
    int64_t best = 0;
    for (int i = 0; i < 3; ++i) {
        const int64_t w = 256 >> i, rounds = ((M + 255) / 256 * ((C + w - 1) / w) + 75) / 76;   // 76 CTA pairs
        const int64_t ns = (i8_swapped(R, N) ? 6500 : 7800) + rounds * steps * kStep[i];
        if (i == 0 || ns < best) {
            best = ns;
            *width = (int)w;
        }
    }
    return best;
}
}  // namespace

int i8_width(int R, int N, int K) {
    int width = 0;
    tiles_ns(R, N, K, &width);
    return width;
}

bool i8_rows_applies(int R, int N, int K) {
    if (R <= 16) return true;
    if (R > 65535 * kRowsPerCta) return false;   // the grid's y: row tiles
    const int64_t ctas = (int64_t)((N + kCols - 1) / kCols) * ((R + kRowsPerCta - 1) / kRowsPerCta);
    int width;
    return 1800 + ctas * (59000 + 31 * (int64_t)K) / 10000 <= tiles_ns(R, N, K, &width);
}

cudaError_t launch_i8_rows(const I8GemmArgs& a, cudaStream_t st) {
    const dim3 grid((unsigned)((a.N + kCols - 1) / kCols), (unsigned)((a.R + kRowsPerCta - 1) / kRowsPerCta));
    const bool longer = a.K > kWarps * kExactK;
    auto k = a.R <= 8 ? k_i8_rows<1, false> : a.R <= 16 ? (longer ? k_i8_rows<2, true> : k_i8_rows<2, false>)
                                                        : (longer ? k_i8_rows<4, true> : k_i8_rows<4, false>);
    return launch_kernel(k, grid, dim3(32 * kWarps), 0, st, a);
}

}  // namespace moe
