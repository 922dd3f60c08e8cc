// The expert FFN's e4m3 gate/up and down GEMMs for calls with few rows per
// expert: the weights are streamed once, and what counts is that HBM never
// waits.
//
// A unit is at most 32 pairs of one expert, taken 16 at a time (the registers
// for more would spill; the second 16's weights come from L2), by 256 weight
// rows (gate/up: 128 gate rows and the up rows of the same 128 intermediate
// indices; down: 256 hidden outputs).  With a handful of pairs per expert the tensor core's 128-row
// tile (fp8_gemm.cu) is nearly empty, yet each block of K still goes through
// TMEM and its promotion.  Here the weights are the MMA's M and the pairs its
// N = 8 (mma.sync m16n8k32): 32 weight rows per warp, the sums of a block of K
// land in registers and are promoted there.
//
// K is permuted inside a block of 128, alike for both operands: lane 4 i + c
// takes bytes 32 c .. 32 c + 31 of its row, and MMA number j of the block's four
// reads bytes 8 j .. 8 j + 7 of them.  So a lane's operands are 16-byte loads.
//
// One CTA per SM, persistent over the unit list, 320 threads:
//   warp 8 lane 0   TMA producer: the block's two weight tiles (2 x 16 KB, 128-byte
//                   swizzle) into a ring of 6 stages, deep enough that it streams
//                   on through the consumers' epilogues
//   warp 9          loader: the pairs' codes (gathered rows of x, or h), swizzled
//                   alike, and the block's scales, by cp.async into the same stage
//   warps 0..7      consumers, which read nothing but the stage
// (Consumers that load the pairs' operands themselves, through L1, wait for L2
// in every block, or hold several blocks of them and spill.  Two CTAs per SM with
// 3 stages each: 99 against 93 us for 32 rows.)  The down GEMM's producer starts
// before the gate/up kernel has ended: its weights and its unit list do not
// depend on it.
// 32 rows of the 2048 x 512 layer with 8 of 256 experts: 60.7 us for the gate/up GEMM's
// 317 MB and 30.8 for the down GEMM's 159, both 5.2 TB/s, start and end included.
// Every wait is bounded, and copies in flight are waited for before the CTA
// exits, as in fp8_gemm.cu.
#include <type_traits>

#include "fp8.cuh"

namespace moe {

namespace {

constexpr uint64_t kWaitLimitNs = 2000000000ull;   // 2 s: far beyond any legal wait
constexpr uint64_t kDrainLimitNs = 200000000ull;   // 0.2 s when draining after an abort

constexpr int kStages = 6;
constexpr int kThreads = 320;
constexpr int kPass = 16;                            // pairs at a time
constexpr int kTile = 128 * 128;
constexpr int kStageBytes = 2 * kTile + kPass * 128;  // weights, pairs' codes
constexpr int kScaleOff = kStages * kStageBytes;      // float [S][32]: pairs' scales, then the weights'
constexpr int kAmaxOff = kScaleOff + kStages * 128;   // uint32 [2 units][8 warps][kPass]
constexpr int kStgOff = kAmaxOff + 2 * 8 * kPass * 4; // per warp: 8 pairs x 64 bytes
constexpr int kBarOff = kStgOff + 8 * 512;
constexpr int kSmem = kBarOff + 256;
static_assert(kStageBytes % 1024 == 0, "swizzle atoms");
static_assert(kSmem <= 227 * 1024, "shared memory budget");
static_assert(8 * (3 * kStages + 1) + 8 <= 256, "barrier region");

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes, of which the first `bytes` (0 or 16) are read and the rest are zeros
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

}  // namespace

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1)
k_fp8_stream(const __grid_constant__ CUtensorMap tmW0, const __grid_constant__ CUtensorMap tmW1,
             const __grid_constant__ CUtensorMap tmS0, const __grid_constant__ CUtensorMap tmS1,
             Fp8GemmArgs a) {
    extern __shared__ __align__(1024) uint8_t base[];   // swizzle atoms are 1 KB
    const uint32_t sbase = smem_u32(base);
    uint64_t* full = reinterpret_cast<uint64_t*>(base + kBarOff);   // [S] tiles landed
    uint64_t* rfull = full + kStages;                                // [S] loader's copies landed
    uint64_t* empty = rfull + kStages;                               // [S] stage free
    uint64_t* xbar = empty + kStages;                                // amax exchange
    volatile int* abort_flag = reinterpret_cast<volatile int*>(xbar + 1);
    volatile int* never = abort_flag + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(rfull + s, 32);
            mbar_init(empty + s, 8);   // the consumer warps
        }
        mbar_init(xbar, 8);
        *abort_flag = 0;
        *never = 0;
        fence_mbar_init();
    }
    __syncthreads();
    // see common.cuh; the down producer reads only weights and the unit list,
    // which the scatter wrote: complete before the gate/up kernel let this one start
    // (its trigger stays behind its wait)
    if (!(MODE == kDown && warp == 8)) {
        pdl_wait();
        pdl_trigger();
    }
    const int E = a.g.E;
    const int nunits = __ldg(a.g.n_units);
    const int nact = active_workers(nunits, (int)gridDim.x);   // balanced rounds
    const int ufirst = (int)blockIdx.x < nact ? (int)blockIdx.x : nunits;
    auto valid = [&](const int4 un) {
        return unit_valid(un, a.g, kFp8StreamRows, MODE == kDown, kFp8GuRows, kFp8DnCols);
    };
    auto blocks = [&](int g) {
        return MODE == kGateUp ? a.g.H / kFp8Block : fp8_blocks(g == E ? a.g.Is : a.g.I);
    };
    auto give_up = [&]() {
        if (!*abort_flag) { *abort_flag = 1; status_add(a.g.status, MOE_STATUS_WAIT_TIMEOUT, 1); }
    };
    const uint64_t kWaitNs = a.g.wait_ns ? a.g.wait_ns : kWaitLimitNs;

    if (warp == 8) {
        if (lane == 0) {
            // ------------------------------------------------------ TMA producer
            int stage = 0, nfills = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int u = ufirst; ok && u < nunits; u += nact) {
                const int4 un = __ldg(a.g.units + u);
                if (!valid(un)) {
                    status_add(a.g.status, MOE_STATUS_BAD_UNIT, 1);
                    continue;
                }
                const int g = un.x, m = un.y;
                const int nkb = blocks(g), nfill = nkb * ((un.w + kPass - 1) / kPass);
                for (int i = 0; i < nfill; ++i) {
                    const int kb = i % nkb;
                    // the ring is full: its consumers start when the gate/up kernel has
                    // ended, and only from then on does the wait's limit count
                    if (MODE == kDown && nfills == kStages) pdl_wait();
                    if (!mbar_wait_bounded(empty + stage, phase ^ 1u, abort_flag, kWaitNs)) {
                        give_up();
                        ok = false;
                        break;
                    }
                    const uint32_t sW = sbase + stage * kStageBytes;
                    uint64_t* bar = full + stage;
                    const int kc = kb * kFp8Block;
                    const int r0 = MODE == kGateUp ? m * 128 : m * 256;
                    const int r1 = MODE == kGateUp ? r0 : r0 + 128;
                    mbar_expect_tx(bar, (uint32_t)(2 * kTile));
                    if (g == E) {
                        tma_load_2d(sW, &tmS0, kc, r0, bar);
                        tma_load_2d(sW + kTile, MODE == kGateUp ? &tmS1 : &tmS0, kc, r1, bar);
                    } else {
                        tma_load_3d(sW, &tmW0, kc, r0, g, bar);
                        tma_load_3d(sW + kTile, MODE == kGateUp ? &tmW1 : &tmW0, kc, r1, g, bar);
                    }
                    ++nfills;
                    if (++stage == kStages) { stage = 0; phase ^= 1u; }
                }
            }
            // drain: the last fill of every stage has landed (consumed or not)
            for (int s = 0; s < kStages; ++s) {
                if (nfills < kStages && s >= nfills) break;
                const uint32_t par = s < stage ? phase : (phase ^ 1u);
                if (!mbar_wait_bounded(full + s, par, never, kDrainLimitNs)) give_up();
            }
        }
        return;   // no later barrier counts this warp
    }
    if (warp == 9) {
        // ---------------------------------------------------------------- loader
        // Pair i's row of 128 codes: 8 lanes, 16 bytes each, chunk ch at ch ^ (i & 7).
        const int ch = lane & 7;
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int u = ufirst; ok && u < nunits; u += nact) {
            const int4 un = __ldg(a.g.units + u);
            if (!valid(un)) continue;
            const int g = un.x, m = un.y;
            const bool sh = g == E;
            const int nkb = blocks(g);
            const int64_t ldx = MODE == kGateUp ? a.g.R : sh ? a.max_rows : a.max_pairs;
            const int ldc = MODE == kGateUp ? a.g.H : sh ? a.g.Is : a.g.I;
            const uint8_t* codes = MODE == kGateUp ? a.xq : sh ? a.shq : a.hq;
            const float* scales = MODE == kGateUp ? a.xs : sh ? a.shs : a.hs;
            const float *pw0, *pw1;
            if (MODE == kGateUp) {
                const int mb = fp8_blocks(sh ? a.g.Is : a.g.I);
                const int64_t o = ((int64_t)(sh ? 0 : g) * mb + m) * nkb;
                pw0 = (sh ? a.sc_sa : a.sc_a) + o;
                pw1 = (sh ? a.sc_sb : a.sc_b) + o;
            } else {
                const int hb = a.g.H / kFp8Block;
                pw0 = (sh ? a.sc_sa : a.sc_a) + ((int64_t)(sh ? 0 : g) * hb + 2 * m) * nkb;
                pw1 = pw0 + nkb;
            }
            for (int i0 = 0; ok && i0 < un.w; i0 += kPass) {
                const int start = un.z + i0, n = min(kPass, un.w - i0);
                // rows past the pass's are not loaded: they feed only columns never stored
                auto row_of = [&](int i) {
                    if (i >= n) return -1;
                    const int p = start + i;
                    if (MODE == kDown) return p;
                    const int r = !sh ? __ldg(a.g.pair_row + p) : (a.g.shared_rows ? __ldg(a.g.shared_rows + p) : p);
                    return r < a.g.R ? r : -1;
                };
                int row[kPass / 4];
#pragma unroll
                for (int j = 0; j < kPass / 4; ++j) row[j] = row_of(4 * j + (lane >> 3));
                const int mine = lane < kPass ? row_of(lane) : -1;
                for (int kb = 0; kb < nkb; ++kb) {
                    const bool free_ok = mbar_wait_bounded(empty + stage, phase ^ 1u, abort_flag, kWaitNs);
                    if (__any_sync(0xffffffffu, !free_ok)) {   // the warp leaves together
                        give_up();
                        ok = false;
                        break;
                    }
                    const uint32_t dst = sbase + stage * kStageBytes + 2 * kTile;
                    const int col = kb * kFp8Block + ch * 16;
                    // K past a row's end (a last block of 64, down only) is zeros, as the
                    // weights are there
                    const int bytes = col < ldc ? 16 : 0;
#pragma unroll
                    for (int j = 0; j < kPass / 4; ++j) {
                        const int i = 4 * j + (lane >> 3);
                        if (row[j] >= 0)
                            cp_async16_or_zero(dst + i * 128 + ((ch ^ (i & 7)) << 4),
                                               codes + (int64_t)row[j] * ldc + (bytes ? col : 0), bytes);
                    }
                    const uint32_t sdst = sbase + kScaleOff + stage * 128 + lane * 4;
                    if (mine >= 0) cp_async4(sdst, scales + kb * ldx + mine);
                    if (lane == kPass || lane == kPass + 1) cp_async4(sdst, (lane == kPass ? pw0 : pw1) + kb);
                    cp_async_arrive(rfull + stage);
                    if (++stage == kStages) { stage = 0; phase ^= 1u; }
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");   // nothing of this thread lands later
        return;
    }

    // ---------------------------------------------------------------- consumers
    const int gi = lane >> 2, c = lane & 3;   // MMA row / pair index, chunk of K and pair columns
    // this lane's rows in the stage: gate/up: rows 16 warp + gi (+ 8) of both
    // tiles; down: rows 32 warp + gi (+ 8, + 16, + 24) of the 256
    const int row0 = MODE == kGateUp ? 16 * warp + gi : (32 * warp) % 128 + gi;
    const uint32_t tile0 = MODE == kGateUp ? 0u : (uint32_t)(warp >> 2) * kTile;
    const uint32_t tile1 = MODE == kGateUp ? (uint32_t)kTile : tile0;
    const int row1 = MODE == kGateUp ? row0 : row0 + 16;
    // chunks 2 c and 2 c + 1 of a row, swizzled by the row (rows 8 apart alike)
    const uint32_t ch0 = (uint32_t)((2 * c) ^ gi) << 4, ch1 = (uint32_t)((2 * c + 1) ^ gi) << 4;
    uint32_t* s_amax = reinterpret_cast<uint32_t*>(base + kAmaxOff);
    uint8_t* stg = base + kStgOff + warp * 512;

    int stage = 0, upar = 0;
    uint32_t phase = 0, xphase = 0;
    bool alive = true;

    // one pass over a unit's weights with NT tiles of 8 pairs
    auto run = [&](auto nt_c, const int4 un) {
        constexpr int NT = decltype(nt_c)::value;
        const int g = un.x, m = un.y, start = un.z, n = un.w;
        const bool sh = g == E;
        const int nkb = blocks(g);
        float acc0[NT][4], acc1[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc0[t][j] = acc1[t][j] = 0.0f;
        for (int kb = 0; kb < nkb; ++kb) {
            const bool ok = mbar_wait_bounded(full + stage, phase, abort_flag, kWaitNs) &&
                            mbar_wait_bounded(rfull + stage, phase, abort_flag, kWaitNs);
            if (__any_sync(0xffffffffu, !ok)) { give_up(); alive = false; return; }
            const uint32_t sW = sbase + stage * kStageBytes, sX = sW + 2 * kTile + gi * 128;
            const uint32_t r0 = sW + tile0 + row0 * 128, r1 = sW + tile1 + row1 * 128;
            const float* sc = reinterpret_cast<const float*>(base + kScaleOff + stage * 128);
            uint4 xl[NT], xh[NT];
            float s0[NT], s1[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                xl[t] = lds16(sX + t * 1024 + ch0);
                xh[t] = lds16(sX + t * 1024 + ch1);
                s0[t] = sc[8 * t + 2 * c];
                s1[t] = sc[8 * t + 2 * c + 1];
            }
            const float sw[2] = {sc[kPass + (MODE == kGateUp ? 0 : warp >> 2)],
                                 sc[kPass + (MODE == kGateUp ? 1 : warp >> 2)]};
#pragma unroll
            for (int half = 0; half < 2; ++half) {   // the two 16-row tiles
                const uint32_t r = half ? r1 : r0;
                const uint4 al = lds16(r + ch0), ah = lds16(r + ch1);
                const uint4 bl = lds16(r + 1024 + ch0), bh = lds16(r + 1024 + ch1);   // row + 8
                if (half == 1) {
                    __syncwarp();   // every lane has read the stage
                    if (lane == 0) mbar_arrive(empty + stage);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    mma_e4m3(d, al.x, bl.x, al.y, bl.y, xl[t].x, xl[t].y);
                    mma_e4m3(d, al.z, bl.z, al.w, bl.w, xl[t].z, xl[t].w);
                    mma_e4m3(d, ah.x, bh.x, ah.y, bh.y, xh[t].x, xh[t].y);
                    mma_e4m3(d, ah.z, bh.z, ah.w, bh.w, xh[t].z, xh[t].w);
                    const float f0 = s0[t] * sw[half], f1 = s1[t] * sw[half];
                    float* ac = half ? acc1[t] : acc0[t];
                    ac[0] = fmaf(f0, d[0], ac[0]);
                    ac[1] = fmaf(f1, d[1], ac[1]);
                    ac[2] = fmaf(f0, d[2], ac[2]);
                    ac[3] = fmaf(f1, d[3], ac[3]);
                }
            }
            if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
        if (MODE == kGateUp) {
            uint32_t* am = s_amax + upar * (8 * kPass);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                uint32_t m0 = 0, m1 = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc0[t][j] = silu_fast(acc0[t][j]) * acc1[t][j];
                    uint32_t& mm = j & 1 ? m1 : m0;
                    mm = max(mm, __float_as_uint(acc0[t][j]) & 0x7FFFFFFFu);
                }
#pragma unroll
                for (int o = 4; o <= 16; o <<= 1) {
                    m0 = max(m0, __shfl_xor_sync(0xffffffffu, m0, o));
                    m1 = max(m1, __shfl_xor_sync(0xffffffffu, m1, o));
                }
                if (gi == 0) {
                    am[warp * kPass + 8 * t + 2 * c] = m0;
                    am[warp * kPass + 8 * t + 2 * c + 1] = m1;
                }
            }
            // two buffers, taken in turn: a warp can be one exchange ahead of another
            __syncwarp();
            if (lane == 0) mbar_arrive(xbar);
            const bool ok = mbar_wait_bounded(xbar, xphase, abort_flag, kWaitNs);
            if (__any_sync(0xffffffffu, !ok)) { give_up(); alive = false; return; }
            upar ^= 1;
            xphase ^= 1u;
            const int ld = sh ? a.g.Is : a.g.I;
            const int i0 = m * 128 + warp * 16;   // I, Is are multiples of 64
            uint8_t* out = (sh ? a.shq : a.hq) + (int64_t)start * ld + i0;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                uint32_t m0 = 0, m1 = 0;
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    m0 = max(m0, am[w * kPass + 8 * t + 2 * c]);
                    m1 = max(m1, am[w * kPass + 8 * t + 2 * c + 1]);
                }
                const float b0 = __uint_as_float(fp8_amax_bits(m0)), b1 = __uint_as_float(fp8_amax_bits(m1));
                const float v0 = __fdiv_rn(448.0f, b0), v1 = __fdiv_rn(448.0f, b1);
                const uint32_t q0 = fp8_pair(acc0[t][0] * v0, acc0[t][1] * v1);   // rows gi: pairs 2c, 2c + 1
                const uint32_t q1 = fp8_pair(acc0[t][2] * v0, acc0[t][3] * v1);   // rows gi + 8
                // 16 codes per pair: staged so that a lane stores them as one chunk
                uint8_t* s0 = stg + (2 * c) * 16 + gi;
                s0[0] = (uint8_t)q0;
                s0[8] = (uint8_t)q1;
                s0[16] = (uint8_t)(q0 >> 8);
                s0[24] = (uint8_t)(q1 >> 8);
                __syncwarp();
                if (lane < 8 && 8 * t + lane < n && i0 < ld)
                    *reinterpret_cast<uint4*>(out + (int64_t)(8 * t + lane) * ld) =
                        *reinterpret_cast<const uint4*>(stg + lane * 16);
                __syncwarp();   // written again
                if (warp == 0 && gi == 0) {
                    float* so = (sh ? a.shs : a.hs) + (int64_t)m * (sh ? a.max_rows : a.max_pairs) + start;
                    if (8 * t + 2 * c < n) so[8 * t + 2 * c] = __fdiv_rn(b0, 448.0f);
                    if (8 * t + 2 * c + 1 < n) so[8 * t + 2 * c + 1] = __fdiv_rn(b1, 448.0f);
                }
            }
        } else {
            const int64_t p0 = (int64_t)(sh ? a.g.shared_row0 : 0) + start;
            const int h0 = m * 256 + warp * 32;   // the warp's 32 columns: one staged quarter
            bool big = false;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int i0 = 8 * t + 2 * c;
                const float w0 = sh ? 1.0f : __ldg(a.g.pair_w + start + min(i0, n - 1));
                const float w1 = sh ? 1.0f : __ldg(a.g.pair_w + start + min(i0 + 1, n - 1));
                float v[8];   // rows gi, + 8, + 16, + 24 of pair 2c, then of pair 2c + 1
                v[0] = acc0[t][0] * w0; v[1] = acc0[t][2] * w0; v[2] = acc1[t][0] * w0; v[3] = acc1[t][2] * w0;
                v[4] = acc0[t][1] * w1; v[5] = acc0[t][3] * w1; v[6] = acc1[t][1] * w1; v[7] = acc1[t][3] * w1;
                // fp16 staging with a power-of-two exponent per quarter (see gemm.cu)
                uint32_t st[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t mb = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t ab = __float_as_uint(v[4 * j + i]) & 0x7FFFFFFFu;
                        mb = max(mb, ab < 0x7F800000u ? ab : 0u);
                    }
#pragma unroll
                    for (int o = 4; o <= 16; o <<= 1) mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, o));
                    const int sft = (int)(mb >> 23) - 141;
                    st[j] = sft > 0 ? (uint32_t)sft : 0u;
                    const float f = __uint_as_float((127u - st[j]) << 23);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[4 * j + i] *= f;
                        reinterpret_cast<__half*>(stg)[(2 * c + j) * 32 + gi + 8 * i] = __float2half_rn(v[4 * j + i]);
                    }
                    if (st[j] && i0 + j < n) big = true;
                    if (gi == 0 && i0 + j < n)
                        a.g.ysx[(int64_t)(h0 >> 5) * a.g.ld_x + p0 + i0 + j] = (uint8_t)st[j];
                }
                __syncwarp();
                if (8 * t + gi < n)
                    *reinterpret_cast<uint4*>(a.g.ys + (p0 + 8 * t + gi) * a.g.H + h0 + c * 8) =
                        *reinterpret_cast<const uint4*>(stg + gi * 64 + c * 16);
                __syncwarp();   // written again
            }
            if (big) *a.g.scaled = 1;
        }
    };

    for (int u = ufirst; alive && u < nunits; u += nact) {
        const int4 un = __ldg(a.g.units + u);
        if (!valid(un)) continue;
        for (int i = 0; alive && i < un.w; i += kPass) {
            const int4 part = make_int4(un.x, un.y, un.z + i, min(kPass, un.w - i));
            if (part.w <= 8) run(std::integral_constant<int, 1>{}, part);
            else run(std::integral_constant<int, 2>{}, part);
        }
    }
}

template <int MODE>
static cudaError_t set_attr() {
    return cudaFuncSetAttribute(k_fp8_stream<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
}

cudaError_t fp8_stream_set_attributes() {
    cudaError_t e = set_attr<kGateUp>();
    return e == cudaSuccess ? set_attr<kDown>() : e;
}

cudaError_t launch_fp8_stream(int mode, const Fp8Maps& m, const Fp8GemmArgs& a, int num_sms,
                              cudaStream_t st) {
    auto k = mode == kGateUp ? k_fp8_stream<kGateUp> : k_fp8_stream<kDown>;
    return launch_kernel(k, dim3(num_sms), dim3(kThreads), kSmem, st, m.w0, m.w1, m.s0, m.s1, a);
}

}  // namespace moe
