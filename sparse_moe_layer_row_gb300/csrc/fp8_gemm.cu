// Block-scaled e4m3 products on the 5th-generation tensor core (sm_103a): the
// dense y = x W^T, and the grouped gate/up and down GEMMs of the expert FFN.
//
//   y[r, n] = sum over blocks b of 128 along K of
//             sx[b, r] * sw[n / 128, b] * sum_{k in b} qx[r, k] qw[n, k]
//
// The scales of a row and of a weight block differ from block to block along
// K, so the tensor core may sum one block of K only (four MMAs of K = 32); the
// eight promotion warps then read that partial sum from TMEM, multiply it by
// sx * sw and add it to accumulators in registers, in fp32.  Two TMEM buffers
// let the tensor core work on the next block of K meanwhile.
//
// A unit of work is 128 rows (the MMA's M, so a TMEM lane is a row, its scale
// one number per thread) by 256 weight rows (N):
//   gate/up  128 gate rows and the 128 up rows of the same intermediate
//            indices.  h = silu(g) u in fp32 is rounded to e4m3 with one scale
//            per row and 128 indices (fp8.cuh): a row's 128 values lie in the
//            two threads of its lane, which exchange their largest magnitude
//            through shared memory.
//   down     256 hidden outputs; the pair's weighted output is staged in fp16
//            with a power-of-two exponent per 32 columns, as k_combine reads it.
//   dense    256 outputs, stored in bf16, fp16 or fp32.
//
// Persistent, one CTA per SM, 384 threads (gate/up: 512):
//   warp 0 lane 0   TMA producer: weight tiles (2 x 16 KB) and, but for
//                   gate/up, the rows' tile (16 KB) into a ring of 3 stages
//   warp 1          TMEM allocation; issues the MMAs
//   warps 4..11     promotion and epilogue: lane quadrant warp & 3, columns by
//                   warpgroup
//   loaders         gate/up: warps 12..15, gather the unit's rows of x by
//                   16-byte cp.async into the swizzled tile (the MMA thread
//                   fences them for the async proxy); else warps 2, 3.  They
//                   also copy the block's scales and, with a unit's last block,
//                   its pair weights, into slots that the promotion warps read;
//                   all of it arrives on the slot's `rfull` when it lands
// Registers are moved from the other warpgroups to the promotion warps, which
// hold 128 accumulators each.  A promotion warp whose 32 rows lie past the
// unit's only passes the buffers on.  Outputs are staged in shared memory, a row
// per lane, and stored 256 consecutive bytes of a row at a time (one bulk copy
// per row instead: the same time).
// Every wait is bounded: a wait that gives up raises a CTA-wide abort flag and
// a device status counter, and all roles leave their loops; before the CTA
// exits its copies and MMAs in flight are waited for (with their own limit),
// and only then is the TMEM released.
//
// What bounds it: 8192 x 4096 x 2048 takes 66.5 us (2.07 PFLOP/s, 1.10 of the measured
// bf16 rate).  A block of K takes some 1030 clocks, of which the tensor core works
// 512 (46% of the cycles): the promotion warps' chain of a barrier, eight TMEM
// reads and 64 packed fmas is as long, and two buffers are all that TMEM holds.
// Four buffers of half the columns, TMEM reads of 32 or 64 columns, polling instead
// of sleeping waits and a test made under the last block's sums changed
// nothing.  The down GEMM's 8192-row call (135 us) writes 302 MB of staged
// outputs beside 300 MB that it reads: near half of a unit is its epilogue.
// All three instances spill a little (8 to 32 bytes stored, 44 to 96 loaded a thread).
#include "fp8.cuh"

namespace moe {

namespace {

constexpr uint64_t kWaitLimitNs = 2000000000ull;   // 2 s: far beyond any legal wait
constexpr uint64_t kDrainLimitNs = 200000000ull;   // 0.2 s when draining after an abort

constexpr int kStages = 3;
constexpr int kThreads = 384, kThreadsGU = 512;
constexpr int kTile = 128 * 128;                 // 128 rows x 128 codes
constexpr int kStageBytes = 3 * kTile;           // rows, weights 0, weights 1
constexpr int kAmaxOff = kStages * kStageBytes;       // uint32 [2 units][2 warpgroups][128 rows]
constexpr int kStgOff = kAmaxOff + 2 * 2 * 128 * 4;   // per promotion warp: 32 rows of 256 bytes,
constexpr int kStgRow = 256 + 16;                     // 16 apart, so that 8 lanes' chunks share no bank
constexpr int kStgWarp = 32 * kStgRow;
// Slots of the loaders' scales, one per fill of a stage, in turn, each with its
// barrier.  The fill kSlots later reuses a slot: it follows the MMA of the fill
// kSlots - kStages later, which follows the promotion (two TMEM buffers) of the
// fill kSlots - kStages - 2 later.
constexpr int kSlots = 8;
static_assert(kSlots - kStages - 2 > 0 && (kSlots & (kSlots - 1)) == 0, "a slot outlives its promotion and epilogue");
constexpr int kSxOff = kStgOff + 8 * kStgWarp;            // float [kSlots][128]: row scales
constexpr int kPwOff = kSxOff + kSlots * 512;         // float [kSlots][128]: pair weights (down)
constexpr int kSwOff = kPwOff + kSlots * 512;         // float [kSlots][2]: weight block scales
constexpr int kBarOff = kSwOff + kSlots * 8;
constexpr int kSmem = kBarOff + 256;
constexpr int kTmemCols = 512;                   // two buffers of 256 columns
// registers per thread after the split: the pool is what the CTA was launched
// with (kThreads x kLaunchRegs), checked on the host before any launch
constexpr int kLaunchRegs = 168, kFewRegs = 56, kManyRegs = 224;
constexpr int kLaunchRegsGU = 128, kFewRegsGU = 56, kManyRegsGU = 200;
static_assert(128 * kFewRegs + 256 * kManyRegs <= kThreads * kLaunchRegs, "register split");
static_assert(256 * kFewRegsGU + 256 * kManyRegsGU <= kThreadsGU * kLaunchRegsGU, "register split");
static_assert(kSmem <= 227 * 1024, "shared memory budget");
static_assert(8 * (2 * kStages + kSlots + 6) + 12 <= 256, "barrier region");

// kind::f8f6f4 with e4m3 A and B (format 0), fp32 accumulator, both K-major.
__device__ __forceinline__ uint32_t idesc_e4m3_f32(int M, int N) {
    return 1u << 4 | (uint32_t)(N >> 3) << 17 | (uint32_t)(M >> 4) << 24;
}

__device__ __forceinline__ void tc_mma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrive on `bar` once this thread's cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// 32 lanes x 16 columns of TMEM into registers; complete after tmem_ld_wait.
__device__ __forceinline__ void tmem_ld16_async(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld_wait() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// acc[j] += f * v[j], two at a time (fma.rn.f32x2: each half as fmaf).
__device__ __forceinline__ void promote16(float* acc, const uint32_t (&v)[16], float f) {
#pragma unroll
    for (int j = 0; j < 16; j += 2)
        asm("{\n\t.reg .b64 a, b, c;\n\t"
            "mov.b64 a, {%2, %3};\n\t"
            "mov.b64 b, {%4, %4};\n\t"
            "mov.b64 c, {%0, %1};\n\t"
            "fma.rn.f32x2 c, a, b, c;\n\t"
            "mov.b64 {%0, %1}, c;\n\t}"
            : "+f"(acc[j]), "+f"(acc[j + 1])
            : "r"(v[j]), "r"(v[j + 1]), "f"(f));
}

__device__ __forceinline__ void store16(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    *reinterpret_cast<uint4*>(p) = make_uint4(a, b, c, d);
}

// Rows of up to 256 staged bytes to global memory by the warp: 16 lanes a row.
__device__ __forceinline__ void copy_rows(const uint8_t* stg, uint8_t* out, int64_t ld, int bytes, int rows,
                                          int lane) {
    __syncwarp();
    const int ch = (lane & 15) * 16;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int r = 2 * i + (lane >> 4);
        if (r < rows && ch < bytes)
            *reinterpret_cast<uint4*>(out + r * ld + ch) = *reinterpret_cast<const uint4*>(stg + r * kStgRow + ch);
    }
    __syncwarp();   // written again
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t bf162_bits(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace

template <int MODE>
__global__ void __launch_bounds__(MODE == kGateUp ? kThreadsGU : kThreads, 1)
k_fp8_gemm(const __grid_constant__ CUtensorMap tmW0, const __grid_constant__ CUtensorMap tmW1,
           const __grid_constant__ CUtensorMap tmS0, const __grid_constant__ CUtensorMap tmS1,
           const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmA1,
           Fp8GemmArgs a) {
    extern __shared__ __align__(1024) uint8_t base[];   // swizzle atoms are 1 KB
    const uint32_t sbase = smem_u32(base);
    uint64_t* full = reinterpret_cast<uint64_t*>(base + kBarOff);  // [S] tiles landed
    uint64_t* rfull = full + kStages;                               // [kSlots] loaders' copies landed
    uint64_t* empty = rfull + kSlots;                               // [S] stage free
    uint64_t* tfull = empty + kStages;                              // [2] partial sums ready
    uint64_t* tempty = tfull + 2;                                   // [2] buffer free
    uint64_t* xbar = tempty + 2;                                    // amax exchange
    uint64_t* dbar = xbar + 1;                                      // MMA drain
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(dbar + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* never = abort_flag + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        for (int s = 0; s < kSlots; ++s) mbar_init(rfull + s, MODE == kGateUp ? 128 : 64);   // the loader threads
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull + i, 1);
            mbar_init(tempty + i, 8);   // the promotion warps
        }
        mbar_init(xbar, 256);
        mbar_init(dbar, 1);
        *abort_flag = 0;
        *never = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(tmem_slot, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();   // see common.cuh
    pdl_trigger();

    const int E = a.g.E;
    const int dense_m = (a.N + 255) / 256;
    const int nunits = MODE == kDense ? dense_m * ((a.R + kFp8Rows - 1) / kFp8Rows)
                                      : __ldg(a.g.n_units);
    const int nact = active_workers(nunits, (int)gridDim.x);   // balanced rounds
    const int ufirst = (int)blockIdx.x < nact ? (int)blockIdx.x : nunits;
    // unit u: group, weight tile, first row, rows
    auto unit = [&](int u) -> int4 {
        if (MODE != kDense) return __ldg(a.g.units + u);
        const int c = u / dense_m, m = u - c * dense_m;
        return make_int4(0, m, c * kFp8Rows, min(kFp8Rows, a.R - c * kFp8Rows));
    };
    auto valid = [&](const int4 un) {
        return MODE == kDense || unit_valid(un, a.g, kFp8Rows, MODE == kDown, kFp8GuRows, kFp8DnCols);
    };
    // blocks of 128 along K of a unit of group g
    auto blocks = [&](int g) {
        return MODE == kDense ? fp8_blocks(a.K)
             : MODE == kGateUp ? a.g.H / kFp8Block : fp8_blocks(g == E ? a.g.Is : a.g.I);
    };
    auto give_up = [&]() {
        if (!*abort_flag) { *abort_flag = 1; status_add(a.g.status, MOE_STATUS_WAIT_TIMEOUT, 1); }
    };
    const uint64_t kWaitNs = a.g.wait_ns ? a.g.wait_ns : kWaitLimitNs;

    // The loaders' loop.  Row i of a gate/up unit is copied by 8 threads, 16 bytes
    // each: chunk c of row i lands at chunk c ^ (i & 7) (the 128-byte swizzle).
    // Rows past the unit's are not loaded: they feed only TMEM lanes never stored.
    auto loader = [&]() {
        constexpr int kLt = MODE == kGateUp ? 128 : 64;
        const int lt = threadIdx.x - (MODE == kGateUp ? 384 : 64);   // 0 .. kLt - 1
        const int r16 = lt >> 3, ch = lt & 7;
        const uint32_t dst0 = sbase + r16 * 128 + ((ch ^ (r16 & 7)) << 4);
        int stage = 0, slot = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int u = ufirst; ok && u < nunits; u += nact) {
            const int4 un = unit(u);
            if (!valid(un)) continue;
            const int g = un.x, m = un.y, start = un.z, n = un.w;
            const bool sh = MODE != kDense && g == E;
            const int nkb = blocks(g);
            const float *px, *pw0, *pw1;   // scales: of row lt, of the two weight blocks
            int64_t ldx;
            int row[8];   // gate/up: the rows of x of this thread's chunks, -1: none
            if (MODE == kGateUp) {
                auto row_of = [&](int i) {
                    if (i >= n) return -1;
                    const int r = !sh ? __ldg(a.g.pair_row + start + i)
                                : (a.g.shared_rows ? __ldg(a.g.shared_rows + start + i) : start + i);
                    return r < a.g.R ? r : -1;
                };
#pragma unroll
                for (int j = 0; j < 8; ++j) row[j] = row_of(16 * j + r16);
                px = a.xs + max(row_of(lt), 0);
                ldx = a.g.R;
                const int mb = fp8_blocks(sh ? a.g.Is : a.g.I);
                const int64_t o = ((int64_t)(sh ? 0 : g) * mb + m) * nkb;
                pw0 = (sh ? a.sc_sa : a.sc_a) + o;
                pw1 = (sh ? a.sc_sb : a.sc_b) + o;
            } else if (MODE == kDown) {
                px = (sh ? a.shs : a.hs) + start;
                ldx = sh ? a.max_rows : a.max_pairs;
                const int hb = a.g.H / kFp8Block;
                pw0 = (sh ? a.sc_sa : a.sc_a) + ((int64_t)(sh ? 0 : g) * hb + 2 * m) * nkb;
                pw1 = pw0 + nkb;
            } else {
                px = a.xs + start;
                ldx = a.R;
                const int nb = fp8_blocks(a.N);
                pw0 = a.sc_a + (int64_t)(2 * m) * nkb;
                pw1 = a.sc_a + (int64_t)min(2 * m + 1, nb - 1) * nkb;
            }
            for (int kb = 0; kb < nkb; ++kb) {
                const bool free_ok = mbar_wait_bounded(empty + stage, phase ^ 1u, abort_flag, kWaitNs);
                if (__any_sync(0xffffffffu, !free_ok)) {   // the warp leaves together
                    give_up();
                    ok = false;
                    break;
                }
                const float* sxk = px + (int64_t)kb * ldx;
                for (int i = lt; i < n; i += kLt) {
                    cp_async4(sbase + kSxOff + (slot * 128 + i) * 4, MODE == kGateUp ? sxk : sxk + i);
                    if (MODE == kDown && kb == nkb - 1 && !sh)
                        cp_async4(sbase + kPwOff + (slot * 128 + i) * 4, a.g.pair_w + start + i);
                }
                if (lt < 2) cp_async4(sbase + kSwOff + (slot * 2 + lt) * 4, (lt ? pw1 : pw0) + kb);
                if (MODE == kGateUp) {
                    const uint32_t dst = dst0 + stage * kStageBytes;
                    const uint8_t* col = a.xq + kb * kFp8Block + ch * 16;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (row[j] >= 0) cp_async16(dst + j * 2048, col + (int64_t)row[j] * a.g.H);
                }
                cp_async_arrive(rfull + slot);
                if (++stage == kStages) { stage = 0; phase ^= 1u; }
                slot = (slot + 1) & (kSlots - 1);
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");   // nothing of this thread lands later
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(MODE == kGateUp ? kFewRegsGU : kFewRegs));
        if (warp == 0 && lane == 0) {
            // ------------------------------------------------------ TMA producer
            int stage = 0, nfills = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int u = ufirst; ok && u < nunits; u += nact) {
                const int4 un = unit(u);
                if (!valid(un)) continue;
                const int g = un.x, m = un.y, start = un.z;
                const bool sh = MODE != kDense && g == E;
                const int nkb = blocks(g);
                for (int kb = 0; kb < nkb; ++kb) {
                    if (!mbar_wait_bounded(empty + stage, phase ^ 1u, abort_flag, kWaitNs)) {
                        give_up();
                        ok = false;
                        break;
                    }
                    const uint32_t sA = sbase + stage * kStageBytes, sW = sA + kTile;
                    uint64_t* bar = full + stage;
                    const int kc = kb * kFp8Block;
                    mbar_expect_tx(bar, (uint32_t)(MODE == kGateUp ? 2 : 3) * kTile);
                    if (MODE == kGateUp) {
                        if (sh) {
                            tma_load_2d(sW, &tmS0, kc, m * 128, bar);
                            tma_load_2d(sW + kTile, &tmS1, kc, m * 128, bar);
                        } else {
                            tma_load_3d(sW, &tmW0, kc, m * 128, g, bar);
                            tma_load_3d(sW + kTile, &tmW1, kc, m * 128, g, bar);
                        }
                    } else if (MODE == kDown) {
                        for (int i = 0; i < 2; ++i) {
                            if (sh) tma_load_2d(sW + i * kTile, &tmS0, kc, m * 256 + i * 128, bar);
                            else tma_load_3d(sW + i * kTile, &tmW0, kc, m * 256 + i * 128, g, bar);
                        }
                        tma_load_2d(sA, sh ? &tmA1 : &tmA0, kc, start, bar);
                    } else {
                        for (int i = 0; i < 2; ++i)
                            tma_load_2d(sW + i * kTile, &tmW0, kc, m * 256 + i * 128, bar);
                        tma_load_2d(sA, &tmA0, kc, start, bar);
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
        } else if (warp == 1) {
            // -------------------------------------------------------- MMA issuer
            // The whole warp runs the loop, so that its values are uniform, and one
            // elected lane issues.  This loop is the kernel's pace-maker: with a lone
            // lane and three waits one after the other it took 1160 clocks per block, of
            // which the tensor core works 512.
            const uint32_t idesc = idesc_e4m3_f32(128, 256);
            const bool leader = elect_one();
            int stage = 0, slot = 0, buf = 0;
            uint32_t phase = 0, rphase = 0, bphase = 0;
            bool ok = true;
            for (int u = ufirst; ok && u < nunits; u += nact) {
                const int4 un = unit(u);
                if (!valid(un)) {
                    if (lane == 0) status_add(a.g.status, MOE_STATUS_BAD_UNIT, 1);
                    continue;
                }
                const int nkb = blocks(un.x);
                for (int kb = 0; kb < nkb; ++kb) {
                    // three tests at once, then the waits for what is not there yet
                    const bool t0 = mbar_test_wait(full + stage, phase);
                    const bool t1 = mbar_test_wait(rfull + slot, rphase);
                    const bool t2 = mbar_test_wait(tempty + buf, bphase ^ 1u);
                    if (!__all_sync(0xffffffffu, t0 && t1 && t2)) {
                        const bool got = mbar_wait_bounded(full + stage, phase, abort_flag, kWaitNs) &&
                                         mbar_wait_bounded(rfull + slot, rphase, abort_flag, kWaitNs) &&
                                         mbar_wait_bounded(tempty + buf, bphase ^ 1u, abort_flag, kWaitNs);
                        if (__any_sync(0xffffffffu, !got)) {
                            if (lane == 0) give_up();
                            ok = false;
                            break;
                        }
                    }
                    if (MODE == kGateUp) fence_proxy_async_smem();   // rows written by cp.async
                    tc_fence_after();
                    const uint32_t sA = sbase + stage * kStageBytes, sW = sA + kTile;
                    const uint32_t d = tmem + (uint32_t)(buf * 256);
                    const uint64_t ad = smem_desc_sw128(sA), bd = smem_desc_sw128(sW);
                    if (leader) {
                        // the two weight tiles follow each other: N = 256 rows of 128 bytes;
                        // 32 bytes along K are 2 in the descriptors' address field
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) tc_mma_e4m3(d, ad + 2 * kk, bd + 2 * kk, idesc, kk != 0);
                        tc_commit(tfull + buf);
                        tc_commit(empty + stage);
                    }
                    __syncwarp();
                    if (++stage == kStages) { stage = 0; phase ^= 1u; }
                    if (++slot == kSlots) { slot = 0; rphase ^= 1u; }
                    buf ^= 1;
                    if (buf == 0) bphase ^= 1u;
                }
            }
            // drain: arrives once every MMA issued above has completed
            if (leader) tc_commit(dbar);
            __syncwarp();
            if (!mbar_wait_bounded(dbar, 0, never, kDrainLimitNs) && lane == 0) give_up();
        } else if (MODE != kGateUp && warp >= 2) {
            loader();
        }
    } else if (MODE == kGateUp && warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegsGU));
        loader();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(MODE == kGateUp ? kManyRegsGU : kManyRegs));
        // ------------------------------------------------ promotion and epilogue
        const int q = warp & 3;           // TMEM lane quadrant this warp may read
        const int wg = (warp - 4) >> 2;   // 0 or 1
        const int t = q * 32 + lane;      // row of the unit
        // the thread's two groups of 64 columns: gate/up: g and u of the same 64
        // intermediate indices; else 128 columns in a row
        const uint32_t col0 = (uint32_t)(MODE == kGateUp ? wg * 64 : wg * 128);
        const uint32_t col1 = (uint32_t)(MODE == kGateUp ? 128 + wg * 64 : wg * 128 + 64);
        const uint32_t tq = tmem + ((uint32_t)(q * 32) << 16);
        uint32_t* s_amax = reinterpret_cast<uint32_t*>(base + kAmaxOff);
        uint8_t* stg = base + kStgOff + (warp - 4) * kStgWarp;
        const volatile float* s_sx = reinterpret_cast<const volatile float*>(base + kSxOff) + t;
        const volatile float* s_sw = reinterpret_cast<const volatile float*>(base + kSwOff);
        int buf = 0, upar = 0, slot = 0;
        uint32_t bphase = 0, xphase = 0;
        bool alive = true;
        int4 next = ufirst < nunits ? unit(ufirst) : make_int4(0, 0, 0, 0);
        for (int u = ufirst; alive && u < nunits; u += nact) {
            const int4 un = next;
            if (u + nact < nunits) next = unit(u + nact);   // long before it is needed
            if (!valid(un)) continue;
            const int g = un.x, m = un.y, start = un.z, n = un.w;
            const bool sh = MODE != kDense && g == E;
            const int nkb = blocks(g);
            const bool act = q * 32 < n;   // the warp has rows of the unit
            float acc[128];
#pragma unroll
            for (int j = 0; j < 128; ++j) acc[j] = 0.0f;
            bool ok;
            for (int kb = 0; kb < nkb; ++kb) {
                ok = mbar_wait_bounded(tfull + buf, bphase, abort_flag, kWaitNs);
                if (__any_sync(0xffffffffu, !ok)) { give_up(); alive = false; break; }
                tc_fence_after();
                const uint32_t tb = tq + (uint32_t)(buf * 256);
                // the block's scales: the MMA thread saw their slot land before it issued
                // the MMAs that this wait was for (a wait of each warp's own for the slot
                // took 13 of 88 us at 8192 x 4096 x 2048)
                const float sx = s_sx[slot * 128];
                const float f0 = sx * s_sw[slot * 2 + (MODE == kGateUp ? 0 : wg)];
                const float f1 = sx * s_sw[slot * 2 + (MODE == kGateUp ? 1 : wg)];
                slot = (slot + 1) & (kSlots - 1);
                if (act) {
                    uint32_t v[2][16];   // the next 16 columns are read while these are added
                    tmem_ld16_async(tb + col0, v[0]);
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        tmem_ld_wait();
                        if (c < 7)
                            tmem_ld16_async(tb + (c < 3 ? col0 + 16 * (c + 1) : col1 + 16 * (c - 3)), v[(c + 1) & 1]);
                        if (c == 7) {   // the buffer has been read: hand it back
                            tc_fence_before();
                            if (lane == 0) mbar_arrive(tempty + buf);
                        }
                        promote16(acc + 16 * c, v[c & 1], c < 4 ? f0 : f1);
                    }
                } else if (lane == 0) {
                    mbar_arrive(tempty + buf);
                }
                buf ^= 1;
                if (buf == 0) bphase ^= 1u;
            }
            if (!alive) break;
            if (MODE == kGateUp) {
                // h of the 64 indices, in place over g
                uint32_t mx = 0;
#pragma unroll
                for (int j = 0; j < 64; ++j) {
                    acc[j] = silu_fast(acc[j]) * acc[64 + j];
                    mx = max(mx, __float_as_uint(acc[j]) & 0x7FFFFFFFu);
                }
                // the row's largest magnitude: the other half is in the other
                // warpgroup.  Two buffers, taken in turn: a warp can be at most one
                // exchange ahead of another.
                uint32_t* am = s_amax + upar * 256;
                am[wg * 128 + t] = mx;
                mbar_arrive(xbar);
                ok = mbar_wait_bounded(xbar, xphase, abort_flag, kWaitNs);
                if (__any_sync(0xffffffffu, !ok)) { give_up(); alive = false; break; }
                mx = max(mx, am[(wg ^ 1) * 128 + t]);
                upar ^= 1;
                xphase ^= 1u;
                const float bm = __uint_as_float(fp8_amax_bits(mx));
                // one more rounding than the quotient of fp8.cuh: h is a sum's rounding away
                // from its exact value anyway
                const float inv = __fdiv_rn(448.0f, bm);
                const int ld = sh ? a.g.Is : a.g.I;
                const int i0 = m * 128 + wg * 64;   // I, Is are multiples of 64
                if (act && i0 < ld) {   // 64 codes of a row, 80 bytes apart
                        uint8_t* row = stg + lane * 80;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float* h = acc + 16 * j + 4 * i;
                            w[i] = fp8_pair(h[0] * inv, h[1] * inv) | fp8_pair(h[2] * inv, h[3] * inv) << 16;
                        }
                        store16(row + 16 * j, w[0], w[1], w[2], w[3]);
                    }
                    __syncwarp();
                    uint8_t* out = (sh ? a.shq : a.hq) + (int64_t)(start + q * 32) * ld + i0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = 8 * i + (lane >> 2), ch = (lane & 3) * 16;
                        if (q * 32 + r < n)
                            *reinterpret_cast<uint4*>(out + (int64_t)r * ld + ch) =
                                *reinterpret_cast<const uint4*>(stg + r * 80 + ch);
                    }
                    __syncwarp();   // written again
                }
                if (wg == 0 && t < n)
                    (sh ? a.shs : a.hs)[(int64_t)m * (sh ? a.max_rows : a.max_pairs) + start + t] =
                        __fdiv_rn(bm, 448.0f);
            } else if (MODE == kDown) {
                if (!act) continue;
                const int64_t p0 = (int64_t)(sh ? a.g.shared_row0 : 0) + start + q * 32;
                // the slot of the unit's last block
                const float w = sh ? 1.0f : reinterpret_cast<const float*>(base + kPwOff)[((slot - 1) & (kSlots - 1)) * 128 + t];
                const int h0 = m * 256 + wg * 128;
                uint8_t* row = stg + lane * kStgRow;
                bool big = false;
#pragma unroll
                for (int c = 0; c < 128; c += 32) {
                    // fp16 holds |v| < 65504: a quarter of 32 columns whose largest
                    // finite magnitude is 2^15 or more is stored as v * 2^-s, s its
                    // exponent above 2^14 (see gemm.cu)
                    float mx = 0.0f;   // fmaxf skips NaN
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        acc[c + j] *= w;
                        mx = fmaxf(mx, fabsf(acc[c + j]));
                    }
                    uint32_t st = 0;
                    if (mx >= 32768.0f) {
                        uint32_t mb = 0;
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const uint32_t ab = __float_as_uint(acc[c + j]) & 0x7FFFFFFFu;
                            mb = max(mb, ab < 0x7F800000u ? ab : 0u);
                        }
                        const int sft = (int)(mb >> 23) - 141;
                        st = sft > 0 ? (uint32_t)sft : 0u;
                        big = big || st != 0;
                        const float f = __uint_as_float((127u - st) << 23);
#pragma unroll
                        for (int j = 0; j < 32; ++j) acc[c + j] *= f;
                    }
                    if (t < n) a.g.ysx[(int64_t)((h0 + c) >> 5) * a.g.ld_x + p0 + lane] = (uint8_t)st;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float* v = acc + c + 8 * j;
                        store16(row + 2 * c + 16 * j, half2_bits(v[0], v[1]), half2_bits(v[2], v[3]),
                                half2_bits(v[4], v[5]), half2_bits(v[6], v[7]));
                    }
                }
                copy_rows(stg, reinterpret_cast<uint8_t*>(a.g.ys + p0 * a.g.H + h0), (int64_t)a.g.H * 2, 256,
                          n - q * 32, lane);
                if (big && t < n) *a.g.scaled = 1;
            } else {
                if (!act) continue;
                const bool f32 = a.ydtype == MOE_F32, bf = a.ydtype == MOE_BF16;
                const int es = f32 ? 4 : 2;
                uint8_t* row = stg + lane * kStgRow;
                // 256 bytes of a row at a time: 64 fp32 or 128 16-bit columns
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    const int n0 = m * 256 + wg * 128 + part * 64;
                    if ((part && !f32) || n0 >= a.N) break;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (f32) {
                                w[i] = __float_as_uint(acc[64 * part + 4 * j + i]);
                            } else {
                                const float* v = acc + 8 * j + 2 * i;
                                w[i] = bf ? bf162_bits(v[0], v[1]) : half2_bits(v[0], v[1]);
                            }
                        }
                        store16(row + 16 * j, w[0], w[1], w[2], w[3]);
                    }
                    uint8_t* out = static_cast<uint8_t*>(a.y) + ((int64_t)(start + q * 32) * a.ldy + n0) * es;
                    const int64_t ldb = a.ldy * es;
                    const int cb = min(256 / es, a.N - n0) * es;   // bytes of each row
                    if (a.y_vec && cb % 16 == 0) {
                        copy_rows(stg, out, ldb, cb, n - q * 32, lane);
                    } else {   // rows at any element: a row at a time, consecutive elements per lane
                        __syncwarp();
                        const int nr = min(32, n - q * 32);
                        for (int r = 0; r < nr; ++r)
                            for (int b = lane * es; b < cb; b += 32 * es) {
                                const uint8_t* src = stg + r * kStgRow + b;
                                if (f32) *reinterpret_cast<uint32_t*>(out + r * ldb + b) = *reinterpret_cast<const uint32_t*>(src);
                                else *reinterpret_cast<uint16_t*>(out + r * ldb + b) = *reinterpret_cast<const uint16_t*>(src);
                            }
                        __syncwarp();   // written again
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int MODE>
static cudaError_t set_attr() {
    cudaError_t e = cudaFuncSetAttribute(k_fp8_gemm<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    // the register split draws on what the CTA is launched with
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, k_fp8_gemm<MODE>)) != cudaSuccess) return e;
    return fa.numRegs == (MODE == kGateUp ? kLaunchRegsGU : kLaunchRegs) ? cudaSuccess : cudaErrorInvalidDeviceFunction;
}

cudaError_t fp8_gemm_set_attributes() {
    cudaError_t e = set_attr<kGateUp>();
    if (e == cudaSuccess) e = set_attr<kDown>();
    return e == cudaSuccess ? set_attr<kDense>() : e;
}

cudaError_t launch_fp8_gemm(int mode, const Fp8Maps& m, const Fp8GemmArgs& a, int num_sms,
                            cudaStream_t st) {
    auto k = mode == kGateUp ? k_fp8_gemm<kGateUp> : mode == kDown ? k_fp8_gemm<kDown> : k_fp8_gemm<kDense>;
    return launch_kernel(k, dim3(num_sms), dim3(mode == kGateUp ? kThreadsGU : kThreads), kSmem, st, m.w0, m.w1, m.s0, m.s1, m.a0,
                         m.a1, a);
}

}  // namespace moe
