// The whole layer for a few rows (up to 8) in one kernel: router, top-k, gate/up,
// SwiGLU, down, weighted sum and shared expert (moe_token_pass); or all but the router
// (moe_token_forward).
//
//   z = x W_r^T + bias;  top-k, w = softmax over the chosen
//   y = S(x) + sum_j w_j E_j(x),   E(x) = W_down (silu(W_gate x) * (W_up x))
//
// A few rows touch a few experts, whose weights take HBM some microseconds (one row of 256 experts
// of 512 x 2048, k = 8: 57 MB, 8.7 us): what a row of kernels costs between them is what there is to
// save.  One CTA per SM, launched cooperatively, goes through three steps:
//   1  a warp per expert and row: its logit, in the order of route_common.cuh
//   2  every CTA: top-k of all rows (in moe_block_route's order and arithmetic, so the same
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
// h lies in global memory between the steps: with bf16 weights rounded as the other paths
// round it (bf16; the shared expert's, which enters every row with weight 1, as two bf16 parts),
// with e4m3 ones in fp32, quantised by every reader with the formula of the other paths.
// Every CTA needs all of it: it is staged in shared memory first, where it fits (STAGED; 8
// rows of 8 experts of 512 do), so that a tile costs no round trip to L2.
//
// Latency is what costs.  So every warp keeps tiles of weights in flight, in shared memory,
// across the ends of units and across the barrier before the down step, and the CTA's down
// weights go to L2 while gate/up runs (the shared expert's while the top-k does; the chosen
// experts' gate/up weights in the microsecond that the list takes changed nothing).  Code that
// runs once is fetched while everything waits for it: loops are not unrolled, nothing is divided.
//
// From step 1 to 2 a logit is one word with the number of its call: who polls it has it with the
// number, where a barrier would cost a fence, a counter's round trip and the read (1.5 us more).
// From step 2 to 3: a counter, to which the CTAs add 1024 in all (the first one what the others,
// 1 each, leave); a CTA waits until it has left the 1024 that it started in.  Each call adds 1024,
// so that the counter needs no clearing, and numbers the calls.  Every wait is bounded; a CTA
// that gives up counts MOE_STATUS_WAIT_TIMEOUT, adds its share to the barrier that it will not
// reach, and leaves.
//
// Measured (replayed in a graph; the calls for any number of rows, which end in the same y, beside):
// one row 19.0 us (43), e4m3 15.8 (32), 2 rows 28 (48), e4m3 23.6 (37), 4 rows 43 (62), e4m3 34 (44), 8
// rows 68 (88; 366 MB, 5.3 TB/s), e4m3 53 (58); under a given routing one row 16.7 and 13.9, 8 rows
// 64 and 48.5.  One row: logits 1.2 us, their way 1.4, top-k 0.8, list 0.8, gate/up 8.2
// (37.7 MB), barrier 2.2 with what CTAs wait for one another, down 2.7.
#include "route_common.cuh"
#include "token.cuh"

namespace moe {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kGroup = 4;                       // warps that share a gate/up unit
constexpr int kGroups = kWarps / kGroup;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr int kMaxPairs = kTokenRows * 32;      // k <= 32
// What goes to L2 ahead, all CTAs' together: of the chosen experts' down weights; of the shared
// expert's gate/up, and of its down weights.  More than L2 holds is read twice: one row of H 8192,
// Is 16384 took 190 us with all of the shared expert's, 151 with 10, 20 or 40 MB of either (H 7168, Is
// 8192 103 and 89; H 2048, Is 512, which is below all of these, 19.2).
constexpr int64_t kPrefetchBytes = 40 << 20, kSharedPrefetchBytes = 20 << 20;

// A tile: 16 weight rows by 128 bytes of K; a lane holds 32 bytes of two rows.
template <bool FP8>
constexpr int kTileK = FP8 ? 128 : 64;
constexpr int kStage = 2048;   // shared memory of a tile in flight, per warp: each lane's 4 x 16 bytes

struct Smem {
    union {
        float part[2][kWarps][kTokenRows][17];  // partial sums (row, weight row)
        struct {                                // before the list is made:
            uint32_t mask[kMaxExperts];         // rows of an expert
            int32_t idx[kMaxPairs];             // [R, k]
            float w[kMaxPairs];
        };
    };
    float wt[kMaxPairs + 1][kTokenRows];        // weight of (listed expert, row); last the shared expert
    uint16_t hrow[kMaxPairs + 1][kTokenRows];   // staged h of (listed expert, row): 64 bytes from its start
    uint8_t slot[kMaxPairs][kTokenRows];        // first slot of (listed expert, row)
    int32_t list[kMaxPairs + 1];                // experts touched, ascending; then the shared one: 0
    uint8_t lmask[kMaxPairs + 1];               // their rows
    uint32_t used[kMaxExperts / 32];            // experts touched, a bit each
    uint32_t scratch[MOE_STATUS_WORDS];         // for status counts that another CTA makes
    int ok;
    uint32_t call;
};

// x in shared memory: rows an odd multiple of 64 bytes apart, so that a quarter-warp's reads (two
// rows, 64 bytes each) share no bank
__host__ __device__ constexpr int odd64(int bytes) { return bytes + (bytes % 128 ? 0 : 64); }
template <bool FP8>
__host__ __device__ constexpr int x_stride(int H) { return odd64(FP8 ? H : 2 * H); }
template <bool FP8>
__host__ __device__ constexpr int x_bytes(int H) {   // a multiple of 128: H % 256 == 0
    return kTokenRows * x_stride<FP8>(H) + (FP8 ? (H / kFp8Block) * kTokenRows * 4 : 0);
}
constexpr int kSmemHead = (int)(sizeof(Smem) + 127) / 128 * 128;
constexpr int kSmemMax = 227 * 1024;
static_assert(kTokenRows * 4 * (kMaxExperts + 96) <= 2 * kWarps * 2048, "keys and candidates fit the ring");
// h in x's place: a row of zeros, routed pairs (row r k + slot), then the shared expert's; bf16: its
// hi, then its lo parts; e4m3: codes, then their scales per block of 128, then a turn's scales of W
template <bool FP8>
__host__ __device__ constexpr int h_stride(int I) { return odd64(FP8 ? I : 2 * I); }
struct HPlan {
    int rstr, sstr, routed, shared, scales, wscales;   // strides and offsets in bytes
    int64_t bytes;
};
template <bool FP8>
__host__ __device__ inline HPlan h_plan(int R, int k, int I, int Is) {
    HPlan p{};
    p.rstr = h_stride<FP8>(I);
    p.sstr = h_stride<FP8>(Is);
    p.routed = p.rstr > p.sstr ? p.rstr : p.sstr;
    const int64_t shared = p.routed + (int64_t)R * k * p.rstr, scales = shared + (int64_t)R * (FP8 ? 1 : 2) * p.sstr;
    const int64_t tiles = (int64_t)R * k * fp8_blocks(I) + fp8_blocks(Is);
    const int64_t wscales = scales + (FP8 ? 4 * ((int64_t)R * k * fp8_blocks(I) + R * fp8_blocks(Is)) : 0);
    p.bytes = (wscales + (FP8 ? 4 * tiles : 0) + 127) / 128 * 128;
    if (p.bytes < kSmemMax) {
        p.shared = (int)shared;
        p.scales = (int)scales;
        p.wscales = (int)wscales;
    }
    return p;
}

__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
// 16 bytes, of which the first `bytes` (all or none) are read and the rest are zeros
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// All but the newest depth - 1 of this thread's copy groups are complete (depth 2 .. 5).
__device__ __forceinline__ void wait_tile(int depth) {
    if (depth == 5) cp_async_wait<4>();
    else if (depth == 4) cp_async_wait<3>();
    else if (depth == 3) cp_async_wait<2>();
    else cp_async_wait<1>();
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

// A lane's part of a tile, rows gi (a) and gi + 8 (b): bytes 16 c .. and 64 + 16 c .., so that
// four lanes read 64 in a row.
// From pa and pb (its first bytes of either row) to the lane's slots; `half`: K ends after 64
// bytes, zeros there.
__device__ __forceinline__ void copy_tile(uint32_t dst, const uint8_t* pa, const uint8_t* pb, bool half) {
    cp_async16(dst, pa);
    cp_async16(dst + 1024, pb);
    if (half) {
        copy16(dst + 512, pa, 0);
        copy16(dst + 1536, pb, 0);
    } else {
        cp_async16(dst + 512, pa + 64);
        cp_async16(dst + 1536, pb + 64);
    }
}
// d += tile . x, the tile in the lane's slots
template <bool FP8>
__device__ __forceinline__ void tile_mma(float (&d)[4], const uint4 (&a)[2], const uint4 (&b)[2], const uint4 (&x)[2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (FP8) {
            mma_e4m3(d, a[i].x, b[i].x, a[i].y, b[i].y, x[i].x, x[i].y);
            mma_e4m3(d, a[i].z, b[i].z, a[i].w, b[i].w, x[i].z, x[i].w);
        } else {
            mma_bf16(d, a[i].x, b[i].x, a[i].y, b[i].y, x[i].x, x[i].y);
            mma_bf16(d, a[i].z, b[i].z, a[i].w, b[i].w, x[i].z, x[i].w);
        }
    }
}

constexpr uint64_t kRound = 1024;
__device__ __forceinline__ uint64_t ld_round(const uint64_t* p) {
    uint64_t v;
    asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v & ~(kRound - 1);
}
// Releases what the CTA wrote before the __syncthreads ahead of it.
__device__ __forceinline__ void arrive(uint64_t* p) {
    const uint64_t n = blockIdx.x == 0 ? kRound - (gridDim.x - 1) : 1;
    asm volatile("red.release.gpu.global.add.u64 [%0], %1;" ::"l"(p), "l"(n) : "memory");
}
// A grid barrier; the whole CTA calls it.  round: the counter's at the start of the kernel (in
// thread 0).  False: gave up, the same in every thread.
__device__ __forceinline__ bool grid_barrier(uint64_t* counter, uint64_t round, uint64_t limit_ns, int* ok) {
    __syncthreads();
    if (threadIdx.x == 0) {
        arrive(counter);
        bool in = true;
        const uint64_t t0 = globaltimer_ns();
        while (in && ld_round(counter) == round) in = globaltimer_ns() - t0 <= limit_ns;
        *ok = in;
    }
    __syncthreads();
    return *ok;
}

// A logit and the call that it is of, in one word: who reads the call's number reads its logit, and
// neither a fence nor a barrier stands between.  Numbers: the rounds that the counter has ended
// modulo 2^32 - 1, plus 1 (0: a word never written).
__device__ __forceinline__ uint32_t call_number(uint64_t round) {
    const uint64_t c = round / kRound;
    uint32_t n = (uint32_t)c + (uint32_t)(c >> 32);   // 2^32 = 1 modulo 2^32 - 1
    if (n < (uint32_t)c) ++n;
    return n == 0xFFFFFFFFu ? 1u : n + 1;
}
__device__ __forceinline__ void store_tagged(uint64_t* p, float z, uint32_t call) {
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"((uint64_t)call << 32 | __float_as_uint(z)) : "memory");
}
__device__ __forceinline__ uint64_t ld_tagged(const uint64_t* p) {
    uint64_t v;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ float warp_sum(float v) {   // the xor butterfly of route_common.cuh
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// The logit of one expert and row, one warp.
__device__ __forceinline__ void expert_logit(const TokenArgs& a, int e, int r, int lane, uint32_t call) {
    constexpr int kS = 8;   // stripes of 256 at a time
    float acc = 0.0f;
    const __nv_bfloat16* w = a.wr + (int64_t)e * a.H + lane * 8;
    const __nv_bfloat16* x = a.x + (int64_t)r * a.H + lane * 8;
    for (int s0 = 0; s0 < a.H; s0 += 256 * kS) {
        uint4 wv[kS], xv[kS];
#pragma unroll
        for (int i = 0; i < kS; ++i) {
            const bool in = s0 + 256 * i < a.H;
            wv[i] = in ? __ldg(reinterpret_cast<const uint4*>(w + s0 + 256 * i)) : make_uint4(0, 0, 0, 0);
            xv[i] = in ? __ldg(reinterpret_cast<const uint4*>(x + s0 + 256 * i)) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kS; ++i)
            if (s0 + 256 * i < a.H) acc = dot8_bf16(xv[i], wv[i], acc);
    }
    const float z = warp_sum(acc);
    if (lane == 0) store_tagged(a.tagged + r * kMaxExperts + e, z, call);
}

// Rows with many equal logits: the top-k of route_common.cuh.  Not inlined: rarely called code.
// It reads logits alone: every CTA writes the same ones.
__device__ __noinline__ void topk_slow(const RouteArgs& ra, const uint64_t* tagged, int row, int lane) {
    for (int e = lane; e < ra.E; e += 32) ra.logits[(int64_t)row * ra.E + e] = __uint_as_float((uint32_t)ld_tagged(tagged + e));
    __syncwarp();
    route_topk(ra, row, row + 1, lane);
}

// How many of the first n keys at `keys` (a multiple of 4 is read) come before this lane's: larger
// ones, and equal ones in lower lanes.
__device__ __forceinline__ int rank_of(const uint32_t* keys, uint32_t mine, int lane, int n) {
    int rank = 0;
#pragma unroll 2
    for (int i = 0; i < n; i += 4) {
        const uint4 o = *reinterpret_cast<const uint4*>(keys + i);
        rank += (o.x > mine || (o.x == mine && i < lane)) + (o.y > mine || (o.y == mine && i + 1 < lane)) +
                (o.z > mine || (o.z == mine && i + 2 < lane)) + (o.w > mine || (o.w == mine && i + 3 < lane));
    }
    return rank;
}
// How many of the 32 keys at `keys` are at least this lane's.
__device__ __forceinline__ int at_least(const uint32_t* keys, uint32_t mine) {
    int n[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint4 o = *reinterpret_cast<const uint4*>(keys + 4 * i);
        n[0] += o.x >= mine;
        n[1] += o.y >= mine;
        n[2] += o.z >= mine;
        n[3] += o.w >= mine;
    }
    return n[0] + n[1] + (n[2] + n[3]);
}

// Top-k of one row, one warp: the order of route_topk, in fewer steps and less code.  Lane j gets the
// j-th chosen expert and its key; the weights can wait (topk_weight).
// The k-th largest of the lanes' own largest keys is a lower bound of the k-th largest key; few keys
// reach it, and their ranks among each other are counted.  tagged: the row's logits, waited for.
// buf: 96 words, then E keys.
enum { kGaveUp = 0, kChosen = 1, kWritten = 2 };   // kWritten: route_topk did it, to ra's outputs
constexpr int kTopkWords = 96;
__device__ __forceinline__ int topk_row(const RouteArgs& ra, const uint64_t* tagged, uint32_t call, uint64_t limit_ns,
                                        int row, int lane, uint32_t* buf, uint32_t& id, uint32_t& key, uint32_t& nonfinite) {
    uint32_t* keys = buf + kTopkWords;
    uint32_t top = 0;
    const uint64_t t0 = globaltimer_ns();
    constexpr int kN = 8;
    for (int e0 = lane; e0 - lane < ra.E; e0 += 32 * kN) {
        float bias[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) bias[i] = ra.bias && e0 + 32 * i < ra.E ? __ldg(ra.bias + e0 + 32 * i) : 0.0f;
        uint64_t v[kN];
        for (;;) {
            bool all = true;
#pragma unroll
            for (int i = 0; i < kN; ++i) v[i] = e0 + 32 * i < ra.E ? ld_tagged(tagged + e0 + 32 * i) : (uint64_t)call << 32;
#pragma unroll
            for (int i = 0; i < kN; ++i) all = all && (uint32_t)(v[i] >> 32) == call;
            if (__all_sync(0xffffffffu, all)) break;
            if (__any_sync(0xffffffffu, globaltimer_ns() - t0 > limit_ns)) return kGaveUp;
        }
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            if (e0 + 32 * i >= ra.E) continue;
            const float z = finish_logit_v(__uint_as_float((uint32_t)v[i]), ra.bias != nullptr, bias[i]);
            nonfinite += !isfinite(z);
            const uint32_t o = order_key(z);
            keys[e0 + 32 * i] = o;
            top = max(top, o);
        }
    }
    buf[lane] = top;
    buf[32 + lane] = 0;   // candidates' keys
    __syncwarp();
    const uint32_t bound = __reduce_max_sync(0xffffffffu, at_least(buf, top) >= ra.k ? top : 0u);
    int count = 0;
    for (int e0 = 0; e0 < ra.E; e0 += 128) {   // in ascending order of the experts
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = e0 + 32 * i + lane < ra.E ? keys[e0 + 32 * i + lane] : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = e0 + 32 * i + lane;
            const bool in = e < ra.E && o[i] >= bound;
            const uint32_t b = __ballot_sync(0xffffffffu, in);
            const int at = count + __popc(b & ((1u << lane) - 1));
            if (in && at < 32) {
                buf[32 + at] = o[i];
                buf[64 + at] = (uint32_t)e;
            }
            count += __popc(b);
        }
    }
    if (count > 32) {
        topk_slow(ra, tagged, row, lane);
        return kWritten;
    }
    __syncwarp();
    const uint32_t k1 = buf[32 + lane], e1 = buf[64 + lane];
    const int rank = rank_of(buf + 32, k1, lane, count);
    __syncwarp();
    if (lane < count) {   // each lane has read its own
        buf[rank] = k1;
        buf[64 + rank] = e1;
    }
    __syncwarp();
    id = buf[64 + lane];
    key = lane < ra.k ? buf[lane] : 0u;
    return kChosen;
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

template <bool FP8, bool STAGED>
__global__ void __launch_bounds__(kThreads, 1) k_token(TokenArgs a) {
    extern __shared__ __align__(128) uint8_t base[];
    Smem& s = *reinterpret_cast<Smem*>(base);
    uint8_t* sx = base + kSmemHead;
    const float* xs = reinterpret_cast<const float*>(sx + kTokenRows * x_stride<FP8>(a.H));
    constexpr int kES = FP8 ? 1 : 2;   // bytes per weight
    constexpr int kTK = kTileK<FP8>;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gi = lane >> 2, c = lane & 3;
    const int G = gridDim.x, cta = blockIdx.x;
    const uint64_t limit = a.wait_ns ? a.wait_ns : kWaitLimitNs;
    // Rounds of the down step's barrier: a counter each for the two calls, as only one of them numbers its
    // logits.  This CTA's own arrival is missing: the round cannot have ended.
    uint64_t* counter = a.counters + (a.given ? 0 : 1);
    const int tasks = a.given ? 0 : ((a.E - cta + G - 1) / G) * a.R;   // logits of this CTA
    const uint64_t round = tid == 0 || (lane == 0 && kWarps - 1 - warp < tasks) ? ld_round(counter) : 0;
    const uint8_t *wg = static_cast<const uint8_t*>(a.wg), *wu = static_cast<const uint8_t*>(a.wu),
                  *wd = static_cast<const uint8_t*>(a.wd), *sg = static_cast<const uint8_t*>(a.sg),
                  *su = static_cast<const uint8_t*>(a.su), *sd = static_cast<const uint8_t*>(a.sd);
    const int utiles = a.I / 8, stiles = a.Is / 8, dtiles = a.H / 16, np = a.R * a.k;

    // ---- step 1: logits
    int my_e = -1;         // given: lane j of warp r holds slot j of row r
    float my_w = 0.0f;
    if (a.given && warp < a.R && lane < a.k) {
        my_e = __ldg(a.topk_idx + warp * a.k + lane);
        my_w = __ldg(a.topk_w + warp * a.k + lane);
    }
    // the last warps first: the first ones stage x meanwhile
    for (int i = kWarps - 1 - warp; i < tasks; i += kWarps)
        expert_logit(a, cta + i / a.R * G, i % a.R, lane, call_number(round));
    stage_x<FP8>(a, sx);
    for (int i = tid; i < a.E; i += kThreads) s.mask[i] = 0;
    const HPlan hp = h_plan<FP8>(a.R, a.k, a.I, a.Is);
    if (STAGED)   // rows that did not choose an expert multiply zeros
        for (int i = tid; i < (kMaxPairs + 1) * kTokenRows; i += kThreads) (&s.hrow[0][0])[i] = 0;
    if (tid < kMaxExperts / 32) s.used[tid] = 0;
    if (tid < MOE_STATUS_WORDS) s.scratch[tid] = 0;
    if (tid == 0) {
        s.ok = 1;
        s.call = call_number(round);
    }
    __syncthreads();

    // the shared expert's weights to L2
    if (tid == kThreads - 1) {
        const uint32_t gb = 8u * a.H * kES, db = 16u * a.Is * kES;
        int left = (int)(kSharedPrefetchBytes / G / (2 * gb));
        for (int t = cta; t < stiles && left > 0; t += G, --left) {
            prefetch_l2(sg + (int64_t)t * gb, gb);
            prefetch_l2(su + (int64_t)t * gb, gb);
        }
        left = (int)(kSharedPrefetchBytes / G / db);
        for (int t = cta; t < dtiles && left > 0; t += G, --left) prefetch_l2(sd + (int64_t)t * db, db);
    }

    // ---- step 2: the experts of each row and the list of all of them
    uint32_t same = 0;     // slots of the row with the same expert
    uint32_t my_key = 0, nonfinite = 0;
    bool weigh = false;    // the row's weights are still to be formed
    int my_l = 0;          // place in the list of experts
    if (warp < a.R) {
        if (!a.given) {
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
            uint32_t* buf = reinterpret_cast<uint32_t*>(sx + a.arena) + warp * (((a.E + 3) & ~3) + kTopkWords);   // the ring is idle
            uint32_t id;
            const int got = topk_row(ra, a.tagged + warp * kMaxExperts, s.call, limit, warp, lane, buf, id, my_key, nonfinite);
            __syncwarp();
            if (got == kGaveUp) {
                s.ok = 0;
            } else if (lane < a.k) {
                my_e = got == kChosen ? (int)id : s.idx[warp * a.k + lane];
                my_w = got == kChosen ? 0.0f : s.w[warp * a.k + lane];
            }
            weigh = got == kChosen;
        }
        const bool good = lane < a.k && my_e >= 0 && my_e < a.E;
        const uint32_t ok = __ballot_sync(0xffffffffu, good);
        same = 1u << lane;
        if (a.given) same = __match_any_sync(0xffffffffu, good ? my_e : -1 - lane);
        if (good && lane == __ffs(same) - 1) {
            atomicOr(&s.mask[my_e], 1u << warp);
            atomicOr(&s.used[my_e >> 5], 1u << (my_e & 31));
        }
        if (a.given && cta == 0 && lane == 0) {
            status_add(a.status, MOE_STATUS_BAD_EXPERT_ID, a.k - __popc(ok));
            status_add(a.status, MOE_STATUS_EMPTY_ROWS, ok == 0);
        }
        if (!good) my_e = -1;
        // an expert in several slots: their weights in slot order, in the first of them
        uint32_t rest = same & (same - 1);
        if (a.given && __any_sync(0xffffffffu, rest != 0)) {
            float sum = my_w;
            for (int j = 0; j < 32; ++j) {
                const float o = __shfl_sync(0xffffffffu, my_w, j);
                if ((rest >> j) & 1u) sum += o;
            }
            my_w = sum;
        }
    }
    __syncthreads();
    if (!s.ok) {
        if (tid == 0) {
            status_add(a.status, MOE_STATUS_WAIT_TIMEOUT, 1);
            arrive(counter);   // the barrier that this CTA will not reach
        }
        return;
    }
    // an expert's place in the list: touched experts below it.  Lane i has word i of `used`.
    const uint32_t word = s.used[lane];
    int upto = __popc(word);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    const int nl = __shfl_sync(0xffffffffu, upto, 31);
    auto place = [&](int e) {   // all lanes take part
        const int i = e >> 5;
        const uint32_t w = __shfl_sync(0xffffffffu, word, i);
        return __shfl_sync(0xffffffffu, upto, i) - __popc(w) + __popc(w & ((1u << (e & 31)) - 1));
    };
    for (int e0 = 32 * warp; e0 < a.E; e0 += kThreads) {
        const int l = place(e0 + lane);
        const uint32_t m = e0 + lane < a.E ? s.mask[e0 + lane] : 0u;
        if (m) {
            s.list[l] = e0 + lane;
            s.lmask[l] = (uint8_t)m;
        }
    }
    if (warp < a.R) {
        my_l = place(my_e >= 0 ? my_e : 0);
        if (my_e >= 0 && lane == __ffs(same) - 1) {
            s.wt[my_l][warp] = my_w;
            s.slot[my_l][warp] = (uint8_t)lane;
            s.hrow[my_l][warp] = (uint16_t)((hp.routed + (warp * a.k + lane) * hp.rstr) / 64);
        }
    }
    if (tid < kTokenRows) {   // the shared expert follows
        s.wt[nl][tid] = 1.0f;
        s.hrow[nl][tid] = tid < a.R ? (uint16_t)((hp.shared + tid * hp.sstr) / 64) : 0;
        s.list[nl] = 0;
        s.lmask[nl] = (uint8_t)((1u << a.R) - 1);
    }
    __syncthreads();
    // The down step's tiles follow gate/up's without a gap: turn by turn 16 hidden outputs; the
    // tiles of all experts (the shared one's last) go round the warps.
    // The lane's slots of the tiles in flight, taken in turn:
    const int depth = a.depth;
    const uint32_t ring = smem_u32(sx) + a.arena + warp * (depth * kStage) + lane * 16;
    const uint32_t ring_end = ring + depth * kStage;
    uint32_t fill = ring, take = ring;
    auto next_slot = [&](uint32_t at) {
        at += kStage;
        return at == ring_end ? ring : at;
    };
    const int kb_r = (a.I + kTK - 1) / kTK, kb_s = (a.Is + kTK - 1) / kTK;   // tiles of an expert's K
    const int nr = nl * kb_r, items = nr + kb_s;
    const int iend = (items + kWarps - 1) / kWarps * kWarps;   // alike for all warps: nothing past the end
    const int dl = kWarps / kb_r, dk = kWarps - dl * kb_r, l0 = warp / kb_r;
    struct Item { int it, l, kb; };   // tile; its expert in the list and place in K
    auto settle = [&](Item& q) {      // tiles past the routed experts' are the shared one's
        if (q.it >= nr) {
            q.l = nl;
            q.kb = q.it - nr;
        }
    };
    auto first = [&](Item& q) {
        q.it = warp;
        q.l = l0;
        q.kb = warp - l0 * kb_r;
        settle(q);
    };
    auto advance = [&](Item& q) {
        q.it += kWarps;
        q.l += dl;
        q.kb += dk;
        if (q.kb >= kb_r) {
            q.kb -= kb_r;
            ++q.l;
        }
        settle(q);
    };
    // the next tile to copy, and the lane's first bytes of the turn's rows of expert 0 and of the shared one
    Item ld;
    first(ld);
    int lt = cta;
    const uint8_t *ldr = wd + (16 * (int64_t)lt + gi) * a.I * kES + 16 * c,
                  *lds = sd + (16 * (int64_t)lt + gi) * a.Is * kES + 16 * c;
    const uint32_t estride = (uint32_t)a.H * a.I * kES, turn_r = 16u * G * a.I * kES, turn_s = 16u * G * a.Is * kES;
    auto copy_down = [&]() {   // without the commit
        if (lt >= dtiles) return;
        if (ld.it < items) {
            const bool sh = ld.l == nl;
            const uint8_t* w = sh ? lds : ldr + (uint64_t)(uint32_t)s.list[ld.l] * estride;
            w += ld.kb * 128;
            const int K = sh ? a.Is : a.I;
            copy_tile(fill, w, w + 8 * K * kES, FP8 && K - ld.kb * 128 < 128);
        }
        if (ld.it + kWarps < iend) {
            advance(ld);
        } else {
            first(ld);
            lt += G;
            ldr += turn_r;
            lds += turn_s;
        }
    };
    // ---- gate/up: units of 8 intermediate indices, the shared expert's first
    __nv_bfloat16* hb = static_cast<__nv_bfloat16*>(a.h);   // bf16: routed, then the shared expert's hi and lo parts
    float* hf = static_cast<float*>(a.h);                   // e4m3: fp32
    const int64_t hpart = (int64_t)np * a.I, spart = (int64_t)a.R * a.Is;
    const uint32_t all = (1u << a.R) - 1;
    {
        const int group = warp / kGroup, gw = warp % kGroup;
        const int nunits = stiles + nl * utiles, ustep = G * kGroups;
        const int tiles = a.H / kTK;                        // of which this warp takes gw, gw + 4, ...
        const int kend = (tiles + kGroup - 1) / kGroup * kGroup + gw;   // as many steps in every warp: none past the end
        int lu = cta + G * group, lk = gw;   // the next tile to copy
        bool prefetched = false;
        const uint8_t *lg = wg, *lv = wu;
        // unit u: its expert (list index; shared: -1) and its tile there
        auto unit = [&](int u, int& ti) {
            if (u < stiles) {
                ti = u;
                return -1;
            }
            const int l = (int)__umulhi(u - stiles, a.inv_utiles);
            ti = u - stiles - l * utiles;
            return l;
        };
        auto copy_next = [&]() {
            if (lu < nunits) {
                if (lk == gw) {   // a new unit
                    int ti;
                    const int l = unit(lu, ti);
                    const int64_t o = ((l < 0 ? 0 : (int64_t)s.list[l] * a.I) + 8 * ti + gi) * a.H * kES + gw * 128 + 16 * c;
                    lg = (l < 0 ? sg : wg) + o;
                    lv = (l < 0 ? su : wu) + o;
                }
                if (lk < tiles) copy_tile(fill, lg, lv, false);
                lg += kGroup * 128;
                lv += kGroup * 128;
                lk += kGroup;
                if (lk >= kend) {
                    lk = gw;
                    lu += ustep;
                }
            } else {
                // then, once, the rest of this CTA's first turns' weights to L2
                if (warp == kWarps - 1 && !prefetched) {
                    prefetched = true;
                    const uint32_t db = 16u * a.I * kES;
                    const int most = (int)(kPrefetchBytes / G / db), mine = (dtiles - cta + G - 1) / G * nl;
#pragma unroll 1
                    for (int i = lane; i < min(most, mine); i += 32)
                        prefetch_l2(wd + ((int64_t)s.list[i % nl] * a.H + 16 * (cta + i / nl * G)) * a.I * kES, db);
                }
                copy_down();
            }
            cp_async_commit();
            fill = next_slot(fill);
        };
        // e4m3: the scales of this warp's tiles of a unit, gate's in lanes 0 .., up's in 16 ..
        // (H / 128 is at most 64, a quarter of it 16)
        auto scales_of = [&](int u) {
            const int k = gw + kGroup * (lane & 15);
            if (!FP8 || u >= nunits || k >= tiles) return 0.0f;
            int ti;
            const int l = unit(u, ti);
            const int64_t o = ((l < 0 ? 0 : (int64_t)s.list[l] * fp8_blocks(a.I)) + (ti >> 4)) * tiles + k;
            return __ldg((l < 0 ? (lane < 16 ? a.csg : a.csu) : (lane < 16 ? a.cg : a.cu)) + o);
        };
        float sc_next = scales_of(lu);
#pragma unroll 1
        for (int i = 0; i < depth - 1; ++i) copy_next();
        // with tiles on their way: the rows' weights, which the down step needs
        if (!a.given && warp < a.R) {
            const float w = weigh ? topk_weight(a.k, lane, my_key) : my_w;
            if (lane < a.k) {
                s.wt[my_l][warp] = w;
                if (cta == 0) {
                    a.topk_idx[warp * a.k + lane] = my_e;
                    a.topk_w[warp * a.k + lane] = w;
                }
            }
            nonfinite = __reduce_add_sync(0xffffffffu, nonfinite);
            if (weigh && cta == 0 && lane == 0) status_add(a.status, MOE_STATUS_NONFINITE_LOGITS, nonfinite);
        }
        const uint32_t xrow = smem_u32(sx) + gi * x_stride<FP8>(a.H) + 16 * c;
        const bool on = gi < a.R;
        int pb = 0;
#pragma unroll 1
        for (int u = cta + G * group; u < nunits; u += ustep) {
            float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            const float sc = sc_next;
            sc_next = scales_of(u + ustep);
#pragma unroll 1
            for (int kt = gw; kt < kend; kt += kGroup) {
                copy_next();
                wait_tile(depth);
                if (kt < tiles) {
                    const uint4 z = make_uint4(0, 0, 0, 0);
                    const uint4 x[2] = {on ? lds16(xrow + kt * 128) : z, on ? lds16(xrow + kt * 128 + 64) : z};
                    const uint4 ta[2] = {lds16(take), lds16(take + 512)}, tb[2] = {lds16(take + 1024), lds16(take + 1536)};
                    if (FP8) {
                        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        tile_mma<FP8>(d, ta, tb, x);
                        const float fa = __shfl_sync(0xffffffffu, sc, kt / kGroup), fb = __shfl_sync(0xffffffffu, sc, 16 + kt / kGroup);
                        // (scales of rows past R are left over: their columns are not read)
                        const float2 f = *reinterpret_cast<const float2*>(xs + kt * kTokenRows + 2 * c);
                        acc[0] = fmaf(f.x * fa, d[0], acc[0]);
                        acc[1] = fmaf(f.y * fa, d[1], acc[1]);
                        acc[2] = fmaf(f.x * fb, d[2], acc[2]);
                        acc[3] = fmaf(f.y * fb, d[3], acc[3]);
                    } else {
                        tile_mma<FP8>(acc, ta, tb, x);
                    }
                }
                take = next_slot(take);
            }
            // the unit's sums over its four warps, and h
#pragma unroll
            for (int j = 0; j < 4; ++j) s.part[pb][warp][2 * c + (j & 1)][gi + 8 * (j >> 1)] = acc[j];
            asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(32 * kGroup) : "memory");
            const int r = (tid & (32 * kGroup - 1)) >> 3, i = tid & 7;   // row, index
            int ti;
            const int l = unit(u, ti);
            const bool sh = l < 0;
            const uint32_t m = sh ? all : s.lmask[l];
            if (r < kTokenRows && ((m >> r) & 1u)) {
                float g = 0.0f, v = 0.0f;
#pragma unroll
                for (int w = 0; w < kGroup; ++w) {
                    g += s.part[pb][group * kGroup + w][r][i];
                    v += s.part[pb][group * kGroup + w][r][8 + i];
                }
                const float h = silu_fast(g) * v;
                const int p = sh ? r : r * a.k + s.slot[l][r];
                const int64_t at = (int64_t)p * (sh ? a.Is : a.I) + 8 * ti + i;
                if (FP8) {
                    hf[(sh ? hpart : 0) + at] = h;
                } else {
                    const __nv_bfloat16 hi = __float2bfloat16_rn(h);
                    __nv_bfloat16* o = hb + (sh ? hpart : 0) + at;
                    o[0] = hi;
                    if (sh) o[spart] = __float2bfloat16_rn(h - __bfloat162float(hi));
                }
            }
            pb ^= 1;   // written again behind the next unit's barrier: read by then
        }
    }

    // ---- step 3: down
    // e4m3: the scale of W for a tile: 16 outputs lie in one block of 128
    auto scale_of = [&](int t, int l, int kb) {
        return __ldg(l == nl ? a.csd + (int64_t)(t >> 3) * kb_s + kb
                             : a.cd + ((int64_t)s.list[l] * (a.H / kFp8Block) + (t >> 3)) * kb_r + kb);
    };
    auto scale_at = [&](int t, int it) {
        const int l = it < nr ? it / kb_r : nl;
        return scale_of(t, l, it < nr ? it - l * kb_r : it - nr);
    };
    float* wsc = reinterpret_cast<float*>(sx + hp.wscales);
    const bool early = FP8 && STAGED && cta < dtiles && tid < items;   // the first turn's are loaded before the barrier
    const float first_sc = early ? scale_at(cta, tid) : 0.0f;
    if (!grid_barrier(counter, round, limit, &s.ok)) {
        cp_async_wait<0>();
        if (tid == 0) status_add(a.status, MOE_STATUS_WAIT_TIMEOUT, 1);
        return;
    }
    if (cta >= dtiles) {
        cp_async_wait<0>();
        return;
    }
    if constexpr (STAGED) {
        for (int i = tid; i < hp.routed / 16; i += kThreads) *reinterpret_cast<uint4*>(sx + 16 * i) = make_uint4(0, 0, 0, 0);
        if constexpr (FP8) {   // a warp per row, half of it per block
            float* hsc = reinterpret_cast<float*>(sx + hp.scales);
            for (int p = warp; p < np + a.R; p += kWarps) {
                const bool sh = p >= np;
                const int K = sh ? a.Is : a.I, nb = sh ? kb_s : kb_r;
                const float* src = hf + (sh ? hpart + (int64_t)(p - np) * K : (int64_t)p * K);
                uint8_t* dst = sx + (sh ? hp.shared + (p - np) * hp.sstr : hp.routed + p * hp.rstr);
                float* sc = hsc + (sh ? np * kb_r + (p - np) * kb_s : p * kb_r);
#pragma unroll 2
                for (int b0 = 0; b0 < nb; b0 += 2) {
                    const int k = 128 * b0 + 8 * lane;
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {   // K % 64 == 0: eight values are all inside or none
                        const float4 f = k < K ? __ldcg(reinterpret_cast<const float4*>(src + k) + i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
                    }
                    uint32_t mx = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) mx = max(mx, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
                    for (int o = 8; o >= 1; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    const float bm = __uint_as_float(fp8_amax_bits(mx));
                    const float inv = __fdiv_rn(448.0f, bm);
                    if (k < K)
                        *reinterpret_cast<uint2*>(dst + k) = make_uint2(
                            fp8_pair(v[0] * inv, v[1] * inv) | fp8_pair(v[2] * inv, v[3] * inv) << 16,
                            fp8_pair(v[4] * inv, v[5] * inv) | fp8_pair(v[6] * inv, v[7] * inv) << 16);
                    if ((lane & 15) == 0 && k < K) sc[k >> 7] = __fdiv_rn(bm, 448.0f);
                }
            }
        } else {
            for (int p = warp; p < np + 2 * a.R; p += kWarps) {
                const bool sh = p >= np;
                const int K = sh ? a.Is : a.I;
                const __nv_bfloat16* src = hb + (sh ? hpart + (int64_t)(p - np) * K : (int64_t)p * K);
                const uint32_t dst = smem_u32(sx) + (sh ? hp.shared + (p - np) * hp.sstr : hp.routed + p * hp.rstr);
                for (int k = 8 * lane; k < K; k += 256) cp_async16(dst + 2 * k, src + k);
            }
            cp_async_commit();
            cp_async_wait<0>();
        }
    }
    {
        constexpr int kHN = FP8 ? 8 : 4;   // not staged: 16-byte pieces of h per lane and tile (bf16: hi, lo)
        // what the lane multiplies of tile q: row gi's part; zeros where the row did not choose the expert
        auto load_h = [&](const Item& q, uint4 (&v)[kHN]) {
            const bool sh = q.l == nl, on = q.it < items && ((s.lmask[q.l] >> gi) & 1u);
            const int K = sh ? a.Is : a.I;
            const int64_t at = on ? (int64_t)(sh ? gi : gi * a.k + s.slot[q.l][gi]) * K + q.kb * kTK : 0;
            const uint4 z = make_uint4(0, 0, 0, 0);
            if constexpr (FP8) {
                const float* src = hf + (sh ? hpart : 0) + at + 16 * c;
#pragma unroll
                for (int i = 0; i < kHN; ++i)   // K % 64 == 0: of 64 values all or none
                    v[i] = on && q.kb * kTK + 64 * (i >> 2) < K
                         ? __ldcg(reinterpret_cast<const uint4*>(src + 64 * (i >> 2)) + (i & 3)) : z;
            } else {
                const __nv_bfloat16* src = hb + (sh ? hpart : 0) + at + 8 * c;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    v[i] = on ? __ldcg(reinterpret_cast<const uint4*>(src + 32 * i)) : z;
                    v[2 + i] = on && sh ? __ldcg(reinterpret_cast<const uint4*>(src + spart + 32 * i)) : z;
                }
            }
        };
        const uint32_t hbase = smem_u32(sx) + 16 * c;
        uint4 h[STAGED ? 1 : kHN], hn[STAGED ? 1 : kHN];
        int pb = 0;
#pragma unroll 1
        for (int t = cta; t < dtiles; t += G) {
            float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            Item cur;
            first(cur);
            if constexpr (STAGED) {
                if (FP8) {
                    if (t == cta && early) wsc[tid] = first_sc;
                    for (int it = tid + (t == cta ? kThreads : 0); it < items; it += kThreads) wsc[it] = scale_at(t, it);
                }
                __syncthreads();   // h and the scales are there
            } else {
                load_h(cur, h);
            }
#pragma unroll 1
            for (; cur.it < iend; ) {
                copy_down();
                cp_async_commit();
                fill = next_slot(fill);
                Item nxt = cur;
                advance(nxt);
                if constexpr (!STAGED) load_h(nxt, hn);
                wait_tile(depth);
                if (cur.it < items) {
                    const bool sh = cur.l == nl;
                    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    const uint32_t m = (uint32_t)s.lmask[cur.l] >> (2 * c);
                    float2 f = *reinterpret_cast<const float2*>(&s.wt[cur.l][2 * c]);
                    const uint4 ta[2] = {lds16(take), lds16(take + 512)}, tb[2] = {lds16(take + 1024), lds16(take + 1536)};
                    if constexpr (STAGED) {
                        const int at = 64 * s.hrow[cur.l][gi];
                        const uint32_t hr = hbase + at + cur.kb * 128;
                        const uint4 x[2] = {lds16(hr), FP8 && (sh ? a.Is : a.I) - cur.kb * 128 < 128 ? make_uint4(0, 0, 0, 0) : lds16(hr + 64)};
                        tile_mma<FP8>(d, ta, tb, x);
                        if constexpr (FP8) {
                            // the scales of the lane's two columns (of a row that did not choose the expert: any)
                            const float* sc = reinterpret_cast<const float*>(sx + hp.scales) + (sh ? np * kb_r : 0) + cur.kb;
                            const int kbn = sh ? kb_s : kb_r, p0 = sh ? 2 * c : 2 * c * a.k + s.slot[cur.l][2 * c];
                            const int p1 = sh ? 2 * c + 1 : (2 * c + 1) * a.k + s.slot[cur.l][2 * c + 1];
                            const float sw = wsc[cur.it];
                            if (m & 1u) f.x *= sc[p0 * kbn] * sw;
                            if (m & 2u) f.y *= sc[p1 * kbn] * sw;
                        } else if (sh) {   // the lo part
                            const uint32_t lo = hr + (at ? a.R * hp.sstr : 0);
                            const uint4 xl[2] = {lds16(lo), lds16(lo + 64)};
                            tile_mma<FP8>(d, ta, tb, xl);
                        }
                    } else if constexpr (FP8) {
                        uint32_t mx = 0;
#pragma unroll
                        for (int i = 0; i < kHN; ++i)
                            mx = max(mx, max(max(h[i].x & 0x7FFFFFFFu, h[i].y & 0x7FFFFFFFu),
                                             max(h[i].z & 0x7FFFFFFFu, h[i].w & 0x7FFFFFFFu)));
                        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                        const float bm = __uint_as_float(fp8_amax_bits(mx));
                        const float inv = __fdiv_rn(448.0f, bm), scale = __fdiv_rn(bm, 448.0f);
                        uint32_t q[8];
#pragma unroll
                        for (int i = 0; i < kHN; ++i)
                            q[i] = fp8_pair(__uint_as_float(h[i].x) * inv, __uint_as_float(h[i].y) * inv) |
                                   fp8_pair(__uint_as_float(h[i].z) * inv, __uint_as_float(h[i].w) * inv) << 16;
                        const uint4 x[2] = {make_uint4(q[0], q[1], q[2], q[3]), make_uint4(q[4], q[5], q[6], q[7])};
                        tile_mma<FP8>(d, ta, tb, x);
                        const float sw = scale_of(t, cur.l, cur.kb);
                        f.x *= __shfl_sync(0xffffffffu, scale, 8 * c) * sw;   // row r's scale is in lanes 4 r ..
                        f.y *= __shfl_sync(0xffffffffu, scale, 8 * c + 4) * sw;
                    } else {
                        const uint4 xh[2] = {h[0], h[1]}, xl[2] = {h[2], h[3]};
                        tile_mma<FP8>(d, ta, tb, xh);
                        if (sh) tile_mma<FP8>(d, ta, tb, xl);
                    }
                    // columns of rows that did not choose the expert stay out (its weights may not be finite)
                    if (m & 1u) { acc[0] = fmaf(f.x, d[0], acc[0]); acc[2] = fmaf(f.x, d[2], acc[2]); }
                    if (m & 2u) { acc[1] = fmaf(f.y, d[1], acc[1]); acc[3] = fmaf(f.y, d[3], acc[3]); }
                }
                take = next_slot(take);
                cur = nxt;
                if constexpr (!STAGED) {
#pragma unroll
                    for (int i = 0; i < kHN; ++i) h[i] = hn[i];
                }
            }
            // the turn's sums over the warps
#pragma unroll
            for (int j = 0; j < 4; ++j) s.part[pb][warp][2 * c + (j & 1)][gi + 8 * (j >> 1)] = acc[j];
            __syncthreads();
            if (warp < kTokenRows / 2) {   // two rows per warp
                const int r = tid >> 4, n = tid & 15;
                float v = s.part[pb][0][r][n];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) v += s.part[pb][w][r][n];
                const uint32_t nf = __ballot_sync(0xffffffffu, !(fabsf(v) < INFINITY));
                if (r < a.R) {
                    const int64_t at = (int64_t)r * a.H + 16 * t + n;
                    a.y[at] = __float2bfloat16_rn(v);
                    if (a.y_f32) a.y_f32[at] = v;
                    if (n == 0) status_add(a.status, MOE_STATUS_NONFINITE_OUTPUT, ((nf >> (lane & 16)) & 0xFFFFu) != 0);
                }
            }
            pb ^= 1;   // written again behind the next turn's barriers: read by then
        }
        cp_async_wait<0>();
    }
}

namespace {

// Where x or h lie, and how many tiles are in flight: up to five, what fits beside them; h is
// staged where two do.
template <bool FP8>
void plan_smem(TokenArgs& a, bool* staged, int* bytes) {
    const int64_t x = x_bytes<FP8>(a.H), h = h_plan<FP8>(a.R, a.k, a.I, a.Is).bytes, room = kSmemMax - kSmemHead;
    *staged = h <= room - 2 * kWarps * kStage;
    a.arena = (int)(*staged && h > x ? h : x);
    const int64_t d = (room - a.arena) / (kWarps * kStage);
    a.depth = d < 5 ? (int)d : 5;
    *bytes = kSmemHead + a.arena + a.depth * kWarps * kStage;
}
static_assert(x_bytes<false>(kTokenMaxH) + 2 * kWarps * kStage <= kSmemMax - kSmemHead &&
              x_bytes<true>(kTokenMaxH) + 2 * kWarps * kStage <= kSmemMax - kSmemHead, "two tiles in flight");

}  // namespace

cudaError_t token_set_attributes() {
    cudaError_t e = cudaSuccess;
    auto set = [&](auto k) {
        if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    };
    set(k_token<false, false>);
    set(k_token<false, true>);
    set(k_token<true, false>);
    set(k_token<true, true>);
    return e;
}

cudaError_t launch_token(bool fp8, TokenArgs a, int num_sms, cudaStream_t st) {
    // u / d = umulhi(u, ceil(2^32 / d)) while u d < 2^32: u below 256 d and d up to 2048
    a.inv_utiles = (uint32_t)((((uint64_t)1 << 32) + a.I / 8 - 1) / (uint64_t)(a.I / 8));
    bool staged;
    int bytes;
    if (fp8) plan_smem<true>(a, &staged, &bytes);
    else plan_smem<false>(a, &staged, &bytes);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)num_sms);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;   // every CTA is resident: they wait for one another
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto k = fp8 ? (staged ? k_token<true, true> : k_token<true, false>)
                 : (staged ? k_token<false, true> : k_token<false, false>);
    return cudaLaunchKernelEx(&cfg, k, a);
}

}  // namespace moe
