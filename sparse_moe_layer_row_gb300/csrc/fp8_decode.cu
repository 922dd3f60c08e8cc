// The expert FFN on e4m3 weights for a single token, or a few on a small layer: a
// call whose weights take HBM a few microseconds, so that latency bounds it.
//
// Few experts are touched, and units of 256 weight rows (fp8_stream.cu) would
// leave most SMs idle: one row has 36 of them for the gate/up GEMM.  Here a CTA
// takes an eighth of a unit and its eight warps share K, as in fp8_rows.cu: one
// round of loads straight to registers, one round of mma.sync m16n8k32 (weights as
// M, pairs as N), one exchange through shared memory.
//
//   gate/up  16 intermediate indices (16 gate rows and 16 up rows).  An eighth of a
//            block of 128 cannot know the block's largest |h|, so h stays fp32.
//   down     32 hidden outputs.  A lane quantises the 32 values of h that it
//            multiplies: the four lanes of a pair hold its block of 128.  The same
//            formula on the same h as the other paths.  Weights and unit list do
//            not depend on the gate/up kernel: they are loaded before the wait for it.
//
// One row of the 2048 x 512 layer with 8 of 256 experts takes 15.7 us with its front and
// combine, four dependent launches of some 4 us each; its 25.8 MB would take 3.9.
#include "fp8.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8;
constexpr int kSub = kFp8DecodeSub;   // CTAs per unit
constexpr int kRowsN = kFp8DecodeRows;
static_assert(kRowsN == 8, "one tile of pairs");

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A lane's operands of one block of K for a 16-row tile: 32 bytes of rows gi and gi + 8.
struct Tile {
    uint4 a[2], b[2];
};
__device__ __forceinline__ Tile load_tile(const uint8_t* w, int64_t ld, int at, int K) {
    Tile t;
#pragma unroll
    for (int i = 0; i < 2; ++i) {   // zeros past the row's end (K % 16 == 0)
        const bool in = at + 16 * i < K;
        const uint4 z = make_uint4(0, 0, 0, 0);
        t.a[i] = in ? __ldg(reinterpret_cast<const uint4*>(w + at + 16 * i)) : z;
        t.b[i] = in ? __ldg(reinterpret_cast<const uint4*>(w + 8 * ld + at + 16 * i)) : z;
    }
    return t;
}
// acc += (tile . pairs) scaled: f0, f1 for the lane's two pairs
__device__ __forceinline__ void block_mma(float (&acc)[4], const Tile& t, const uint4 (&x)[2], float f0, float f1) {
    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    mma_e4m3(d, t.a[0].x, t.b[0].x, t.a[0].y, t.b[0].y, x[0].x, x[0].y);
    mma_e4m3(d, t.a[0].z, t.b[0].z, t.a[0].w, t.b[0].w, x[0].z, x[0].w);
    mma_e4m3(d, t.a[1].x, t.b[1].x, t.a[1].y, t.b[1].y, x[1].x, x[1].y);
    mma_e4m3(d, t.a[1].z, t.b[1].z, t.a[1].w, t.b[1].w, x[1].z, x[1].w);
    acc[0] = fmaf(f0, d[0], acc[0]);
    acc[1] = fmaf(f1, d[1], acc[1]);
    acc[2] = fmaf(f0, d[2], acc[2]);
    acc[3] = fmaf(f1, d[3], acc[3]);
}

}  // namespace

__global__ void __launch_bounds__(32 * kWarps) k_fp8_decode_gu(Fp8DecodeArgs a) {
    pdl_wait();  // see common.cuh: nothing global is touched before
    pdl_trigger();   // not earlier: the down kernel reads the unit list before its wait
    __shared__ float part[kWarps][2][kRowsN][17];
    const int u = blockIdx.x / kSub, sub = blockIdx.x % kSub;
    const GemmArgs& ga = a.f.g;
    // both loads at once: entry u is inside the list's memory, if not always written
    const int4 un = __ldg(ga.units + u);
    if (u >= __ldg(ga.n_units)) return;
    if (!unit_valid(un, ga, kRowsN, false, kFp8GuRows)) {
        if (sub == 0 && threadIdx.x == 0) status_add(ga.status, MOE_STATUS_BAD_UNIT, 1);
        return;
    }
    const int g = un.x, m = un.y, start = un.z, n = un.w;
    const bool sh = g == ga.E;
    const int ld = sh ? ga.Is : ga.I, i0 = m * 128 + sub * 16;
    if (i0 >= ld) return;   // I, Is are multiples of 64
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gi = lane >> 2, c = lane & 3;
    const int H = ga.H, kb_n = H / kFp8Block;
    const int64_t wo = ((int64_t)(sh ? 0 : g) * ld + i0 + gi) * H + 32 * c;
    const uint8_t* wg = (sh ? a.w_sa : a.w_a) + wo;
    const uint8_t* wu = (sh ? a.w_sb : a.w_b) + wo;
    const int64_t so = ((int64_t)(sh ? 0 : g) * fp8_blocks(ld) + m) * kb_n;
    const float* pg = (sh ? a.f.sc_sa : a.f.sc_a) + so;
    const float* pu = (sh ? a.f.sc_sb : a.f.sc_b) + so;
    // pairs past the unit's repeat its last: they feed columns that are not stored
    auto row_of = [&](int i) {
        const int p = start + min(i, n - 1);
        const int r = !sh ? __ldg(ga.pair_row + p) : (ga.shared_rows ? __ldg(ga.shared_rows + p) : p);
        return min(max(r, 0), ga.R - 1);
    };
    const uint8_t* px = a.f.xq + (int64_t)row_of(gi) * H + 32 * c;
    const float* ps0 = a.f.xs + row_of(2 * c);
    const float* ps1 = a.f.xs + row_of(2 * c + 1);
    float ag[4] = {0.0f, 0.0f, 0.0f, 0.0f}, au[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int kb = warp; kb < kb_n; kb += 2 * kWarps) {
        Tile tg[2], tu[2];
        uint4 x[2][2];
        float s0[2], s1[2], sg[2], su[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {   // every load first
            const int k = kb + h * kWarps;
            const int end = k < kb_n ? H : 0;   // none past the last block
            const int at = k * kFp8Block;
            tg[h] = load_tile(wg, H, at, end);
            tu[h] = load_tile(wu, H, at, end);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                x[h][i] = at < end ? __ldg(reinterpret_cast<const uint4*>(px + at + 16 * i)) : make_uint4(0, 0, 0, 0);
            s0[h] = at < end ? __ldg(ps0 + (int64_t)k * ga.R) : 0.0f;
            s1[h] = at < end ? __ldg(ps1 + (int64_t)k * ga.R) : 0.0f;
            sg[h] = at < end ? __ldg(pg + k) : 0.0f;
            su[h] = at < end ? __ldg(pu + k) : 0.0f;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            block_mma(ag, tg[h], x[h], s0[h] * sg[h], s1[h] * sg[h]);
            block_mma(au, tu[h], x[h], s0[h] * su[h], s1[h] * su[h]);
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {   // D: rows gi, gi + 8 of pairs 2c, 2c + 1
        part[warp][0][2 * c + (j & 1)][gi + 8 * (j >> 1)] = ag[j];
        part[warp][1][2 * c + (j & 1)][gi + 8 * (j >> 1)] = au[j];
    }
    __syncthreads();
    const int t = threadIdx.x >> 4, i = threadIdx.x & 15;   // pair, index
    if (t < n) {
        float gv = part[0][0][t][i], uv = part[0][1][t][i];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            gv += part[w][0][t][i];
            uv += part[w][1][t][i];
        }
        (sh ? a.sh32 : a.h32)[(int64_t)(start + t) * ld + i0 + i] = silu_fast(gv) * uv;
    }
}

__global__ void __launch_bounds__(32 * kWarps) k_fp8_decode_dn(Fp8DecodeArgs a) {
    __shared__ float part[4][2][kRowsN][17];
    const int u = blockIdx.x / kSub, sub = blockIdx.x % kSub;
    const GemmArgs& ga = a.f.g;
    // the unit list was written by the scatter, complete before the gate/up kernel
    // let this one start (common.cuh)
    const int4 un = __ldg(ga.units + u);
    const bool on = u < __ldg(ga.n_units);
    const bool good = on && unit_valid(un, ga, kRowsN, true, kFp8GuRows, kFp8DnCols);
    if (!good) {
        if (on && sub == 0 && threadIdx.x == 0) status_add(ga.status, MOE_STATUS_BAD_UNIT, 1);
        pdl_wait();
        pdl_trigger();
        return;
    }
    const int g = un.x, m = un.y, start = un.z, n = un.w;
    const bool sh = g == ga.E;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gi = lane >> 2, c = lane & 3, tile = warp & 1, kpart = warp >> 1;
    const int K = sh ? ga.Is : ga.I, kb_n = fp8_blocks(K), H = ga.H;
    const int h0 = m * 256 + sub * 32;
    const uint8_t* w = (sh ? a.w_sa : a.w_a) + ((int64_t)(sh ? 0 : g) * H + h0 + 16 * tile + gi) * K;
    const float* pw = (sh ? a.f.sc_sa : a.f.sc_a) + ((int64_t)(sh ? 0 : g) * (H / kFp8Block) + h0 / kFp8Block) * kb_n;
    const float* ph = (sh ? a.sh32 : a.h32) + (int64_t)(start + min(gi, n - 1)) * K;
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    bool waited = false;
    for (int kb = kpart; kb < kb_n || !waited; kb += 4) {
        const int at = kb * kFp8Block + 32 * c;
        const Tile t = load_tile(w, K, at, K);
        const float sw = kb < kb_n ? __ldg(pw + kb) : 0.0f;
        if (!waited) {   // the weights are on their way; now h
            pdl_wait();
            pdl_trigger();
            waited = true;
        }
        if (kb >= kb_n) break;
        float4 v[8];
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {   // K % 64 == 0: a lane's 32 values are all inside or none
            v[i] = at < K ? __ldcg(reinterpret_cast<const float4*>(ph + at) + i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
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
        // pair p's scale is in lanes 4 p ..
        block_mma(acc, t, x, __shfl_sync(0xffffffffu, scale, 8 * c) * sw,
                  __shfl_sync(0xffffffffu, scale, 8 * c + 4) * sw);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) part[kpart][tile][2 * c + (j & 1)][gi + 8 * (j >> 1)] = acc[j];
    __syncthreads();
    // warp = pair, lane = column: one staged quarter of 32 columns (see gemm.cu)
    if (warp >= n) return;
    float v = part[0][lane >> 4][warp][lane & 15];
#pragma unroll
    for (int k = 1; k < 4; ++k) v += part[k][lane >> 4][warp][lane & 15];
    v *= sh ? 1.0f : __ldg(ga.pair_w + start + warp);
    const uint32_t ab = __float_as_uint(v) & 0x7FFFFFFFu;
    const int sft = (int)(__reduce_max_sync(0xffffffffu, ab < 0x7F800000u ? ab : 0u) >> 23) - 141;
    const uint32_t st = sft > 0 ? (uint32_t)sft : 0u;
    v *= __uint_as_float((127u - st) << 23);
    const int64_t p = (int64_t)(sh ? ga.shared_row0 : 0) + start + warp;
    ga.ys[p * H + h0 + lane] = __float2half_rn(v);
    if (lane == 0) {
        ga.ysx[(int64_t)(h0 >> 5) * ga.ld_x + p] = (uint8_t)st;
        if (st) *ga.scaled = 1;
    }
}

cudaError_t launch_fp8_decode(int mode, const Fp8DecodeArgs& a, int units, cudaStream_t st) {
    auto k = mode == kGateUp ? k_fp8_decode_gu : k_fp8_decode_dn;
    return launch_kernel(k, dim3((unsigned)(units * kSub)), dim3(32 * kWarps), 0, st, a);
}

}  // namespace moe
