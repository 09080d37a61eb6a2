// NVFP4 x NVFP4 linear for B200 (sm_100a): C = A_hat B_hat^T straight from the
// 4-bit codes, on the block-scaled tensor cores.
//
// With q the E2M1 values and s the E4M3 block scales of groups of 16 along K,
//   C[m, n] = out( fl(a_ts * b_ts) *
//                  sum_g a_s[m, g] b_s[n, g] sum_{i<16} a_q[m, 16 g + i] b_q[n, 16 g + i] ).
// tcgen05.mma kind::mxf4nvf4 with a scale per 16 elements evaluates the double
// sum from the codes as they are stored (two per byte, the first in the low
// nibble, K contiguous) and the scale bytes as UE4M3, accumulating in binary32
// in tensor memory: no operand is decoded, and a step of K = 64 takes the time
// that K = 16 takes in fp16.
//
// What the codes' row-major scale layout costs: the MMA reads the scales of
// one K step of 64 from tensor memory, the 4 bytes of operand row m in lane
// m % 32 of column m / 32.  tcgen05.cp (32x128b, repeated for the four lane
// quarters) fills that from 512 contiguous bytes of shared memory, row m's 4
// bytes at (m % 32) * 16 + (m / 32) * 4.  The scales of a row lie K / 16
// bytes apart from the next row's, so no tiled copy makes this order from
// them: they go through registers, 16 bytes per row and 256 of K, and leave as
// four words, one per K step.  Work comes in units of 512 of K, so that the
// two lanes of a row use a whole 32-byte sector.  With few rows the kernel's
// own warps do that beside the MMAs; with many rows a kernel in front of it does,
// once for all the tiles that share a row.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/if4.h"
#include "if4_device.cuh"
#include "if4_host.cuh"
#include "if4_tc.cuh"
#include "nvfp4_scales.cuh"

namespace {

using namespace if4dev;

constexpr int SK = 256;               // K per stage: 128 bytes of codes, one swizzle row
constexpr int MMA_K = 64;             // K per tcgen05.mma of 4-bit operands
constexpr int KSTEPS = SK / MMA_K;
constexpr int UNIT = 2 * SK;          // K per unit of the scale ring
constexpr int SF_STEP = 512;          // scale bytes of 128 rows x one K step
constexpr int SF_BLOCK = KSTEPS * SF_STEP;   // 128 rows x one stage

// instruction descriptor, kind::mxf4nvf4: A and B E2M1 (1), both K-major,
// UE4M3 scales (bit 23 clear), scale ids 0, K = 64
__host__ __device__ constexpr uint32_t mxf4_idesc(int m, int n)
{
    return (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// Shared-memory descriptor of one 512-byte scale block for tcgen05.cp: four
// 8-row groups of 16-byte rows, 128 bytes apart, not swizzled.
__device__ __forceinline__ uint64_t smem_desc_scales(uint32_t addr)
{
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)(128u >> 4) << 32 | (uint64_t)1u << 46;
}

// The issuing warp stays converged and one elected lane issues: the operands
// of tcgen05 instructions are then warp-uniform values that the compiler keeps
// in uniform registers.  With one lane in a branch of its own the 16
// instructions of a stage took twice the MMAs' time (124 against 63 us at
// 8192 x 4096 x 4096 with the copies of codes and scales left out).
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(p));
    return p != 0;
}

// mbar_wait by a whole warp, with one answer for all its lanes.
template <bool CLUSTER = false>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag)
{
    return __all_sync(0xFFFFFFFFu, mbar_wait<CLUSTER>(bar, parity, abort_flag));
}

template <int CG>
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t d)
{
    if constexpr (CG == 1)
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" :: "r"(tmem), "l"(d));
    else
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" :: "r"(tmem), "l"(d));
}

template <int CG>
__device__ __forceinline__ void umma_nvfp4(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                           uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                           uint32_t accumulate)
{
    if constexpr (CG == 1)
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "setp.ne.b32 p, %6, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X"
                     " [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
                     :: "r"(tmem_d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb),
                        "r"(accumulate));
    else
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "setp.ne.b32 p, %6, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X"
                     " [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
                     :: "r"(tmem_d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb),
                        "r"(accumulate));
}

__device__ __forceinline__ void sts_u32(uint32_t addr, uint32_t v)
{
    asm volatile("st.shared.b32 [%0], %1;" :: "r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ void fence_async_smem()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Loader of load_scales16: behind the launch wait.
struct AfterWait {
    __device__ __forceinline__ uint32_t u16(const uint8_t *p) const { return ld_after_wait_u16(p); }
    __device__ __forceinline__ uint32_t u32(const uint8_t *p) const { return ld_after_wait_u32(p); }
    __device__ __forceinline__ void v4(const uint8_t *p, uint32_t &a, uint32_t &b, uint32_t &c,
                                       uint32_t &d) const
    {
        ld_after_wait_v4(p, a, b, c, d);
    }
};

template <int VEC>
__device__ __forceinline__ void load_scales16(const uint8_t *p, int nb, uint32_t (&w)[4])
{
    load_scales16<VEC>(p, nb, w, AfterWait());
}

// One accumulator value to its output type.
template <int ODT>
__device__ __forceinline__ void store_c(void *c, int64_t i, float v)
{
    if constexpr (ODT == IF4_F32) {
        static_cast<float *>(c)[i] = v;
    } else if constexpr (ODT == IF4_BF16) {
        static_cast<__nv_bfloat16 *>(c)[i] = __float2bfloat16_rn(v);
    } else {
        static_cast<__half *>(c)[i] = __float2half_rn(v);
    }
}

// --------------------------------------------------- one or two tokens ----
//
// A warp computes ROWS output columns for all tokens.  Its lanes take pieces
// of 32 along K (16 code bytes, 2 scale bytes) in turn.  Codes become f16x2
// values by conversion; the 8 products of each half of a group are multiples
// of 1/4 of at most 36, so their sum in f16 (at most 288, 11 bits) is exact;
// the product of the two scales (8 bits) and its product with the group's sum
// (20 bits) are exact in binary32, which takes one rounding per group.
//
// Nothing here waits for anything but the loads: no tensor memory, barrier
// or cluster stands between the launch and them.  A token of 4096 x 4096 takes
// 3.0 to 3.8 us from run to run (5.7 with the kernel below; the weight's bytes
// are 1.5), two tokens 4.2 (5.8).  The conversions bound it: four tokens take 7.3 us (5.8), and a
// token of 16384 x 4096 11.1 (10.0).  Two columns per warp and eight warps per
// block, all loads of a chunk up front: four columns took 4.5 us, one 3.7, four
// warps 3.4.

namespace few {

constexpr int ROWS = 2;                        // output columns per warp
constexpr int CHUNK = 4;                       // pieces per lane under way
constexpr int WARPS = 8;

// Sizes it is faster for than the split kernel (us here / there, one token
// unless said otherwise): 8192 x 4096 4.8 / 6.2, 4096 x 8192 6.3 / 6.4, two of 4096 x
// 4096 4.2 / 5.7; but two of 8192 x 4096 7.2 / 6.2, 16384 x 4096 11.1 / 10.0,
// 14336 x 2048 7.1 / 6.2 and 2048 x 14336 9.4 / 6.9.
inline bool takes(int64_t M, int64_t N, int64_t K)
{
    return M <= 2 && N <= 8192 && K <= 8192 && M * N * K <= (1 << 25);
}

}  // namespace few

__device__ __forceinline__ void e2m1x8_to_f16(uint32_t word, uint32_t (&h)[4])
{
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(word));
}

// Two scale bytes as floats (bit 7 is reported elsewhere).
__device__ __forceinline__ void e4m3x2_to_f32(uint32_t two, float (&s)[2])
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    s[0] = f16lo_to_f32(h);
    s[1] = f16hi_to_f32(h);
}

template <int MT, int ODT>
__global__ void __launch_bounds__(few::WARPS * 32)
nvfp4_linear_few(const uint8_t *x_codes, const uint8_t *x_scales, const float *x_ts,
                 const uint8_t *w_codes, const uint8_t *w_scales, const float *w_ts, void *c, int M,
                 int N, int K, int *err)
{
    using namespace few;
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int n0 = (blockIdx.x * WARPS + (threadIdx.x >> 5)) * ROWS;
    if (n0 >= N) return;
    const int pieces = K / 32;
    const int64_t cb = K / 2, sb = K / 16;         // bytes of a row
    float acc[ROWS][MT];
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[r][m] = 0.0f;
    uint32_t bad = 0;
    auto load = [&](const uint8_t *codes, const uint8_t *scales, int64_t row, int piece, bool in,
                    uint32_t (&w)[4], uint32_t &s) {
        w[0] = w[1] = w[2] = w[3] = s = 0u;
        if (in) {
            ld_after_wait_v4(codes + row * cb + (int64_t)piece * 16, w[0], w[1], w[2], w[3]);
            s = ld_after_wait_u16(scales + row * sb + (int64_t)piece * 2);
        }
    };
    for (int p0 = lane; p0 < pieces; p0 += 32 * CHUNK) {
        uint32_t w[CHUNK][ROWS][4], ws[CHUNK][ROWS], x[CHUNK][MT][4], xsc[CHUNK][MT];
#pragma unroll
        for (int q = 0; q < CHUNK; ++q)
#pragma unroll
            for (int m = 0; m < MT; ++m)
                load(x_codes, x_scales, m, p0 + 32 * q, p0 + 32 * q < pieces && m < M, x[q][m],
                     xsc[q][m]);
#pragma unroll
        for (int q = 0; q < CHUNK; ++q)
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
                load(w_codes, w_scales, n0 + r, p0 + 32 * q,
                     p0 + 32 * q < pieces && n0 + r < N, w[q][r], ws[q][r]);
#pragma unroll
        for (int q = 0; q < CHUNK; ++q) {
            uint32_t xh[MT][4][4];
            float xs[MT][2];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
#pragma unroll
                for (int j = 0; j < 4; ++j) e2m1x8_to_f16(x[q][m][j], xh[m][j]);
                e4m3x2_to_f32(xsc[q][m], xs[m]);
                bad |= xsc[q][m];
            }
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                uint32_t wh[4][4];
                float sw[2];
#pragma unroll
                for (int j = 0; j < 4; ++j) e2m1x8_to_f16(w[q][r][j], wh[j]);
                e4m3x2_to_f32(ws[q][r], sw);
                bad |= ws[q][r];
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        uint32_t d = 0u;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            asm("fma.rn.f16x2 %0, %1, %2, %0;"
                                : "+r"(d) : "r"(wh[2 * g + j / 4][j % 4]),
                                  "r"(xh[m][2 * g + j / 4][j % 4]));
                        const float dot = __fadd_rn(f16lo_to_f32(d), f16hi_to_f32(d));
                        acc[r][m] = __fmaf_rn(dot, __fmul_rn(sw[g], xs[m][g]), acc[r][m]);
                    }
            }
        }
    }
    const float scale = __fmul_rn(ld_after_wait(x_ts), ld_after_wait(w_ts));
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            float v = acc[r][m];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
            if (lane == r * MT + m && m < M && n0 + r < N)
                store_c<ODT>(c, (int64_t)m * N + n0 + r, __fmul_rn(v, scale));
        }
    if ((bad & 0x8080u) && err) atomicOr(err, IF4_DEV_BAD_SCALE);
}

// -------------------------------------------- small products: split over K ----
//
// Few tokens, or few output tiles.  The weight rows take the MMA's M side (128
// per CTA) and NT tokens its N side, so D is C transposed: a lane holds one
// output column and a warp's stores are contiguous along N.  A cluster of S
// CTAs splits K into whole units; each CTA leaves its binary32 partial tile in
// its shared memory, and the CTAs add the S partials in rank order through
// distributed shared memory, each for its share of the tokens: no workspace,
// no atomics, the same sum every time.
//
// One tile and one unit of K (16 x 128 x 512) take 3.4 us: launch, tensor memory,
// the first loads' latency and the epilogue.  A cluster's reduction adds 0.8 (16
// x 128 x 1024 to 4096 4.2 to 4.3).  Above that a CTA waits for its own chain of
// loads: 48 x 8192 x 4096 takes 9.2 us with DRAM 17 %, L2 16 % and the tensor pipe
// 5 % busy, 100 x 4096 x 14336 14.9.  (Scales loaded two, three or four units ahead
// instead of one: 1 to 10 % slower.)

namespace split {

constexpr int WR = 128;                        // weight rows per CTA
constexpr int W_BYTES = WR * SK / 2;           // 16 KB per stage
constexpr int THREADS = 192;                   // TMA, MMA, four scale / epilogue warps
constexpr int SF_UNITS = 3;
constexpr int SF_UNIT_BYTES = 4 * SF_BLOCK;    // two stages x (weights, tokens)
constexpr int SF_COLS = 2 * 2 * KSTEPS * 4;    // two stages of scale columns
constexpr int MAX_RANKS = 8;                   // the portable cluster size
constexpr int PER_SM = 2;                      // CTAs per SM

template <int NT>
struct Cfg {
    static constexpr int X_BYTES = NT * SK / 2;
    static constexpr int STAGE = W_BYTES + X_BYTES;
    static constexpr int STAGES = NT <= 32 ? 4 : 3;      // 97-106 KB: two CTAs per SM
    static constexpr int SF_OFF = STAGES * STAGE;
    static constexpr int BAR_OFF = SF_OFF + SF_UNITS * SF_UNIT_BYTES;
    static constexpr int SMEM = BAR_OFF + 256 + 1024;
    static constexpr int TMEM_COLS = 128;
    static_assert(NT + SF_COLS <= TMEM_COLS, "tensor memory");
    static_assert(NT * WR * 4 <= SF_OFF, "the partial tile fits the stages");
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

}  // namespace split

template <int NT, int VEC, int ODT>
__global__ void __launch_bounds__(split::THREADS, 1)
nvfp4_linear_split(const __grid_constant__ CUtensorMap tmap_w,
                   const __grid_constant__ CUtensorMap tmap_x,
                   const uint8_t *__restrict__ w_scales, const uint8_t *__restrict__ x_scales,
                   const float *__restrict__ w_ts, const float *__restrict__ x_ts,
                   void *__restrict__ c, int M, int N, int K, int *err)
{
    using namespace split;
    using C = Cfg<NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *smem_w = smem;
    uint8_t *smem_x = smem + C::STAGES * W_BYTES;
    uint8_t *smem_sf = smem + C::SF_OFF;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF);
    uint64_t *empty = full + C::STAGES;
    uint64_t *sf_full = empty + C::STAGES;
    uint64_t *sf_empty = sf_full + SF_UNITS;
    uint64_t *acc_full = sf_empty + SF_UNITS;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_full + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0);   // warp-uniform
    const int lane = threadIdx.x & 31;
    uint32_t ranks;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
    const uint32_t rank = cta_rank();
    const int n0 = blockIdx.y * WR;
    const int m0 = (int)(blockIdx.x / ranks) * NT;
    const int units = (K + UNIT - 1) / UNIT;
    const int u0 = (int)((int64_t)units * rank / ranks);
    const int u1 = (int)((int64_t)units * (rank + 1) / ranks);
    const int kb0 = u0 * 2;                                  // stages of this CTA
    const int kb1 = min(u1 * 2, (K + SK - 1) / SK);

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int s = 0; s < SF_UNITS; ++s) {
            mbar_init(smem_u32(&sf_full[s]), 128);
            mbar_init(smem_u32(&sf_empty[s]), 1);
        }
        mbar_init(smem_u32(acc_full), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_tmap(&tmap_w);
        prefetch_tmap(&tmap_x);
    }
    if (warp == 1) {
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(tmem_slot)), "r"(C::TMEM_COLS));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    // programmatic launch: nothing above reads a kernel input
    pdl_enter();

    if (warp == 0 && lane == 0) {
        // ---------------------------------------------------- TMA producer
        int stage = 0;
        uint32_t phase = 0;
        int issued = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, abort_flag)) break;
            const uint32_t fb = smem_u32(&full[stage]);
            mbar_expect_tx(fb, C::STAGE);
            tma_load_2d(smem_u32(smem_w + stage * W_BYTES), &tmap_w, kb * (SK / 2), n0, fb);
            tma_load_2d(smem_u32(smem_x + stage * C::X_BYTES), &tmap_x, kb * (SK / 2), m0, fb);
            ++issued;
            if (++stage == C::STAGES) { stage = 0; phase ^= 1u; }
        }
        // every copy issued here lands before the shared memory is reused or
        // the CTA exits (bounded)
        const int pending = issued < C::STAGES ? issued : C::STAGES;
        for (int i = 0; i < pending; ++i) {
            if (--stage < 0) { stage = C::STAGES - 1; phase ^= 1u; }
            const unsigned long long t0 = globaltimer();
            while (!mbar_try_wait(smem_u32(&full[stage]), phase))
                if (globaltimer() - t0 > WAIT_LIMIT_NS) break;
        }
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issuer
        const bool issue = elect_one();
        const uint64_t w_desc = smem_desc_sw128(smem_u32(smem_w));
        const uint64_t x_desc = smem_desc_sw128(smem_u32(smem_x));
        const uint64_t sf_desc = smem_desc_scales(smem_u32(smem_sf));
        int stage = 0, slot = 0;
        uint32_t phase = 0, sf_phase = 0;
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb) {
            const int half = (kb - kb0) & 1;
            if (half == 0 && !warp_wait(smem_u32(&sf_full[slot]), sf_phase, abort_flag)) {
                ok = false;
                break;
            }
            if (!warp_wait(smem_u32(&full[stage]), phase, abort_flag)) { ok = false; break; }
            tc_fence_after();
            const uint64_t wd = w_desc + (uint64_t)(stage * (W_BYTES >> 4));
            const uint64_t xd = x_desc + (uint64_t)(stage * (C::X_BYTES >> 4));
            const uint64_t sd = sf_desc + (uint64_t)((slot * SF_UNIT_BYTES + half * SF_BLOCK) >> 4);
            const uint32_t tsf = tmem_base + NT + half * (SF_COLS / 2);
            const int steps = min(KSTEPS, (K - kb * SK + MMA_K - 1) / MMA_K);
            if (issue) {
#pragma unroll
                for (int kk = 0; kk < KSTEPS; ++kk) {
                    if (kk < steps) {
                        const uint32_t tw = tsf + kk * 4, tx = tsf + 16 + kk * 4;
                        copy_scales<1>(tw, sd + kk * (SF_STEP >> 4));
                        copy_scales<1>(tx, sd + ((2 * SF_BLOCK + kk * SF_STEP) >> 4));
                        umma_nvfp4<1>(tmem_base, wd + 2 * kk, xd + 2 * kk, mxf4_idesc(WR, NT), tw,
                                      tx, kb != kb0 || kk != 0 ? 1u : 0u);
                    }
                }
                umma_commit(smem_u32(&empty[stage]));
                if (half == 1) umma_commit(smem_u32(&sf_empty[slot]));
            }
            __syncwarp();
            if (++stage == C::STAGES) { stage = 0; phase ^= 1u; }
            if (half == 1 && ++slot == SF_UNITS) { slot = 0; sf_phase ^= 1u; }
        }
        // MMAs and scale copies complete before anyone reads the accumulator,
        // reuses the shared memory or frees tensor memory
        if (issue) {
            umma_commit(smem_u32(acc_full));
            if (!ok) {
                const unsigned long long t0 = globaltimer();
                while (!mbar_try_wait(smem_u32(acc_full), 0))
                    if (globaltimer() - t0 > WAIT_LIMIT_NS) break;
            }
        }
    } else if (warp >= 2) {
        // ---------------------------------------------------- block scales
        // thread t: chunk t & 1 (one stage) of rows 32 p + 16 i + 4 v + q
        const int t = threadIdx.x - 64;
        const int ch = t & 1, q = (t >> 1) & 3, p = (t >> 3) & 3, v = t >> 5;
        const int row0 = 32 * p + 4 * v + q;                 // and row0 + 16
        const int kg = K / 16;
        const uint32_t so = (uint32_t)((row0 & 31) * 16 + p * 4);
        int slot = 0;
        uint32_t phase = 0;
        uint32_t bad = 0;
        uint32_t ww[2][4], xw[2][4];
        auto fetch = [&](int u) {
            const int g0 = u * (UNIT / 16) + ch * 16;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = row0 + 16 * i;
                load_scales16<VEC>(w_scales + (int64_t)(n0 + r) * kg + g0,
                                   n0 + r < N ? kg - g0 : 0, ww[i]);
                if (r < NT)
                    load_scales16<VEC>(x_scales + (int64_t)(m0 + r) * kg + g0,
                                       m0 + r < M ? kg - g0 : 0, xw[i]);
            }
        };
        if (u0 < u1) fetch(u0);
        for (int u = u0; u < u1; ++u) {
            if (!mbar_wait(smem_u32(&sf_empty[slot]), phase ^ 1u, abort_flag)) break;
            const uint32_t d = smem_u32(smem_sf + slot * SF_UNIT_BYTES) + ch * SF_BLOCK + so;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    sts_u32(d + i * 256 + j * SF_STEP, ww[i][j]);
                    bad |= ww[i][j];
                }
                if (row0 + 16 * i < NT) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        sts_u32(d + 2 * SF_BLOCK + i * 256 + j * SF_STEP, xw[i][j]);
                        bad |= xw[i][j];
                    }
                }
            }
            fence_async_smem();
            mbar_arrive(smem_u32(&sf_full[slot]));
            if (++slot == SF_UNITS) { slot = 0; phase ^= 1u; }
            if (u + 1 < u1) fetch(u + 1);
        }
        if ((bad & 0x80808080u) && err) atomicOr(err, IF4_DEV_BAD_SCALE);
        // -------------------------------------------------------- epilogue
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(acc_full), 0, abort_flag));
        tc_fence_after();
        if (ok && u0 < u1) {
            const float scale = __fmul_rn(ld_after_wait(x_ts), ld_after_wait(w_ts));
            float *part = reinterpret_cast<float *>(smem);
#pragma unroll 1
            for (int mc = 0; mc < NT && m0 + mc < M; mc += 16) {
                uint32_t r[16];
                tmem_ld16(tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)mc, r);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int m = m0 + mc + j;
                    if (ranks > 1)
                        part[(mc + j) * WR + row] = __uint_as_float(r[j]);
                    else if (m < M && n0 + row < N)
                        store_c<ODT>(c, (int64_t)m * N + n0 + row,
                                     __fmul_rn(__uint_as_float(r[j]), scale));
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (ranks > 1) {
        cluster_sync();
        // rank r adds tokens r, r + ranks, ...: a warp per token, four rows per
        // lane, the partials of all ranks loaded before they are added in order
        if (!*abort_flag) {
            const float scale = __fmul_rn(ld_after_wait(x_ts), ld_after_wait(w_ts));
            uint32_t part[MAX_RANKS];
#pragma unroll
            for (uint32_t s = 0; s < MAX_RANKS; ++s)
                part[s] = map_to(smem_u32(smem) + lane * 16, s < ranks ? s : 0);
            const int n = n0 + 4 * lane;
            const int tokens = min(NT, M - m0);
            for (int m = (int)rank + (int)ranks * warp; m < tokens; m += (int)ranks * (THREADS / 32)) {
                float v[MAX_RANKS][4];
#pragma unroll
                for (uint32_t s = 0; s < MAX_RANKS; ++s)
                    if (s < ranks)
                        asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                                     : "=f"(v[s][0]), "=f"(v[s][1]), "=f"(v[s][2]), "=f"(v[s][3])
                                     : "r"(part[s] + m * WR * 4) : "memory");
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float sum = v[0][i];
#pragma unroll
                    for (uint32_t s = 1; s < MAX_RANKS; ++s)
                        if (s < ranks) sum = __fadd_rn(sum, v[s][i]);
                    if (n + i < N)
                        store_c<ODT>(c, (int64_t)(m0 + m) * N + n + i, __fmul_rn(sum, scale));
                }
            }
        }
        cluster_sync();                  // no CTA leaves while another reads its partials
    }
    if (threadIdx.x == 0 && *abort_flag && err) atomicOr(err, IF4_DEV_TIMEOUT);
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;"
                     :: "r"(tmem_base), "r"(C::TMEM_COLS));
    }
}

// --------------------------------------------------- many rows: CTA pairs ----
//
// A pair of CTAs on two SMs computes 256 x BN tiles with tcgen05.mma of
// cta_group::2, persistent over the tiles: CTA r holds rows r * 128..+127 of
// A's slab and half of B's, the leader's MMAs read both halves, and each CTA
// keeps its own 128 rows of the product.  The MMA reads a row's scales from
// the tensor memory of the CTA that holds the accumulator, so each CTA brings
// the scales of its own A rows and of all BN rows of B.
//
// Scales: a small kernel first puts both operands' scales into the workspace
// in the order that tcgen05.cp reads (pack_scales), so that here they are two
// more tiles of the stage's TMA copies.  Loading and reordering them in this
// kernel instead (four warps, a second ring) was measured at 8192 x 4096 x
// 4096: 135 us, the ring's round trips and the loads' latency in the way of
// every stage.
//
// Tensor memory: two accumulators of BN columns, so that the epilogue of one
// tile runs under the MMAs of the next, and the scale columns of two K steps:
// 2 * 240 + 32 = 512.  (256 columns with the accumulators overlapping, the
// overlap drained first: the wait for it cost 0.6 us a tile, and over the
// sizes tried it was 5 % faster to 9 % slower.)  A wide tile reads less shared memory
// per product; narrow ones use more SMs when there are few tiles.  Measured, BN =
// 240 against 128, us: 8192 x 4096 x 4096 68.6 / 86.5, 1024 x 4096 x 4096
// 12.7 / 15.8 (72 and 128 tiles), 512 x 4096 x 4096 11.9 / 11.5 (36 and 64),
// 1001 x 1555 x 4128 22.0 / 16.6 (28 and 52; 13.8 with the stores of flush_pairs): 128
// while its tiles fit the pairs.
//
// Long runs are bound by the board's power: 8192 x 4096 x 4096 takes 58 us in bursts
// of 1.2 ms at 1965 MHz, and 67 us over 3 s, at 1500 MHz and 985 W with sw_power_cap
// the one active reason.  binary32 C takes 84: its rows leave as each lane's own
// stores, not as boxes.

namespace duo {

constexpr int PM = 128;                        // rows per CTA
constexpr int A_BYTES = PM * SK / 2;           // 16 KB per stage
constexpr int SFA_BYTES = SF_BLOCK;            // 2 KB
constexpr int THREADS = 192;                   // TMA, MMA, 4 epilogue warps
constexpr int OUT_BYTES = 4608;                // staged output per epilogue warp
constexpr int OUT_BOX = 32 * 64;               // 32 rows x 32 two-byte columns, two buffers

template <int BN>
struct Cfg {
    static constexpr int B_BYTES = BN / 2 * SK / 2;
    static constexpr int SFB_BLOCKS = (BN + 127) / 128;
    static constexpr int SFB_BYTES = SFB_BLOCKS * SF_BLOCK;
    static constexpr int STAGE = A_BYTES + B_BYTES + SFA_BYTES + SFB_BYTES;
    static constexpr int STAGES = BN > 128 ? 5 : 7;
    static constexpr int SF_STEP_COLS = 4 + 4 * SFB_BLOCKS;      // scale columns of a K step
    static constexpr int SF_COL0 = 512 - 32;                     // two K steps in turn
    static constexpr int OUT_OFF = STAGES * STAGE;
    static constexpr int BAR_OFF = OUT_OFF + 4 * OUT_BYTES;
    static constexpr int SMEM = BAR_OFF + 256 + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static_assert(2 * BN <= SF_COL0 && SF_STEP_COLS <= 16, "tensor memory");
    static_assert(BN % 16 == 0 && STAGE % 1024 == 0 && B_BYTES % 1024 == 0, "alignment");
};

}  // namespace duo

// The scales of one operand: [rows, K / 16] as stored, and [tiles of `tile`
// rows][`blocks` blocks of 128][K steps of 64, a multiple of 4][512 bytes] as
// tcgen05.cp reads them; rows past a tile's end are 0.
struct ScalePack {
    const uint8_t *src;
    uint8_t *dst;
    int rows, tile, blocks;
    __host__ __device__ int64_t row_blocks() const
    {
        return (int64_t)((rows + tile - 1) / tile) * blocks;
    }
};

// A thread takes one stage (four K steps) of the rows m, m + 32, m + 64 and
// m + 96 of a block, 16 bytes each, and writes their words as four 16-byte
// lines, one per K step.  Rows and K past the end become 0.  A warp covers 16
// rows m x 2 stages: whole 32-byte sectors read, 256-byte runs written.
template <int VEC>
__global__ void __launch_bounds__(256)
pack_scales(ScalePack a, ScalePack b, int K, int *err)
{
    pdl_enter();
    const int kg = K / 16, stages = (K + SK - 1) / SK, pairs = (stages + 1) / 2;
    const int64_t na = a.row_blocks() * pairs * 2;           // warps' work items
    const int64_t nb = b.row_blocks() * pairs * 2;
    const int lane = threadIdx.x & 31;
    uint32_t bad = 0;
    for (int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); w < na + nb;
         w += (int64_t)gridDim.x * 8) {
        const bool first = w < na;
        const uint8_t *src = first ? a.src : b.src;
        uint8_t *dst = first ? a.dst : b.dst;
        const int rows = first ? a.rows : b.rows, tile_rows = first ? a.tile : b.tile;
        const int blocks = first ? a.blocks : b.blocks;
        // (row blocks x stages fit 32 bits: 2^15 blocks of rows, 2^12 stages)
        const uint32_t i = (uint32_t)(first ? w : w - na);
        const int m = (int)(i & 1) * 16 + (lane >> 1);
        const uint32_t block = (i >> 1) / (uint32_t)pairs;
        const int stage = (int)((i >> 1) - block * (uint32_t)pairs) * 2 + (lane & 1);
        if (stage >= stages) continue;
        const uint32_t tile = block / (uint32_t)blocks;
        const int in_tile0 = (int)(block - tile * (uint32_t)blocks) * 128;
        uint32_t v[4][4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int in_tile = in_tile0 + m + 32 * p;
            const int64_t row = (int64_t)tile * tile_rows + in_tile;
            load_scales16<VEC>(src + row * kg + stage * 16,
                               in_tile < tile_rows && row < rows ? kg - stage * 16 : 0, v[p]);
#pragma unroll
            for (int j = 0; j < 4; ++j) bad |= v[p][j];
        }
        uint8_t *d = dst + ((int64_t)block * stages + stage) * SF_BLOCK + m * 16;
#pragma unroll
        for (int j = 0; j < 4; ++j) st_v4(d + j * SF_STEP, v[0][j], v[1][j], v[2][j], v[3][j]);
    }
    if ((bad & 0x80808080u) && err) atomicOr(err, IF4_DEV_BAD_SCALE);
}

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap *map, int x, int y,
                                                 int z, uint32_t bar_cluster)
{
    asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global"
                 ".mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4}], [%5];"
                 :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z),
                    "r"(bar_cluster)
                 : "memory");
}

// COLS (16 or 32) accumulator columns of a warp's 32 rows (lane: row), scaled,
// to C's type.  width: bytes that C's base and row length allow per store, 32
// or 16; 0: elements only.  Then a lane's stores would touch a sector each for
// two or four bytes, so the block goes through the warp's shared memory (rows
// of 33 words) and leaves row by row, lanes along the columns.  (Two-byte C: only
// the last 16 columns of a 240-wide tile come here, its other blocks leave as
// boxes or pairs, below.)
template <int ODT, int COLS>
__device__ __forceinline__ void store_cols(void *c, const uint32_t *r, float scale, int row0, int M,
                                           int N, int col0, int width, uint32_t *stage)
{
    const int lane = threadIdx.x & 31;
    constexpr int ES = ODT == IF4_F32 ? 4 : 2;
    if (width >= 16 && col0 + COLS <= N) {
        if (row0 + lane >= M) return;
        uint32_t w[COLS * ES / 4];
#pragma unroll
        for (int i = 0; i < COLS; i += 2) {
            const float lo = __fmul_rn(__uint_as_float(r[i]), scale);
            const float hi = __fmul_rn(__uint_as_float(r[i + 1]), scale);
            if constexpr (ODT == IF4_F32) {
                w[i] = __float_as_uint(lo);
                w[i + 1] = __float_as_uint(hi);
            } else {
                w[i / 2] = ODT == IF4_BF16 ? bf16x2_from_f32(lo, hi) : f16x2_from_f32(lo, hi);
            }
        }
        uint8_t *p = static_cast<uint8_t *>(c) + ((int64_t)(row0 + lane) * N + col0) * ES;
        if (width == 32) {
#pragma unroll
            for (int q = 0; q < COLS * ES / 32; ++q)
                st_v8(p + 32 * q, *reinterpret_cast<const uint32_t(*)[8]>(w + 8 * q));
        } else {
#pragma unroll
            for (int q = 0; q < COLS * ES / 16; ++q)
                st_v4(p + 16 * q, w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
        }
    } else {
        __syncwarp();                      // the previous block has been read
#pragma unroll
        for (int i = 0; i < COLS; ++i) stage[lane * 33 + i] = r[i];
        __syncwarp();
        // 32 / COLS rows at a time
        const int col = lane % COLS, sub = lane / COLS;
        const int rows = min(32, M - row0);
        if (col0 + col < N)
            for (int q = sub; q < rows; q += 32 / COLS)
                store_c<ODT>(c, (int64_t)(row0 + q) * N + col0 + col,
                             __fmul_rn(__uint_as_float(stage[q * 33 + col]), scale));
    }
}

// Two-byte C whose rows begin anywhere: COLS columns of the warp's 32 rows
// (lane: row) into its shared memory as pairs, from column `off` of 64 ...
template <int ODT, int COLS>
__device__ __forceinline__ void stage_pairs(const uint32_t *r, float scale, int off, uint32_t *stage)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < COLS / 2; ++i) {
        const float lo = __fmul_rn(__uint_as_float(r[2 * i]), scale);
        const float hi = __fmul_rn(__uint_as_float(r[2 * i + 1]), scale);
        stage[lane * 33 + off / 2 + i] =
            ODT == IF4_BF16 ? bf16x2_from_f32(lo, hi) : f16x2_from_f32(lo, hi);
    }
}

// ... and out row by row, a four-byte store per lane: pairs as they lie where
// the row's first element is on a four-byte boundary, else pairs shifted by
// one element and the two ends by themselves.  Four warps write the whole tile,
// so what counts is that eight rows' reads are under way at once: 8192 x 4097 x
// 4096 88 us; row after row 126, an element per lane and store 105.
__device__ __forceinline__ void flush_pairs(void *c, int row0, int M, int N, int col0, int cols,
                                            uint32_t *stage)
{
    const int lane = threadIdx.x & 31;
    const int rows = min(32, M - row0);
    cols = min(cols, N - col0);
    __syncwarp();
    uint16_t *p = static_cast<uint16_t *>(c) + (int64_t)row0 * N + col0;
    const uint32_t *in = stage + lane;
    const int next = lane < 31 ? 1 : 0;
#pragma unroll 1
    for (int q = 0; q < rows; q += 8) {
        uint32_t w0[8], w1[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w0[i] = in[(q + i) * 33];
            w1[i] = in[(q + i) * 33 + next];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint16_t *d = p + (int64_t)(q + i) * N;
            const uint32_t odd = (uint32_t)(reinterpret_cast<uintptr_t>(d) >> 1) & 1u;
            const int first = 2 * lane + (int)odd;
            const uint32_t v = __funnelshift_r(w0[i], w1[i], 16 * odd);
            const bool in_row = q + i < rows;
            if (in_row && first + 1 < cols) *reinterpret_cast<uint32_t *>(d + first) = v;
            // the last element alone, and (lane 0) the first
            if (in_row && first + 1 == cols) d[first] = (uint16_t)v;
            if (in_row && odd && lane == 0 && cols > 0) d[0] = (uint16_t)w0[i];
        }
    }
    __syncwarp();
}

// The same for two-byte C whose rows are multiples of 16 bytes, 32 whole
// columns: through shared memory (64-byte rows, swizzled as the tensor map
// says) and a TMA store, which writes whole lines and clips at C's edges
// (direct 32-byte stores of a row per lane: 16384 x 8192 x 8192 553 against
// 524 us, 512 x 4096 x 4096 12.4 against 11.9 us).
template <int ODT>
__device__ __forceinline__ void store_box(const CUtensorMap *map, const uint32_t *r, float scale,
                                          int row0, int col0, uint32_t buf)
{
    const int lane = threadIdx.x & 31;
    // the store two boxes ago has read this buffer
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float lo = __fmul_rn(__uint_as_float(r[8 * q + 2 * i]), scale);
            const float hi = __fmul_rn(__uint_as_float(r[8 * q + 2 * i + 1]), scale);
            w[i] = ODT == IF4_BF16 ? bf16x2_from_f32(lo, hi) : f16x2_from_f32(lo, hi);
        }
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};"
                     :: "r"(buf + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)), "r"(w[0]), "r"(w[1]),
                        "r"(w[2]), "r"(w[3])
                     : "memory");
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) {
        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];"
                     :: "l"(reinterpret_cast<uint64_t>(map)), "r"(col0), "r"(row0), "r"(buf)
                     : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
}

template <int BN, int ODT>
__global__ void __launch_bounds__(duo::THREADS, 1)
nvfp4_linear_pair(const __grid_constant__ CUtensorMap tmap_a,
                  const __grid_constant__ CUtensorMap tmap_b,
                  const __grid_constant__ CUtensorMap tmap_sa,
                  const __grid_constant__ CUtensorMap tmap_sb,
                  const __grid_constant__ CUtensorMap tmap_c, int box_stores,
                  const float *__restrict__ a_ts, const float *__restrict__ b_ts,
                  void *__restrict__ c, int M, int N, int K, int *err)
{
    using namespace duo;
    using C = Cfg<BN>;
    constexpr int STAGES = C::STAGES, STAGE = C::STAGE, B_BYTES = C::B_BYTES;
    constexpr int SFB_BYTES = C::SFB_BYTES, SFB_BLOCKS = C::SFB_BLOCKS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *smem_a = smem;
    uint8_t *smem_b = smem_a + STAGES * A_BYTES;
    uint8_t *smem_sa = smem_b + STAGES * B_BYTES;
    uint8_t *smem_sb = smem_sa + STAGES * SFA_BYTES;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF);   // leader
    uint64_t *empty = full + STAGES;               // both
    uint64_t *acc_full = empty + STAGES;           // both
    uint64_t *acc_free = acc_full + 2;             // leader, [2]
    uint64_t *drain = acc_free + 2;                // leader
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0);   // warp-uniform
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cta_rank();
    const bool leader = rank == 0;
    const int m_tiles = (M + 2 * PM - 1) / (2 * PM);
    const int tiles = m_tiles * ((N + BN - 1) / BN);
    const int pair_id = blockIdx.x >> 1;
    const int num_pairs = gridDim.x >> 1;
    const int k_blocks = (K + SK - 1) / SK;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        mbar_init(smem_u32(&acc_full[0]), 1);
        mbar_init(smem_u32(&acc_full[1]), 1);
        mbar_init(smem_u32(&acc_free[0]), 2 * 4);
        mbar_init(smem_u32(&acc_free[1]), 2 * 4);
        mbar_init(smem_u32(drain), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_tmap(&tmap_a);
        prefetch_tmap(&tmap_b);
        prefetch_tmap(&tmap_sa);
        prefetch_tmap(&tmap_sb);
        if (box_stores) prefetch_tmap(&tmap_c);
    }
    if (warp == 1) {
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(tmem_slot)), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();                      // peer barriers initialised before any remote use
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    // programmatic launch: nothing above reads a kernel input
    pdl_enter();

    if (warp == 0 && lane == 0) {
        // ---------------------------------------------------- TMA producer
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int t = pair_id; t < tiles && ok; t += num_pairs) {
            const int mt = t % m_tiles, nt = t / m_tiles;
            const int m0 = mt * 2 * PM + (int)rank * PM;
            const int n0 = nt * BN + (int)rank * (BN / 2);
            for (int kb = 0; kb < k_blocks; ++kb) {
                if (!mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, abort_flag)) { ok = false; break; }
                const uint32_t fb = map_to(smem_u32(&full[stage]), 0);
                if (leader) mbar_expect_tx(smem_u32(&full[stage]), 2 * STAGE);
                tma_load_2d_pair(smem_u32(smem_a + stage * A_BYTES), &tmap_a, kb * (SK / 2), m0, fb);
                tma_load_2d_pair(smem_u32(smem_b + stage * B_BYTES), &tmap_b, kb * (SK / 2), n0, fb);
                tma_load_3d_pair(smem_u32(smem_sa + stage * SFA_BYTES), &tmap_sa, 0, kb * KSTEPS,
                                 mt * 2 + (int)rank, fb);
                tma_load_3d_pair(smem_u32(smem_sb + stage * SFB_BYTES), &tmap_sb, 0, kb * KSTEPS,
                                 nt * SFB_BLOCKS, fb);
                if (++stage == STAGES) { stage = 0; phase ^= 1u; }
            }
        }
        // every copy issued here has been consumed by the leader's MMAs when
        // the loops end normally; after an abort, give them a bounded time
        const unsigned long long t0 = globaltimer();
        if (*abort_flag)
            while (globaltimer() - t0 < 2000000ull) { }
    } else if (warp == 1 && leader) {
        // ------------------------------------------- MMA issuer (leader)
        const bool issue = elect_one();
        const uint64_t a_desc = smem_desc_sw128(smem_u32(smem_a));
        const uint64_t b_desc = smem_desc_sw128(smem_u32(smem_b));
        const uint64_t sa_desc = smem_desc_scales(smem_u32(smem_sa));
        const uint64_t sb_desc = smem_desc_scales(smem_u32(smem_sb));
        const uint32_t sf_tmem = tmem_base + C::SF_COL0;
        int stage = 0, acc = 0;
        uint32_t phase = 0, free_phase = 1;
        bool ok = true;
        for (int t = pair_id; t < tiles && ok; t += num_pairs) {
            // the epilogue of two tiles ago has drained this accumulator
            if (!warp_wait<true>(smem_u32(&acc_free[acc]), free_phase, abort_flag)) break;
            free_phase ^= (uint32_t)acc;
            tc_fence_after();
            const uint32_t d_tmem = tmem_base + (uint32_t)(acc * BN);
            for (int kb = 0; kb < k_blocks; ++kb) {
                if (!warp_wait(smem_u32(&full[stage]), phase, abort_flag)) { ok = false; break; }
                tc_fence_after();
                const uint64_t ad = a_desc + (uint64_t)(stage * (A_BYTES >> 4));
                const uint64_t bd = b_desc + (uint64_t)(stage * (B_BYTES >> 4));
                const uint64_t sad = sa_desc + (uint64_t)(stage * (SFA_BYTES >> 4));
                const uint64_t sbd = sb_desc + (uint64_t)(stage * (SFB_BYTES >> 4));
                const int steps = min(KSTEPS, (K - kb * SK + MMA_K - 1) / MMA_K);
                if (issue) {
#pragma unroll
                    for (int kk = 0; kk < KSTEPS; ++kk) {
                        if (kk < steps) {
                            const uint32_t ta = sf_tmem + (kk & 1) * 16, tb = ta + 4;
                            copy_scales<2>(ta, sad + kk * (SF_STEP >> 4));
#pragma unroll
                            for (int j = 0; j < SFB_BLOCKS; ++j)
                                copy_scales<2>(tb + 4 * j, sbd + ((j * SF_BLOCK + kk * SF_STEP) >> 4));
                            umma_nvfp4<2>(d_tmem, ad + 2 * kk, bd + 2 * kk, mxf4_idesc(2 * PM, BN),
                                          ta, tb, (kb | kk) != 0 ? 1u : 0u);
                        }
                    }
                    umma_commit_both(smem_u32(&empty[stage]));
                    if (kb + 1 == k_blocks) umma_commit_both(smem_u32(&acc_full[acc]));
                }
                __syncwarp();
                if (++stage == STAGES) { stage = 0; phase ^= 1u; }
            }
            acc ^= 1;
        }
        if (issue) {
            asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                         :: "r"(smem_u32(drain)) : "memory");
            const unsigned long long t0 = globaltimer();
            while (!mbar_try_wait(smem_u32(drain), 0))
                if (globaltimer() - t0 > WAIT_LIMIT_NS) break;
        }
    } else if (warp >= 2) {
        // -------------------------------------------------------- epilogue
        const int quarter = warp & 3;
        const float scale = __fmul_rn(ld_after_wait(a_ts), ld_after_wait(b_ts));
        constexpr int ES = ODT == IF4_F32 ? 4 : 2;
        const uintptr_t al = reinterpret_cast<uintptr_t>(c) | (uintptr_t)((int64_t)N * ES);
        const int width = al % 32 == 0 ? 32 : al % 16 == 0 ? 16 : 0;
        const uint32_t free_bar[2] = {map_to(smem_u32(&acc_free[0]), 0),
                                      map_to(smem_u32(&acc_free[1]), 0)};
        uint32_t *stage = reinterpret_cast<uint32_t *>(smem + C::OUT_OFF + quarter * OUT_BYTES);
        const uint32_t boxes = smem_u32(stage);
        int box = 0;
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int t = pair_id; t < tiles; t += num_pairs) {
            const int row0 = (t % m_tiles) * 2 * PM + (int)rank * PM + quarter * 32;
            const int n0 = (t / m_tiles) * BN;
            if (!warp_wait(smem_u32(&acc_full[acc]), acc_phase, abort_flag)) break;
            tc_fence_after();
            const uint32_t lanes = tmem_base + ((uint32_t)(quarter * 32) << 16);
            auto put32 = [&](const uint32_t (&r)[32], int col) {
                if (ODT != IF4_F32 && box_stores) {
                    if (row0 < M && n0 + col < N) {
                        store_box<ODT>(&tmap_c, r, scale, row0, n0 + col, boxes + box * OUT_BOX);
                        box ^= 1;          // only a box that was stored takes a buffer
                    }
                } else if (ODT != IF4_F32) {
                    stage_pairs<ODT, 32>(r, scale, col & 32, stage);
                    if ((col & 32) || col + 32 == BN)
                        flush_pairs(c, row0, M, N, n0 + (col & ~32), (col & 32) + 32, stage);
                } else {
                    store_cols<ODT, 32>(c, r, scale, row0, M, N, n0 + col, width, stage);
                }
            };
            const uint32_t base = lanes + (uint32_t)(acc * BN);
#pragma unroll 1
            for (int ch = 0; ch < BN / 32; ++ch) {
                uint32_t r[32];
                tmem_ld32(base + ch * 32, r);
                put32(r, ch * 32);
            }
            if constexpr (BN % 32 != 0) {
                uint32_t q[16];
                tmem_ld16(base + BN / 32 * 32, q);
                constexpr int LAST = BN / 32 * 32;
                if (ODT != IF4_F32 && !box_stores) {
                    // with the 32 columns that wait, if any do
                    stage_pairs<ODT, 16>(q, scale, LAST & 32, stage);
                    flush_pairs(c, row0, M, N, n0 + (LAST & ~32), (LAST & 32) + 16, stage);
                } else {
                    // element stores at C's edge go through the boxes' memory
                    if (box_stores && n0 + LAST + 16 > N) {
                        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                        __syncwarp();
                    }
                    store_cols<ODT, 16>(c, q, scale, row0, M, N, n0 + LAST, width, stage);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_remote(free_bar[acc]);
            acc_phase ^= (uint32_t)acc;
            acc ^= 1;
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();                      // the peer's MMAs and copies are done
    if (threadIdx.x == 0 && *abort_flag && err) atomicOr(err, IF4_DEV_TIMEOUT);
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;"
                     :: "r"(tmem_base), "r"(512));
    }
}

// ------------------------------------------------------------ host side ----

constexpr int64_t MAX_MN = 1 << 22, MAX_K = 1 << 20;

// Codes [rows, K / 2] -> tensor map with a (128 bytes x box_rows) box.
bool make_codes_map(CUtensorMap *map, const void *base, int64_t rows, int64_t K, int box_rows)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)(K / 2), (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(K / 2)};
    const cuuint32_t box[2] = {(cuuint32_t)(SK / 2), (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Problem {
    const uint8_t *a_codes, *a_scales, *b_codes, *b_scales;
    const float *a_ts, *b_ts;
    int64_t M, N, K;
    void *workspace;
    void *c;
    int *err;
    cudaStream_t st;
};

template <int MT, int ODT>
int launch_few(const Problem &p)
{
    const int64_t per_block = few::WARPS * few::ROWS;
    return launch_k(nvfp4_linear_few<MT, ODT>, (unsigned)((p.N + per_block - 1) / per_block),
                    (unsigned)few::WARPS * 32u, p.st, p.a_codes, p.a_scales, p.a_ts, p.b_codes,
                    p.b_scales, p.b_ts, p.c, (int)p.M, (int)p.N, (int)p.K, p.err);
}

template <int NT, int VEC, int ODT>
int launch_split(const Problem &p, const DeviceInfo &d, int ranks)
{
    using C = split::Cfg<NT>;
    auto kernel = nvfp4_linear_split<NT, VEC, ODT>;
    static OncePerDevice done;
    const int rc = allow_smem(kernel, C::SMEM, d, done);
    if (rc != IF4_OK) return rc;
    CUtensorMap mw, mx;
    if (!make_codes_map(&mw, p.b_codes, p.N, p.K, split::WR) ||
        !make_codes_map(&mx, p.a_codes, p.M, p.K, NT))
        return IF4_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    // token tiles next to each other, so that they share a weight tile in L2
    cfg.gridDim = dim3((unsigned)(ranks * ((p.M + NT - 1) / NT)),
                       (unsigned)((p.N + split::WR - 1) / split::WR), 1);
    cfg.blockDim = dim3(split::THREADS, 1, 1);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = p.st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ranks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return launched(cudaLaunchKernelEx(&cfg, kernel, mw, mx, p.b_scales, p.a_scales, p.b_ts, p.a_ts,
                                       p.c, (int)p.M, (int)p.N, (int)p.K, p.err));
}

// Two-byte C [M, N] -> tensor map with a box of 32 columns x 32 rows.
bool make_out_map(CUtensorMap *map, void *c, int64_t M, int64_t N)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)M};
    const cuuint64_t strides[1] = {(cuuint64_t)N * 2};
    const cuuint32_t box[2] = {32, 32};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, c, dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Packed scales [row blocks][K steps][512 bytes] -> tensor map with a box of
// one stage (4 K steps) x `blocks` row blocks.
bool make_scales_map(CUtensorMap *map, const void *base, int64_t row_blocks, int64_t K, int blocks)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t steps = (cuuint64_t)((K + SK - 1) / SK) * KSTEPS;
    const cuuint64_t dims[3] = {SF_STEP / 4, steps, (cuuint64_t)row_blocks};
    const cuuint64_t strides[2] = {SF_STEP, steps * SF_STEP};
    const cuuint32_t box[3] = {SF_STEP / 4, KSTEPS, (cuuint32_t)blocks};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void *>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Bytes of one operand's packed scales (row blocks of 128).
size_t packed_bytes(int64_t row_blocks, int64_t K)
{
    return (size_t)row_blocks * (size_t)((K + SK - 1) / SK) * SF_BLOCK;
}

// The pair kernel takes what has more than 64 rows and more tiles of 64 tokens x
// 128 columns than the split kernel runs at once (148 SMs x 2 CTAs; above 128
// rows, which fill a pair's tile, with two K ranks).  us split / pair, weights
// from memory: 128 x 2048 x 2048 6.5 / 8.4, 512 x 1024 x 4096 9.2 / 10.6, 128 x
// 14336 x 4096 (224 tiles) 14.0 / 15.1, 256 x 4096 x 4096 (128) 10.7 / 11.2, 256 x
// 4096 x 14336 20.3 / 23.5, and with 64 rows 64 x 28672 x 4096 17.8 / 23.5; from L2
// 256 x 256 x 512 3.6 / 5.5, 512 x 512 x 16384 12.6 / 23.4, 256 x 256 x 65536 18 /
// 75; but 320 x 4096 x 4096 (160) 12.7 / 11.4, 160 x 8192 x 4096 (192) 12.7 / 11.4,
// 96 x 28672 x 4096 (448) 26.5 / 23.9, 65536 x 128 x 4096 53 / 42.  Rows of scales
// on 2-byte boundaries cost the split kernel more, which loads them once per
// tile: 300 x 1555 x 4128 (65) 12.3 / 13.2, 500 x 1555 x 4128 (104) 16.4 / 13.2,
// 1000 x 1000 x 1056 (128) 8.2 / 7.6.
bool use_pair(int64_t M, int64_t N, int64_t K)
{
    const int64_t most = (M <= 128 ? 296 : 148) / (K % 64 ? 2 : 1);
    return M > 64 && (N + 127) / 128 * ((M + 63) / 64) > most;
}

template <int BN, int VEC, int ODT>
int launch_pair(const Problem &p, const DeviceInfo &d)
{
    using C = duo::Cfg<BN>;
    auto kernel = nvfp4_linear_pair<BN, ODT>;
    static OncePerDevice done;
    static std::atomic<int> resident[MAX_DEVICES];
    const int rc = allow_smem(kernel, C::SMEM, d, done);
    if (rc != IF4_OK) return rc;
    ScalePack sa{p.a_scales, static_cast<uint8_t *>(p.workspace), (int)p.M, 2 * duo::PM, 2};
    ScalePack sb{p.b_scales, nullptr, (int)p.N, BN, C::SFB_BLOCKS};
    sb.dst = sa.dst + packed_bytes(sa.row_blocks(), p.K);
    const bool boxes = ODT != IF4_F32 && p.N % 8 == 0 && reinterpret_cast<uintptr_t>(p.c) % 16 == 0;
    CUtensorMap ma, mb, msa, msb, mc = {};
    if (!make_codes_map(&ma, p.a_codes, p.M, p.K, duo::PM) ||
        !make_codes_map(&mb, p.b_codes, p.N, p.K, BN / 2) ||
        !make_scales_map(&msa, sa.dst, sa.row_blocks(), p.K, 1) ||
        !make_scales_map(&msb, sb.dst, sb.row_blocks(), p.K, C::SFB_BLOCKS) ||
        (boxes && !make_out_map(&mc, p.c, p.M, p.N)))
        return IF4_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = p.st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int64_t warps = (sa.row_blocks() + sb.row_blocks()) * ((p.K + UNIT - 1) / UNIT) * 2;
    const int64_t blocks = (warps + 7) / 8, most = (int64_t)d.sm_count * 8;
    cfg.gridDim = dim3((unsigned)(blocks < most ? blocks : most), 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    const int packed = launched(cudaLaunchKernelEx(&cfg, pack_scales<VEC>, sa, sb, (int)p.K, p.err));
    if (packed != IF4_OK) return packed;

    cfg.gridDim = dim3((unsigned)(2 * (d.sm_count / 2)), 1, 1);
    cfg.blockDim = dim3(duo::THREADS, 1, 1);
    cfg.dynamicSmemBytes = C::SMEM;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    // persistent: as many pairs as can be resident at once (the SMs of a pair
    // share a GPC, so this can be below sms / 2)
    int pairs_max = resident[d.id].load(std::memory_order_relaxed);
    if (pairs_max == 0) {
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
            (void)cudaGetLastError();
            n = 0;
        }
        pairs_max = n > 0 && n < d.sm_count / 2 ? n : d.sm_count / 2;
        resident[d.id].store(pairs_max, std::memory_order_relaxed);
    }
    const int64_t tiles = ((p.M + 2 * duo::PM - 1) / (2 * duo::PM)) * ((p.N + BN - 1) / BN);
    const int64_t pairs = tiles < pairs_max ? tiles : pairs_max;
    cfg.gridDim = dim3((unsigned)(2 * pairs), 1, 1);
    return launched(cudaLaunchKernelEx(&cfg, kernel, ma, mb, msa, msb, mc, boxes ? 1 : 0, p.a_ts,
                                       p.b_ts, p.c, (int)p.M, (int)p.N, (int)p.K, p.err));
}

template <int VEC, int ODT>
int launch_linear(const Problem &p, const DeviceInfo &d)
{
    if (use_pair(p.M, p.N, p.K)) {
        // narrow tiles while each has a pair of SMs of its own, or if one spans C
        const int64_t narrow = ((p.M + 2 * duo::PM - 1) / (2 * duo::PM)) * ((p.N + 127) / 128);
        return narrow <= d.sm_count / 2 || p.N <= 128
                   ? launch_pair<128, VEC, ODT>(p, d)
                   : launch_pair<240, VEC, ODT>(p, d);
    }
    if (few::takes(p.M, p.N, p.K))
        return p.M == 1 ? launch_few<1, ODT>(p) : launch_few<2, ODT>(p);
    // The largest power of two of K ranks that still runs in one wave: a second
    // wave costs more than all the splitting gains (32 x 4096 x 4096 6.5 against
    // 11.4 us).
    const int64_t wt = (p.N + split::WR - 1) / split::WR;
    const int64_t units = (p.K + UNIT - 1) / UNIT;
    auto tiles = [&](int nt) { return wt * ((p.M + nt - 1) / nt); };
    const int64_t slots = (int64_t)d.sm_count * split::PER_SM;
    auto run = [&](auto nt) {
        constexpr int NT = decltype(nt)::value;
        int s = 1;
        while (s < split::MAX_RANKS && 2 * s <= units && tiles(NT) * 2 * s <= slots) s *= 2;
        return launch_split<NT, VEC, ODT>(p, d, s);
    };
    // Few tokens per CTA make the reduction and the epilogue short, many read
    // the weights fewer times; the tiles' units of K say which counts.  us with 16
    // / 32 / 64 tokens per CTA: 32 x 4096 x 4096 6.5 / 7.3 / 7.4, 128 x 2048 x 2048
    // 6.4 / 6.8 / 8.1 (512 units each with 16); 64 x 4096 x 4096 8.1 / 7.7 / 9.4
    // (1024 with 16), 128 x 8192 x 4096 19.4 / 10.9 / 11.3 (2048 with 32); 128 x
    // 4096 x 14336 23.5 / 16.9 / 15.1 (3584 with 32), 128 x 14336 x 4096 35.3 /
    // 20.6 / 14.2.  And one wave whatever K is: 4096 x 256 x 512 8.4 / 4.9 / 6.1.
    auto suits = [&](int nt, int64_t most) {
        return p.M <= nt || (tiles(nt) <= slots && tiles(nt) * units <= most);
    };
    if (suits(16, 768)) return run(std::integral_constant<int, 16>{});
    if (suits(32, 2048)) return run(std::integral_constant<int, 32>{});
    return run(std::integral_constant<int, 64>{});
}

}  // namespace

extern "C" size_t nvfp4_linear_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    if (M < 1 || N < 1 || K < 32 || K % 32 != 0 || M > MAX_MN || N > MAX_MN || K > MAX_K) return 0;
    // B in tiles of 240 columns, two blocks each; tiles of 128 columns, one block
    // each, never need more: 2 ceil(N / 240) >= ceil(N / 128)
    return use_pair(M, N, K) ? packed_bytes((M + 255) / 256 * 2 + (N + 239) / 240 * 2, K) : 0;
}

extern "C" int nvfp4_linear(const uint8_t *a_codes, const uint8_t *a_scales, const float *a_ts,
                            const uint8_t *b_codes, const uint8_t *b_scales, const float *b_ts,
                            int64_t M, int64_t N, int64_t K, void *workspace, size_t ws_bytes,
                            void *c, int c_dtype, int *err_flag, void *stream)
{
    if (M < 0 || N < 0 || K < 32 || K % 32 != 0) return IF4_ERR_SHAPE;
    if (M > MAX_MN || N > MAX_MN || K > MAX_K) return IF4_ERR_SHAPE;
    if (c_dtype != IF4_F32 && c_dtype != IF4_BF16 && c_dtype != IF4_F16) return IF4_ERR_DTYPE;
    if (!err_flag) return IF4_ERR_NULL;
    if (M == 0 || N == 0) return IF4_OK;
    if (!a_codes || !a_scales || !a_ts || !b_codes || !b_scales || !b_ts || !c) return IF4_ERR_NULL;
    auto misaligned = [](const void *q, uintptr_t n) { return reinterpret_cast<uintptr_t>(q) % n != 0; };
    if (misaligned(a_codes, 16) || misaligned(b_codes, 16) || misaligned(a_scales, 2) ||
        misaligned(b_scales, 2) || misaligned(a_ts, 4) || misaligned(b_ts, 4) ||
        misaligned(err_flag, 4) || misaligned(c, c_dtype == IF4_F32 ? 4 : 2))
        return IF4_ERR_ALIGN;
    const size_t need = nvfp4_linear_workspace_bytes(M, N, K);
    if (need && (!workspace || ws_bytes < need)) return IF4_ERR_WORKSPACE;
    if (need && misaligned(workspace, 256)) return IF4_ERR_ALIGN;
    DeviceInfo d;
    const int rc = check_device(d);
    if (rc != IF4_OK) return rc;
    const Problem p{a_codes, a_scales, b_codes, b_scales, a_ts, b_ts, M, N, K, workspace, c, err_flag,
                    static_cast<cudaStream_t>(stream)};
    const int vec = K % 256 == 0 && !misaligned(a_scales, 16) && !misaligned(b_scales, 16) ? 16
                    : K % 64 == 0 && !misaligned(a_scales, 4) && !misaligned(b_scales, 4) ? 4 : 2;
    auto typed = [&](auto v) {
        constexpr int V = decltype(v)::value;
        return c_dtype == IF4_F32    ? launch_linear<V, IF4_F32>(p, d)
               : c_dtype == IF4_BF16 ? launch_linear<V, IF4_BF16>(p, d)
                                     : launch_linear<V, IF4_F16>(p, d);
    };
    return vec == 16  ? typed(std::integral_constant<int, 16>{})
           : vec == 4 ? typed(std::integral_constant<int, 4>{})
                      : typed(std::integral_constant<int, 2>{});
}
