// RMS norm with the residual's addition and a 4-bit output, and its gradient
// (sm_100a).
//
// Forward, per row of x [R, C]:
//   h    = RN(x + r)                     the residual stream, in x's type
//   rstd = fl32(1 / sqrt(sum(h^2) / C + eps))    the sum and the root in binary64
//   y    = fl(fl(h * rstd) * w)          binary32
//   codes, scales = IF4 or NVFP4 of y under the given tensor scale
// y never reaches memory.  The binary64 sum makes rstd the correctly rounded
// value whatever the order of the additions, up to ties that a binary64 sum
// cannot resolve: a row's codes then depend on nothing but the row, and equal
// those of quantizing y computed any other way that takes the same roundings.
// (A binary32 sum moves rstd by a few steps, and with it values next to a
// rounding border of the 4-bit grid by a whole step.)
//
// Backward, with n = h * rstd the normalized row, g = dy * w:
//   dx = RN(dres + rstd * (g - n * mean(g * n))),   dw = sum over rows of dy * n.
// The quantizer passes gradients straight through.  dw's sum over the rows, as
// long as a batch, keeps more than binary32: each term n rounds once, a block's
// sum of its rows is rounded once, and the sum of the blocks' once.

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/if4.h"
#include "if4_device.cuh"
#include "if4_encode.cuh"
#include "if4_host.cuh"
#include "if4_load.cuh"

namespace {

constexpr int NORM_THREADS = 256;

// A group's 16 raw values as binary32 pairs.
template <int DT>
__device__ __forceinline__ void to_pairs(const Raw<DT> &r, f2_t (&x)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if constexpr (DT == DT_F32)
            x[j] = f2_pack(__uint_as_float(r.w[2 * j]), __uint_as_float(r.w[2 * j + 1]));
        else if constexpr (DT == DT_BF16)
            x[j] = f2_from_bf16x2(r.w[j]);
        else
            x[j] = f2_pack(f16lo_to_f32(r.w[j]), f16hi_to_f32(r.w[j]));
    }
}

// Binary32 pairs rounded to the type's raw bits.
template <int DT>
__device__ __forceinline__ void to_raw(const f2_t (&x)[8], Raw<DT> &r)
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float lo, hi;
        f2_unpack(x[j], lo, hi);
        if constexpr (DT == DT_F32) {
            r.w[2 * j] = __float_as_uint(lo);
            r.w[2 * j + 1] = __float_as_uint(hi);
        } else {
            r.w[j] = DT == DT_BF16 ? bf16x2_from_f32(lo, hi) : f16x2_from_f32(lo, hi);
        }
    }
}

template <int DT>
__device__ __forceinline__ void store_group(char *p, const Raw<DT> &r)
{
#pragma unroll
    for (int q = 0; q < (DT == DT_F32 ? 4 : 2); ++q)
        st_v4(p + 16 * q, r.w[4 * q], r.w[4 * q + 1], r.w[4 * q + 2], r.w[4 * q + 3]);
}

// Sum over a block of NORM_THREADS; every thread gets it.
template <typename T>
__device__ __forceinline__ T block_sum(T v, T *buf)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    __syncthreads();                       // buf may still be read
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    T s = buf[0];
#pragma unroll
    for (int i = 1; i < NORM_THREADS / 32; ++i) s += buf[i];
    return s;
}

struct NormArgs {
    const char *x, *res, *w;        // w: binary32 or x's type
    char *h;
    int64_t ld_x, ld_res, ld_h;     // bytes
    uint8_t *codes, *scales;
    const float *ts;
    float *rstd;
    unsigned int *amax;
    int *err;
    int64_t rows;
    int gpr;                        // groups per row
    bool v8;                        // x, residual and h on 32-byte boundaries
    double inv_cols, eps;
};

// s + v * v in binary64 for a binary32 value's bits.  The conversion instruction
// runs at a quarter of the rate of the multiply-add beside it, so the value is
// rebiased by hand: |v|'s bits moved down by 3 plus 896 exponents.  That takes
// 0 and subnormals for numbers of about 2^-127, whose squares vanish beside
// any eps, and Inf and NaN for finite ones, which the codes' check reports.
// Values of 16-bit types leave the low word empty.
template <int DT>
__device__ __forceinline__ double add_square(double s, float v)
{
    const uint32_t b = __float_as_uint(v);
    uint32_t hi;
    asm("mad.hi.u32 %0, %1, %2, %3;"
        : "=r"(hi) : "r"(b & 0x7FFFFFFFu), "r"(0x20000000u), "r"(0x38000000u));
    const double x = __hiloint2double((int)hi, DT == DT_F32 ? (int)(b << 29) : 0);
    return fma(x, x, s);
}

// rstd of a row from its binary64 sum of squares.  The binary32 reciprocal root
// (2^-22 off at most) and two Newton steps in binary64 leave 2^-52, so the one
// rounding to binary32 is the rounding of the definition's value (which has
// the same freedom in its last binary64 bits); the division and root in
// binary64 took as long as a sixth of the row.  Outside binary32's comfortable
// range they are used as they stand.
__device__ __noinline__ float row_rstd_general(double v) { return (float)(1.0 / sqrt(v)); }

__device__ __forceinline__ float row_rstd(double s, double inv_cols, double eps)
{
    const double v = fma(s, inv_cols, eps);
    if (!(v > 1e-30 && v < 1e30)) return row_rstd_general(v);
    double r = (double)rsqrtf((float)v);
#pragma unroll
    for (int i = 0; i < 2; ++i) r = fma(r * 0.5, fma(-v * r, r, 1.0), r);
    return (float)r;
}

// The same for stores, 256 bits where the addresses allow it.
template <int DT>
__device__ __forceinline__ void store_group(char *p, const Raw<DT> &r, bool v8)
{
    if (v8) {
#pragma unroll
        for (int q = 0; q < (DT == DT_F32 ? 2 : 1); ++q)
            st_v8(p + 32 * q, *reinterpret_cast<const uint32_t(*)[8]>(r.w + 8 * q));
    } else {
        store_group<DT>(p, r);
    }
}

template <int DT>
__device__ __forceinline__ void zero_group(Raw<DT> &r)
{
#pragma unroll
    for (uint32_t &w : r.w) w = 0u;
}

// A group of the weight (L1 keeps it for the next rows).
template <int WT>
__device__ __forceinline__ void load_weight(const char *w, int g, Raw<WT> &r)
{
    const char *p = w + (int64_t)g * 16 * elem_bytes<WT>();
#pragma unroll
    for (int q = 0; q < (WT == DT_F32 ? 4 : 2); ++q)
        ld_after_wait_v4(p + 16 * q, r.w[4 * q], r.w[4 * q + 1], r.w[4 * q + 2], r.w[4 * q + 3]);
}

// h = RN(x + r), into x.  16-bit types add in their own type: the sum of two
// such values either is exact in binary32 or has one operand below a quarter
// step of the other, so rounding once or through binary32 is the same.
template <int DT>
__device__ __forceinline__ void add_residual(Raw<DT> &x, const Raw<DT> &r)
{
    if constexpr (DT == DT_F32) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            x.w[j] = __float_as_uint(__fadd_rn(__uint_as_float(x.w[j]), __uint_as_float(r.w[j])));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (DT == DT_BF16)
                asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(x.w[j]) : "r"(r.w[j]));
            else
                asm("add.rn.f16x2 %0, %0, %1;" : "+r"(x.w[j]) : "r"(r.w[j]));
        }
    }
}

// A group's sum of squares added to s, s + s1 in two chains.  bf16 goes from its
// packed words to the rebiased binary64 words directly (see add_square).
template <int DT>
__device__ __forceinline__ double add_group_squares(double s, const Raw<DT> &h)
{
    double s1 = 0.0;
    if constexpr (DT == DT_BF16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t w = h.w[j];
            const uint32_t lo = (w & 0x7FFFu) * 8192u + 0x38000000u;
            uint32_t hi;
            asm("mad.hi.u32 %0, %1, %2, %3;"
                : "=r"(hi) : "r"(w & 0x7FFF0000u), "r"(0x20000000u), "r"(0x38000000u));
            const double x = __hiloint2double((int)lo, 0), y = __hiloint2double((int)hi, 0);
            s = fma(x, x, s);
            s1 = fma(y, y, s1);
        }
    } else {
        f2_t v[8];
        to_pairs<DT>(h, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float lo, hi;
            f2_unpack(v[j], lo, hi);
            s = add_square<DT>(s, lo);
            s1 = add_square<DT>(s1, hi);
        }
    }
    return s + s1;
}

// Rings in shared memory, one per warp: a warp copies the pieces that its
// lanes will need of later rows there with cp.async and reads back only those,
// so its lanes' wait_group and a __syncwarp order everything.  Loads in flight
// then hold no registers, which the encoder needs.
//
// A warp's lanes own PP consecutive 16-byte pieces each.  They are copied with
// neighbouring lanes on neighbouring pieces (each lane copying its own fetched every
// 32-byte sector twice: 124 against 86 us for the norm of 8192 x 8192), and
// placed so that eight lanes reading their q-th pieces hit different banks.
template <int PP>
__device__ __forceinline__ uint32_t piece_pos(uint32_t p)
{
    static_assert(PP == 1 || PP == 2 || PP == 4, "pieces per lane");
    return 16u * (PP == 1 ? p : p ^ ((p >> 3) & (PP - 1)));
}

// Pieces p < valid of a warp's span, from src to ring (both the warp's).
template <int PP>
__device__ __forceinline__ void ring_copy(uint32_t ring, const char *src, int valid)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int q = 0; q < PP; ++q) {
        const int p = q * 32 + lane;
        if (p < valid)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                         :: "r"(ring + piece_pos<PP>(p)), "l"(src + p * 16) : "memory");
    }
}

// This lane's PP pieces.
template <int PP>
__device__ __forceinline__ void ring_read(uint32_t ring, uint32_t *w)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int q = 0; q < PP; ++q)
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[4 * q]), "=r"(w[4 * q + 1]), "=r"(w[4 * q + 2]), "=r"(w[4 * q + 3])
                     : "r"(ring + piece_pos<PP>(lane * PP + q)) : "memory");
}

__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// until at most N of the warp's newest groups are under way
template <int N>
__device__ __forceinline__ void ring_wait()
{
    asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory");
    __syncwarp();
}

// h of one group: x, or RN(x + residual).
template <int DT>
__device__ __forceinline__ void load_h(const NormArgs &a, int64_t row, int g, Raw<DT> &h)
{
    constexpr int GB = 16 * elem_bytes<DT>();
    load_group_rw<DT>(a.x + row * a.ld_x + (int64_t)g * GB, h, a.v8);
    if (a.res) {
        Raw<DT> r;
        load_group_rw<DT>(a.res + row * a.ld_res + (int64_t)g * GB, r, a.v8);
        add_residual<DT>(h, r);
    }
}

// Rows of up to G groups per thread of the block: one pass, h kept in
// registers between the sum and the encode (the weight comes from L1 each
// time).  A block takes rows blockIdx.x, + gridDim.x, ...; PREFETCH: the next
// row's loads are issued as soon as h of a row is formed.
//
// The encoder's and the norm's instructions bound it as much as memory does (IF4
// 8192 x 8192 bf16: 402 per group, 61 % of the issue slots with DRAM 59 % busy;
// NVFP4 280, 54 and 73 %), so two groups per thread, which
// share the row's sum, with loads straight to registers (128 of them, 512
// threads per SM) beat one group (64 registers, 1024 threads: 92 us) and rows
// under way in shared memory (85 us).
template <int DT, int WT, int MODE, int G, bool PREFETCH>
__global__ void __launch_bounds__(PREFETCH ? 512 : 1024, 1)
rms_norm_quantize_rows_kernel(const __grid_constant__ NormArgs a)
{
    pdl_enter();
    __shared__ float inv_tab[128];
    __shared__ double sums[2][32];
    constexpr int GB = 16 * elem_bytes<DT>();
    const float ts = ld_after_wait(a.ts);
    const float rts = __frcp_rn(ts);
    if (blockIdx.x == 0 && threadIdx.x == 0 && !ts_valid(ts) && a.err)
        atomicOr(a.err, IF4_DEV_BAD_SCALE);
    for (int i = threadIdx.x; i < 128; i += blockDim.x)
        inv_tab[i] = i == 0 ? 0.0f : __frcp_rn(__fmul_rn(f32_from_e4m3(i), ts));
    Raw<DT> x[PREFETCH ? G : 1], r[PREFETCH ? G : 1];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int k = 0; k < (PREFETCH ? G : 0); ++k) {
            const int g = threadIdx.x + k * blockDim.x;
            if (g < a.gpr) {
                load_group_rw<DT>(a.x + row * a.ld_x + (int64_t)g * GB, x[k], a.v8);
                if (a.res) load_group_rw<DT>(a.res + row * a.ld_res + (int64_t)g * GB, r[k], a.v8);
            }
        }
    };
#pragma unroll
    for (int k = 0; k < (PREFETCH ? G : 0); ++k) {
        zero_group(x[k]);
        zero_group(r[k]);
    }
    bool nonfinite = false;
    uint32_t top = 0;
    int par = 0;
    const int warps = blockDim.x >> 5;
    int64_t row = blockIdx.x;
    if (PREFETCH && row < a.rows) fetch(row);
    __syncthreads();                        // inv_tab
    for (; row < a.rows; row += gridDim.x, par ^= 1) {
        double s = 0.0;
        Raw<DT> h[G];
#pragma unroll
        for (int k = 0; k < G; ++k) {
            if constexpr (PREFETCH) {
                h[k] = x[k];
                if (a.res) add_residual<DT>(h[k], r[k]);
            } else {
                const int g = threadIdx.x + k * blockDim.x;
                zero_group(h[k]);
                if (g < a.gpr) load_h<DT>(a, row, g, h[k]);
            }
            s = add_group_squares<DT>(s, h[k]);
        }
        // h may be x's or the residual's memory: this row's store only comes
        // after this row's loads, and no other block reads this row
#pragma unroll
        for (int k = 0; k < G; ++k) {
            const int g = threadIdx.x + k * blockDim.x;
            if (a.h && g < a.gpr)
                store_group<DT>(a.h + row * a.ld_h + (int64_t)g * GB, h[k], a.v8);
        }
        if (PREFETCH && row + gridDim.x < a.rows) fetch(row + gridDim.x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        if (warps > 1) {
            // two buffers in turn: a warp writes row i + 2's only after the
            // barrier of row i + 1, which every reader of row i's has passed
            if ((threadIdx.x & 31) == 0) sums[par][threadIdx.x >> 5] = s;
            __syncthreads();
            const int i = threadIdx.x & 31;
            s = i < warps ? sums[par][i] : 0.0;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        }
        const float rstd = row_rstd(s, a.inv_cols, a.eps);
        if (threadIdx.x == 0 && a.rstd) a.rstd[row] = rstd;
        const f2_t RS = f2_pack(rstd, rstd);
#pragma unroll
        for (int k = 0; k < G; ++k) {
            const int g = threadIdx.x + k * blockDim.x;
            if (g < a.gpr) {
                f2_t v[8], wv[8];
                Raw<WT> w;
                load_weight<WT>(a.w, g, w);
                to_pairs<DT>(h[k], v);
                to_pairs<WT>(w, wv);
                float mx = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[j] = f2_mul(f2_mul(v[j], RS), wv[j]);
                    float lo, hi;
                    f2_unpack(v[j], lo, hi);
                    mx = absmax3_f32(mx, lo, hi);
                }
                const uint32_t m = __float_as_uint(mx);
                nonfinite |= m >= 0x7F800000u;
                top = max(top, m);
                const GroupCode c = encode_registers<MODE>(v, __uint_as_float(m), ts, rts, inv_tab);
                const int64_t gi = row * a.gpr + g;
                st_v2(a.codes + gi * 8, c.c0, c.c1);
                st_u8(a.scales + gi, c.scale);
            }
        }
    }
    if (a.amax) {
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        if ((threadIdx.x & 31) == 0) atomicMax(a.amax, top);
    }
    if (nonfinite && a.err) atomicOr(a.err, IF4_DEV_NONFINITE);
}

// More columns than the rows kernel holds in registers: a block per row, h
// formed twice (the second time mostly from L2).
template <int DT, int WT, int MODE>
__global__ void __launch_bounds__(NORM_THREADS)
rms_norm_quantize_kernel(const __grid_constant__ NormArgs a)
{
    pdl_enter();
    __shared__ float inv_tab[128];
    __shared__ double sums[NORM_THREADS / 32];
    const float ts = ld_after_wait(a.ts);
    const float rts = __frcp_rn(ts);
    if (blockIdx.x == 0 && threadIdx.x == 0 && !ts_valid(ts) && a.err)
        atomicOr(a.err, IF4_DEV_BAD_SCALE);
    fill_inv_tab(inv_tab, ts);
    constexpr int GB = 16 * elem_bytes<DT>();
    bool nonfinite = false;
    uint32_t top = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        double s = 0.0;
        for (int g = threadIdx.x; g < a.gpr; g += NORM_THREADS) {
            Raw<DT> h;
            f2_t v[8];
            load_h<DT>(a, row, g, h);
            to_pairs<DT>(h, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float lo, hi;
                f2_unpack(v[j], lo, hi);
                s = add_square<DT>(s, lo);
                s = add_square<DT>(s, hi);
            }
        }
        s = block_sum(s, sums);
        const float rstd = row_rstd(s, a.inv_cols, a.eps);
        if (threadIdx.x == 0 && a.rstd) a.rstd[row] = rstd;
        const f2_t RS = f2_pack(rstd, rstd);
        for (int g = threadIdx.x; g < a.gpr; g += NORM_THREADS) {
            Raw<DT> h;
            Raw<WT> wr;
            f2_t v[8], w[8];
            load_h<DT>(a, row, g, h);
            if (a.h) store_group<DT>(a.h + row * a.ld_h + (int64_t)g * GB, h);
            load_weight<WT>(a.w, g, wr);
            to_pairs<DT>(h, v);
            to_pairs<WT>(wr, w);
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = f2_mul(f2_mul(v[j], RS), w[j]);
                float lo, hi;
                f2_unpack(v[j], lo, hi);
                m = absmax_f32(m, lo);
                m = absmax_f32(m, hi);
            }
            m &= 0x7FFFFFFFu;
            nonfinite |= m >= 0x7F800000u;
            top = max(top, m);
            const GroupCode c = encode_registers<MODE>(v, __uint_as_float(m), ts, rts, inv_tab);
            const int64_t gi = row * a.gpr + g;
            st_v2(a.codes + gi * 8, c.c0, c.c1);
            st_u8(a.scales + gi, c.scale);
        }
    }
    if (a.amax) {
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        if ((threadIdx.x & 31) == 0) atomicMax(a.amax, top);
    }
    if (nonfinite && a.err) atomicOr(a.err, IF4_DEV_NONFINITE);
}

// -------------------------------------------------------------- gradient ----

constexpr int BACK_BLOCKS = 296;     // partial sums of dw at most
constexpr int BACK_THREADS = 512;

struct BackArgs {
    const char *dy, *h, *w, *dres;
    char *dx;
    int64_t ld_dy, ld_h, ld_dres, ld_dx;   // bytes
    const float *rstd;
    float *part;                    // [BACK_BLOCKS][cols]
    int64_t rows;
    int gpr;
    bool v8;                        // every matrix on 32-byte boundaries
    float inv_cols;
};

// Sums of dw over many rows: s + c is the sum, s its binary32 value and c what
// s's additions rounded away.  With p = x * y exact, t = RN(s + p) and d = RN(s - t),
// d + p is the rounding error of t whenever s - t is exact, which it is unless
// |p| > |s| / 2; then d is off by at most 2^-24 |p|.  So a term costs at most one
// rounding of its own size, and in a long sum almost none does, where a plain
// chain's roundings are of the size of the sum.
__device__ __forceinline__ void add_product(f2_t &s, f2_t &c, f2_t x, f2_t y)
{
    const f2_t t = f2_fma(x, y, s);
    c = f2_add(c, f2_fma(x, y, f2_sub(s, t)));
    s = t;
}

// s + c += s1 + c1, with the rounding error of s + s1 whatever their sizes.
__device__ __forceinline__ void add_sums(f2_t &s, f2_t &c, f2_t s1, f2_t c1)
{
    const f2_t t = f2_add(s, s1), b = f2_sub(t, s);
    const f2_t e = f2_add(f2_sub(s, f2_sub(t, b)), f2_sub(s1, b));
    c = f2_add(c, f2_add(e, c1));
    s = t;
}

// The sum, rounded once.  A c that is not finite says nothing: it comes from an
// s that is Inf or NaN, or was on the way.
__device__ __forceinline__ float sum_of(float s, float c)
{
    return fabsf(c) <= 3.402823466e38f ? __fadd_rn(s, c) : s;
}

// The gradient's rows kernel works in units of 8 elements.
template <int DT>
struct Unit {
    static constexpr int BYTES = 8 * elem_bytes<DT>();
    uint32_t w[DT == DT_F32 ? 8 : 4];
};

// Pair j (elements 2j, 2j + 1) in binary32.
template <int DT>
__device__ __forceinline__ f2_t pair_of(const Unit<DT> &r, int j)
{
    if constexpr (DT == DT_F32)
        return f2_pack(__uint_as_float(r.w[2 * j]), __uint_as_float(r.w[2 * j + 1]));
    else if constexpr (DT == DT_BF16)
        return f2_from_bf16x2(r.w[j]);
    else
        return f2_pack(f16lo_to_f32(r.w[j]), f16hi_to_f32(r.w[j]));
}

template <int DT, int U>
struct BackRing {
    static constexpr int S = DT != DT_F32 && U == 2 ? 4 : 2;     // rows under way
    static constexpr int BYTES = S * 3 * U * Unit<DT>::BYTES;    // per thread: h, dy, dres
};

// Rows of up to U * T units: one pass over dy, h and dres.  A block of 512 =
// `slots` x T threads holds `slots` rows at a time, T threads each (a power of
// two, at least a warp), with the next S rows of each slot under way in its
// threads' rings (192 KB, one block per SM); a thread keeps its columns' part of
// dw in registers over all its rows, in twice binary32's precision.  The row sums
// meet at a barrier of the row's own threads.  At the end the block's row slots
// add their parts through shared memory, and the block writes one partial row of
// binary32 values.
//
// Memory (73 % busy) and its instructions (195 per unit, 57 % of the issue slots)
// bound it together: 16384 x 4096 bf16 87 to 94 us from board to board, where memory
// needs 82.  dw's sums take four of the seven arithmetic instructions per pair of
// columns in front of the row's sum.  What two units per thread share of a row (its
// sum, barrier and addresses) pays for them: one unit per thread took 101 (64
// registers, 1024 threads per SM), and 126 with a row's inputs held in registers
// over the sum, which spilled, instead of read from the ring again.  Above 8192
// columns four units, whose weight comes from L1 each time: 4096 x 12288 95 us, and
// 121 with the weight in registers, which spilled.
template <int DT, int WT, int U>
__global__ void __launch_bounds__(BACK_THREADS, 1)
rms_norm_backward_rows_kernel(const __grid_constant__ BackArgs a, int T)
{
    pdl_enter();
    using R = BackRing<DT, U>;
    constexpr int UP = elem_bytes<DT>() / 2;        // pieces of a unit
    __shared__ float sums[2][32];
    extern __shared__ __align__(16) uint8_t back_smem[];   // the rings, then the slots' dw
    const int slots = blockDim.x / T, slot = threadIdx.x / T, t = threadIdx.x % T;
    const int warps = T >> 5, warp0 = slot * warps;
    const int units = a.gpr * 2;
    const int64_t step = (int64_t)gridDim.x * slots;
    // the weight: in registers with two units per thread, from L1 with four
    auto weight = [&](int u) {
        Unit<WT> r;
#pragma unroll
        for (uint32_t &z : r.w) z = 0u;
        if (u < units) {
#pragma unroll
            for (int q = 0; q < (WT == DT_F32 ? 2 : 1); ++q)
                ld_after_wait_v4(a.w + (int64_t)u * Unit<WT>::BYTES + 16 * q, r.w[4 * q],
                                 r.w[4 * q + 1], r.w[4 * q + 2], r.w[4 * q + 3]);
        }
        return r;
    };
    Unit<WT> held[2];
    if constexpr (U == 2)
#pragma unroll
        for (int k = 0; k < 2; ++k) held[k] = weight(t + k * T);
    auto weight_of = [&](int k) {
        if constexpr (U == 2) return held[k];
        else return weight(t + k * T);
    };
    f2_t dw[U][4], dc[U][4];
#pragma unroll
    for (int k = 0; k < U; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) dw[k][j] = dc[k][j] = f2_pack(0.0f, 0.0f);
    // a warp's ring: [stage][h, dy, dres][unit of the lane][span of 32 units]
    constexpr uint32_t SPAN = 32 * Unit<DT>::BYTES;
    const int u0 = t & ~31;                         // the warp's first unit
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(back_smem) +
                          (threadIdx.x >> 5) * (32 * R::BYTES);
    auto fetch = [&](int64_t row, int stage) {
        __syncwarp();                      // the lanes have read what this overwrites
        if (row < a.rows) {
            auto copy = [&](const char *src, int64_t ld, int which) {
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int u = u0 + k * T;
                    ring_copy<UP>(ring + ((stage * 3 + which) * U + k) * SPAN,
                                  src + row * ld + (int64_t)u * Unit<DT>::BYTES, (units - u) * UP);
                }
            };
            copy(a.h, a.ld_h, 0);
            copy(a.dy, a.ld_dy, 1);
            if (a.dres) copy(a.dres, a.ld_dres, 2);
        }
        ring_commit();                     // also when empty: the waits count groups
    };
    int par = 0, stage = 0;
    int64_t row = (int64_t)blockIdx.x * slots + slot;
    // dx may be dy's or dres's memory: a warp stores only what it has copied
    // itself, and no other warp reads that
#pragma unroll
    for (int i = 0; i < R::S; ++i) fetch(row + i * step, i);
    float rstd_next = row < a.rows ? a.rstd[row] : 0.0f;
    for (; row < a.rows; row += step, par ^= 1) {
        ring_wait<R::S - 1>();
        const float rstd = rstd_next;
        if (row + step < a.rows) rstd_next = a.rstd[row + step];
        Unit<DT> h, d, e;
        auto read = [&](int k, bool with_e) {
            const uint32_t r = ring + (stage * 3 * U + k) * SPAN;
            ring_read<UP>(r, h.w);
            ring_read<UP>(r + U * SPAN, d.w);
            if (with_e && a.dres) ring_read<UP>(r + 2 * U * SPAN, e.w);
        };
        f2_t acc = f2_pack(0.0f, 0.0f);
        const f2_t RS = f2_pack(rstd, rstd);
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (t + k * T < units) {
                read(k, false);
                const Unit<WT> w = weight_of(k);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // (n first: dy * h may leave binary32's range where dy * n does not)
                    const f2_t n = f2_mul(pair_of(h, j), RS), dy = pair_of(d, j);
                    add_product(dw[k][j], dc[k][j], dy, n);
                    acc = f2_fma(f2_mul(dy, pair_of(w, j)), n, acc);
                }
            }
        float s, hi;
        f2_unpack(acc, s, hi);
        s += hi;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        if (warps > 1) {
            // two buffers in turn: see the forward kernel
            if ((threadIdx.x & 31) == 0) sums[par][threadIdx.x >> 5] = s;
            // (barrier 0 is __syncthreads', below)
            asm volatile("bar.sync %0, %1;" :: "r"(slot + 1), "r"(T) : "memory");
            const int i = threadIdx.x & 31;
            s = i < warps ? sums[par][warp0 + i] : 0.0f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        }
        // mean(g * n) * rstd, n = h * rstd
        const float c = s * rstd * a.inv_cols;
        const f2_t NC = f2_pack(-c, -c);
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int u = t + k * T;
            if (u < units) {
                read(k, true);
                const Unit<WT> w = weight_of(k);
                uint32_t o[DT == DT_F32 ? 8 : 4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    f2_t v = f2_mul(f2_fma(pair_of(h, j), NC,
                                           f2_mul(pair_of(d, j), pair_of(w, j))), RS);
                    if (a.dres) v = f2_add(v, pair_of(e, j));
                    float lo, up;
                    f2_unpack(v, lo, up);
                    if constexpr (DT == DT_F32) {
                        o[2 * j] = __float_as_uint(lo);
                        o[2 * j + 1] = __float_as_uint(up);
                    } else {
                        o[j] = DT == DT_BF16 ? bf16x2_from_f32(lo, up) : f16x2_from_f32(lo, up);
                    }
                }
                char *p = a.dx + row * a.ld_dx + (int64_t)u * Unit<DT>::BYTES;
#pragma unroll
                for (int q = 0; q < (DT == DT_F32 ? 2 : 1); ++q)
                    st_v4(p + 16 * q, o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
            }
        }
        fetch(row + R::S * step, stage);
        if (++stage == R::S) stage = 0;
    }
    // the block's partial row: the slots' parts added in order, two columns per
    // thread, through the rings' memory (every copy has landed and been read; a
    // thread's sums take 64 * U of its 192 * U bytes)
    const int cols = a.gpr * 16;
    float *slot_s = reinterpret_cast<float *>(back_smem), *slot_c = slot_s + slots * cols;
    float *out = a.part + (int64_t)blockIdx.x * cols;
    auto put = [&](int at, f2_t s, f2_t c) {
        float s0, s1, c0, c1;
        f2_unpack(s, s0, s1);
        f2_unpack(c, c0, c1);
        *reinterpret_cast<f2_t *>(out + at) = f2_pack(sum_of(s0, c0), sum_of(s1, c1));
    };
    if (slots > 1) __syncthreads();
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int u = t + k * T;
        if (u < units)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int at = u * 8 + 2 * j;
                if (slots == 1) {
                    put(at, dw[k][j], dc[k][j]);
                } else {
                    *reinterpret_cast<f2_t *>(slot_s + slot * cols + at) = dw[k][j];
                    *reinterpret_cast<f2_t *>(slot_c + slot * cols + at) = dc[k][j];
                }
            }
    }
    if (slots > 1) {
        __syncthreads();
        for (int at = 2 * threadIdx.x; at < cols; at += 2 * blockDim.x) {
            f2_t s = *reinterpret_cast<const f2_t *>(slot_s + at);
            f2_t c = *reinterpret_cast<const f2_t *>(slot_c + at);
            for (int q = 1; q < slots; ++q)
                add_sums(s, c, *reinterpret_cast<const f2_t *>(slot_s + q * cols + at),
                         *reinterpret_cast<const f2_t *>(slot_c + q * cols + at));
            put(at, s, c);
        }
    }
}

// More columns than the rows kernel holds: dx with a block per row, dy and h
// read twice, and dw's partial sums by a kernel of their own.
template <int DT, int WT>
__global__ void __launch_bounds__(NORM_THREADS)
rms_norm_dx_kernel(const __grid_constant__ BackArgs a)
{
    pdl_enter();
    __shared__ float sums[NORM_THREADS / 32];
    constexpr int GB = 16 * elem_bytes<DT>();
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float rstd = a.rstd[row];
        const f2_t RS = f2_pack(rstd, rstd);
        float s = 0.0f;
        for (int g = threadIdx.x; g < a.gpr; g += NORM_THREADS) {
            Raw<DT> hr, dr;
            Raw<WT> wr;
            f2_t h[8], d[8], w[8];
            load_group_rw<DT>(a.h + row * a.ld_h + (int64_t)g * GB, hr, a.v8);
            load_group_rw<DT>(a.dy + row * a.ld_dy + (int64_t)g * GB, dr, a.v8);
            load_weight<WT>(a.w, g, wr);
            to_pairs<DT>(hr, h);
            to_pairs<DT>(dr, d);
            to_pairs<WT>(wr, w);
            f2_t acc = f2_pack(0.0f, 0.0f);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc = f2_fma(f2_mul(d[j], w[j]), f2_mul(h[j], RS), acc);
            float lo, hi;
            f2_unpack(acc, lo, hi);
            s += lo + hi;
        }
        s = block_sum(s, sums);
        // mean(g * n) * rstd, n = h * rstd
        const float k = s * rstd * a.inv_cols;
        const f2_t NK = f2_pack(-k, -k);
        for (int g = threadIdx.x; g < a.gpr; g += NORM_THREADS) {
            Raw<DT> hr, dr, er;
            Raw<WT> wr;
            f2_t h[8], d[8], w[8], e[8];
            load_group_rw<DT>(a.h + row * a.ld_h + (int64_t)g * GB, hr, a.v8);
            load_group_rw<DT>(a.dy + row * a.ld_dy + (int64_t)g * GB, dr, a.v8);
            load_weight<WT>(a.w, g, wr);
            to_pairs<DT>(hr, h);
            to_pairs<DT>(dr, d);
            to_pairs<WT>(wr, w);
            if (a.dres) {
                load_group_rw<DT>(a.dres + row * a.ld_dres + (int64_t)g * GB, er, a.v8);
                to_pairs<DT>(er, e);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                f2_t v = f2_mul(f2_fma(h[j], NK, f2_mul(d[j], w[j])), RS);
                d[j] = a.dres ? f2_add(v, e[j]) : v;
            }
            Raw<DT> o;
            to_raw<DT>(d, o);
            store_group<DT>(a.dx + row * a.ld_dx + (int64_t)g * GB, o);
        }
    }
}

// Partial sums of dw: block (i, c) adds rows i, i + n, ... for 512 columns, two
// per thread.
template <int DT>
__global__ void __launch_bounds__(256)
rms_norm_dw_kernel(const __grid_constant__ BackArgs a)
{
    pdl_enter();
    constexpr int ES = elem_bytes<DT>();
    const int col = (blockIdx.y * 256 + threadIdx.x) * 2;
    if (col >= a.gpr * 16) return;
    auto pair = [&](const char *p) {
        if constexpr (DT == DT_F32) {
            const float2 v = *reinterpret_cast<const float2 *>(p);
            return f2_pack(v.x, v.y);
        } else {
            const uint32_t v = *reinterpret_cast<const uint32_t *>(p);
            return DT == DT_BF16 ? f2_from_bf16x2(v) : f2_pack(f16lo_to_f32(v), f16hi_to_f32(v));
        }
    };
    f2_t s = f2_pack(0.0f, 0.0f), c = s;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float rstd = a.rstd[row];
        add_product(s, c, pair(a.dy + row * a.ld_dy + (int64_t)col * ES),
                    f2_mul(pair(a.h + row * a.ld_h + (int64_t)col * ES), f2_pack(rstd, rstd)));
    }
    float s0, s1, c0, c1;
    f2_unpack(s, s0, s1);
    f2_unpack(c, c0, c1);
    *reinterpret_cast<f2_t *>(a.part + (int64_t)blockIdx.x * a.gpr * 16 + col) =
        f2_pack(sum_of(s0, c0), sum_of(s1, c1));
}

// dw: n <= BACK_BLOCKS partial rows, added in binary64 and rounded once.  A block
// takes 32 columns; warp v adds rows v, v + 32, ..., all loaded before they are
// added, then one warp adds the warps' sums.  Few rows take little of its code: a
// straight line of 41 additions cost a single row 1 us.
__global__ void __launch_bounds__(1024)
rms_norm_dw_sum_kernel(const float *part, int n, int cols, float *dw)
{
    pdl_enter();
    __shared__ double sums[32][33];
    constexpr int PER = (BACK_BLOCKS + 31) / 32;
    const int lane = threadIdx.x & 31, v = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    const float *p = part + (int64_t)v * cols + col;
    const bool in = col < cols;
    double s = in && v < n ? (double)ld_after_wait(p) : 0.0;
    if (n > 32) {
        float x[PER - 1];
#pragma unroll
        for (int i = 0; i < PER - 1; ++i)
            x[i] = in && v + 32 * (i + 1) < n ? ld_after_wait(p + (int64_t)(i + 1) * 32 * cols) : 0.0f;
#pragma unroll
        for (int i = 0; i < PER - 1; ++i) s = __dadd_rn(s, (double)x[i]);
    }
    sums[v][lane] = s;
    __syncthreads();
    if (v == 0 && in) {
        const int m = (min(n, 32) + 3) & ~3;
        double y[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 1
        for (int i = 0; i < m; i += 4)
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = __dadd_rn(y[k], sums[i + k][lane]);
        dw[col] = (float)__dadd_rn(__dadd_rn(y[0], y[1]), __dadd_rn(y[2], y[3]));
    }
}

// ------------------------------------------------------------ host side ----

bool misaligned(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

constexpr int64_t MAX_NORM_COLS = 1 << 22;

int check_weight(const void *w, int w_dtype, int x_dtype)
{
    if (w_dtype != x_dtype && w_dtype != IF4_F32) return IF4_ERR_DTYPE;
    return misaligned(w, 16) ? IF4_ERR_ALIGN : IF4_OK;
}

// f(std::integral_constant<DT>, std::integral_constant<WT>) for a pair of types
template <typename F>
int by_types(int x_dtype, int w_dtype, F f)
{
    using F32 = std::integral_constant<int, DT_F32>;
    using BF = std::integral_constant<int, DT_BF16>;
    using HF = std::integral_constant<int, DT_F16>;
    if (x_dtype == IF4_F32) return f(F32{}, F32{});
    if (x_dtype == IF4_BF16) return w_dtype == IF4_F32 ? f(BF{}, F32{}) : f(BF{}, BF{});
    return w_dtype == IF4_F32 ? f(HF{}, F32{}) : f(HF{}, HF{});
}

template <int MODE>
int rms_norm_quantize_entry(const void *x, int64_t ld_x, const void *res, int64_t ld_res,
                            const void *w, int w_dtype, int x_dtype, int64_t rows, int64_t cols,
                            float eps, void *h, int64_t ld_h, float *rstd, uint8_t *codes,
                            uint8_t *scales, const float *ts, float *amax, int *err_flag,
                            void *stream)
{
    Shape s, sr, sh;
    int rc = check_tensor(x, x_dtype, rows, cols, ld_x, s);
    if (rc != IF4_OK) return rc;
    if (res && (rc = check_tensor(res, x_dtype, rows, cols, ld_res, sr)) != IF4_OK) return rc;
    if (h && (rc = check_tensor(h, x_dtype, rows, cols, ld_h, sh)) != IF4_OK) return rc;
    if (cols > MAX_NORM_COLS) return IF4_ERR_SHAPE;
    if ((rc = check_weight(w, w_dtype, x_dtype)) != IF4_OK) return rc;
    if (!(eps > 0.0f && eps <= 3.402823466e38f)) return IF4_ERR_MODE;
    if (!ts || (s.ngroups > 0 && (!w || !codes || !scales))) return IF4_ERR_NULL;
    if (misaligned(codes, 16) || misaligned(ts, 4) || misaligned(rstd, 4) || misaligned(amax, 4) ||
        misaligned(err_flag, 4))
        return IF4_ERR_ALIGN;
    DeviceInfo d;
    rc = check_device(d);
    if (rc != IF4_OK) return rc;
    if (s.ngroups == 0) return IF4_OK;
    const NormArgs a{static_cast<const char *>(x), static_cast<const char *>(res),
                     static_cast<const char *>(w), static_cast<char *>(h), s.ld_bytes, sr.ld_bytes,
                     sh.ld_bytes, codes, scales, ts, rstd, reinterpret_cast<unsigned int *>(amax),
                     err_flag, rows, (int)(cols / 16),
                     s.v8 && (!res || sr.v8) && (!h || sh.v8), 1.0 / (double)cols, (double)eps};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t n = cols / 16;
    return by_types(x_dtype, w_dtype, [&](auto dt, auto wt) {
        constexpr int DT = decltype(dt)::value, WT = decltype(wt)::value;
        const int64_t warps = (n + 31) / 32;
        auto rows_kernel = [&](auto k, int g, unsigned per_sm) {
            // the fewest whole warps that hold a row; blocks for one wave
            const unsigned threads = (unsigned)((warps + g - 1) / g * 32);
            const int64_t wave = (int64_t)d.sm_count * std::min<unsigned>(per_sm / threads, 32);
            return launch_k(k, (unsigned)std::min(rows, wave), threads, st, a);
        };
        if constexpr (DT == DT_F32) {
            if (n <= 1024)
                return rows_kernel(rms_norm_quantize_rows_kernel<DT, WT, MODE, 1, false>, 1, 1024);
        } else {
            if (n <= 32)
                return rows_kernel(rms_norm_quantize_rows_kernel<DT, WT, MODE, 1, false>, 1, 1024);
            if (n <= 1024)
                return rows_kernel(rms_norm_quantize_rows_kernel<DT, WT, MODE, 2, true>, 2, 512);
            if (n <= 2048)
                return rows_kernel(rms_norm_quantize_rows_kernel<DT, WT, MODE, 2, false>, 2, 1024);
        }
        return launch_k(rms_norm_quantize_kernel<DT, WT, MODE>,
                        (unsigned)std::min<int64_t>(rows, (int64_t)d.sm_count * 8),
                        (unsigned)NORM_THREADS, st, a);
    });
}

}  // namespace

extern "C" {

int if4_rms_norm_quantize(const void *x, int64_t ld_x, const void *residual, int64_t ld_res,
                          const void *weight, int w_dtype, int x_dtype, int64_t rows, int64_t cols,
                          float eps, void *h, int64_t ld_h, float *rstd, uint8_t *codes,
                          uint8_t *scales, const float *ts, float *amax, int *err_flag, void *stream)
{
    return rms_norm_quantize_entry<Q_IF4>(x, ld_x, residual, ld_res, weight, w_dtype, x_dtype, rows,
                                          cols, eps, h, ld_h, rstd, codes, scales, ts, amax,
                                          err_flag, stream);
}

int nvfp4_rms_norm_quantize(const void *x, int64_t ld_x, const void *residual, int64_t ld_res,
                            const void *weight, int w_dtype, int x_dtype, int64_t rows,
                            int64_t cols, float eps, void *h, int64_t ld_h, float *rstd,
                            uint8_t *codes, uint8_t *scales, const float *ts, float *amax,
                            int *err_flag, void *stream)
{
    return rms_norm_quantize_entry<Q_NVFP4>(x, ld_x, residual, ld_res, weight, w_dtype, x_dtype,
                                            rows, cols, eps, h, ld_h, rstd, codes, scales, ts, amax,
                                            err_flag, stream);
}

size_t if4_rms_norm_backward_workspace_bytes(int64_t rows, int64_t cols)
{
    if (rows < 1 || cols < 16 || cols % 16 != 0 || cols > MAX_NORM_COLS ||
        rows > 0x7FFFFFFF / (cols / 16))
        return 0;
    return (size_t)std::min<int64_t>(rows, BACK_BLOCKS) * (size_t)cols * sizeof(float);
}

int if4_rms_norm_backward(const void *dy, int64_t ld_dy, const void *h, int64_t ld_h,
                          const void *weight, int w_dtype, const float *rstd, const void *dres,
                          int64_t ld_dres, int x_dtype, int64_t rows, int64_t cols, void *dx,
                          int64_t ld_dx, float *dweight, void *workspace, size_t ws_bytes,
                          void *stream)
{
    Shape sy, sh, sr, sx;
    int rc = check_tensor(dy, x_dtype, rows, cols, ld_dy, sy);
    if (rc == IF4_OK) rc = check_tensor(h, x_dtype, rows, cols, ld_h, sh);
    if (rc == IF4_OK) rc = check_tensor(dx, x_dtype, rows, cols, ld_dx, sx);
    if (rc == IF4_OK && dres) rc = check_tensor(dres, x_dtype, rows, cols, ld_dres, sr);
    if (rc == IF4_OK && cols > MAX_NORM_COLS) rc = IF4_ERR_SHAPE;
    if (rc == IF4_OK) rc = check_weight(weight, w_dtype, x_dtype);
    if (rc != IF4_OK) return rc;
    if (cols > 0 && !dweight) return IF4_ERR_NULL;
    if (sy.ngroups > 0 && (!weight || !rstd)) return IF4_ERR_NULL;
    if (misaligned(rstd, 4) || misaligned(dweight, 4)) return IF4_ERR_ALIGN;
    const size_t need = if4_rms_norm_backward_workspace_bytes(rows, cols);
    if (need && (!workspace || ws_bytes < need)) return IF4_ERR_WORKSPACE;
    if (need && misaligned(workspace, 256)) return IF4_ERR_ALIGN;
    DeviceInfo d;
    rc = check_device(d);
    if (rc != IF4_OK) return rc;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (sy.ngroups == 0) {                // no rows: dweight is an empty sum
        return cols > 0 ? launched(cudaMemsetAsync(dweight, 0, (size_t)cols * 4, st)) : IF4_OK;
    }
    const BackArgs a{static_cast<const char *>(dy), static_cast<const char *>(h),
                     static_cast<const char *>(weight), static_cast<const char *>(dres),
                     static_cast<char *>(dx), sy.ld_bytes, sh.ld_bytes, sr.ld_bytes, sx.ld_bytes,
                     rstd, static_cast<float *>(workspace), rows, (int)(cols / 16),
                     sy.v8 && sh.v8 && sx.v8 && (!dres || sr.v8), 1.0f / (float)cols};
    const int64_t n = cols / 16;
    auto sum_dw = [&](int parts) {
        return launch_k(rms_norm_dw_sum_kernel, (unsigned)((cols + 31) / 32), 1024u, st,
                        (const float *)workspace, parts, (int)cols, dweight);
    };
    return by_types(x_dtype, w_dtype, [&](auto dt, auto wt) {
        constexpr int DT = decltype(dt)::value, WT = decltype(wt)::value;
        if (n <= (DT == DT_F32 ? 512 : 1024)) {
            // the fewest threads per row (a power of two) that hold it, two units
            // each up to 8192 columns, four above
            const int64_t units = 2 * n;
            const int per = units <= 1024 ? 2 : 4;
            int T = 32;
            while (T * per < units) T *= 2;
            const int slots = BACK_THREADS / T;
            const int parts = (int)std::min<int64_t>((rows + slots - 1) / slots, BACK_BLOCKS / 2);
            auto rows_kernel = [&](auto V) {
                constexpr int U = decltype(V)::value;
                auto kernel = rms_norm_backward_rows_kernel<DT, WT, U>;
                static OncePerDevice done;
                constexpr int SMEM = BACK_THREADS * BackRing<DT, U>::BYTES;
                const int ok = allow_smem(kernel, SMEM, d, done);
                if (ok != IF4_OK) return ok;
                cudaLaunchConfig_t cfg = {};
                cfg.gridDim = dim3((unsigned)parts, 1, 1);
                cfg.blockDim = dim3(BACK_THREADS, 1, 1);
                cfg.dynamicSmemBytes = SMEM;
                cfg.stream = st;
                cudaLaunchAttribute attr[1];
                attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
                attr[0].val.programmaticStreamSerializationAllowed = 1;
                cfg.attrs = attr;
                cfg.numAttrs = 1;
                return launched(cudaLaunchKernelEx(&cfg, kernel, a, T));
            };
            int r;
            if constexpr (DT == DT_F32)
                r = rows_kernel(std::integral_constant<int, 2>{});
            else
                r = per == 2 ? rows_kernel(std::integral_constant<int, 2>{})
                             : rows_kernel(std::integral_constant<int, 4>{});
            if (r != IF4_OK) return r;
            return sum_dw(parts);
        }
        const int parts = (int)std::min<int64_t>(rows, BACK_BLOCKS);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)parts, (unsigned)((cols + 511) / 512), 1);
        cfg.blockDim = dim3(256, 1, 1);
        cfg.stream = st;
        int r = launched(cudaLaunchKernelEx(&cfg, rms_norm_dw_kernel<DT>, a));
        if (r != IF4_OK) return r;
        r = sum_dw(parts);
        if (r != IF4_OK) return r;
        return launch_k(rms_norm_dx_kernel<DT, WT>,
                        (unsigned)std::min<int64_t>(rows, (int64_t)d.sm_count * 8),
                        (unsigned)NORM_THREADS, st, a);
    });
}

}  // extern "C"
