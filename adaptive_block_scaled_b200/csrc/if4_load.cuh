// Raw loads of groups of 16 values and their unpacking to binary32 pairs with
// the group's max |x|, shared by the quantizer kernels.
#pragma once

#include <cstdint>

#include "if4_device.cuh"
#include "if4_encode.cuh"

namespace {

using namespace if4dev;

// Raw bits of one group: 16-bit types fill w[0..7], f32 fills w[0..15].
template <int DT>
struct Raw {
    uint32_t w[DT == DT_F32 ? 16 : 8];
};

template <int DT, bool V8>
__device__ __forceinline__ void load_group(const char *p, Raw<DT> &r)
{
    if constexpr (DT == DT_F32) {
        if constexpr (V8) {
            uint32_t a[8], b[8];
            ld_v8(p, a);
            ld_v8(p + 32, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) { r.w[i] = a[i]; r.w[8 + i] = b[i]; }
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                ld_v4(p + 16 * q, r.w[4 * q], r.w[4 * q + 1], r.w[4 * q + 2], r.w[4 * q + 3]);
        }
    } else {
        if constexpr (V8) {
            ld_v8(p, r.w);
        } else {
            ld_v4(p, r.w[0], r.w[1], r.w[2], r.w[3]);
            ld_v4(p + 16, r.w[4], r.w[5], r.w[6], r.w[7]);
        }
    }
}

// The same with the width chosen at run time, also for values that this kernel
// overwrites itself.  v8: 32-byte aligned, 256 bits at once.
template <int DT>
__device__ __forceinline__ void load_group_rw(const char *p, Raw<DT> &r, bool v8)
{
    if (v8) {
#pragma unroll
        for (int q = 0; q < (DT == DT_F32 ? 2 : 1); ++q)
            asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                         : "=r"(r.w[8 * q]), "=r"(r.w[8 * q + 1]), "=r"(r.w[8 * q + 2]),
                           "=r"(r.w[8 * q + 3]), "=r"(r.w[8 * q + 4]), "=r"(r.w[8 * q + 5]),
                           "=r"(r.w[8 * q + 6]), "=r"(r.w[8 * q + 7])
                         : "l"(p + 32 * q));
    } else {
#pragma unroll
        for (int q = 0; q < (DT == DT_F32 ? 4 : 2); ++q)
            asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(r.w[4 * q]), "=r"(r.w[4 * q + 1]), "=r"(r.w[4 * q + 2]),
                           "=r"(r.w[4 * q + 3])
                         : "l"(p + 16 * q));
    }
}

// Unpack to 8 float pairs (element 2j low, 2j+1 high) and the group's max |x|
// as float bits; *nonfinite is set for Inf/NaN.
template <int DT>
__device__ __forceinline__ float unpack_group(const Raw<DT> &r, f2_t (&x)[8], bool &nonfinite)
{
    if constexpr (DT == DT_F32) {
        // max |x| in two chains of one instruction per element (NaN
        // propagates; the sign bit it leaves is masked off)
        uint32_t m0 = 0, m1 = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t a = r.w[2 * j], b = r.w[2 * j + 1];
            m0 = absmax_f32(m0, __uint_as_float(a));
            m1 = absmax_f32(m1, __uint_as_float(b));
            x[j] = f2_pack(__uint_as_float(a), __uint_as_float(b));
        }
        const uint32_t m = absmax_f32(m0, __uint_as_float(m1)) & 0x7FFFFFFFu;
        nonfinite = m >= 0x7F800000u;
        return __uint_as_float(m);
    } else {
        // max(|a|, |b|) per 16-bit lane in one instruction (the sign bit it
        // leaves is ignored); NaN propagates, so Inf/NaN show up in the max
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t w = r.w[j];
            m = (DT == DT_BF16) ? absmax_bf16x2(m, w) : absmax_f16x2(m, w);
            if constexpr (DT == DT_BF16)
                x[j] = f2_from_bf16x2(w);
            else
                x[j] = f2_pack(f16lo_to_f32(w), f16hi_to_f32(w));
        }
        const uint32_t m16 = max(m & 0x7FFFu, (m >> 16) & 0x7FFFu);
        if constexpr (DT == DT_BF16) {
            nonfinite = m16 >= 0x7F80u;
            return __uint_as_float(m16 << 16);
        } else {
            nonfinite = m16 >= 0x7C00u;
            return f16lo_to_f32(m16);
        }
    }
}

__device__ __forceinline__ bool ts_valid(float ts)
{
    return ts >= kTsFloor && ts <= kTsCeil;   // false for NaN
}

template <int DT>
__host__ __device__ constexpr int elem_bytes() { return DT == DT_F32 ? 4 : 2; }

// IF4 (lower-error candidate) or NVFP4 codes of one group held in registers:
// its 8 pairs x and max |x|, under the tensor scale ts.  rts = fl(1 / ts),
// inv_tab[c] = fl(1 / fl(E4M3(c) * ts)), inv_tab[0] = 0.  The results are
// those of if4_quantize and nvfp4_quantize.
template <int MODE>
__device__ __forceinline__ GroupCode encode_registers(const f2_t (&x)[8], float amax, float ts,
                                                      float rts, const float *inv_tab)
{
    if constexpr (MODE == Q_IF4) {
        const If4Fast f = if4_fast(x, amax, ts, rts, inv_tab);
        return if4_finish(f, amax, ts, rts, inv_tab, [&](float (&y)[16]) {
#pragma unroll
            for (int j = 0; j < 8; ++j) f2_unpack(x[j], y[2 * j], y[2 * j + 1]);
        });
    } else {
        const uint32_t sb = e4m3_from_f32(block_scale(amax, ts, rts)) & 0x7Fu;
        GroupCode out = encode_group<Q_NVFP4, false>(x, sb, inv_tab[sb], nullptr);
        if (sb == 0) out.c0 = out.c1 = out.scale = 0u;
        return out;
    }
}

// ts = amax / 2688, 1 for amax == 0, floored at 2^-117 (NaN stays NaN).
__device__ __forceinline__ float tensor_scale_of(float a)
{
    float t = 1.0f;
    if (a != 0.0f) {
        t = __fdiv_rn(a, 2688.0f);
        if (t < kTsFloor) t = kTsFloor;
    }
    return t;
}

// inv_tab of encode_registers, by threads 0..127 of a block (no barrier).
__device__ __forceinline__ void fill_inv_tab(float *inv_tab, float ts)
{
    if (threadIdx.x < 128)
        inv_tab[threadIdx.x] =
            threadIdx.x == 0 ? 0.0f : __frcp_rn(__fmul_rn(f32_from_e4m3(threadIdx.x), ts));
}

}  // namespace
