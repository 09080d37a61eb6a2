// The 16 scale bytes of a row and 256 of K, as four words: which loads bring
// them in.  Plain C++ over a loader, so that a host program can check every
// address.
#pragma once

#include <cstdint>

namespace {

// The 16 scale bytes at p, of which the first nb exist (nb <= 0: none); the
// others read as 0, and no load touches a byte outside the first nb.  VEC: the
// bytes that p's and nb's alignment allows per load: 16 (K % 256 == 0, aligned
// base), 4 (K % 64 == 0, aligned base) or 2.
template <int VEC, typename Load>
__device__ __forceinline__ void load_scales16(const uint8_t *p, int nb, uint32_t (&w)[4], Load ld)
{
    w[0] = w[1] = w[2] = w[3] = 0u;
    if constexpr (VEC == 16) {
        if (nb > 0) ld.v4(p, w[0], w[1], w[2], w[3]);
    } else if constexpr (VEC == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (nb > 4 * j) w[j] = ld.u32(p + 4 * j);
    } else if (nb >= 16) {
        // rows on 4-byte and on 2-byte boundaries in turn: the whole aligned
        // words, and in rows on 2-byte boundaries both ends by themselves,
        // shifted together
        const uint32_t off = (uint32_t)reinterpret_cast<uintptr_t>(p) & 2u;
        uint32_t a[4], prev = off ? ld.u16(p) << 16 : 0u;
#pragma unroll
        for (int j = 0; j < 3; ++j) a[j] = ld.u32(p + off + 4 * j);
        a[3] = off ? ld.u16(p + 14) : ld.u32(p + 12);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[j] = off ? prev >> 16 | a[j] << 16 : a[j];
            prev = a[j];
        }
    } else {
        uint32_t h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = nb > 2 * j ? ld.u16(p + 2 * j) : 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = h[2 * j] | h[2 * j + 1] << 16;
    }
}

}  // namespace
