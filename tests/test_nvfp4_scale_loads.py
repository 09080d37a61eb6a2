"""The loads of a row's scale bytes (nvfp4_scales.cuh), compiled for the host:
every address inside the bytes that exist, aligned to its load, and the four
words those bytes."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "adaptive_block_scaled_b200", "csrc")

PROGRAM = r"""
#define __device__
#define __forceinline__ inline
#include "nvfp4_scales.cuh"
#include <cstdio>
#include <cstring>

alignas(64) static uint8_t mem[128];
static const uint8_t *lo, *hi;         // the bytes that exist
static int faults = 0;

struct Checked {
    void touch(const uint8_t *p, int n) const
    {
        if (p < lo || p + n > hi || reinterpret_cast<uintptr_t>(p) % n) ++faults;
    }
    uint32_t u16(const uint8_t *p) const { touch(p, 2); uint16_t v; memcpy(&v, p, 2); return v; }
    uint32_t u32(const uint8_t *p) const { touch(p, 4); uint32_t v; memcpy(&v, p, 4); return v; }
    void v4(const uint8_t *p, uint32_t &a, uint32_t &b, uint32_t &c, uint32_t &d) const
    {
        touch(p, 16);
        memcpy(&a, p, 4); memcpy(&b, p + 4, 4); memcpy(&c, p + 8, 4); memcpy(&d, p + 12, 4);
    }
};

template <int VEC> static int check()
{
    int bad = 0;
    for (int start = 32; start < 64; start += VEC)
        for (int nb = -VEC; nb <= 32; nb += VEC) {
            const uint8_t *p = mem + start;
            const int n = nb < 0 ? 0 : nb > 16 ? 16 : nb;
            lo = p, hi = p + n, faults = 0;
            uint32_t w[4];
            load_scales16<VEC>(p, nb, w, Checked());
            uint8_t want[16] = {}, got[16];
            memcpy(want, p, n);
            memcpy(got, w, 16);
            if (faults || memcmp(want, got, 16)) {
                printf("VEC %d start %d bytes %d: %d accesses out of place\n", VEC, start, nb, faults);
                ++bad;
            }
        }
    return bad;
}

int main()
{
    for (int i = 0; i < 128; ++i) mem[i] = (uint8_t)(i * 37 + 11);
    return check<2>() + check<4>() + check<16>() != 0;
}
"""


def test_every_load_stays_inside_the_row(tmp_path):
    src, exe = tmp_path / "loads.cc", tmp_path / "loads"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wno-unknown-pragmas", f"-I{CSRC}", str(src),
                    "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout
