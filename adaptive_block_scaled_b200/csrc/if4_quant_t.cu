// Quantizers along the rows (sm_100a): groups of 16 consecutive rows of one
// column of x [R, C], i.e. the quantization of x^T along its last axis, as
// codes [C, R / 2] and scales [C, R / 16]; optionally also the quantization
// of x along its own last axis, from the same read.
//
// Why: a linear's gradients contract over the axes its forward pass does not
// group.  With Y = X W^T (X [M, K], W [N, K], both grouped along K),
//   dX = dY W     contracts over N: dY grouped along N, W^T along N,
//   dW = dY^T X   contracts over M: dY^T and X^T grouped along M,
// so each of X, W and dY is needed both ways.
//
// A block takes a tile of 128 x 128 (64 x 64 for small tensors) into shared
// memory with asynchronous 16-byte copies, which hold no registers while they
// are under way.  Row form: a thread reads whole row groups (16 values, 32 or
// 64 bytes) and encodes them.  Column form: a thread reads 16 rows of two
// neighbouring columns (one conflict-free word per row), which are two whole
// column groups in registers, and encodes them with the same group encoder.
// The column codes are put back in order through shared memory, so that a
// tile's code bytes of a column leave as one run.
//
// With both forms the encoder's instructions bound it: 511 per 16 values in IF4
// (two encodes and all around them), 281 in NVFP4.  8192 x 8192 bf16 with the tensor
// scale given takes 74 and 46 to 47 us, four blocks per SM issuing in 81 and 78 % of
// the cycles.  Holding the tile's loads in registers instead allowed two: IF4 83 us.

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/if4.h"
#include "if4_device.cuh"
#include "if4_encode.cuh"
#include "if4_host.cuh"
#include "if4_load.cuh"

namespace {

constexpr int THREADS_T = 256;

// A block's tile of T x T.
template <int DT, int T>
struct Tile {
    static constexpr int PITCH = T * (DT == DT_F32 ? 4 : 2);     // bytes of a row
    static constexpr int GROUPS = T / 16;                        // along one side
    static constexpr int CODE_PITCH = T / 2 + 8;                 // staged code bytes per column
    static constexpr int CODE_OFF = T * PITCH;
    static constexpr int SCALE_OFF = CODE_OFF + T * CODE_PITCH;
    static constexpr int SMEM = SCALE_OFF + T * GROUPS;
};

// Tensor scale, first step: block i's max |x| as float bits to parts[i] (NaN and
// Inf compare above every finite value).  A float per block needs no zeroed
// word and no atomics; the parts lie in the column codes' own memory, which the
// quantizer writes only after the second step has read them.
template <int DT>
__global__ void __launch_bounds__(256)
amax_parts_kernel(const char *x, int64_t ld_bytes, uint32_t gpr, uint32_t ngroups, bool v8,
                  uint32_t *parts)
{
    pdl_enter();
    constexpr int U = DT == DT_F32 ? 4 : 8;       // loads in flight
    const uint32_t stride = gridDim.x * blockDim.x;
    uint32_t m = 0;
    for (uint64_t g0 = blockIdx.x * blockDim.x + threadIdx.x; g0 < ngroups;
         g0 += (uint64_t)U * stride) {
        Raw<DT> r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint64_t g = g0 + (uint64_t)u * stride;
            if (g < ngroups) {
                const uint32_t row = (uint32_t)g / gpr;
                load_group_rw<DT>(x + (int64_t)row * ld_bytes +
                                      (int64_t)((uint32_t)g - row * gpr) * 16 * elem_bytes<DT>(),
                                  r[u], v8);
            } else {
#pragma unroll
                for (uint32_t &w : r[u].w) w = 0u;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            f2_t xv[8];
            bool bad;
            m = max(m, __float_as_uint(unpack_group<DT>(r[u], xv, bad)));
        }
    }
    __shared__ uint32_t warp_max[8];
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 1; i < 8; ++i) m = max(m, warp_max[i]);
        parts[blockIdx.x] = m;
    }
}

// Second step: ts of n parts, by one block.
__global__ void __launch_bounds__(256)
scale_parts_kernel(const uint32_t *parts, int n, float *ts)
{
    pdl_enter();
    __shared__ uint32_t warp_max[8];
    uint32_t m = 0;
    for (int i = threadIdx.x; i < n; i += 256) {
        uint32_t v;
        asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(parts + i) : "memory");
        m = max(m, v);
    }
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 1; i < 8; ++i) m = max(m, warp_max[i]);
        *ts = tensor_scale_of(__uint_as_float(m));
    }
}

// Byte offset of 16-byte piece k of a tile row.  The pieces are permuted inside
// each 128 bytes so that the eight lanes that read the same piece of eight
// neighbouring row groups hit different banks; a whole row read by columns is
// a permutation of the same banks.
template <int DT>
__device__ __forceinline__ int piece_at(int k)
{
    return 16 * (DT == DT_F32 ? k ^ ((k >> 3) & 3) : k ^ ((k >> 3) & 1));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool in)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 :: "r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}

template <int DT, int MODE, bool ROWS, int T>
__global__ void __launch_bounds__(THREADS_T, DT == DT_F32 ? 2 : 4)
quantize_t_kernel(const char *__restrict__ x, int64_t ld_bytes, int64_t rows, int64_t cols,
                  uint8_t *__restrict__ codes, uint8_t *__restrict__ scales,
                  uint8_t *__restrict__ codes_t, uint8_t *__restrict__ scales_t,
                  const float *__restrict__ ts_ptr, int *err, int check_ts)
{
    pdl_enter();
    constexpr int ES = elem_bytes<DT>();
    using L = Tile<DT, T>;
    constexpr int TILE = T, TG = L::GROUPS, CODE_PITCH = L::CODE_PITCH, PITCH = L::PITCH;
    constexpr int PIECES = PITCH / 16;      // 16-byte pieces of a tile row
    constexpr int GP = ES;                  // pieces of a group: 2 or 4
    extern __shared__ __align__(16) uint8_t smem_t[];
    uint8_t *tile = smem_t;
    uint8_t *code_out = smem_t + L::CODE_OFF;
    uint8_t *scale_out = smem_t + L::SCALE_OFF;
    __shared__ float inv_tab[128];

    const int64_t col_tiles = (cols + TILE - 1) / TILE;
    const int64_t r0 = (int64_t)(blockIdx.x / (uint32_t)col_tiles) * TILE;
    const int64_t c0 = (int64_t)(blockIdx.x % (uint32_t)col_tiles) * TILE;
    const int tile_rows = (int)min((int64_t)TILE, rows - r0);
    const int tile_cols = (int)min((int64_t)TILE, cols - c0);
    {
        const uint32_t dst = (uint32_t)__cvta_generic_to_shared(tile);
        const char *src = x + r0 * ld_bytes + c0 * ES;
        const int k = threadIdx.x % PIECES;
#pragma unroll
        for (int i = 0; i < TILE * PIECES / THREADS_T; ++i) {
            const int r = threadIdx.x / PIECES + i * (THREADS_T / PIECES);
            // past the tensor: zero fill, the address stays inside it
            const bool in = r < tile_rows && k * 16 < tile_cols * ES;
            cp_async16(dst + r * PITCH + piece_at<DT>(k),
                       in ? src + (int64_t)r * ld_bytes + k * 16 : x, in);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    const float ts = ld_after_wait(ts_ptr);
    const float rts = __frcp_rn(ts);
    if (check_ts && blockIdx.x == 0 && threadIdx.x == 0 && !ts_valid(ts) && err)
        atomicOr(err, IF4_DEV_BAD_SCALE);
    fill_inv_tab(inv_tab, ts);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();

    if constexpr (ROWS) {
        // a thread takes one group of every (256 / groups)-th row
        const int lg = threadIdx.x & (TG - 1);
#pragma unroll 1
        for (int row = threadIdx.x / TG; row < tile_rows; row += THREADS_T / TG) {
            if (16 * lg >= tile_cols) break;
            Raw<DT> raw;
#pragma unroll
            for (int q = 0; q < GP; ++q) {
                const uint4 v = *reinterpret_cast<const uint4 *>(tile + row * PITCH +
                                                                 piece_at<DT>(lg * GP + q));
                raw.w[4 * q] = v.x;
                raw.w[4 * q + 1] = v.y;
                raw.w[4 * q + 2] = v.z;
                raw.w[4 * q + 3] = v.w;
            }
            f2_t xv[8];
            bool bad;                       // the column form reports it
            const float amax = unpack_group<DT>(raw, xv, bad);
            const GroupCode g = encode_registers<MODE>(xv, amax, ts, rts, inv_tab);
            const int64_t gi = (r0 + row) * (cols / 16) + c0 / 16 + lg;
            st_v2(codes + gi * 8, g.c0, g.c1);
            st_u8(scales + gi, g.scale);
        }
    }

    // column groups: warp w takes row group w, a lane two neighbouring
    // columns of each 64 (a tile of 64 x 64 leaves half the warps idle here)
    bool nonfinite = false;
    const int rg = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (16 * rg < tile_rows) {
#pragma unroll 1
        for (int col = 2 * lane; col < tile_cols; col += 64) {
            const uint8_t *p = tile + rg * 16 * PITCH + piece_at<DT>(col * ES / 16) + col * ES % 16;
            // 16 rows of the two columns, as pairs of rows, and their max |x|
            f2_t xa[8], xb[8];
            float amax_a, amax_b;
            if constexpr (DT == DT_F32) {
                float ma = 0.0f, mb = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 u = *reinterpret_cast<const float2 *>(p + 2 * i * PITCH);
                    const float2 v = *reinterpret_cast<const float2 *>(p + (2 * i + 1) * PITCH);
                    ma = absmax3_f32(ma, u.x, v.x);
                    mb = absmax3_f32(mb, u.y, v.y);
                    xa[i] = f2_pack(u.x, v.x);
                    xb[i] = f2_pack(u.y, v.y);
                }
                amax_a = ma;
                amax_b = mb;
            } else {
                uint32_t m = 0;            // column a in the low half, b in the high
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t u = *reinterpret_cast<const uint32_t *>(p + 2 * i * PITCH);
                    const uint32_t v = *reinterpret_cast<const uint32_t *>(p + (2 * i + 1) * PITCH);
                    if constexpr (DT == DT_BF16) {
                        m = absmax_bf16x2(absmax_bf16x2(m, u), v);
                        xa[i] = f2_pack(__uint_as_float(u << 16), __uint_as_float(v << 16));
                        xb[i] = f2_pack(__uint_as_float(u & 0xFFFF0000u),
                                        __uint_as_float(v & 0xFFFF0000u));
                    } else {
                        m = absmax_f16x2(absmax_f16x2(m, u), v);
                        xa[i] = f2_pack(f16lo_to_f32(u), f16lo_to_f32(v));
                        xb[i] = f2_pack(f16hi_to_f32(u), f16hi_to_f32(v));
                    }
                }
                m &= 0x7FFF7FFFu;          // the sign bits the maxima leave
                amax_a = DT == DT_BF16 ? __uint_as_float(m << 16) : f16lo_to_f32(m);
                amax_b = DT == DT_BF16 ? __uint_as_float(m & 0xFFFF0000u) : f16hi_to_f32(m);
            }
            // Inf or NaN in a column
            nonfinite |= !(amax_a <= 3.402823466e38f) || !(amax_b <= 3.402823466e38f);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const GroupCode g = encode_registers<MODE>(k ? xb : xa, k ? amax_b : amax_a, ts, rts,
                                                           inv_tab);
                *reinterpret_cast<uint2 *>(code_out + (col + k) * CODE_PITCH + rg * 8) =
                    make_uint2(g.c0, g.c1);
                scale_out[(col + k) * TG + rg] = (uint8_t)g.scale;
            }
        }
    }
    __syncthreads();
    const int row_groups = tile_rows / 16;
#pragma unroll
    for (int i = 0; i < TILE * TG / THREADS_T; ++i) {
        const int k = threadIdx.x + i * THREADS_T;
        const int col = k / TG, g = k & (TG - 1);
        if (col < tile_cols && g < row_groups) {
            const uint2 w = *reinterpret_cast<const uint2 *>(code_out + col * CODE_PITCH + g * 8);
            const int64_t gi = (c0 + col) * (rows / 16) + r0 / 16 + g;
            st_v2(codes_t + gi * 8, w.x, w.y);
            st_u8(scales_t + gi, scale_out[col * TG + g]);
        }
    }
    if (nonfinite && err) atomicOr(err, IF4_DEV_NONFINITE);
}

// ------------------------------------------------------------ host side ----

struct OutT {
    uint8_t *codes, *scales, *codes_t, *scales_t;
};

template <int DT, int MODE, bool ROWS, int T>
int launch_quantize_t(const Shape &s, const void *x, int64_t rows, int64_t cols, const OutT &o,
                      const float *ts, int *err, int check_ts, cudaStream_t st, const DeviceInfo &d)
{
    auto kernel = quantize_t_kernel<DT, MODE, ROWS, T>;
    constexpr int SMEM = Tile<DT, T>::SMEM;
    static OncePerDevice done;
    const int rc = allow_smem(kernel, SMEM, d, done);
    if (rc != IF4_OK) return rc;
    const int64_t tiles = ((rows + T - 1) / T) * ((cols + T - 1) / T);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)tiles, 1, 1);
    cfg.blockDim = dim3(THREADS_T, 1, 1);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launched(cudaLaunchKernelEx(&cfg, kernel, static_cast<const char *>(x), s.ld_bytes, rows,
                                       cols, o.codes, o.scales, o.codes_t, o.scales_t, ts, err,
                                       check_ts));
}

template <int DT, int MODE>
int dispatch_quantize_t(const Shape &s, const void *x, int64_t rows, int64_t cols, const OutT &o,
                        const float *ts, int *err, int check_ts, cudaStream_t st,
                        const DeviceInfo &d)
{
    // Small tiles while large ones make less than two blocks per SM (IF4 both
    // ways, bf16, us with tiles of 64 / 128: 1024 x 1024 4.4 / 5.7, 2048 x 2048 7.7 / 10.0,
    // 4096 x 2048 13.5 / 12.7, 4096 x 4096 27.0 / 22.1).
    const int64_t large = ((rows + 127) / 128) * ((cols + 127) / 128);
    auto run = [&](auto t) {
        constexpr int T = decltype(t)::value;
        return o.codes
            ? launch_quantize_t<DT, MODE, true, T>(s, x, rows, cols, o, ts, err, check_ts, st, d)
            : launch_quantize_t<DT, MODE, false, T>(s, x, rows, cols, o, ts, err, check_ts, st, d);
    };
    return large <= 2 * d.sm_count ? run(std::integral_constant<int, 64>{})
                                   : run(std::integral_constant<int, 128>{});
}

// ts of x, with `parts` (the column codes: 8 bytes per group) as scratch.
int launch_scale(int x_dtype, const Shape &s, const void *x, uint32_t *parts,
                 float *ts, cudaStream_t st, const DeviceInfo &d)
{
    // a block per 256 threads' first groups, up to four blocks per SM; never
    // more than there are groups
    const uint32_t want = (s.ngroups + 255) / 256, most = (uint32_t)d.sm_count * 4;
    const uint32_t grid = want < most ? want : most;
    auto amax = [&](auto k) {
        return launch_k(k, grid, 256u, st, static_cast<const char *>(x), s.ld_bytes, s.gpr,
                        s.ngroups, s.v8, parts);
    };
    int rc;
    if (x_dtype == IF4_F32)
        rc = amax(amax_parts_kernel<DT_F32>);
    else if (x_dtype == IF4_BF16)
        rc = amax(amax_parts_kernel<DT_BF16>);
    else
        rc = amax(amax_parts_kernel<DT_F16>);
    if (rc != IF4_OK) return rc;
    return launch_k(scale_parts_kernel, 1u, 256u, st, (const uint32_t *)parts, (int)grid, ts);
}

template <int MODE>
int quantize_t_entry(const void *x, int x_dtype, int64_t rows, int64_t cols, int64_t ld_x,
                     const OutT &o, float *ts, int ts_mode, int *err_flag, void *stream)
{
    Shape s;
    int rc = check_tensor(x, x_dtype, rows, cols, ld_x, s);
    if (rc != IF4_OK) return rc;
    if (rows % 16 != 0) return IF4_ERR_SHAPE;
    if (ts_mode != IF4_TS_COMPUTE && ts_mode != IF4_TS_GIVEN) return IF4_ERR_MODE;
    if (!ts || !o.codes != !o.scales) return IF4_ERR_NULL;
    if (s.ngroups > 0 && (!o.codes_t || !o.scales_t)) return IF4_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(o.codes) % 16 || reinterpret_cast<uintptr_t>(o.codes_t) % 16 ||
        reinterpret_cast<uintptr_t>(ts) % 4 || reinterpret_cast<uintptr_t>(err_flag) % 4)
        return IF4_ERR_ALIGN;
    DeviceInfo d;
    rc = check_device(d);
    if (rc != IF4_OK) return rc;
    if (s.ngroups == 0)                // ts of an empty tensor is 1
        return ts_mode == IF4_TS_COMPUTE
                   ? if4_tensor_amax(x, x_dtype, rows, cols, ld_x, ts, err_flag, stream) == IF4_OK
                         ? if4_tensor_scale(ts, ts, stream)
                         : (int)IF4_ERR_CUDA
                   : (int)IF4_OK;
    const int check_ts = ts_mode == IF4_TS_GIVEN ? 1 : 0;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (ts_mode == IF4_TS_COMPUTE) {
        rc = launch_scale(x_dtype, s, x, reinterpret_cast<uint32_t *>(o.codes_t), ts, st, d);
        if (rc != IF4_OK) return rc;
    }
    switch (x_dtype) {
    case IF4_F32:
        return dispatch_quantize_t<DT_F32, MODE>(s, x, rows, cols, o, ts, err_flag, check_ts, st, d);
    case IF4_BF16:
        return dispatch_quantize_t<DT_BF16, MODE>(s, x, rows, cols, o, ts, err_flag, check_ts, st, d);
    default:
        return dispatch_quantize_t<DT_F16, MODE>(s, x, rows, cols, o, ts, err_flag, check_ts, st, d);
    }
}

}  // namespace

extern "C" {

int if4_quantize_t(const void *x, int x_dtype, int64_t rows, int64_t cols, int64_t ld_x,
                   uint8_t *codes, uint8_t *scales, uint8_t *codes_t, uint8_t *scales_t, float *ts,
                   int ts_mode, int *err_flag, void *stream)
{
    return quantize_t_entry<Q_IF4>(x, x_dtype, rows, cols, ld_x, {codes, scales, codes_t, scales_t},
                                   ts, ts_mode, err_flag, stream);
}

int nvfp4_quantize_t(const void *x, int x_dtype, int64_t rows, int64_t cols, int64_t ld_x,
                     uint8_t *codes, uint8_t *scales, uint8_t *codes_t, uint8_t *scales_t,
                     float *ts, int ts_mode, int *err_flag, void *stream)
{
    return quantize_t_entry<Q_NVFP4>(x, x_dtype, rows, cols, ld_x,
                                     {codes, scales, codes_t, scales_t}, ts, ts_mode, err_flag,
                                     stream);
}

}  // extern "C"
