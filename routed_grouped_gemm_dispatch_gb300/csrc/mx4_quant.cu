// Conversion to and from 4-bit microscaled values.
//
// A block is 32 consecutive values of a row.  With a = max |x| over the block and
// e = floor(log2 a) − 2 (2 is the exponent of 4, the largest power of two of
// e2m1), clamped to at least −127, its scale byte is e + 127 and each code is
// x·2^−e rounded to nearest even in e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and signs),
// saturated at ±6: the conversion of the OCP Microscaling Formats
// specification 1.0, section 6.3.  e + 127 is the exponent field of a as an fp32
// number minus 2 (at least 0), and the product with 2^−e is exact, so codes and
// scales are the same on any machine.  A block with an infinity or NaN gets the
// scale byte 255, which reads back as NaN.
//
// Both kernels move each value once: 2 (or 4) bytes one way, 17/32 of a byte the
// other, so device memory bounds them.  Four lanes share a block, 8 values each:
// the loads are 16 bytes a lane and consecutive across the warp, two shuffles
// give the block's maximum, and a lane's 8 codes are one 4-byte store.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/moe_gb300.h"
#include "moe_internal.h"
#include "mx4_internal.h"
#include "sm103_ptx.cuh"
#include "tile_store.cuh"

namespace moe {
namespace {

constexpr int THREADS = 256;
constexpr int SEG = 256;          // values of a row that a warp takes at a time
constexpr int UNROLL = 4;         // such pieces in flight per warp

// Byte offset of the 4-byte word with the scales of row `row`, blocks 4*kt .. 4*kt + 3.
__device__ __forceinline__ int64_t scale_word(int64_t row, int32_t kt, int32_t k_tiles) {
    return ((row >> 7) * k_tiles + kt) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4;
}

template <int DTYPE>
struct Eight {                    // 8 values as loaded
    uint4 v[DTYPE == MOE_DTYPE_F32 ? 2 : 1];
};

template <int DTYPE>
__device__ __forceinline__ Eight<DTYPE> load8(const void* x, int64_t at) {
    Eight<DTYPE> r;
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(x) + at * (DTYPE == MOE_DTYPE_F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (DTYPE == MOE_DTYPE_F32 ? 2 : 1); ++i) r.v[i] = __ldg(p + i);
    return r;
}

template <int DTYPE>
__device__ __forceinline__ void widen(const Eight<DTYPE>& e, float (&f)[8]) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(e.v);
    if (DTYPE == MOE_DTYPE_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 t = unpack_16bit2<DTYPE == MOE_DTYPE_BF16>(w[i]);
            f[2 * i] = t.x;
            f[2 * i + 1] = t.y;
        }
    }
}

// Two codes, `lo` in the low half of the byte.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\tcvt.u32.u8 %0, b;\n\t}"
        : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// One warp per (row, run of SEG * UNROLL values); runs of a row are adjacent warps.
// Rows n_rows .. pad_rows - 1 (without row maps: the rest of the last scale
// tile) only get zero scales.
template <int DTYPE>
__global__ void __launch_bounds__(THREADS)
quantize_kernel(const Mx4Quantize a, int64_t pad_rows, int32_t runs) {
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t warp = static_cast<int64_t>(blockIdx.x) * (THREADS / 32) + (threadIdx.x >> 5);
    const int64_t row = warp / runs;
    const int32_t c0 = static_cast<int32_t>(warp - row * runs) * (SEG * UNROLL) + lane * 8;
    if (row >= pad_rows) return;
    const int32_t k_tiles = a.cols / 128;
    const bool given = row < a.n_rows;
    int64_t src = row;
    if (given && a.src_rows) {
        src = __ldg(a.src_rows + row);
        if (src >= a.n_src && a.status && lane == 0) atomicOr(a.status, MOE_DEV_BAD_TABLE);
        if (src < 0 || src >= a.n_src) return;             // negative rows are skipped
    }

    Eight<DTYPE> raw[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
        if (given && c0 + u * SEG < a.cols) raw[u] = load8<DTYPE>(a.x, src * a.cols + c0 + u * SEG);
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const int32_t c = c0 + u * SEG;
        // a piece of 128 values is 16 lanes: lanes past the row's end only take part in the shuffles
        const bool in = c < a.cols;
        uint32_t codes = 0, byte = 0;
        float f[8] = {};
        if (given && in) widen<DTYPE>(raw[u], f);
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const uint32_t ex = m >> 23;
        byte = ex == 255u ? 255u : (ex > 2u ? ex - 2u : 0u);
        if (ex != 255u) {
            const float inv = __uint_as_float((254u - byte) << 23);        // 2^−e, a normal number
#pragma unroll
            for (int i = 0; i < 4; ++i) codes |= e2m1x2(f[2 * i] * inv, f[2 * i + 1] * inv) << (8 * i);
        }
        // the four blocks' scale bytes, gathered in the first of their 16 lanes
        uint32_t word = byte << (8 * ((lane >> 2) & 3));
        word |= __shfl_xor_sync(0xffffffffu, word, 4);
        word |= __shfl_xor_sync(0xffffffffu, word, 8);
        if (!in) continue;
        for (int32_t j = 0; j < (given ? a.copies : 1); ++j) {
            int64_t dst = row;
            if (a.dest_rows) {
                dst = __ldg(a.dest_rows + row * a.copies + j);
                if (dst >= a.n_dest && a.status && lane == 0) atomicOr(a.status, MOE_DEV_BAD_TABLE);
                if (dst < 0 || dst >= a.n_dest) continue;
            }
            if (given) *reinterpret_cast<uint32_t*>(a.codes + (dst * a.cols + c) / 2) = codes;
            if ((lane & 15) == 0)
                *reinterpret_cast<uint32_t*>(a.scales + scale_word(dst, c >> 7, k_tiles)) = given ? word : 0u;
        }
    }
}

// Eight values from four bytes of codes and the block's scale byte.
template <int DTYPE>
__device__ __forceinline__ void store8(void* out, int64_t at, uint32_t codes, uint32_t byte) {
    // 2^(byte − 127); byte 0 is the subnormal 2^−127, byte 255 is NaN
    const float s = byte == 0u ? __uint_as_float(0x00400000u) : (byte == 255u ? __uint_as_float(0x7fc00000u)
                                                                           : __uint_as_float(byte << 23));
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h;
        const uint16_t two = static_cast<uint16_t>((codes >> (8 * i)) & 0xffu);
        asm("{\n\t.reg .b8 lo, hi;\n\tmov.b16 {lo, hi}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, lo;\n\t}" : "=r"(h) : "h"(two));
        const float2 v = unpack_16bit2<false>(h);
        f[2 * i] = v.x * s;
        f[2 * i + 1] = v.y * s;
    }
    if (DTYPE == MOE_DTYPE_F32) {
        uint4* p = reinterpret_cast<uint4*>(static_cast<float*>(out) + at);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            p[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                              __float_as_uint(f[4 * i + 3]));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pack_16bit2<DTYPE == MOE_DTYPE_BF16>(f[2 * i], f[2 * i + 1]);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <int DTYPE>
__global__ void __launch_bounds__(THREADS)
dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t rows, int32_t cols,
                  void* __restrict__ out, int32_t runs) {
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t warp = static_cast<int64_t>(blockIdx.x) * (THREADS / 32) + (threadIdx.x >> 5);
    const int64_t row = warp / runs;
    const int32_t c0 = static_cast<int32_t>(warp - row * runs) * (SEG * UNROLL) + lane * 8;
    if (row >= rows) return;
    uint32_t w[UNROLL], b[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const int32_t c = c0 + u * SEG;
        if (c < cols) {
            w[u] = __ldg(reinterpret_cast<const uint32_t*>(codes + (row * cols + c) / 2));
            b[u] = __ldg(scales + scale_word(row, c >> 7, cols / 128) + ((c >> 5) & 3));
        }
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
        if (c0 + u * SEG < cols) store8<DTYPE>(out, row * cols + c0 + u * SEG, w[u], b[u]);
}

cudaError_t config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, int64_t warps, cudaStream_t stream) {
    const int64_t blocks = (warps + THREADS / 32 - 1) / (THREADS / 32);
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_mx4_quantize(const Mx4Quantize& a, cudaStream_t stream) {
    const int32_t runs = (a.cols + SEG * UNROLL - 1) / (SEG * UNROLL);
    const int64_t pad_rows = a.dest_rows ? a.n_rows : (a.n_rows + 127) / 128 * 128;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    if (cudaError_t e = config(cfg, attr, pad_rows * runs, stream)) return e;
    switch (a.dtype) {
        case MOE_DTYPE_F16: return cudaLaunchKernelEx(&cfg, quantize_kernel<MOE_DTYPE_F16>, a, pad_rows, runs);
        case MOE_DTYPE_BF16: return cudaLaunchKernelEx(&cfg, quantize_kernel<MOE_DTYPE_BF16>, a, pad_rows, runs);
        default: return cudaLaunchKernelEx(&cfg, quantize_kernel<MOE_DTYPE_F32>, a, pad_rows, runs);
    }
}

cudaError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t cols,
                                  int32_t dtype, void* out, cudaStream_t stream) {
    const int32_t runs = (cols + SEG * UNROLL - 1) / (SEG * UNROLL);
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    if (cudaError_t e = config(cfg, attr, rows * runs, stream)) return e;
    switch (dtype) {
        case MOE_DTYPE_F16:
            return cudaLaunchKernelEx(&cfg, dequantize_kernel<MOE_DTYPE_F16>, codes, scales, rows, cols, out, runs);
        case MOE_DTYPE_BF16:
            return cudaLaunchKernelEx(&cfg, dequantize_kernel<MOE_DTYPE_BF16>, codes, scales, rows, cols, out, runs);
        default:
            return cudaLaunchKernelEx(&cfg, dequantize_kernel<MOE_DTYPE_F32>, codes, scales, rows, cols, out, runs);
    }
}

}  // namespace moe
