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
// other, so device memory bounds them as long as the arithmetic stays at a few
// instructions a value: the maximum is taken on packed pairs, and the
// hardware's conversion rounds two values at a time.  Four lanes share a block,
// 8 values each: the loads are 16 bytes a lane and consecutive across the warp,
// two shuffles give the block's maximum, and a lane's 8 codes are one 4-byte
// store.  16384 x 7168: bf16 to 4 bits 53 us (5.6 TB/s, instructions 70% busy), fp32
// 78 us (6.8 TB/s), 4 bits to bf16 48 us (6.2 TB/s), to fp32 86 us (6.2 TB/s).
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

// Eight codes of eight values, the first in the lowest four bits.
__device__ __forceinline__ uint32_t e2m1x8(const float (&f)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
    return r;
}

// Exponent field, as an fp32 number, of the largest magnitude of eight values;
// 255 if one of them is infinite or NaN.  Lanes of a group of four agree on it.
template <int DTYPE>
__device__ __forceinline__ uint32_t max_exponent(const Eight<DTYPE>& e) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(e.v);
    uint32_t m = 0;
    if constexpr (DTYPE == MOE_DTYPE_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7fffffffu);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        return m >> 23;
    } else {
        // magnitudes of 16-bit floats order like whole numbers, NaN above infinity
#pragma unroll
        for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
        m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
        m = max(m & 0xffffu, m >> 16);
        if (DTYPE == MOE_DTYPE_BF16) return m >> 7;
        return m >= 0x7c00u ? 255u : __float_as_uint(__half2float(__ushort_as_half(static_cast<uint16_t>(m)))) >> 23;
    }
}

// A warp takes one row's run of SEG * UNROLL values: rows along the grid's x,
// runs along y.  Without destination rows, rows n_rows .. pad_rows - 1 (the rest
// of the last scale tile) get zero scales; with them pad_rows is n_rows.  LISTS:
// there is a list of source or of destination rows.
template <int DTYPE, bool LISTS>
__global__ void __launch_bounds__(THREADS, 6)
quantize_kernel(const Mx4Quantize a, int64_t pad_rows) {
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (THREADS / 32) + (threadIdx.x >> 5);
    const int32_t c0 = static_cast<int32_t>(blockIdx.y) * (SEG * UNROLL) + lane * 8;
    if (row >= pad_rows) return;
    const int32_t k_tiles = a.cols / 128;
    const bool given = row < a.n_rows;
    int64_t src = row;
    if (LISTS && given && a.src_rows) {
        src = __ldg(a.src_rows + row);
        if (src >= a.n_src && a.status && lane == 0) atomicOr(a.status, MOE_DEV_BAD_TABLE);
        if (src < 0 || src >= a.n_src) return;             // negative rows are skipped
    }

    Eight<DTYPE> raw[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        raw[u] = Eight<DTYPE>{};
        if (given && c0 + u * SEG < a.cols) raw[u] = load8<DTYPE>(a.x, src * a.cols + c0 + u * SEG);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const int32_t c = c0 + u * SEG;
        if (c - lane * 8 >= a.cols) break;                 // the whole warp is past the row's end
        const uint32_t ex = max_exponent<DTYPE>(raw[u]);
        const uint32_t byte = ex == 255u ? 255u : (ex > 2u ? ex - 2u : 0u);
        // 2^−e, a normal number (of no use in a bad block, whose codes are 0)
        const float inv = __uint_as_float((254u - byte) << 23);
        float f[8];
        widen<DTYPE>(raw[u], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= inv;
        uint32_t codes = e2m1x8(f);
        if (ex == 255u) codes = 0;
        // the four blocks' scale bytes, gathered in the first of their 16 lanes
        uint32_t word = byte << (8 * ((lane >> 2) & 3));
        word |= __shfl_xor_sync(0xffffffffu, word, 4);
        word |= __shfl_xor_sync(0xffffffffu, word, 8);
        if (c >= a.cols) continue;                         // a last piece of 128 values is 16 lanes
        auto put = [&](int64_t dst) {
            MOE_DCHECK(dst >= 0 && dst < (given ? a.n_dest : (a.n_dest + 127) / 128 * 128) && c + 8 <= a.cols, a.status);
            MOE_DCHECK(!given || (src >= 0 && src < a.n_src), a.status);
            if (given) *reinterpret_cast<uint32_t*>(a.codes + (dst * a.cols + c) / 2) = codes;
            if ((lane & 15) == 0)
                *reinterpret_cast<uint32_t*>(a.scales + scale_word(dst, c >> 7, k_tiles)) = given ? word : 0u;
        };
        if (LISTS && a.dest_rows) {
            for (int32_t j = 0; j < a.copies; ++j) {
                const int64_t dst = __ldg(a.dest_rows + row * a.copies + j);
                if (dst >= a.n_dest && a.status && lane == 0) atomicOr(a.status, MOE_DEV_BAD_TABLE);
                if (dst >= 0 && dst < a.n_dest) put(dst);
            }
        } else {
            put(row);                                      // the padding's rows too: their scale words alone
        }
    }
}

// 2^(byte − 127); byte 0 is the subnormal 2^−127, byte 255 is NaN.
__device__ __forceinline__ float scale_of(uint32_t byte) {
    return __uint_as_float(byte == 0u ? 0x00400000u : (byte == 255u ? 0x7fc00000u : byte << 23));
}

// Four values from two bytes of codes.
__device__ __forceinline__ void decode4(uint32_t codes, float s, float (&f)[4]) {
    uint32_t lo, hi;
    const uint16_t two = static_cast<uint16_t>(codes);
    asm("{\n\t.reg .b8 a, b;\n\tmov.b16 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t}" : "=r"(lo), "=r"(hi) : "h"(two));
    const float2 a = unpack_16bit2<false>(lo), b = unpack_16bit2<false>(hi);
    f[0] = a.x * s;
    f[1] = a.y * s;
    f[2] = b.x * s;
    f[3] = b.y * s;
}

// As quantize_kernel; a lane's store is 16 bytes in every type: 8 values of 16
// bits, or twice 4 of fp32, 128 columns apart.
template <int DTYPE>
__global__ void __launch_bounds__(THREADS)
dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t rows, int32_t cols,
                  void* __restrict__ out) {
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    constexpr int PARTS = DTYPE == MOE_DTYPE_F32 ? 2 : 1;
    constexpr int VALUES = 8 / PARTS;                     // of a lane's piece
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (THREADS / 32) + (threadIdx.x >> 5);
    const int32_t c0 = static_cast<int32_t>(blockIdx.y) * (SEG * UNROLL) + lane * VALUES;
    if (row >= rows) return;
    uint32_t w[UNROLL * PARTS], b[UNROLL * PARTS];
#pragma unroll
    for (int u = 0; u < UNROLL * PARTS; ++u) {
        const int32_t c = c0 + u * (SEG / PARTS);
        if (c < cols) {
            const uint8_t* p = codes + (row * cols + c) / 2;
            w[u] = PARTS == 1 ? __ldg(reinterpret_cast<const uint32_t*>(p)) : __ldg(reinterpret_cast<const uint16_t*>(p));
            b[u] = __ldg(scales + scale_word(row, c >> 7, cols / 128) + ((c >> 5) & 3));
        }
    }
#pragma unroll
    for (int u = 0; u < UNROLL * PARTS; ++u) {
        const int32_t c = c0 + u * (SEG / PARTS);
        if (c >= cols) break;
        const float s = scale_of(b[u]);
        float f[4], g[4];
        decode4(w[u] & 0xffffu, s, f);
        if (DTYPE == MOE_DTYPE_F32) {
            reinterpret_cast<float4*>(static_cast<float*>(out) + row * cols + c)[0] = make_float4(f[0], f[1], f[2], f[3]);
        } else {
            constexpr bool BF16 = DTYPE == MOE_DTYPE_BF16;
            decode4(w[u] >> 16, s, g);
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + row * cols + c) =
                make_uint4(pack_16bit2<BF16>(f[0], f[1]), pack_16bit2<BF16>(f[2], f[3]), pack_16bit2<BF16>(g[0], g[1]),
                           pack_16bit2<BF16>(g[2], g[3]));
        }
    }
}

// Eight rows a block along x, runs of SEG * UNROLL columns along y.
void config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, int64_t rows, int32_t cols, cudaStream_t stream) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>((rows + THREADS / 32 - 1) / (THREADS / 32)),
                       static_cast<unsigned>((cols + SEG * UNROLL - 1) / (SEG * UNROLL)));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
}

template <int DTYPE>
cudaError_t quantize(const Mx4Quantize& a, cudaStream_t stream) {
    const int64_t pad_rows = a.dest_rows ? a.n_rows : (a.n_rows + 127) / 128 * 128;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    config(cfg, attr, pad_rows, a.cols, stream);
    return a.src_rows || a.dest_rows ? cudaLaunchKernelEx(&cfg, quantize_kernel<DTYPE, true>, a, pad_rows)
                                     : cudaLaunchKernelEx(&cfg, quantize_kernel<DTYPE, false>, a, pad_rows);
}

template <int DTYPE>
cudaError_t dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t cols, void* out,
                       cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    config(cfg, attr, rows, cols, stream);
    return cudaLaunchKernelEx(&cfg, dequantize_kernel<DTYPE>, codes, scales, rows, cols, out);
}

}  // namespace

cudaError_t launch_mx4_quantize(const Mx4Quantize& a, cudaStream_t stream) {
    switch (a.dtype) {
        case MOE_DTYPE_F16: return quantize<MOE_DTYPE_F16>(a, stream);
        case MOE_DTYPE_BF16: return quantize<MOE_DTYPE_BF16>(a, stream);
        default: return quantize<MOE_DTYPE_F32>(a, stream);
    }
}

cudaError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t cols,
                                  int32_t dtype, void* out, cudaStream_t stream) {
    switch (dtype) {
        case MOE_DTYPE_F16: return dequantize<MOE_DTYPE_F16>(codes, scales, rows, cols, out, stream);
        case MOE_DTYPE_BF16: return dequantize<MOE_DTYPE_BF16>(codes, scales, rows, cols, out, stream);
        default: return dequantize<MOE_DTYPE_F32>(codes, scales, rows, cols, out, stream);
    }
}

}  // namespace moe
