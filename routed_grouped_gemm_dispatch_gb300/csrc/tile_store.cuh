// 16-bit rounding and whole-line stores of accumulator rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace moe {

// Two fp32 values rounded to nearest even in the output's 16-bit type.
template <bool BF16>
__device__ __forceinline__ uint32_t pack_16bit2(float lo, float hi) {
    if (BF16) {
        __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<uint32_t*>(&v);
    }
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

template <bool BF16>
__device__ __forceinline__ float2 unpack_16bit2(uint32_t v) {
    if (BF16) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    return __half22float2(*reinterpret_cast<__half2*>(&v));
}

// 8 x 8 transpose of 16-byte pieces inside every group of 8 lanes, in three
// butterfly rounds: piece k of lane i moves to piece i of lane k.
__device__ __forceinline__ void transpose_pieces(uint4 (&el)[8], int lane) {
#pragma unroll
    for (int m = 4; m >= 1; m >>= 1) {
        const bool hi = (lane & m) != 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (e & m) continue;
            const int f = e | m;
            const uint4 send = hi ? el[e] : el[f];
            uint4 recv;
            recv.x = __shfl_xor_sync(0xffffffffu, send.x, m);
            recv.y = __shfl_xor_sync(0xffffffffu, send.y, m);
            recv.z = __shfl_xor_sync(0xffffffffu, send.z, m);
            recv.w = __shfl_xor_sync(0xffffffffu, send.w, m);
            if (hi) el[e] = recv;
            else el[f] = recv;
        }
    }
}

// Store 64 columns of 32 rows: thread `lane` holds row `lane` of the warp, el[k]
// its columns 8k .. 8k + 7.  `dst0` is the first column of the warp's first
// row.  The first `rows` rows and the first `cols` columns (a multiple of 8)
// are written.  With at least 16 rows the pieces are transposed first, so that
// 8 lanes write one whole 128-byte line and a warp instruction four of them,
// instead of 32 half-filled sectors.
__device__ __forceinline__ void store_rows_64(uint4 (&el)[8], uint16_t* dst0, int64_t stride, int lane, int32_t rows,
                                              int32_t cols) {
    if (rows >= 16) {
        transpose_pieces(el, lane);
        const int g8 = lane & ~7;
#pragma unroll
        for (int r = 0; r < 8; ++r)
            if (g8 + r < rows && (lane & 7) * 8 < cols)
                *reinterpret_cast<uint4*>(dst0 + static_cast<int64_t>(g8 + r) * stride + (lane & 7) * 8) = el[r];
    } else if (lane < rows) {
        uint16_t* d = dst0 + static_cast<int64_t>(lane) * stride;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k * 8 < cols) *reinterpret_cast<uint4*>(d + k * 8) = el[k];
    }
}

// The same exchange through 4 KB of the warp's own shared memory: 32 rows of 128
// bytes, a row's 16-byte pieces permuted by its index so that neither side has
// bank conflicts.  It moves as many bytes through shared memory as the
// shuffles and spares their selects: about 16 instructions instead of 190.
__device__ __forceinline__ void stage_rows(const uint4 (&el)[8], uint8_t* buf, int lane) {
#pragma unroll
    for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4*>(buf + lane * 128 + ((k ^ (lane & 7)) * 16)) = el[k];
    __syncwarp();
}

// store_rows_64 by way of `buf`.
__device__ __forceinline__ void store_staged_64(const uint4 (&el)[8], uint8_t* buf, uint16_t* dst0, int64_t stride,
                                                int lane, int32_t rows, int32_t cols) {
    stage_rows(el, buf, lane);
    const int piece = lane & 7, g = lane >> 3;
    uint16_t* d = dst0 + static_cast<int64_t>(g) * stride + piece * 8;
    if (piece * 8 < cols) {
#pragma unroll
        for (int r = 0; r < 8; ++r) {                     // rows 4r + g: a warp's store is four whole lines
            const int at = 4 * r + g;
            if (at < rows)
                *reinterpret_cast<uint4*>(d + static_cast<int64_t>(4 * r) * stride) =
                    *reinterpret_cast<const uint4*>(buf + at * 128 + ((piece ^ (at & 7)) * 16));
        }
    }
    __syncwarp();
}

// Lines of 64 columns as read from memory (lane 8g + i: piece i of rows g, 4 + g, ...), and
// their exchange into rows: thread `lane` ends with row `lane`.  Rows and columns
// outside the given extents read as zero.
__device__ __forceinline__ void load_lines_64(uint4 (&el)[8], const uint16_t* src0, int64_t stride, int lane,
                                              int32_t rows, int32_t cols) {
    const int piece = lane & 7, g = lane >> 3;
    const uint16_t* p = src0 + static_cast<int64_t>(g) * stride + piece * 8;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        el[r] = make_uint4(0, 0, 0, 0);
        if (4 * r + g < rows && piece * 8 < cols)
            el[r] = __ldg(reinterpret_cast<const uint4*>(p + static_cast<int64_t>(4 * r) * stride));
    }
}

__device__ __forceinline__ void lines_to_rows(uint4 (&el)[8], uint8_t* buf, int lane) {
    const int piece = lane & 7, g = lane >> 3;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        const int at = 4 * r + g;
        *reinterpret_cast<uint4*>(buf + at * 128 + ((piece ^ (at & 7)) * 16)) = el[r];
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 8; ++k) el[k] = *reinterpret_cast<const uint4*>(buf + lane * 128 + ((k ^ (lane & 7)) * 16));
    __syncwarp();
}

}  // namespace moe
