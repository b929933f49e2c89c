// 4-bit microscaled operators: arguments of their launchers (host side).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace moe {

struct Mx4Quantize {
    int32_t dtype;                // MOE_DTYPE_*
    const void* x;                // [src rows, cols]
    int64_t n_src;
    int64_t n_rows;               // rows converted
    int32_t cols;
    const int32_t* src_rows;      // [n_rows], or nullptr: row i
    const int32_t* dest_rows;     // [n_rows, copies], or nullptr: row i
    int32_t copies;
    int64_t n_dest;
    uint8_t* codes;               // [n_dest, cols / 2]
    uint8_t* scales;              // tiles of [n_dest, cols / 32]
    int32_t* status;
};

enum Mx4Form { MX4_MATMUL = 0, MX4_GATE_UP = 1, MX4_DOWN = 2 };

struct Mx4Product {
    Mx4Form form;
    bool bf16;
    const uint8_t* a;             // [rows, k / 2]
    const uint8_t* a_scales;
    int64_t rows;
    int32_t k;
    const uint8_t* b;             // [n_experts * n, k / 2] (gate for MX4_GATE_UP)
    const uint8_t* b_scales;
    const uint8_t* b2;            // up
    const uint8_t* b2_scales;
    int32_t n_experts, n;
    const float* weights;         // MX4_DOWN: [valid_total]
    int64_t valid_total;
    const int32_t* sizes;
    const int32_t* offsets;       // MX4_DOWN only
    const int32_t* padded;
    const int32_t* gidx;
    int64_t num_blocks;           // MX4_MATMUL: ceil(rows / 128)
    uint16_t* out;                // [rows, n]
    int32_t* status;
};

// Arguments already validated; at least one row (block) of work.
cudaError_t launch_mx4_quantize(const Mx4Quantize& a, cudaStream_t stream);
cudaError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t cols,
                                  int32_t dtype, void* out, cudaStream_t stream);
cudaError_t launch_mx4_product(const Mx4Product& a, cudaStream_t stream);

}  // namespace moe
