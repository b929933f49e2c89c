// Orthogonalised update: for each matrix G of a stack
//     X₀ = G / max(‖G‖, eps)   (Frobenius norm)
//     A = X·Xᵀ,  B = b·A + c·A²,  X ← a·X + B·X      `steps` times
// with X taken with the fewer rows (a tall G is transposed on the way in and out; the
// polynomial is the same from either side).  A and B are symmetric, so only the tiles on and
// below the diagonal are multiplied, and the others are stored from them.
//
// One launch for all steps of all matrices: a list of tiles, 256 rows high, that pairs of CTAs
// take in order (pair_tiles.cuh).  A tile starts when the panels (256 rows) of what it multiplies
// are complete, which counters in memory say:
//     A(i, j)  of step k   X's panels i and j          all B(i, ·)·X of step k − 1
//     B(i, j)              A's panels i and j          every A(i, ·) and A(·, i)
//     X(i, n)              B's panel i                 every B(i, ·) and B(·, i)
// The order makes them complete early: A by rows, B by columns, X by rows.  Nothing is
// overwritten while it is read: X has two buffers, and a tile that may write a panel of A, B
// or the older X has waited, through that chain, for all that read it.  A stack is walked in groups of
// matrices, large enough that a tile's panels were finished a while ago, small enough that
// what a group passes from product to product is still in L2.
//
// Numbers.  All operands are fp16 (11 bits at the rate of bf16's 8), times powers of two that
// keep them normal: X·2^6, A·2^10, B·2^6; sums are fp32.  X₀ is G times a power of two, which
// is exact for 16-bit values but for those below 2^-20 of the norm (fp16 holds them in steps of 2^-24, 2^-30 of the
// norm: less than the result's own rounding in any matrix whose norm is at least eps), and the rest of 1/‖G‖ enters the
// first step's fp32 sums.  Values whose norm
// grows past 2^9 in a step (coefficients that diverge) overflow.
//
// What a tile needs besides its sums would come from L2 beside the operands, whose way from there is
// the bound, so as little as possible does:
//  * B = c·(A + s)² − c·s², s = b/2c: A is stored with s on its diagonal, and B(i, j) is a product of its
//    rows.  What the diagonal's rounding makes of B's own diagonal is put right from A's
//    diagonal in fp32; off it, it is a relative 2^-12.  (c = 0: A's product gives B at once.)
//  * a is on B's diagonal.  Its rounding scales a row of X by 1 ± 2^-12, which leaves the rank as it is.
//  * Rounding X to 11 bits does not: it adds noise in directions that a low-rank G does not have,
//    and a multiplies it by 3.44 a step.  So a·X takes X with some 15 bits: hi + lo·2^-13, fp16
//    and e4m3 (hi alone is the products' operand).
// Bound.  A stack: the operands' way from L2, whose 0.2 us for 64 along K of a 256 x 128 tile is 1.6 PFLOP/s
// on all pairs (0.326 and 2.0 for 256 x 256), and the tiles' empty rows (1408 are 5.5 panels); 64 x
// 1408 x 2048 takes 3.7 ms where its operations are 2.45 at the measured rate of bf16, and 4.1 to 4.3 back to back under the
// power cap.  One matrix: besides, each product waits for the one before, with some 6.3 us from its
// operands' completion to its own where it has few tiles (a poll that sees it 1.4, copies and K loop 2 to 3.5,
// epilogue 1.5, publishing 0.7), and few whole rounds of tiles: 2816 x 2048 257 us (operations 113),
// 2048 x 7168 425 to 445 (253), 3 x 333 x 1001 104 (2.8).
//
// In 64-bit simulation with these roundings, the root mean square error of five steps relative to that
// of the result:
//                                        Gaussian   rank M/4    rank 1
//     X as hi alone                       0.9e-3     1.4e-2     3.2e-2
//     as here                             1.3e-3     1.8e-3     2.8e-3
//     A and X read, X as two fp16         1.5e-3     1.2e-3     1.4e-3
//     all operands bf16                   1.1e-2     1.4e-1     3.4e-1
// The last step's X is rounded to bf16 (1.7e-3 by itself).
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/moe_gb300.h"
#include "moe_internal.h"
#include "pair_tiles.cuh"
#include "train_internal.h"

namespace moe {
namespace {

using pairs::Tile;

constexpr float X_SCALE = 64.0f;            // 2^6
constexpr int X_EXPONENT = 6;
constexpr float B_SCALE = 64.0f;
constexpr float LO_SCALE = 8192.0f;         // lo = (x - hi)·2^13
constexpr float MAX_A_SCALE = 1024.0f;      // of A, less where s is large
constexpr int SUM_THREADS = 256;
constexpr int SUM_VALUES = 2048;            // that a block sums at least
constexpr int MAX_SUM_BLOCKS = 512;         // of one matrix

// ---------------------------------------------------------------------------
// norms, and X₀
// ---------------------------------------------------------------------------

template <int DTYPE>
__device__ __forceinline__ float value_at(const void* base, int64_t i) {
    if (DTYPE == MOE_DTYPE_F32) return __ldg(static_cast<const float*>(base) + i);
    const uint16_t v = __ldg(static_cast<const uint16_t*>(base) + i);
    if (DTYPE == MOE_DTYPE_BF16) return __uint_as_float(static_cast<uint32_t>(v) << 16);
    return __half2float(__ushort_as_half(v));
}

// 16 bytes of values.
template <int DTYPE>
__device__ __forceinline__ void values_of(const uint4& w, float (&v)[DTYPE == MOE_DTYPE_F32 ? 4 : 8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DTYPE == MOE_DTYPE_F32) {
            v[i] = __uint_as_float(u[i]);
        } else {
            const float2 f = unpack_16bit2<DTYPE == MOE_DTYPE_BF16>(u[i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}

// Two remainders as e4m3 bytes (largest magnitude 448), the first in the low one, and back.
__device__ __forceinline__ uint32_t pack_lo2(float x, float y) {
    return __nv_cvt_float2_to_fp8x2(make_float2(x * LO_SCALE, y * LO_SCALE), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 unpack_lo2(uint32_t v) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    return make_float2(f.x * (1.0f / LO_SCALE), f.y * (1.0f / LO_SCALE));
}

struct Prepare {
    const void* update;
    int64_t elements;             // of a matrix
    int32_t M, N, ld, ld_lo;      // X is [M, ld], N of the columns in use
    int32_t sum_blocks;
    float least_norm;
    float* sums;                  // [batch, sum_blocks]
    float* rest;                  // [batch]: what X₀ still has to be times
    uint16_t* hi;                 // [batch, M, ld]
    uint8_t* lo;                  // [batch, M, ld_lo], nullable
    int32_t* ready;               // [batch, counters], zeroed here for the products
    int32_t* queue;
    int32_t counters;
};

// Σ v² of a piece of a matrix.
template <int DTYPE, bool VEC>
__global__ void __launch_bounds__(SUM_THREADS) square_sum_kernel(const Prepare p) {
    __shared__ float part[SUM_THREADS / 32];
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    constexpr int PER = DTYPE == MOE_DTYPE_F32 ? 4 : 8;
    constexpr int BYTES = DTYPE == MOE_DTYPE_F32 ? 4 : 2;
    const uint8_t* base = static_cast<const uint8_t*>(p.update) + static_cast<int64_t>(blockIdx.y) * p.elements * BYTES;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * SUM_THREADS + threadIdx.x;
    const int64_t step = static_cast<int64_t>(gridDim.x) * SUM_THREADS;
    float sum = 0.0f;
    if (VEC) {
#pragma unroll 8
        for (int64_t i = first; i < p.elements / PER; i += step) {
            float v[PER];
            values_of<DTYPE>(__ldg(reinterpret_cast<const uint4*>(base) + i), v);
#pragma unroll
            for (int j = 0; j < PER; ++j) sum += v[j] * v[j];
        }
    } else {
#pragma unroll 8
        for (int64_t i = first; i < p.elements; i += step) {
            const float v = value_at<DTYPE>(base, i);
            sum += v * v;
        }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < SUM_THREADS / 32; ++w) sum += part[w];
        p.sums[static_cast<int64_t>(blockIdx.y) * p.sum_blocks + blockIdx.x] = sum;
    }
}

// What the norm makes of the values of a matrix: times `power`, a power of two, they are X₀·2^6 / `rest`.
struct Norm {
    float power, rest;
};
__device__ __forceinline__ Norm norm_of(const Prepare& p, int64_t matrix, float* part) {
    float sum = 0.0f;
    for (int i = threadIdx.x; i < p.sum_blocks; i += SUM_THREADS) sum += __ldg(p.sums + matrix * p.sum_blocks + i);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = 0.0f;
    for (int w = 0; w < SUM_THREADS / 32; ++w) sum += part[w];
    float norm = sqrtf(sum);
    if (norm < p.least_norm) norm = p.least_norm;             // a NaN stays
    int e = 0;
    Norm n;
    n.rest = __int_as_float(0x7fffffff);                      // infinite (or NaN): so is the result, NaN
    if (norm <= 3.4e38f) n.rest = 1.0f / frexpf(norm, &e);    // norm = f·2^e, f in [0.5, 1), e >= -69
    n.power = ldexpf(1.0f, X_EXPONENT - e);
    return n;
}

// Eight values of X₀, as hi and (where it is kept) lo.
__device__ __forceinline__ void store_x0(const Prepare& p, int64_t row, int32_t col, const float (&v)[8], float power) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float x = v[2 * j] * power, y = v[2 * j + 1] * power;
        h[j] = pack_16bit2<false>(x, y);
        const float2 back = unpack_16bit2<false>(h[j]);
        l[j] = pack_lo2(x - back.x, y - back.y);
    }
    *reinterpret_cast<uint4*>(p.hi + row * p.ld + col) = make_uint4(h[0], h[1], h[2], h[3]);
    if (p.lo) *reinterpret_cast<uint2*>(p.lo + row * p.ld_lo + col) = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
}

// Eight values from element i on, `n` of them there (the others zero).
template <int DTYPE, bool VEC>
__device__ __forceinline__ void load_eight(float (&v)[8], const void* base, int64_t i, int32_t n) {
    if constexpr (VEC && DTYPE == MOE_DTYPE_F32) {
        float a[4], b[4];
        values_of<DTYPE>(__ldg(reinterpret_cast<const uint4*>(static_cast<const float*>(base) + i)), a);
        values_of<DTYPE>(__ldg(reinterpret_cast<const uint4*>(static_cast<const float*>(base) + i + 4)), b);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = a[j];
            v[4 + j] = b[j];
        }
    } else if constexpr (VEC) {
        values_of<DTYPE>(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i)), v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < n ? value_at<DTYPE>(base, i + j) : 0.0f;
    }
}

// X₀ up to the factor `rest`.  Grid: blocks x matrices.  VEC: the update's rows are whole 8 values.
template <int DTYPE, bool VEC>
__global__ void __launch_bounds__(SUM_THREADS) prepare_kernel(const Prepare p) {
    __shared__ float part[SUM_THREADS / 32];
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int64_t matrix = blockIdx.y;
    const Norm n = norm_of(p, matrix, part);
    if (blockIdx.x == 0) {
        for (int i = threadIdx.x; i < p.counters; i += SUM_THREADS) p.ready[matrix * p.counters + i] = 0;
        if (threadIdx.x == 0) {
            p.rest[matrix] = n.rest;
            if (matrix == 0) *p.queue = 0;
        }
    }
    constexpr int BYTES = DTYPE == MOE_DTYPE_F32 ? 4 : 2;
    const uint8_t* base = static_cast<const uint8_t*>(p.update) + matrix * p.elements * BYTES;
    const int32_t pieces = p.ld / 8;
    const int64_t all = static_cast<int64_t>(p.M) * pieces, step = static_cast<int64_t>(gridDim.x) * SUM_THREADS;
    // four pieces' loads ahead of their stores
    for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * SUM_THREADS + threadIdx.x; i0 < all; i0 += 4 * step) {
        float v[4][8];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t i = i0 + u * step;
            if (i >= all) break;
            const int64_t row = VEC && p.lo == nullptr ? 0 : i / pieces;
            const int32_t col = static_cast<int32_t>(i - row * pieces) * 8;
            if (VEC) load_eight<DTYPE, true>(v[u], base, i * 8, 8);
            else load_eight<DTYPE, false>(v[u], base, row * p.N + col, p.N - col);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t i = i0 + u * step;
            if (i >= all) break;
            if (VEC && p.lo == nullptr) {
                // rows one after the other, as in the update
                uint32_t h[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) h[j] = pack_16bit2<false>(v[u][2 * j] * n.power, v[u][2 * j + 1] * n.power);
                reinterpret_cast<uint4*>(p.hi)[matrix * all + i] = make_uint4(h[0], h[1], h[2], h[3]);
            } else {
                const int64_t row = i / pieces;
                store_x0(p, matrix * p.M + row, static_cast<int32_t>(i - row * pieces) * 8, v[u], n.power);
            }
        }
    }
}

// The same from a tall update [N, M], in tiles of 64 rows x 64 columns of X.
template <int DTYPE, bool VEC>
__global__ void __launch_bounds__(SUM_THREADS) prepare_tall_kernel(const Prepare p) {
    __shared__ float tile[64][65];
    __shared__ float part[SUM_THREADS / 32];
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int64_t matrix = blockIdx.y;
    const Norm n = norm_of(p, matrix, part);
    if (blockIdx.x == 0) {
        for (int i = threadIdx.x; i < p.counters; i += SUM_THREADS) p.ready[matrix * p.counters + i] = 0;
        if (threadIdx.x == 0) {
            p.rest[matrix] = n.rest;
            if (matrix == 0) *p.queue = 0;
        }
    }
    constexpr int BYTES = DTYPE == MOE_DTYPE_F32 ? 4 : 2;
    const uint8_t* base = static_cast<const uint8_t*>(p.update) + matrix * p.elements * BYTES;
    const int32_t tiles_m = (p.M + 63) / 64, tiles = tiles_m * ((p.ld + 63) / 64);
    for (int32_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int32_t n0 = t / tiles_m * 64, m0 = t % tiles_m * 64;
        float v[2][8];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = (threadIdx.x >> 3) + 32 * u, c = (threadIdx.x & 7) * 8;
            const int32_t left = n0 + r < p.N ? p.M - m0 - c : 0;
            if (VEC && left >= 8) load_eight<DTYPE, true>(v[u], base, static_cast<int64_t>(n0 + r) * p.M + m0 + c, 8);
            else load_eight<DTYPE, false>(v[u], base, static_cast<int64_t>(n0 + r) * p.M + m0 + c, left);
        }
        __syncthreads();                          // the tile before is out
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < 8; ++j) tile[(threadIdx.x & 7) * 8 + j][(threadIdx.x >> 3) + 32 * u] = v[u][j];
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = (threadIdx.x >> 3) + 32 * u, c = (threadIdx.x & 7) * 8;
            if (m0 + r >= p.M || n0 + c >= p.ld) continue;
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = tile[r][c + j];
            store_x0(p, matrix * p.M + m0 + r, n0 + c, x, n.power);
        }
    }
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------

enum Kind { GRAM = 0, POLY = 1, APPLY = 2 };
enum Map { X_ROWS, X_COLS = X_ROWS + 2, X_RIGHT = X_COLS + 2, A_ROWS = X_RIGHT + 2, A_COLS, B_ROWS, MAPS };
static_assert(MAPS <= pairs::MAX_MAPS, "maps fit");

struct OrthoProducts {
    int32_t total_tiles, n_maps;
    int32_t* status;
    int32_t* queue;               // the next tile to take
    int32_t* ready;               // [batch][3][panels]: CTAs that have stored their part of a tile of a panel
    int32_t batch, group;         // matrices; of a group
    int32_t M, N;                 // X [M, N]
    int32_t ld_x, ld_a, ld_lo;    // elements between rows of X's hi; of A and B; of X's lo
    int32_t panels;               // of 256 rows
    int32_t width_a, width_x;     // columns of a tile of A and B, of X
    int32_t cols_a, cols_x;       // tile columns
    int32_t tri;                  // tiles of A (or B)
    int32_t steps;
    float a, b, c;
    float a_scale, shift;         // of A; on its diagonal
    int32_t square;               // c is not 0: B is a product
    int32_t has_lo;               // X₀ has one
    const float* rest;            // [batch] what X₀ still has to be times
    uint16_t* hi[2];              // X, in turn
    uint8_t* lo[2];
    float* diagonal;              // [batch, M] A's, as the sums have it
    uint16_t* A;
    uint16_t* B;
    uint16_t* out;
    int32_t tall;                 // out is transposed
};

// Tiles of A (or B) in 256-row panel q that lie on or below the diagonal.
__device__ __forceinline__ int32_t row_tiles(const OrthoProducts& p, int32_t q) {
    const int32_t n = p.width_a == 256 ? q + 1 : 2 * q + 2;
    return n < p.cols_a ? n : p.cols_a;
}
// The panel across the diagonal of tile column j.
__device__ __forceinline__ int32_t panel_of(const OrthoProducts& p, int32_t j) { return p.width_a == 256 ? j : j >> 1; }
// Tiles that store a part of panel q of A (or B).
__device__ __forceinline__ int32_t panel_tiles(const OrthoProducts& p, int32_t q) {
    const int32_t below = p.panels - 1 - q;
    return row_tiles(p, q) + (p.width_a == 256 ? below : 2 * below);
}

// The transpose of a warp's 32 rows x 64 columns (el: a row per lane): column n goes to row n of dst0, rows `stride`
// elements apart, as far as there are `cols` of them, and of each the first `rows` elements (a multiple of 2, and
// dst0 and stride so that pairs are aligned, unless ODD).  Neighbouring lanes exchange halves of
// their words, so that each has two rows of one column; 16 lanes write 64 bytes.  (By way of the staging memory,
// with 16-byte stores, 3 x 333 x 1001 took 115 us instead of 108, 2816 x 2048 272 instead of 263.)
template <bool ODD>
__device__ __forceinline__ void store_columns_64(const uint4 (&el)[8], uint16_t* dst0, int64_t stride, int lane, int32_t rows,
                                                 int32_t cols) {
    const int m = lane & ~1, odd = lane & 1;
    uint16_t* d = dst0 + odd * stride + m;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t u[4] = {el[k].x, el[k].y, el[k].z, el[k].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t other = __shfl_xor_sync(0xffffffffu, u[j], 1);
            const uint32_t v = odd ? __byte_perm(other, u[j], 0x7632) : __byte_perm(u[j], other, 0x5410);
            if (8 * k + 2 * j + odd < cols) {
                if (!ODD) {
                    if (m < rows) *reinterpret_cast<uint32_t*>(d) = v;
                } else {
                    if (m < rows) d[0] = static_cast<uint16_t>(v);
                    if (m + 1 < rows) d[1] = static_cast<uint16_t>(v >> 16);
                }
            }
            d += 2 * stride;
        }
    }
}

// 64 bytes of each of a warp's 32 rows, as lines (lane 4g + i: piece i of rows g, 8 + g, ...)
// from L2, where this launch itself has put them, and by way of `buf` as rows; and back.
__device__ __forceinline__ void load_bytes_64(uint4 (&el)[4], const uint8_t* src0, int64_t stride, int lane, int32_t rows,
                                              int32_t cols) {
    const int piece = lane & 3, g = lane >> 2;
    const uint8_t* s = src0 + static_cast<int64_t>(g) * stride + piece * 16;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        el[r] = make_uint4(0, 0, 0, 0);
        if (8 * r + g < rows && piece * 16 < cols)
            el[r] = __ldcg(reinterpret_cast<const uint4*>(s + static_cast<int64_t>(8 * r) * stride));
    }
}
__device__ __forceinline__ uint4* byte_piece(uint8_t* buf, int row, int piece) {
    return reinterpret_cast<uint4*>(buf + row * 64 + ((piece ^ ((row >> 1) & 3)) * 16));
}
__device__ __forceinline__ void bytes_to_rows(uint4 (&el)[4], uint8_t* buf, int lane) {
#pragma unroll
    for (int r = 0; r < 4; ++r) *byte_piece(buf, 8 * r + (lane >> 2), lane & 3) = el[r];
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) el[k] = *byte_piece(buf, lane, k);
    __syncwarp();
}
__device__ __forceinline__ void store_bytes_64(const uint4 (&el)[4], uint8_t* buf, uint8_t* dst0, int64_t stride, int lane,
                                               int32_t rows, int32_t cols) {
#pragma unroll
    for (int k = 0; k < 4; ++k) *byte_piece(buf, lane, k) = el[k];
    __syncwarp();
    const int piece = lane & 3, g = lane >> 2;
    uint8_t* d = dst0 + static_cast<int64_t>(g) * stride + piece * 16;
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (8 * r + g < rows && piece * 16 < cols)
            *reinterpret_cast<uint4*>(d + static_cast<int64_t>(8 * r) * stride) = *byte_piece(buf, 8 * r + g, piece);
    __syncwarp();
}

template <int BN_>
struct OrthoOp {
    static constexpr int BN = BN_;
    static constexpr bool BF16 = false;
    static constexpr bool MASKABLE = false;
    static constexpr bool QUEUE = true;
    using Params = OrthoProducts;

    struct Place {
        int32_t kind, step, matrix, i, j;          // panel of rows, tile column
    };
    using Code = int2;                             // a Place
    static_assert(MOE_ORTHO_MAX_SIZE <= 1 << 16 && MOE_ORTHO_MAX_STEPS <= 64, "a Place in 47 bits");
    static __device__ __forceinline__ Code code(const Params& p, int32_t t) {
        const Place at = number(p, t);
        return make_int2(at.kind | at.step << 2 | at.i << 8 | at.j << 17, at.matrix);
    }
    static __device__ __forceinline__ void pack(const Code& c, int32_t& x, int32_t& y) {
        x = c.x;
        y = c.y;
    }
    static __device__ __forceinline__ Code unpack(int32_t x, int32_t y) { return make_int2(x, y); }
    static __device__ __forceinline__ Place place(const Code& c) {
        return Place{c.x & 3, c.x >> 2 & 63, c.y, c.x >> 8 & 511, c.x >> 17 & 1023};
    }
    // Order: groups of matrices, their steps, the three products of a step, the group's matrices, tiles.
    static __device__ __forceinline__ Place number(const Params& p, int32_t t) {
        Place at;
        const int32_t symmetric = (1 + p.square) * p.tri;
        const int32_t per_matrix = symmetric + p.panels * p.cols_x;
        const int32_t per_group = p.group * p.steps * per_matrix;
        const int32_t g = t / per_group;
        int32_t r = t - g * per_group;
        const int32_t first = g * p.group;
        const int32_t n = p.batch - first < p.group ? p.batch - first : p.group;
        at.step = r / (n * per_matrix);
        r -= at.step * n * per_matrix;
        int32_t m, l;
        if (r < n * symmetric) {
            at.kind = r < n * p.tri ? GRAM : POLY;
            if (at.kind == POLY) r -= n * p.tri;
            m = r / p.tri;
            l = r - m * p.tri;
            if (at.kind == GRAM) {
                at.i = 0;
                for (int32_t w; l >= (w = row_tiles(p, at.i)); ++at.i) l -= w;
                at.j = l;
            } else {
                // column j starts in the panel that holds the diagonal
                at.j = 0;
                for (int32_t h; l >= (h = p.panels - panel_of(p, at.j)); ++at.j) l -= h;
                at.i = panel_of(p, at.j) + l;
            }
        } else {
            at.kind = APPLY;
            r -= n * symmetric;
            const int32_t per = p.panels * p.cols_x;
            m = r / per;
            l = r - m * per;
            at.i = l / p.cols_x;
            at.j = l - at.i * p.cols_x;
        }
        at.matrix = first + m;
        return at;
    }
    static __device__ __forceinline__ Tile tile(const Params& p, const Code& code) {
        const Place at = place(code);
        Tile ti{};
        const int32_t x = at.step & 1;
        ti.a_map = at.kind == GRAM ? X_ROWS + x : at.kind == POLY ? A_ROWS : B_ROWS;
        ti.b_map = at.kind == GRAM ? X_COLS + x : at.kind == POLY ? A_COLS : X_RIGHT + x;
        ti.b_mn = at.kind == APPLY;                // B·X: rows of X are K
        ti.a_row = at.i * 256;
        ti.width = at.kind == APPLY ? p.width_x : p.width_a;
        ti.b_row = at.j * ti.width;
        ti.batch = at.matrix;
        ti.steps = ((at.kind == GRAM ? p.ld_x : p.M) + pairs::BK - 1) / pairs::BK;
        return ti;
    }
    static __device__ __forceinline__ bool dirty(const Params&) { return false; }

    static __device__ __forceinline__ int32_t* counter(const Params& p, int32_t matrix, int32_t kind, int32_t panel) {
        return p.ready + (static_cast<int64_t>(matrix) * 3 + kind) * p.panels + panel;
    }
    // By a whole warp: returns when what the tile reads is complete (false: not in time).
    static __device__ __forceinline__ bool wait(const Params& p, const Code& code, volatile int* abort) {
        const Place at = place(code);
        if (at.kind == GRAM && at.step == 0) return true;
        const int lane = threadIdx.x & 31;
        const int32_t from = at.kind == GRAM ? APPLY : at.kind == POLY || !p.square ? GRAM : POLY;
        const int32_t q = lane == 0 || at.kind == APPLY ? at.i : panel_of(p, at.j);
        // both CTAs of every tile count, in every step so far
        const int32_t need = 2 * (at.kind == GRAM ? at.step * p.cols_x : (at.step + 1) * panel_tiles(p, q));
        bool ok = true;
        if (lane < 2) {
            const int32_t* c = counter(p, at.matrix, from, q);
            auto reached = [&] {
                int32_t v;
                asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(c) : "memory");
                return v >= need;
            };
            if (!reached()) {
                const uint64_t t0 = global_timer_ns();
                while (ok && !reached()) {
                    if (*abort) {
                        ok = false;
                    } else if (global_timer_ns() - t0 > pairs::WAIT_LIMIT_NS) {
                        *abort = 1;
                        ok = false;
                    }
                }
            }
        }
        ok = __all_sync(0xffffffffu, ok);
        __syncwarp();
        return ok;
    }
    // By one thread, which has waited for those that stored: this CTA's part of the tile is there, for TMA
    // loads and for the other SMs.  (One fence for both counters: two releases, 3 x 333 x 1001 107 us instead of 104.)
    static __device__ __forceinline__ void publish(const Params& p, const Code& code) {
        const Place at = place(code);
        if (at.kind == APPLY && at.step + 1 == p.steps) return;
        auto add_one = [&](int32_t panel) {
            asm volatile("red.relaxed.gpu.global.add.s32 [%0], 1;" ::"l"(counter(p, at.matrix, at.kind, panel)) : "memory");
        };
        asm volatile("fence.proxy.async.global;\n\tfence.acq_rel.gpu;" ::: "memory");
        add_one(at.i);
        const int32_t across = panel_of(p, at.j);
        if (at.kind != APPLY && across != at.i) add_one(across);
    }

    struct Finish {
        const Params& p;
        uint8_t* staging;
        int32_t row, odd, lane;
        Place at;
        int32_t tile_width;
        int32_t col0;                      // the tile's first column
        int32_t r0, rows;                  // the warp's first row, and how many of its 32 exist
        bool first, last, with_lo, store_lo;
        float rest;
        uint4 lo[4];                       // X's, asked for ahead of the tile

        __device__ __forceinline__ Finish(const Params& p_, uint8_t* staging_, int32_t row_, int odd_, int lane_)
            : p(p_), staging(staging_), row(row_), odd(odd_), lane(lane_) {}

        __device__ __forceinline__ int width_of() const { return tile_width; }
        __device__ __forceinline__ int32_t width() const { return at.kind == APPLY ? p.ld_x : p.ld_a; }
        __device__ __forceinline__ int64_t element(int c, int32_t ld) const {
            return (static_cast<int64_t>(at.matrix) * p.M + r0) * ld + col0 + c * 64;
        }
        __device__ __forceinline__ void ask(int c) {
            const int32_t cols = p.ld_lo - col0 - c * 64;
            if (with_lo && rows > 0 && cols > 0)
                load_bytes_64(lo, p.lo[at.step & 1] + element(c, p.ld_lo), p.ld_lo, lane, rows, cols);
        }
        __device__ __forceinline__ bool before(const Code& code) {
            at = place(code);
            tile_width = at.kind == APPLY ? p.width_x : p.width_a;
            col0 = at.j * tile_width;
            r0 = at.i * 256 + row;
            rows = p.M - r0;
            rows = rows > 32 ? 32 : rows;
            first = at.step == 0;
            last = at.step + 1 == p.steps;
            with_lo = at.kind == APPLY && !last && (!first || p.has_lo);
            store_lo = at.kind == APPLY && at.step + 2 < p.steps;          // the last step reads hi alone
            rest = first ? __ldg(p.rest + at.matrix) : 1.0f;
            ask(odd);
            return true;
        }
        __device__ __forceinline__ void pass(int c, uint32_t taddr) {
            const int32_t cols = width() - col0 - c * 64;
            if (rows <= 0 || cols <= 0) return;
            MOE_DCHECK(at.matrix < p.batch && at.i < p.panels && at.step < p.steps && r0 >= 0 && r0 < p.M && col0 >= 0,
                       p.status);
            if (at.kind == APPLY) {
                if (c != odd) ask(c);
                finish_x(c, taddr, cols);
            } else {
                finish_symmetric(c, taddr, cols);
            }
            __syncwarp();                          // (TMEM is read by whole warps)
        }
        // A or B: the sums, and on the diagonal what it takes to have B as (A + s)².
        __device__ __forceinline__ void finish_symmetric(int c, uint32_t taddr, int32_t cols) {
            const bool b_now = at.kind == POLY || !p.square;
            const float to_a = rest * rest * (1.0f / (X_SCALE * X_SCALE));       // GRAM: the sums as A's values
            const float unscale = 1.0f / (p.a_scale * p.a_scale);                // POLY: the sums as values
            const float scale = at.kind == POLY ? p.c * B_SCALE * unscale : b_now ? p.b * B_SCALE * to_a : p.a_scale * to_a;
            // does the diagonal pass through the warp's 32 rows and these 64 columns; which of mine is on it
            const int32_t on = r0 + lane - col0 - c * 64;
            const bool diagonal = static_cast<uint32_t>(r0 - col0 - c * 64) < 64u;
            float* d_at = p.diagonal + static_cast<int64_t>(at.matrix) * p.M + r0 + lane;
            const bool mine = diagonal && lane < rows;
            const float a_ii = mine && at.kind == POLY ? __ldcg(d_at) : 0.0f;
            uint4 el[8];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(taddr + hh * 32, v);
                tmem_ld_wait();
                float fixed = 0.0f;
                if (diagonal) {
                    // every lane's own diagonal element (of another half: unused)
                    float sum = 0.0f;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (hh * 32 + i == on) sum = __uint_as_float(v[i]);
                    const bool here = mine && (on >> 5) == hh;
                    if (at.kind == POLY) {
                        const float q = __half2float(__float2half_rn((a_ii + p.shift) * p.a_scale)) / p.a_scale;
                        const float s = q - a_ii;            // what the rounding made of the shift
                        fixed = (p.b * a_ii + p.c * (sum * unscale - 2.0f * s * a_ii - s * s) + p.a) * B_SCALE;
                    } else {
                        const float a = sum * to_a;
                        if (here && !b_now) *d_at = a;
                        fixed = b_now ? (p.b * a + p.a) * B_SCALE : (a + p.shift) * p.a_scale;
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float x = __uint_as_float(v[8 * k + 2 * j]) * scale;
                        float y = __uint_as_float(v[8 * k + 2 * j + 1]) * scale;
                        if (diagonal) {
                            if (hh * 32 + 8 * k + 2 * j == on) x = fixed;
                            if (hh * 32 + 8 * k + 2 * j + 1 == on) y = fixed;
                        }
                        w[j] = pack_16bit2<false>(x, y);
                    }
                    el[4 * hh + k] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            uint16_t* dst = b_now ? p.B : p.A;
            store_staged_64(el, staging, dst + element(c, p.ld_a), p.ld_a, lane, rows, cols);
            if (col0 + tile_width <= at.i * 256) {
                // the tile across the diagonal
                const int32_t n = col0 + c * 64;
                store_columns_64<false>(el, dst + (static_cast<int64_t>(at.matrix) * p.M + n) * p.ld_a + r0, p.ld_a, lane,
                                        p.ld_a - r0, p.M - n);
            }
        }
        // X, or the result: the sums (B has a on its diagonal) and a·lo.
        __device__ __forceinline__ void finish_x(int c, uint32_t taddr, int32_t cols) {
            const float scale = rest * (last ? 1.0f / (B_SCALE * X_SCALE) : 1.0f / B_SCALE);
            const float add = rest * p.a;
            if (with_lo) bytes_to_rows(lo, staging, lane);
            uint4 el[8];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(taddr + hh * 32, v);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t w[4], l[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float x = __uint_as_float(v[8 * k + 2 * j]) * scale;
                        float y = __uint_as_float(v[8 * k + 2 * j + 1]) * scale;
                        // columns 32 hh + 8 k + 2 j: bytes 8 k + 2 j of the half's 32
                        uint32_t& word = reinterpret_cast<uint32_t*>(&lo[2 * hh + (k >> 1)])[2 * (k & 1) + (j >> 1)];
                        if (with_lo) {
                            const float2 f = unpack_lo2((word >> (16 * (j & 1))) & 0xffffu);
                            x += add * f.x;
                            y += add * f.y;
                        }
                        w[j] = last ? pack_16bit2<true>(x, y) : pack_16bit2<false>(x, y);
                        if (store_lo) {
                            const float2 back = unpack_16bit2<false>(w[j]);
                            l[j] = pack_lo2(x - back.x, y - back.y);
                        }
                        if (store_lo && (j & 1)) word = l[j - 1] | l[j] << 16;
                    }
                    el[4 * hh + k] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            if (last) {
                store_result(el, c);
                return;
            }
            store_staged_64(el, staging, p.hi[(at.step + 1) & 1] + element(c, p.ld_x), p.ld_x, lane, rows, cols);
            if (store_lo)
                store_bytes_64(lo, staging, p.lo[(at.step + 1) & 1] + element(c, p.ld_lo), p.ld_lo, lane, rows,
                               p.ld_lo - col0 - c * 64);
        }
        // 64 columns of the warp's rows of the result [M, N], or [N, M] where it is tall.
        __device__ __forceinline__ void store_result(const uint4 (&el)[8], int c) {
            const int32_t n0 = col0 + c * 64;
            if (n0 >= p.N) return;
            uint16_t* out = p.out + static_cast<int64_t>(at.matrix) * p.M * p.N;
            if (!p.tall) {
                if ((p.N & 7) == 0) {
                    store_staged_64(el, staging, out + static_cast<int64_t>(r0) * p.N + n0, p.N, lane, rows, p.N - n0);
                    return;
                }
                stage_rows(el, staging, lane);
                for (int r = 0; r < rows; ++r) {
                    const uint32_t w = *reinterpret_cast<const uint32_t*>(staging + r * 128 + (((lane >> 2) ^ (r & 7)) * 16) + (lane & 3) * 4);
                    uint16_t* d = out + static_cast<int64_t>(r0 + r) * p.N + n0 + 2 * lane;
                    if (n0 + 2 * lane < p.N) d[0] = static_cast<uint16_t>(w);
                    if (n0 + 2 * lane + 1 < p.N) d[1] = static_cast<uint16_t>(w >> 16);
                }
                __syncwarp();
                return;
            }
            uint16_t* d = out + static_cast<int64_t>(n0) * p.M + r0;
            if ((p.M & 1) == 0) store_columns_64<false>(el, d, p.M, lane, p.M - r0, p.N - n0);
            else store_columns_64<true>(el, d, p.M, lane, p.M - r0, p.N - n0);
        }
    };
};

struct OrthoLayout {
    bool tall;
    int32_t M, N, ld_x, ld_a, ld_lo, sum_blocks;
    int64_t hi[2], lo[2], A, B, diagonal, sums, rest, ready, queue, bytes;
    int32_t panels;
};

OrthoLayout ortho_layout(int64_t batch, int32_t rows, int32_t cols) {
    OrthoLayout l;
    l.tall = rows > cols;
    l.M = l.tall ? cols : rows;
    l.N = l.tall ? rows : cols;
    l.ld_x = (l.N + 7) / 8 * 8;
    l.ld_a = (l.M + 7) / 8 * 8;
    l.ld_lo = (l.N + 15) / 16 * 16;
    // by the matrix alone, so that its norm is summed the same way in any stack
    const int64_t blocks = (static_cast<int64_t>(rows) * cols + SUM_VALUES - 1) / SUM_VALUES;
    l.sum_blocks = static_cast<int32_t>(blocks < MAX_SUM_BLOCKS ? blocks : MAX_SUM_BLOCKS);
    int64_t at = 0;
    auto take = [&at](int64_t n) {
        const int64_t r = at;
        at += (n + 255) / 256 * 256;
        return r;
    };
    const int64_t x = batch * l.M * l.ld_x * 2, a = batch * l.M * l.ld_a * 2;
    for (int i = 0; i < 2; ++i) {
        l.hi[i] = take(x);
        l.lo[i] = take(batch * l.M * l.ld_lo);
    }
    l.A = take(a);
    l.B = take(a);
    l.diagonal = take(batch * l.M * 4);
    l.sums = take(batch * l.sum_blocks * 4);
    l.rest = take(batch * 4);
    l.panels = (l.M + 255) / 256;
    l.ready = take(batch * 3 * l.panels * 4);
    l.queue = take(4);
    l.bytes = at;
    return l;
}

template <class Kernel>
cudaError_t launch_pdl(Kernel kernel, dim3 grid, int threads, cudaStream_t stream, const Prepare& p) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int DTYPE>
cudaError_t launch_prepare(const Prepare& p, int64_t batch, bool tall, cudaStream_t stream) {
    constexpr int PER = DTYPE == MOE_DTYPE_F32 ? 4 : 8;
    const dim3 sum_grid(static_cast<unsigned>(p.sum_blocks), static_cast<unsigned>(batch));
    cudaError_t err = p.elements % PER == 0
                          ? launch_pdl(square_sum_kernel<DTYPE, true>, sum_grid, SUM_THREADS, stream, p)
                          : launch_pdl(square_sum_kernel<DTYPE, false>, sum_grid, SUM_THREADS, stream, p);
    if (err != cudaSuccess) return err;
    // as many blocks as for the sums
    const bool rows8 = (tall ? p.M : p.N) % 8 == 0;
    if (tall)
        return rows8 ? launch_pdl(prepare_tall_kernel<DTYPE, true>, sum_grid, SUM_THREADS, stream, p)
                     : launch_pdl(prepare_tall_kernel<DTYPE, false>, sum_grid, SUM_THREADS, stream, p);
    return rows8 ? launch_pdl(prepare_kernel<DTYPE, true>, sum_grid, SUM_THREADS, stream, p)
                 : launch_pdl(prepare_kernel<DTYPE, false>, sum_grid, SUM_THREADS, stream, p);
}

// How wide the tiles are, by the time that a product should take.  As measured (us): a stage of 64 along
// K 0.2 for 256 x 128 tiles and 0.326 for 256 x 256 (both at the rate at which operands come from L2),
// a tile at least 4 and 5.5, its epilogue 2.5 and 6 where no other tile hides it.  One matrix's products
// wait for one another in whole rounds, a stack's overlap.  16 x 512 x 512 takes 125 us with
// narrow tiles and 207 with wide ones, 64 x 300 x 1000 415 and 350, 2048 x 7168 456 with narrow ones and
// 412 where X has wide ones.  Where A and X both want narrow ones they have a kernel of their own with
// eight stages instead of six.
struct Widths {
    int a, x;
};
Widths widths(const OrthoLayout& l, int64_t batch, int n_pairs) {
    auto time = [n_pairs, batch](int64_t tiles, int32_t k, bool wide) {
        const float mma = static_cast<float>(pairs::ceil_div(k, pairs::BK)) * (wide ? 0.326f : 0.2f);
        const float least = wide ? 5.5f : 4.0f, epilogue = wide ? 6.0f : 2.5f;
        float rounds = static_cast<float>(tiles) / static_cast<float>(n_pairs);
        if (batch == 1 || rounds < 1.0f) rounds = static_cast<float>((tiles + n_pairs - 1) / n_pairs);
        return rounds * (mma > least ? mma : least) + epilogue;
    };
    const int64_t narrow = pairs::ceil_div(l.M, 128);
    int64_t wide_a = 0, narrow_a = 0;
    for (int32_t q = 0; q < l.panels; ++q) {
        wide_a += q + 1;
        narrow_a += 2 * q + 2 < narrow ? 2 * q + 2 : narrow;
    }
    const int64_t wide_x = static_cast<int64_t>(l.panels) * pairs::ceil_div(l.ld_x, 256);
    const int64_t narrow_x = static_cast<int64_t>(l.panels) * pairs::ceil_div(l.ld_x, 128);
    const float a_wide = time(batch * wide_a, l.ld_x, true) + time(batch * wide_a, l.M, true);
    const float a_narrow = time(batch * narrow_a, l.ld_x, false) + time(batch * narrow_a, l.M, false);
    return Widths{a_narrow < 0.9f * a_wide ? 128 : 256,
                  time(batch * narrow_x, l.M, false) < time(batch * wide_x, l.M, true) ? 128 : 256};
}

template <int BN>
cudaError_t launch_products(const OrthoLayout& l, int64_t batch, const Widths& w, OrthoProducts& p, cudaStream_t stream) {
    using Op = OrthoOp<BN>;
    pairs::Maps maps;
    // rows with the columns up to their 16-byte boundary, which hold zeros
    auto map = [&](int i, const void* base, int32_t ld, int box_rows) {
        return pairs::map_3d(&maps.m[i], base, batch, l.M, ld, ld, box_rows);
    };
    for (int i = 0; i < 2; ++i)
        if (!map(X_ROWS + i, p.hi[i], l.ld_x, pairs::BM) || !map(X_COLS + i, p.hi[i], l.ld_x, w.a / 2) ||
            !map(X_RIGHT + i, p.hi[i], l.ld_x, pairs::BK))
            return cudaErrorInvalidValue;
    if (!map(A_ROWS, p.A, l.ld_a, pairs::BM) || !map(A_COLS, p.A, l.ld_a, w.a / 2) || !map(B_ROWS, p.B, l.ld_a, pairs::BM))
        return cudaErrorInvalidValue;
    const int n_pairs = pairs::resident_pairs<Op>();
    if (n_pairs == 0) return cudaErrorNoDevice;
    p.n_maps = MAPS;
    p.panels = l.panels;
    p.width_a = w.a;
    p.width_x = w.x;
    p.cols_a = pairs::ceil_div(l.M, w.a);
    p.cols_x = pairs::ceil_div(l.ld_x, w.x);
    p.tri = 0;
    for (int32_t q = 0; q < p.panels; ++q) {
        const int32_t n = (q + 1) * (256 / w.a);
        p.tri += n < p.cols_a ? n : p.cols_a;
    }
    // Groups of matrices with about twice as many tiles of A as there are pairs.  (64 x 1408 x 2048 in groups of
    // 4: 4.5 ms; 8: 3.8; 16: 3.8 to 4.0; 64: 4.1 to 4.2.)
    const int64_t tiles = batch * p.tri / (2 * n_pairs);
    const int64_t groups = tiles > 1 ? tiles : 1;
    p.group = static_cast<int32_t>((batch + groups - 1) / groups);
    p.total_tiles = static_cast<int32_t>(batch) * p.steps * ((1 + p.square) * p.tri + p.panels * p.cols_x);
    return pairs::launch<Op>(maps, p, stream);
}

}  // namespace

int64_t orthogonalize_workspace_bytes(int64_t batch, int32_t rows, int32_t cols) {
    return ortho_layout(batch, rows, cols).bytes;
}

cudaError_t launch_orthogonalize(const Orthogonalize& a, cudaStream_t stream) {
    if (orthogonalize_is_small(a.rows, a.cols)) {
        const cudaError_t err = launch_orthogonalize_small(a, stream);
        if (err != cudaErrorNotSupported) return err;
    }
    if (!tensor_map_encoder()) return cudaErrorNotSupported;
    const OrthoLayout l = ortho_layout(a.batch, a.rows, a.cols);
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    auto u16 = [ws](int64_t at) { return reinterpret_cast<uint16_t*>(ws + at); };
    const bool f32 = a.dtype == MOE_DTYPE_F32;
    Prepare pr{};
    pr.update = a.update;
    pr.elements = static_cast<int64_t>(a.rows) * a.cols;
    pr.M = l.M;
    pr.N = l.N;
    pr.ld = l.ld_x;
    pr.ld_lo = l.ld_lo;
    pr.sum_blocks = l.sum_blocks;
    pr.least_norm = a.least_norm;
    pr.sums = reinterpret_cast<float*>(ws + l.sums);
    pr.rest = reinterpret_cast<float*>(ws + l.rest);
    pr.hi = u16(l.hi[0]);
    pr.lo = f32 ? ws + l.lo[0] : nullptr;         // 16-bit values are hi by themselves
    pr.ready = reinterpret_cast<int32_t*>(ws + l.ready);
    pr.queue = reinterpret_cast<int32_t*>(ws + l.queue);
    pr.counters = 3 * l.panels;
    cudaError_t err = f32 ? launch_prepare<MOE_DTYPE_F32>(pr, a.batch, l.tall, stream)
                    : a.dtype == MOE_DTYPE_BF16 ? launch_prepare<MOE_DTYPE_BF16>(pr, a.batch, l.tall, stream)
                                                : launch_prepare<MOE_DTYPE_F16>(pr, a.batch, l.tall, stream);
    if (err != cudaSuccess) return err;
    OrthoProducts p{};
    p.status = a.status;
    p.queue = pr.queue;
    p.ready = pr.ready;
    p.batch = static_cast<int32_t>(a.batch);
    p.M = l.M;
    p.N = l.N;
    p.ld_x = l.ld_x;
    p.ld_a = l.ld_a;
    p.ld_lo = l.ld_lo;
    p.steps = a.steps;
    p.a = a.a;
    p.b = a.b;
    p.c = a.c;
    p.square = a.c != 0.0f ? 1 : 0;
    p.shift = p.square ? a.b / (2.0f * a.c) : 0.0f;
    // A + s is at most about 2^14 in fp16
    p.a_scale = MAX_A_SCALE;
    while (p.a_scale * fabsf(p.shift) > 16384.0f) p.a_scale *= 0.5f;
    p.has_lo = f32 ? 1 : 0;
    p.rest = pr.rest;
    for (int i = 0; i < 2; ++i) {
        p.hi[i] = u16(l.hi[i]);
        p.lo[i] = ws + l.lo[i];
    }
    p.diagonal = reinterpret_cast<float*>(ws + l.diagonal);
    p.A = u16(l.A);
    p.B = u16(l.B);
    p.out = a.out;
    p.tall = l.tall ? 1 : 0;
    const int n_pairs = pairs::resident_pairs<OrthoOp<256>>();
    if (n_pairs == 0) return cudaErrorNoDevice;
    const Widths w = widths(l, a.batch, n_pairs);
    return w.a == 128 && w.x == 128 ? launch_products<128>(l, a.batch, w, p, stream)
                                    : launch_products<256>(l, a.batch, w, p, stream);
}

}  // namespace moe
