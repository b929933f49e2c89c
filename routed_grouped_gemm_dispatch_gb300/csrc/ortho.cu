// Orthogonalised update: for each matrix G of a stack
//     X₀ = G / max(‖G‖, eps)   (Frobenius norm)
//     A = X·Xᵀ,  B = b·A + c·A²,  X ← a·X + B·X      `steps` times
// with X taken with the fewer rows (a tall G is transposed on the way in and out; the
// polynomial is the same from either side).  Three launches a step, each a list of 256-row
// tiles over the whole stack (pair_tiles.cuh); A and B are symmetric, so only the
// tiles on and below the diagonal are multiplied, and the others are stored from them.
//
// Numbers.  All operands are fp16 (11 bits at the rate of bf16's 8), times fixed powers of two
// that keep them normal: X·2^6, A·2^10, B·2^6; sums are fp32.  X₀ is G times a power of
// two, which is exact, and the rest of 1/‖G‖ enters the first step's fp32 sums.  Values whose
// norm grows past 2^9 in a step (coefficients that diverge) overflow.
//
// Rounding X to 11 bits adds noise in directions that a low-rank G does not have, and
// a·X multiplies it by a = 3.44 a step.  So that term takes X with 22 bits: as
// hi + lo·2^-11, two fp16 arrays (hi alone is the products' operand).  In 64-bit simulation
// with these roundings, the root mean square error of five steps relative to that of the result:
//                             Gaussian   rank M/4    rank 1
//     X as hi alone            1.3e-3     1.4e-2     3.2e-2
//     X as hi + lo             1.5e-3     1.3e-3     1.4e-3
//     all operands bf16        1.1e-2     1.4e-1     3.4e-1
// The last step adds `a` to B's diagonal instead: nothing amplifies its rounding any more, and
// it spares the tile of X.  The result is rounded to bf16 (1.7e-3 by itself).
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

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
constexpr float A_SCALE = 1024.0f;
constexpr float B_SCALE = 64.0f;
constexpr float LO_SCALE = 2048.0f;         // lo = (x - hi)·2^11
constexpr int SUM_THREADS = 256;
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

struct Prepare {
    const void* update;
    int64_t elements;             // of a matrix
    int32_t M, N, ld;             // X is [M, ld], N of the columns in use
    int32_t sum_blocks;
    float eps;
    float* sums;                  // [batch, sum_blocks]
    float* rest;                  // [batch]: what X₀ still has to be times
    uint16_t* hi;                 // [batch, M, ld]
    uint16_t* lo;                 // nullable
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
#pragma unroll 4
        for (int64_t i = first; i < p.elements / PER; i += step) {
            float v[PER];
            values_of<DTYPE>(__ldg(reinterpret_cast<const uint4*>(base) + i), v);
#pragma unroll
            for (int j = 0; j < PER; ++j) sum += v[j] * v[j];
        }
    } else {
#pragma unroll 4
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

// X₀ up to the factor `rest`, in tiles of 64 rows x 64 columns of X.
template <int DTYPE, bool TALL>
__global__ void __launch_bounds__(256) prepare_kernel(const Prepare p) {
    __shared__ float tile[64][65];
    __shared__ float part[8];
    __shared__ float power;
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int64_t matrix = blockIdx.z;
    float sum = 0.0f;
    for (int i = threadIdx.x; i < p.sum_blocks; i += 256) sum += p.sums[matrix * p.sum_blocks + i];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 8; ++w) sum += part[w];
        float norm = sqrtf(sum);
        if (norm < p.eps) norm = p.eps;                       // a NaN stays
        float two_e = 0.0f, rest = 0.0f;
        if (norm != 0.0f) {
            int e = 0;
            rest = __int_as_float(0x7fffffff);                // infinite (or NaN): so is the result, NaN
            if (norm <= 3.4e38f) rest = 1.0f / frexpf(norm, &e);   // norm = f·2^e, f in [0.5, 1)
            two_e = ldexpf(1.0f, X_EXPONENT - e);
        }
        power = two_e;
        if (blockIdx.x == 0 && blockIdx.y == 0) p.rest[matrix] = rest;
    }
    const int32_t m0 = static_cast<int32_t>(blockIdx.y) * 64, n0 = static_cast<int32_t>(blockIdx.x) * 64;
    const int32_t rows = TALL ? p.N : p.M, cols = TALL ? p.M : p.N;
    const int32_t r0 = TALL ? n0 : m0, c0 = TALL ? m0 : n0;
    constexpr int BYTES = DTYPE == MOE_DTYPE_F32 ? 4 : 2;
    const uint8_t* base = static_cast<const uint8_t*>(p.update) + matrix * p.elements * BYTES;
    for (int i = threadIdx.x; i < 64 * 64; i += 256) {
        const int r = i >> 6, c = i & 63;
        float v = 0.0f;
        if (r0 + r < rows && c0 + c < cols) v = value_at<DTYPE>(base, static_cast<int64_t>(r0 + r) * cols + c0 + c);
        if (TALL) tile[c][r] = v;
        else tile[r][c] = v;
    }
    __syncthreads();
    const float s = power;
    for (int i = threadIdx.x; i < 64 * 8; i += 256) {
        const int r = i >> 3, c = (i & 7) * 8;
        if (m0 + r >= p.M || n0 + c >= p.ld) continue;
        uint32_t h[4], l[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float x = tile[r][c + 2 * j] * s, y = tile[r][c + 2 * j + 1] * s;
            h[j] = pack_16bit2<false>(x, y);
            const float2 back = unpack_16bit2<false>(h[j]);
            l[j] = pack_16bit2<false>((x - back.x) * LO_SCALE, (y - back.y) * LO_SCALE);
        }
        const int64_t at = (matrix * p.M + m0 + r) * p.ld + n0 + c;
        *reinterpret_cast<uint4*>(p.hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
        if (p.lo) *reinterpret_cast<uint4*>(p.lo + at) = make_uint4(l[0], l[1], l[2], l[3]);
    }
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------

enum Kind { GRAM = 0, POLY = 1, APPLY = 2 };

struct OrthoProducts {
    int32_t total_tiles, n_maps;
    int32_t* status;
    int32_t M, N;                 // X [M, N]
    int32_t ld_x, ld_a;           // elements between rows of X; of A and B
    int32_t tiles;                // of a matrix
    int32_t n_tiles;              // APPLY: tile columns
    int32_t steps;                // K steps of a tile
    float scale;                  // of the sums
    float add;                    // POLY: of A; APPLY: of X
    float diagonal;               // POLY: added on the diagonal
    const float* rest;            // per matrix, first step: GRAM times its square, APPLY times it (nullable)
    const uint16_t* in_hi;        // POLY: A; APPLY: X (nullable)
    const uint16_t* in_lo;        // APPLY: nullable
    uint16_t* dst;                // A, B, X's hi, or the result
    uint16_t* dst_lo;             // APPLY: nullable
    int32_t final_step;           // APPLY: dst is the result, in bf16
    int32_t tall;                 // ... transposed
};

// Tile l of the ones on and below the diagonal, row by row.
__device__ __forceinline__ void triangle(int32_t l, int32_t& i, int32_t& j) {
    i = static_cast<int32_t>((sqrtf(8.0f * static_cast<float>(l) + 1.0f) - 1.0f) * 0.5f);
    while (i * (i + 1) / 2 > l) --i;
    while ((i + 1) * (i + 2) / 2 <= l) ++i;
    j = l - i * (i + 1) / 2;
}

// The transpose of a warp's 32 rows x 64 columns (el: a row per lane), through its 4 KB of staging:
// afterwards piece k of lane 4c + q is rows 8q .. 8q + 7 of column 8k + c.
__device__ __forceinline__ void transpose_32x64(const uint4 (&el)[8], uint4 (&out)[8], uint8_t* buf, int lane) {
    stage_rows(el, buf, lane);
    uint32_t even[16], odd[16];                  // columns 2·lane and 2·lane + 1
#pragma unroll
    for (int r = 0; r < 32; r += 2) {
        const uint32_t x = *reinterpret_cast<const uint32_t*>(buf + r * 128 + (((lane >> 2) ^ (r & 7)) * 16) + (lane & 3) * 4);
        const uint32_t y =
            *reinterpret_cast<const uint32_t*>(buf + (r + 1) * 128 + (((lane >> 2) ^ ((r + 1) & 7)) * 16) + (lane & 3) * 4);
        even[r / 2] = __byte_perm(x, y, 0x5410);
        odd[r / 2] = __byte_perm(x, y, 0x7632);
    }
    __syncwarp();
    // lane's two columns are 128 contiguous bytes; its pieces permuted against bank conflicts
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        *reinterpret_cast<uint4*>(buf + lane * 128 + ((k ^ (lane & 7)) * 16)) =
            make_uint4(even[4 * k], even[4 * k + 1], even[4 * k + 2], even[4 * k + 3]);
        *reinterpret_cast<uint4*>(buf + lane * 128 + (((k + 4) ^ (lane & 7)) * 16)) =
            make_uint4(odd[4 * k], odd[4 * k + 1], odd[4 * k + 2], odd[4 * k + 3]);
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int col = 8 * k + (lane >> 2), q = lane & 3;
        const int owner = col >> 1;
        out[k] = *reinterpret_cast<const uint4*>(buf + owner * 128 + (((q + 4 * (col & 1)) ^ (owner & 7)) * 16));
    }
    __syncwarp();
}

template <int KIND>
struct OrthoOp {
    static constexpr int BN = 256;
    static constexpr bool BF16 = false;
    static constexpr bool MASKABLE = false;
    using Params = OrthoProducts;
    enum { LEFT, RIGHT, MAPS };

    struct Place {
        int32_t matrix, row, col;          // of the tile in its matrix
    };
    static __device__ __forceinline__ Place place(const Params& p, int32_t t) {
        Place at;
        at.matrix = t / p.tiles;
        const int32_t l = t - at.matrix * p.tiles;
        int32_t i, j;
        if (KIND == APPLY) {
            i = l / p.n_tiles;
            j = l - i * p.n_tiles;
        } else {
            triangle(l, i, j);
        }
        at.row = i * 256;
        at.col = j * BN;
        return at;
    }
    static __device__ __forceinline__ Tile tile(const Params& p, int32_t t) {
        const Place at = place(p, t);
        Tile ti{};
        ti.a_map = LEFT;
        ti.b_map = RIGHT;
        ti.b_mn = KIND == APPLY;           // B·X: rows of X are K
        ti.a_row = at.row;
        ti.b_row = at.col;
        ti.batch = at.matrix;
        ti.steps = p.steps;
        return ti;
    }
    static __device__ __forceinline__ bool dirty(const Params&) { return false; }

    struct Finish {
        const Params& p;
        uint8_t* staging;
        int32_t row, odd, lane;
        Place at;
        int32_t r0, rows;                  // the warp's first row, and how many of its 32 exist
        float scale, add;
        uint4 hi[KIND == GRAM ? 1 : 8], lo[KIND == APPLY ? 8 : 1];   // asked for ahead of the tile

        __device__ __forceinline__ Finish(const Params& p_, uint8_t* staging_, int32_t row_, int odd_, int lane_)
            : p(p_), staging(staging_), row(row_), odd(odd_), lane(lane_) {}

        __device__ __forceinline__ int32_t width() const { return KIND == APPLY ? p.ld_x : p.ld_a; }
        __device__ __forceinline__ int64_t element(int c) const {
            return (static_cast<int64_t>(at.matrix) * p.M + r0) * width() + at.col + c * 64;
        }
        __device__ __forceinline__ void ask(int c) {
            if constexpr (KIND != GRAM) {
                const int32_t cols = width() - at.col - c * 64;
                if (rows <= 0 || cols <= 0) return;
                if (p.in_hi) load_lines_64(hi, p.in_hi + element(c), width(), lane, rows, cols);
                if constexpr (KIND == APPLY)
                    if (p.in_lo) load_lines_64(lo, p.in_lo + element(c), width(), lane, rows, cols);
            }
        }
        __device__ __forceinline__ bool before(int32_t t) {
            at = place(p, t);
            r0 = at.row + row;
            rows = p.M - r0;
            rows = rows > 32 ? 32 : rows;
            scale = p.scale;
            add = p.add;
            if (p.rest) {
                const float f = __ldg(p.rest + at.matrix);
                scale *= KIND == GRAM ? f * f : f;
                add *= f;
            }
            ask(odd);
            return true;
        }
        __device__ __forceinline__ void pass(int c, uint32_t taddr) {
            const int32_t cols = width() - at.col - c * 64;
            if (rows <= 0 || cols <= 0) return;
            MOE_DCHECK(at.row >= 0 && r0 < p.M && at.col + c * 64 < width() &&
                           (static_cast<int64_t>(at.matrix) + 1) * p.tiles <= p.total_tiles,
                       p.status);
            if constexpr (KIND != GRAM) {
                if (c != odd) ask(c);
                if (p.in_hi) lines_to_rows(hi, staging, lane);
                if constexpr (KIND == APPLY)
                    if (p.in_lo) lines_to_rows(lo, staging, lane);
            }
            const bool bf16 = KIND == APPLY && p.final_step;
            uint4 el[8], rest[KIND == APPLY ? 8 : 1];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(taddr + hh * 32, v);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t w[4], wl[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float x = __uint_as_float(v[8 * k + 2 * j]) * scale;
                        float y = __uint_as_float(v[8 * k + 2 * j + 1]) * scale;
                        if constexpr (KIND != GRAM) {
                            if (p.in_hi) {
                                const uint32_t hw = reinterpret_cast<const uint32_t*>(&hi[4 * hh + k])[j];
                                float2 f = unpack_16bit2<false>(hw);
                                if constexpr (KIND == APPLY) {
                                    if (p.in_lo) {
                                        const float2 g = unpack_16bit2<false>(reinterpret_cast<const uint32_t*>(&lo[4 * hh + k])[j]);
                                        f.x += g.x * (1.0f / LO_SCALE);
                                        f.y += g.y * (1.0f / LO_SCALE);
                                    }
                                }
                                x += add * f.x;
                                y += add * f.y;
                            }
                        }
                        if constexpr (KIND == POLY) {
                            const int32_t col = at.col + c * 64 + hh * 32 + 8 * k + 2 * j;
                            if (col == r0 + lane) x += p.diagonal;
                            if (col + 1 == r0 + lane) y += p.diagonal;
                        }
                        w[j] = bf16 ? pack_16bit2<true>(x, y) : pack_16bit2<false>(x, y);
                        if constexpr (KIND == APPLY) {
                            if (p.dst_lo) {
                                const float2 back = unpack_16bit2<false>(w[j]);
                                wl[j] = pack_16bit2<false>((x - back.x) * LO_SCALE, (y - back.y) * LO_SCALE);
                            }
                        }
                    }
                    el[4 * hh + k] = make_uint4(w[0], w[1], w[2], w[3]);
                    if constexpr (KIND == APPLY)
                        if (p.dst_lo) rest[4 * hh + k] = make_uint4(wl[0], wl[1], wl[2], wl[3]);
                }
            }
            if (KIND == APPLY && p.final_step) {
                store_result(el, c);
                return;
            }
            store_staged_64(el, staging, p.dst + element(c), width(), lane, rows, cols);
            if constexpr (KIND == APPLY)
                if (p.dst_lo) store_staged_64(rest, staging, p.dst_lo + element(c), width(), lane, rows, cols);
            if constexpr (KIND != APPLY) {
                if (at.col + BN <= at.row) {
                    // the tile across the diagonal
                    uint4 tr[8];
                    transpose_32x64(el, tr, staging, lane);
                    const int32_t m = r0 + (lane & 3) * 8;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int32_t n = at.col + c * 64 + 8 * k + (lane >> 2);
                        if (n < p.M && m < p.ld_a)
                            *reinterpret_cast<uint4*>(p.dst + (static_cast<int64_t>(at.matrix) * p.M + n) * p.ld_a + m) = tr[k];
                    }
                }
            }
        }
        // 64 columns of the warp's rows of the result [M, N], or [N, M] where it is tall.
        __device__ __forceinline__ void store_result(const uint4 (&el)[8], int c) {
            const int32_t n0 = at.col + c * 64;
            if (n0 >= p.N) return;
            uint16_t* out = p.dst + static_cast<int64_t>(at.matrix) * p.M * p.N;
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
            uint4 tr[8];
            transpose_32x64(el, tr, staging, lane);
            const int32_t m = r0 + (lane & 3) * 8;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int32_t n = n0 + 8 * k + (lane >> 2);
                if (n >= p.N || m >= p.M) continue;
                uint16_t* d = out + static_cast<int64_t>(n) * p.M + m;
                if ((p.M & 7) == 0) {
                    *reinterpret_cast<uint4*>(d) = tr[k];
                } else {
                    const uint32_t w[4] = {tr[k].x, tr[k].y, tr[k].z, tr[k].w};
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (m + j < p.M) d[j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
                }
            }
        }
    };
};

struct OrthoLayout {
    bool tall;
    int32_t M, N, ld_x, ld_a, sum_blocks;
    int64_t hi[2], lo[2], A, B, sums, rest, bytes;
};

OrthoLayout ortho_layout(int64_t batch, int32_t rows, int32_t cols) {
    OrthoLayout l;
    l.tall = rows > cols;
    l.M = l.tall ? cols : rows;
    l.N = l.tall ? rows : cols;
    l.ld_x = (l.N + 7) / 8 * 8;
    l.ld_a = (l.M + 7) / 8 * 8;
    const int64_t blocks = (static_cast<int64_t>(rows) * cols + SUM_THREADS * 64 - 1) / (SUM_THREADS * 64);
    l.sum_blocks = static_cast<int32_t>(blocks > MAX_SUM_BLOCKS ? MAX_SUM_BLOCKS : blocks);
    int64_t at = 0;
    auto take = [&at](int64_t n) {
        const int64_t r = at;
        at += (n + 255) / 256 * 256;
        return r;
    };
    const int64_t x = batch * l.M * l.ld_x * 2, a = batch * l.M * l.ld_a * 2;
    for (int i = 0; i < 2; ++i) {
        l.hi[i] = take(x);
        l.lo[i] = take(x);
    }
    l.A = take(a);
    l.B = take(a);
    l.sums = take(batch * l.sum_blocks * 4);
    l.rest = take(batch * 4);
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
    const dim3 grid(static_cast<unsigned>((p.ld + 63) / 64), static_cast<unsigned>((p.M + 63) / 64),
                    static_cast<unsigned>(batch));
    return tall ? launch_pdl(prepare_kernel<DTYPE, true>, grid, 256, stream, p)
                : launch_pdl(prepare_kernel<DTYPE, false>, grid, 256, stream, p);
}

template <int KIND>
cudaError_t launch_product(const void* left, const void* right, const OrthoLayout& l, int64_t batch, OrthoProducts p,
                           cudaStream_t stream) {
    using Op = OrthoOp<KIND>;
    pairs::Maps maps;
    const int32_t ld_left = KIND == GRAM ? l.ld_x : l.ld_a, ld_right = KIND == POLY ? l.ld_a : l.ld_x;
    // rows and their lengths in memory: columns up to the 16-byte boundary hold zeros
    if (!pairs::map_3d(&maps.m[Op::LEFT], left, batch, l.M, ld_left, ld_left, pairs::BM) ||
        !pairs::map_3d(&maps.m[Op::RIGHT], right, batch, l.M, ld_right, ld_right, KIND == APPLY ? pairs::BK : Op::BN / 2))
        return cudaErrorInvalidValue;
    const int32_t m_tiles = pairs::ceil_div(l.M, 256);
    p.n_maps = Op::MAPS;
    p.M = l.M;
    p.N = l.N;
    p.ld_x = l.ld_x;
    p.ld_a = l.ld_a;
    p.n_tiles = pairs::ceil_div(l.ld_x, Op::BN);
    p.tiles = KIND == APPLY ? m_tiles * p.n_tiles : m_tiles * (m_tiles + 1) / 2;
    p.total_tiles = static_cast<int32_t>(batch) * p.tiles;
    p.steps = pairs::ceil_div(KIND == GRAM ? l.ld_x : l.M, pairs::BK);
    return pairs::launch<Op>(maps, p, stream);
}

}  // namespace

int64_t orthogonalize_workspace_bytes(int64_t batch, int32_t rows, int32_t cols) {
    return ortho_layout(batch, rows, cols).bytes;
}

cudaError_t launch_orthogonalize(const Orthogonalize& a, cudaStream_t stream) {
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
    pr.sum_blocks = l.sum_blocks;
    pr.eps = a.eps;
    pr.sums = reinterpret_cast<float*>(ws + l.sums);
    pr.rest = reinterpret_cast<float*>(ws + l.rest);
    pr.hi = u16(l.hi[0]);
    pr.lo = f32 ? u16(l.lo[0]) : nullptr;         // 16-bit values are hi by themselves
    cudaError_t err = f32 ? launch_prepare<MOE_DTYPE_F32>(pr, a.batch, l.tall, stream)
                    : a.dtype == MOE_DTYPE_BF16 ? launch_prepare<MOE_DTYPE_BF16>(pr, a.batch, l.tall, stream)
                                                : launch_prepare<MOE_DTYPE_F16>(pr, a.batch, l.tall, stream);
    if (err != cudaSuccess) return err;
    for (int32_t k = 0; k < a.steps; ++k) {
        const bool last = k + 1 == a.steps;
        uint16_t* hi = u16(l.hi[k & 1]);
        OrthoProducts g{};
        g.status = a.status;
        g.scale = A_SCALE / (X_SCALE * X_SCALE);
        g.rest = k == 0 ? pr.rest : nullptr;
        g.dst = u16(l.A);
        if ((err = launch_product<GRAM>(hi, hi, l, a.batch, g, stream)) != cudaSuccess) return err;
        OrthoProducts q{};
        q.status = a.status;
        q.scale = a.c * B_SCALE / (A_SCALE * A_SCALE);
        q.add = a.b * B_SCALE / A_SCALE;
        q.diagonal = last ? a.a * B_SCALE : 0.0f;
        q.in_hi = u16(l.A);
        q.dst = u16(l.B);
        if ((err = launch_product<POLY>(u16(l.A), u16(l.A), l, a.batch, q, stream)) != cudaSuccess) return err;
        OrthoProducts x{};
        x.status = a.status;
        x.scale = last ? 1.0f / (B_SCALE * X_SCALE) : 1.0f / B_SCALE;
        x.rest = k == 0 ? pr.rest : nullptr;
        if (last) {
            x.final_step = 1;
            x.tall = l.tall ? 1 : 0;
            x.dst = a.out;
        } else {
            x.add = a.a;
            x.in_hi = hi;
            x.in_lo = k > 0 || f32 ? u16(l.lo[k & 1]) : nullptr;
            x.dst = u16(l.hi[(k + 1) & 1]);
            x.dst_lo = k + 2 < a.steps ? u16(l.lo[(k + 1) & 1]) : nullptr;
        }
        if ((err = launch_product<APPLY>(u16(l.B), hi, l, a.batch, x, stream)) != cudaSuccess) return err;
    }
    return cudaSuccess;
}

}  // namespace moe
