// Orthogonalised updates of matrices with at most 128 rows or columns (a router's weights, an
// adapter's), each by one cluster in one launch: see ortho.cu for the iteration.
//
// With so few rows the products take next to no time, and passing A, B and X through L2
// between them costs 4 to 8 us a product.  Here X, [M, N] with M <= 128, stays on chip: a cluster of C CTAs
// has N / C of its columns each, as the fp16 operand hi·2^6 in shared memory and, times a, in fp32
// in TMEM, where B·hi is added to it.  A step is
//     each CTA's part of X·Xᵀ (its columns are K), rows of it to the CTA that adds them up,
//     rows of A from there to all CTAs,                    two exchanges of the cluster
//     A², B = b·A + c·A² in every CTA, a·X + B·X of its columns.
// The same bytes are a K-major operand for X·Xᵀ and an M/N-major one for B·X.
//
// 64 x 2048 takes 32.4 us, 6 a step, against 100 of the tiles in L2.  Bound: the chain of
// three products, two exchanges and three passes over registers, with one warp's latency
// in each (the tensor pipe is busy for 0.7% of it).  Roundings: X as an operand (fp16) and the result (bf16); a·X is fp32, and A and B are each the
// sum of two fp16 matrices: with few rows there are few singular values, whose errors do not
// average out, and a single B was most of it (20 x 2000: 2.4e-3 of the result, with two terms of A and B
// 0.8e-3; the result's rounding by itself is 1.7e-3).
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "../../include/moe_gb300.h"
#include "moe_internal.h"
#include "sm103_products.cuh"
#include "tile_store.cuh"
#include "train_internal.h"

namespace moe {
namespace {

constexpr int ROWS = 128;
constexpr int THREADS = 256;                  // a row of TMEM per thread, columns halved between warps w and w + 4
// Columns of X per CTA at most: beside A's (64 or 128) in 512 columns of TMEM.
__host__ __device__ constexpr int a_columns(int M) { return M <= 64 ? 64 : 128; }
__host__ __device__ constexpr int max_columns(int M) { return 512 - a_columns(M); }
constexpr int MAX_CLUSTER = 16;
constexpr float X_SCALE = 64.0f;              // operands times powers of two, as in ortho.cu
constexpr float A_SCALE = 1024.0f;
constexpr float B_SCALE = 64.0f;
constexpr int BOX_BYTES = ROWS * 128;         // 64 columns of 128 rows, 128-byte swizzle
constexpr uint64_t WAIT_LIMIT_NS = 2000000000ull;
constexpr uint64_t DRAIN_LIMIT_NS = 200000000ull;
// All that an SM has, whatever is used of it: no other CTA that wants TMEM may be beside this one, as
// two clusters that hold it on one SM each and wait for it on the other would wait for ever.
constexpr int SMEM_BYTES = 225 * 1024;
// X, two terms of A, and the parts of A's rows on their way.
constexpr int shared_bytes(int M, int cols) {
    return 1024 + cols / 64 * BOX_BYTES + 2 * a_columns(M) / 64 * BOX_BYTES + ROWS * a_columns(M) * 4;
}

constexpr int TMEM_A = 0, TMEM_COLS = 512;

static_assert(shared_bytes(64, max_columns(64)) <= SMEM_BYTES && shared_bytes(128, max_columns(128)) <= SMEM_BYTES,
              "the widest parts fit");

struct Small {
    const void* update;
    int64_t batch;
    int32_t M, N;                 // of X
    int32_t cols;                 // a CTA's columns, a multiple of 64
    int32_t steps;
    float a, b, c, least_norm;
    int32_t tall;                 // update is [N, M]
    uint16_t* out;
    int32_t* status;
};

__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
          "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
          "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
          "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void store_cluster4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Byte offset of the 16-byte piece that holds columns col .. col + 7 (a multiple of 8) of a row.
__device__ __forceinline__ uint32_t piece_at(int row, int col) {
    return static_cast<uint32_t>((col >> 6) * BOX_BYTES + row * 128 + ((((col >> 3) & 7) ^ (row & 7)) * 16));
}

// Two values as the sum of two fp16 pairs: their rounding, and that of what it left.
__device__ __forceinline__ void two_terms(float x, float y, uint32_t& hi, uint32_t& lo) {
    hi = pack_16bit2<false>(x, y);
    const float2 f = unpack_16bit2<false>(hi);
    lo = pack_16bit2<false>(x - f.x, y - f.y);
}

template <int DTYPE>
__device__ __forceinline__ float value_at(const void* base, int64_t i) {
    if (DTYPE == MOE_DTYPE_F32) return __ldg(static_cast<const float*>(base) + i);
    const uint16_t v = __ldg(static_cast<const uint16_t*>(base) + i);
    if (DTYPE == MOE_DTYPE_BF16) return __uint_as_float(static_cast<uint32_t>(v) << 16);
    return __half2float(__ushort_as_half(v));
}

template <int DTYPE>
__global__ void __launch_bounds__(THREADS, 1) ortho_small_kernel(const Small p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem =
        reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ uint64_t bar_mem;
    __shared__ uint32_t tmem_mem;
    __shared__ int abort_mem;
    __shared__ float part[THREADS / 32];
    __shared__ float sums[MAX_CLUSTER];
    const int an = a_columns(p.M);                        // A's rows and columns that there is room for
    const int x_bytes = p.cols / 64 * BOX_BYTES, a_bytes = an / 64 * BOX_BYTES;
    const uint32_t TMEM_X = static_cast<uint32_t>(an);
    uint8_t* xs = smem;                                   // hi
    uint8_t* as = smem + x_bytes;                         // A, then B: its rounding, and what that left
    uint8_t* ex = as + 2 * a_bytes;                       // [C][an / C][an] fp32: parts of this CTA's rows of A
    const uint32_t bar = smem_u32(&bar_mem);
    volatile int* abort_flag = &abort_mem;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    uint32_t C;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(C));
    const uint32_t rank = cluster_cta_rank();
    const int64_t matrix = blockIdx.x / C;
    const int row = (warp & 3) * 32 + lane, half = warp >> 2;
    const int own = an / static_cast<int>(C);             // rows of A that a CTA adds up

    if (tid == 0) {
        mbar_init(bar, 1);
        abort_mem = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(&tmem_mem), TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    cluster_arrive_relaxed();      // this CTA runs; the others may write into its shared memory
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_mem, 0);
    const uint32_t taddr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);

    // ---- X₀: this CTA's columns, and the norm of all of them
    const int64_t elements = static_cast<int64_t>(p.M) * p.N;
    const void* g = static_cast<const uint8_t*>(p.update) + matrix * elements * (DTYPE == MOE_DTYPE_F32 ? 4 : 2);
    const int c0 = static_cast<int>(rank) * p.cols;
    const int n_cols = p.N - c0 < 0 ? 0 : (p.N - c0 < p.cols ? p.N - c0 : p.cols);
    // read once: the values as they are wait in TMEM for the norm
    const bool whole = !p.tall && (p.N & 7) == 0;         // rows of whole 16-byte pieces
    float sum = 0.0f;
    for (int col = half * 32; col < p.cols; col += 64) {
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = 0.0f;
        if (row < p.M && col < n_cols) {
            if (whole) {
                const int64_t first = static_cast<int64_t>(row) * p.N + c0 + col;
                constexpr int PER = DTYPE == MOE_DTYPE_F32 ? 4 : 8;
#pragma unroll
                for (int k = 0; k < 32 / PER; ++k) {
                    if (col + k * PER >= n_cols) break;
                    const uint4 w = __ldg(reinterpret_cast<const uint4*>(
                        static_cast<const uint8_t*>(g) + (first + k * PER) * (DTYPE == MOE_DTYPE_F32 ? 4 : 2)));
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if constexpr (DTYPE == MOE_DTYPE_F32) {
                            v[4 * k + j] = __uint_as_float(u[j]);
                        } else {
                            const float2 f = unpack_16bit2<DTYPE == MOE_DTYPE_BF16>(u[j]);
                            v[8 * k + 2 * j] = f.x;
                            v[8 * k + 2 * j + 1] = f.y;
                        }
                    }
                }
            } else {
                // (tall: lanes have neighbouring values)
                const int64_t first = p.tall ? static_cast<int64_t>(c0 + col) * p.M + row : static_cast<int64_t>(row) * p.N + c0 + col;
                const int64_t step = p.tall ? p.M : 1;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (col + i < n_cols) v[i] = value_at<DTYPE>(g, first + i * step);
            }
        }
        uint32_t t[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            sum += v[i] * v[i];
            t[i] = __float_as_uint(v[i]);
        }
        tmem_st_32x32b_x32(taddr + TMEM_X + col, t);
    }
    tmem_st_wait();
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    cluster_wait_acquire();        // all CTAs of the cluster run (asked for ahead of the loads of X)
    if (tid < static_cast<int>(C)) {
        sum = 0.0f;
        for (int w = 0; w < THREADS / 32; ++w) sum += part[w];
        const uint32_t to = mapa_shared(smem_u32(&sums[rank]), static_cast<uint32_t>(tid));
        asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(to), "r"(__float_as_uint(sum)) : "memory");
    }
    __syncwarp();
    cluster_sync_all();
    sum = 0.0f;
    for (uint32_t i = 0; i < C; ++i) sum += sums[i];
    float norm = sqrtf(sum);
    if (norm < p.least_norm) norm = p.least_norm;         // a NaN stays
    float to_x = X_SCALE / norm;                          // times a value: X₀·2^6 (at most 2^75)
    if (!(norm <= 3.4e38f)) to_x = __int_as_float(0x7fffffff);
    // a chunk of 32 columns: the operand to shared memory, and a times it (as the sums of B·hi come: times
    // B_SCALE) to TMEM
    // (For the last step a times the operand itself: nothing multiplies its rounding any more, and it then
    // enters both terms, whose slopes near 1 have opposite signs.)
    auto keep = [&](int col, const float (&v)[32], bool for_last) {
        uint32_t t[32];
        MOE_DCHECK(col >= 0 && col + 32 <= p.cols && p.cols <= max_columns(p.M) && matrix < p.batch, p.status);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = pack_16bit2<false>(v[8 * k + 2 * j], v[8 * k + 2 * j + 1]);
            *reinterpret_cast<uint4*>(xs + piece_at(row, col + 8 * k)) = make_uint4(w[0], w[1], w[2], w[3]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = for_last ? unpack_16bit2<false>(w[j]) : make_float2(v[8 * k + 2 * j], v[8 * k + 2 * j + 1]);
                t[8 * k + 2 * j] = __float_as_uint(f.x * (p.a * B_SCALE));
                t[8 * k + 2 * j + 1] = __float_as_uint(f.y * (p.a * B_SCALE));
            }
        }
        tmem_st_32x32b_x32(taddr + TMEM_X + col, t);
    };
    for (int col = half * 32; col < p.cols; col += 64) {
        uint32_t t[32];
        tmem_ld_32x32b_x32(taddr + TMEM_X + col, t);
        tmem_ld_wait();
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(t[i]) * to_x;
        keep(col, v, p.steps == 1);
    }

    // rows of A that no CTA owns stay zero (the products take 128)
    if (an < ROWS)
        for (int i = tid; i < 2 * (ROWS - an) * 8; i += THREADS) {
            const int r = an + (i >> 3) % (ROWS - an), term = (i >> 3) / (ROWS - an);
            *reinterpret_cast<uint4*>(as + term * a_bytes + r * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
    uint32_t phase = 0;
    // The MMAs that thread 0 has issued are done.
    auto finished = [&]() {
        if (!mbar_wait_bounded(bar, phase, abort_flag, WAIT_LIMIT_NS)) abort_mem = 1;
        phase ^= 1u;
        __syncwarp();
        tc_fence_after_sync();
    };
    // Shared memory and TMEM that threads wrote are operands from here on.
    auto hand_over = [&]() {
        tmem_st_wait();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_before_sync();
        __syncthreads();
        tc_fence_after_sync();
    };
    const uint32_t xb = smem_u32(xs), ab = smem_u32(as);
    const int m16 = (p.M + 15) / 16 * 16;                 // K and N of products over rows
    const uint32_t n_a = m16 < 32 ? 32u : static_cast<uint32_t>(m16);
    for (int step = 0; step < p.steps; ++step) {
        hand_over();
        // ---- this CTA's part of X·Xᵀ
        if (tid == 0) {
            const uint32_t idesc = idesc_16bit_f32acc(ROWS, n_a, false, false, false);
            for (int k = 0; k < p.cols / 16; ++k) {
                const uint64_t d = smem_desc_k_sw128(xb + (k >> 2) * BOX_BYTES) + (k & 3) * 2;
                tc_mma_f16(tmem + TMEM_A, d, d, idesc, k > 0 ? 1u : 0u);
            }
            tc_commit(bar);
        }
        __syncwarp();
        finished();
        // ---- its rows to the CTAs that add them up
        {
            const uint32_t owner = row < an ? static_cast<uint32_t>(row / own) : 0u;
            MOE_DCHECK(owner < C && static_cast<int>(rank) * own + row % own < an, p.status);
            const uint32_t to = mapa_shared(smem_u32(ex), owner) +
                                4u * static_cast<uint32_t>((static_cast<int>(rank) * own + row % own) * an);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int col = half * 32 + c * 64;
                if (col >= static_cast<int>(n_a)) break;
                uint32_t v[32];
                tmem_ld_32x32b_x32(taddr + TMEM_A + col, v);
                tmem_ld_wait();
                if (row < p.M) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        store_cluster4(to + 4u * (col + 4 * i), v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                }
            }
        }
        __syncwarp();
        cluster_sync_all();
        // ---- this CTA's rows of A, in rank order, to all CTAs
        const int per_row = an == 64 ? 3 : 4;              // log2 of a row's pieces
        for (int i = tid; i < own << per_row; i += THREADS) {
            const int r = i >> per_row, col = (i & ((1 << per_row) - 1)) * 8;
            const int m = static_cast<int>(rank) * own + r;
            MOE_DCHECK(m < an && piece_at(m, col) + 16 <= static_cast<uint32_t>(a_bytes), p.status);
            float s[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] = 0.0f;
            if (m < p.M && col < static_cast<int>(n_a)) {
                for (uint32_t q = 0; q < C; ++q) {
                    const float4* src = reinterpret_cast<const float4*>(ex + 4 * ((static_cast<int>(q) * own + r) * an + col));
                    const float4 lo = src[0], hi = src[1];
                    s[0] += lo.x;
                    s[1] += lo.y;
                    s[2] += lo.z;
                    s[3] += lo.w;
                    s[4] += hi.x;
                    s[5] += hi.y;
                    s[6] += hi.z;
                    s[7] += hi.w;
                }
            }
            uint32_t w[4], l[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                constexpr float F = A_SCALE / (X_SCALE * X_SCALE);
                two_terms(s[2 * j] * F, s[2 * j + 1] * F, w[j], l[j]);
            }
            const uint32_t off = smem_u32(as) + piece_at(m, col);
            for (uint32_t q = 0; q < C; ++q) {
                const uint32_t to = mapa_shared(off, (rank + q) % C);
                store_cluster4(to, w[0], w[1], w[2], w[3]);
                store_cluster4(to + a_bytes, l[0], l[1], l[2], l[3]);
            }
        }
        __syncwarp();
        cluster_sync_all();
        hand_over();
        // ---- A²
        if (tid == 0) {
            const uint32_t idesc = idesc_16bit_f32acc(ROWS, n_a, false, false, false);
            for (int k = 0; k < m16 / 16; ++k) {
                const uint64_t hi = smem_desc_k_sw128(ab + (k >> 2) * BOX_BYTES) + (k & 3) * 2;
                const uint64_t lo = smem_desc_k_sw128(ab + a_bytes + (k >> 2) * BOX_BYTES) + (k & 3) * 2;
                tc_mma_f16(tmem + TMEM_A, hi, hi, idesc, k > 0 ? 1u : 0u);
                tc_mma_f16(tmem + TMEM_A, hi, lo, idesc, 1u);
                tc_mma_f16(tmem + TMEM_A, lo, hi, idesc, 1u);
            }
            tc_commit(bar);
        }
        __syncwarp();
        finished();
        // ---- B, in A's place (its reads are done)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int col = half * 32 + c * 64;
            if (col >= static_cast<int>(n_a)) break;
            uint32_t v[32];
            tmem_ld_32x32b_x32(taddr + TMEM_A + col, v);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint4* piece = reinterpret_cast<uint4*>(as + piece_at(row, col + 8 * k));
                uint4* rest = reinterpret_cast<uint4*>(as + a_bytes + piece_at(row, col + 8 * k));
                const uint4 old = *piece, old_rest = *rest;
                const uint32_t ow[4] = {old.x, old.y, old.z, old.w};
                const uint32_t ol[4] = {old_rest.x, old_rest.y, old_rest.z, old_rest.w};
                uint32_t w[4], l[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = unpack_16bit2<false>(ow[j]), e = unpack_16bit2<false>(ol[j]);
                    const float sq = p.c * (B_SCALE / (A_SCALE * A_SCALE)), lin = p.b * (B_SCALE / A_SCALE);
                    two_terms(lin * (f.x + e.x) + sq * __uint_as_float(v[8 * k + 2 * j]),
                              lin * (f.y + e.y) + sq * __uint_as_float(v[8 * k + 2 * j + 1]), w[j], l[j]);
                }
                *piece = make_uint4(w[0], w[1], w[2], w[3]);
                *rest = make_uint4(l[0], l[1], l[2], l[3]);
            }
        }
        hand_over();
        // ---- a·X + B·X, 64 columns at a time
        if (tid == 0) {
            const uint32_t idesc = idesc_16bit_f32acc(ROWS, 64, false, false, true);
            for (int box = 0; box < p.cols / 64; ++box)
                for (int k = 0; k < m16 / 16; ++k) {
                    const uint64_t x = smem_desc_mn_sw128(xb + box * BOX_BYTES, BOX_BYTES) + k * (2048 >> 4);
#pragma unroll
                    for (int term = 0; term < 2; ++term)
                        tc_mma_f16(tmem + TMEM_X + box * 64,
                                   smem_desc_k_sw128(ab + term * a_bytes + (k >> 2) * BOX_BYTES) + (k & 3) * 2, x, idesc, 1u);
                }
            tc_commit(bar);
        }
        __syncwarp();
        finished();
        const bool last = step + 1 == p.steps;
        for (int col = half * 32; col < p.cols; col += 64) {
            uint32_t t[32];
            tmem_ld_32x32b_x32(taddr + TMEM_X + col, t);
            tmem_ld_wait();
            float v[32];
            const float f = last ? 1.0f / (B_SCALE * X_SCALE) : 1.0f / B_SCALE;
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(t[i]) * f;
            if (!last) {
                keep(col, v, step + 2 == p.steps);
            } else if (row < p.M) {
                uint16_t* out = p.out + matrix * elements;
                if (p.tall) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (col + i < n_cols)
                            out[static_cast<int64_t>(c0 + col + i) * p.M + row] =
                                static_cast<uint16_t>(pack_16bit2<true>(v[i], 0.0f) & 0xffffu);
                } else if ((p.N & 7) == 0) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) w[j] = pack_16bit2<true>(v[8 * k + 2 * j], v[8 * k + 2 * j + 1]);
                        if (col + 8 * k < n_cols)
                            *reinterpret_cast<uint4*>(out + static_cast<int64_t>(row) * p.N + c0 + col + 8 * k) =
                                make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (col + i < n_cols)
                            out[static_cast<int64_t>(row) * p.N + c0 + col + i] =
                                static_cast<uint16_t>(pack_16bit2<true>(v[i], 0.0f) & 0xffffu);
                }
            }
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (tid == 0 && abort_mem) {
        // MMAs still in flight end before their TMEM is given back
        volatile int never = 0;
        mbar_wait_bounded(bar, phase ^ 1u, &never, DRAIN_LIMIT_NS);
    }
    __syncwarp();
    cluster_sync_all();
    if (tid == 0 && abort_mem && p.status) atomicOr(p.status, MOE_DEV_TIMEOUT);
    if (warp == 0) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// Clusters of `size` CTAs (a power of two) that fit on the device at once (0: none), asked once per
// device and size.
template <int DTYPE>
int resident_clusters(int size) {
    struct Entry {
        std::once_flag once;
        int clusters = 0;
    };
    constexpr int MAX_DEVICES = 16;
    static Entry table[MAX_DEVICES][MAX_CLUSTER];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= MAX_DEVICES || size > MAX_CLUSTER) return 0;
    Entry& r = table[dev][size - 1];
    std::call_once(r.once, [&r, size] {
        if (cudaFuncSetAttribute(ortho_small_kernel<DTYPE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 SMEM_BYTES) == cudaSuccess &&
            cudaFuncSetAttribute(ortho_small_kernel<DTYPE>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
                cudaSuccess) {
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = static_cast<unsigned>(size);
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(static_cast<unsigned>(size));
            cfg.blockDim = dim3(THREADS);
            cfg.dynamicSmemBytes = SMEM_BYTES;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, ortho_small_kernel<DTYPE>, &cfg) == cudaSuccess) r.clusters = n;
        }
        cudaGetLastError();
    });
    return r.clusters;
}

int32_t columns_of(int32_t N, int cluster) { return ((N + cluster - 1) / cluster + 63) / 64 * 64; }

template <int DTYPE>
cudaError_t launch_small(const Orthogonalize& o, cudaStream_t stream) {
    const bool tall = o.rows > o.cols;
    const int32_t M = tall ? o.cols : o.rows, N = tall ? o.rows : o.cols;
    // The fewest CTAs that hold X; then more of them while each still gets 64 columns and all
    // matrices of the stack run at once.
    int cluster = 1;
    while (cluster < MAX_CLUSTER && columns_of(N, cluster) > max_columns(M)) cluster *= 2;
    while (cluster < MAX_CLUSTER && columns_of(N, cluster) > 64 &&
           o.batch <= resident_clusters<DTYPE>(2 * cluster))
        cluster *= 2;
    if (columns_of(N, cluster) > max_columns(M) || resident_clusters<DTYPE>(cluster) == 0)
        return cudaErrorNotSupported;
    Small p{};
    p.update = o.update;
    p.batch = o.batch;
    p.M = M;
    p.N = N;
    p.cols = columns_of(N, cluster);
    p.steps = o.steps;
    p.a = o.a;
    p.b = o.b;
    p.c = o.c;
    p.least_norm = o.least_norm;
    p.tall = tall ? 1 : 0;
    p.out = o.out;
    p.status = o.status;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(o.batch * cluster));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, ortho_small_kernel<DTYPE>, p);
}

}  // namespace

bool orthogonalize_is_small(int32_t rows, int32_t cols) {
    const int32_t M = rows < cols ? rows : cols, N = rows < cols ? cols : rows;
    return M <= ROWS && N <= MAX_CLUSTER * max_columns(M);
}

cudaError_t launch_orthogonalize_small(const Orthogonalize& o, cudaStream_t stream) {
    return o.dtype == MOE_DTYPE_F32    ? launch_small<MOE_DTYPE_F32>(o, stream)
           : o.dtype == MOE_DTYPE_BF16 ? launch_small<MOE_DTYPE_BF16>(o, stream)
                                       : launch_small<MOE_DTYPE_F16>(o, stream);
}

}  // namespace moe
