// Matrix products of the dense gated feed-forward block and of its gradients.
//
// Forward, x [T, H], gate_w / up_w [I, H], down_w [H, I], all of one 16-bit type:
//     G = x·gate_wᵀ, U = x·up_wᵀ (fp32), h = G·sigmoid(G)·U      first launch
//     y = h·down_wᵀ                                              second launch
// Backward, from d_y and the stored G, U, h, with s = sigmoid(G):
//     d_h = d_y·down_w (fp32), d_U = d_h·G·s, d_G = d_h·U·s·(1 + G·(1 − s))   first launch
//     d_x = d_G·gate_w + d_U·up_w;  d_gate_w = d_Gᵀ·x;  d_up_w = d_Uᵀ·x;
//     d_down_w = d_yᵀ·h                                          second launch
//
// One kernel serves them all: C[m, n] = Σ_k A[m, k]·B[n, k] over up to four
// problems a launch, each with its own extents, operands and order of operands:
// an operand is K-major (K contiguous: x, h, d_y, d_G as A; the forward's
// weights as B) or M/N-major (M or N contiguous: the transposed ones), which
// the tensor cores read from shared memory as TMA leaves it, so nothing is ever
// transposed in memory.  d_x sums over two K segments (gate, then up) in one
// accumulator, and the four products of the backward's second half share one
// launch, so that its last wave is one and not four.
//
//  * Persistent clusters of two CTAs, one 2-SM MMA tile of M = 256 x N = 256 at
//    a time: each CTA holds 128 rows of A and 128 of B per stage (K = 128, 64 KB,
//    ring of three), warp 0 feeds the ring by TMA, warp 1 of the even CTA issues
//    the MMAs into one of two TMEM accumulators, and warps 2-5 of both CTAs turn
//    the other one into 16-bit rows meanwhile.  With 128 x 256 tiles on one SM
//    the operands' way into and out of shared memory, not the tensor core, is
//    the bound; the pair halves the bytes of B each SM moves.
//  * Rows past T, columns past H or I and the end of K are zeros that TMA fills
//    in: no size needs padding, only whole 16-byte rows (H and I multiples of 8).
//  * First forward launch: a tile is 128 columns of gate (held by the even CTA)
//    and the same 128 of up (the odd one), so both projections and h come from
//    one pass over x, and h is formed in registers from the fp32 accumulators.
//  * First backward launch: d_h stays in TMEM; the epilogue reads G and U of the
//    tile and writes d_G and d_U.
//
// Roundings to 16 bits: h, y and every gradient once from fp32; G and U when the
// caller stores them for the backward (half the bytes of fp32 and the type the
// backward's products need); d_G and d_U, which are operands of products.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <map>
#include <mutex>

#include "../../include/moe_gb300.h"
#include "ffn_internal.h"
#include "moe_internal.h"
#include "sm103_ptx.cuh"
#include "tensor_map.h"
#include "tile_store.cuh"

namespace moe {
namespace {

constexpr int BM = 128;                        // rows of A (and of B) per CTA
constexpr int BN = 256;                        // columns of a tile
constexpr int BK = 128;                        // K per stage
constexpr int STAGES = 3;
constexpr int OP_BYTES = BM * BK * 2;          // one operand's stage: two boxes of 16 KB
constexpr int BOX_BYTES = OP_BYTES / 2;
constexpr int STAGE_BYTES = 2 * OP_BYTES;
constexpr int TMEM_COLS = 2 * BN;
constexpr int NUM_THREADS = 192;
constexpr int NUM_EPI_THREADS = 128;
constexpr int CLUSTER = 2;
constexpr uint16_t CLUSTER_MASK = 0x3;
constexpr int GROUP_M = 8;                     // tile rows (of 256) that are walked together
constexpr uint64_t WAIT_LIMIT_NS = 2000000000ull;
constexpr uint64_t DRAIN_LIMIT_NS = 200000000ull;

constexpr int OFF_BARS = STAGES * STAGE_BYTES;
constexpr int NUM_BARS = 2 * STAGES + 2 + 2 + 1;   // full, empty, tfull, tempty, drain
constexpr int OFF_TMEM_SLOT = OFF_BARS + NUM_BARS * 8;
constexpr int OFF_ABORT = OFF_TMEM_SLOT + 4;
constexpr int SMEM_BYTES = 1024 + OFF_ABORT + 4;

constexpr int MAX_MAPS = 10;
constexpr int MAX_PROBLEMS = 4;

enum Epilogue { EPI_STORE = 0, EPI_GATE_UP = 1, EPI_GRAD = 2 };

struct Maps {
    CUtensorMap m[MAX_MAPS];
};

struct Problem {
    uint16_t* dst;                 // C [m, n]
    int64_t m;
    int32_t n;
    int32_t m_tiles, n_tiles;
    int32_t first_tile;
    int32_t steps[2];              // stages along K of the two K segments
    int8_t a_map[2];               // per segment
    int8_t b_map[2][2];            // per segment and CTA of the pair
    int8_t a_mn, b_mn;             // operand is M/N-major
};

struct Plan {
    Problem pr[MAX_PROBLEMS];
    int32_t n_problems;
    int32_t total_tiles;
    int32_t tile_cols;             // output columns of a tile: 128 (gate and up side by side) or 256
    const uint16_t* gate_in;       // EPI_GRAD: stored G, U [m, n]
    const uint16_t* up_in;
    uint16_t* dst_gate;            // EPI_GRAD: d_G, d_U; EPI_GATE_UP: G, U when stored (nullable)
    uint16_t* dst_up;
    int32_t* status;
};

struct Tile {
    int32_t q, m, n;
};

// Tiles of a problem run in groups of GROUP_M tile rows, column by column inside
// a group: concurrent clusters then work on a near-square patch of C and share
// both operands' slices in L2.
__device__ __forceinline__ Tile tile_at(const Plan& p, int32_t t) {
    Tile ti;
    ti.q = 0;
#pragma unroll
    for (int i = 1; i < MAX_PROBLEMS; ++i)
        if (i < p.n_problems && t >= p.pr[i].first_tile) ti.q = i;
    const Problem& pr = p.pr[ti.q];
    const int32_t l = t - pr.first_tile;
    const int32_t per_group = GROUP_M * pr.n_tiles;
    const int32_t g = l / per_group;
    const int32_t r = l - g * per_group;
    const int32_t left = pr.m_tiles - g * GROUP_M;
    const int32_t gs = left < GROUP_M ? left : GROUP_M;
    ti.n = r / gs;
    ti.m = g * GROUP_M + (r - ti.n * gs);
    return ti;
}

template <int EPI, bool BF16>
__global__ void __launch_bounds__(NUM_THREADS, 1)
ffn_gemm_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Plan p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem =
        reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar_full = sbase + OFF_BARS;                  // [STAGES] (used in the even CTA)
    const uint32_t bar_empty = bar_full + 8 * STAGES;            // [STAGES]
    const uint32_t bar_tfull = bar_empty + 8 * STAGES;           // [2]
    const uint32_t bar_tempty = bar_tfull + 16;                  // [2] (used in the even CTA)
    const uint32_t bar_drain = bar_tempty + 16;                  // [1]
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + OFF_TMEM_SLOT);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_ABORT);

    const int tid = threadIdx.x;
    const int warp = tid >> 5;
    const int lane = tid & 31;
    const uint32_t rank = cluster_cta_rank();
    const bool leader = rank == 0;

    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar_full + 8 * s, 1);           // the even CTA's arrive.expect_tx
            mbar_init(bar_empty + 8 * s, 1);          // the MMAs' commit, multicast to both CTAs
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(bar_tfull + 8 * a, 1);
            mbar_init(bar_tempty + 8 * a, CLUSTER * NUM_EPI_THREADS);
        }
        mbar_init(bar_drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(sbase + OFF_TMEM_SLOT, TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    // Everything above overlaps the kernel before; every global access is below.
    // The next kernel may start only now that this CTA holds its TMEM.
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const uint32_t tmem_base = *tmem_slot;
    cluster_sync_all();            // both CTAs' barriers exist before copies and commits cross

    const int32_t cluster_id = static_cast<int32_t>(blockIdx.x) / CLUSTER;
    const int32_t n_clusters = static_cast<int32_t>(gridDim.x) / CLUSTER;

    if (warp == 0) {
        // ===================== TMA producer (both CTAs) =====================
        if (lane == 0) {
            const uint64_t policy = l2_policy_evict_normal();
            const uint32_t leader_full = mapa_shared(bar_full, 0);
            uint32_t stage = 0, phase = 0;
            int64_t issued = 0;
            bool ok = true;
            for (int32_t t = cluster_id; t < p.total_tiles && ok; t += n_clusters) {
                const Tile ti = tile_at(p, t);
                const Problem& pr = p.pr[ti.q];
                const int32_t arow = ti.m * 2 * BM + static_cast<int32_t>(rank) * BM;
                // gate and up side by side: both CTAs take the same 128 columns, of different weights
                const int32_t brow = EPI == EPI_GATE_UP ? ti.n * BM : ti.n * BN + static_cast<int32_t>(rank) * BM;
                for (int seg = 0; seg < 2 && ok; ++seg) {
                    const CUtensorMap* am = &maps.m[pr.a_map[seg]];
                    const CUtensorMap* bm = &maps.m[pr.b_map[seg][rank]];
                    for (int32_t kb = 0; kb < pr.steps[seg]; ++kb) {
                        if (!mbar_wait_bounded(bar_empty + 8 * stage, phase ^ 1u, abort_flag, WAIT_LIMIT_NS)) {
                            ok = false;
                            break;
                        }
                        const uint32_t fb = leader_full + 8 * stage;
                        const uint32_t sa = sbase + stage * STAGE_BYTES;
                        const uint32_t sb = sa + OP_BYTES;
                        const int32_t k0 = kb * BK;
                        if (leader) mbar_arrive_expect_tx(bar_full + 8 * stage, CLUSTER * STAGE_BYTES);
                        // K-major: two boxes of 64 along K x 128 rows; M/N-major:
                        // two boxes of 64 along M/N x 128 rows of K
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            if (pr.a_mn) tma_load_2d_pair(sa + b * BOX_BYTES, am, fb, arow + b * 64, k0, policy);
                            else tma_load_2d_pair(sa + b * BOX_BYTES, am, fb, k0 + b * 64, arow, policy);
                            if (pr.b_mn) tma_load_2d_pair(sb + b * BOX_BYTES, bm, fb, brow + b * 64, k0, policy);
                            else tma_load_2d_pair(sb + b * BOX_BYTES, bm, fb, k0 + b * 64, brow, policy);
                        }
                        ++issued;
                        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                    }
                }
            }
            if (!ok) {
                // Let the copies already in flight land before the CTA exits.
                volatile int never = 0;
                if (leader) {
                    const int64_t n = issued < STAGES ? issued : STAGES;
                    for (int64_t i = 0; i < n; ++i) {
                        const int64_t idx = issued - 1 - i;
                        mbar_wait_bounded(bar_full + 8 * static_cast<uint32_t>(idx % STAGES),
                                          static_cast<uint32_t>((idx / STAGES) & 1), &never, DRAIN_LIMIT_NS);
                    }
                } else {
                    // the odd CTA's copies report to the even CTA's barriers
                    const uint64_t t0 = global_timer_ns();
                    while (global_timer_ns() - t0 < 1000000ull) { }
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ===================== MMA issuer (even CTA only) =====================
        if (lane == 0 && leader) {
            uint32_t stage = 0, phase = 0, acc = 0, aphase = 0;
            bool ok = true;
            for (int32_t t = cluster_id; t < p.total_tiles && ok; t += n_clusters) {
                if (!mbar_wait_bounded(bar_tempty + 8 * acc, aphase ^ 1u, abort_flag, WAIT_LIMIT_NS)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const Problem& pr = p.pr[tile_at(p, t).q];
                const uint32_t d_tmem = tmem_base + acc * BN;
                const bool a_mn = pr.a_mn != 0, b_mn = pr.b_mn != 0;
                const uint32_t idesc = idesc_16bit_f32acc(2 * BM, BN, BF16, a_mn, b_mn);
                const int32_t steps = pr.steps[0] + pr.steps[1];
                for (int32_t kb = 0; kb < steps; ++kb) {
                    if (!mbar_wait_bounded(bar_full + 8 * stage, phase, abort_flag, WAIT_LIMIT_NS)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint32_t sa = sbase + stage * STAGE_BYTES;
                    const uint32_t sb = sa + OP_BYTES;
                    const uint64_t da = a_mn ? smem_desc_mn_sw128(sa, BOX_BYTES) : smem_desc_k_sw128(sa);
                    const uint64_t db = b_mn ? smem_desc_mn_sw128(sb, BOX_BYTES) : smem_desc_k_sw128(sb);
#pragma unroll
                    for (int kk = 0; kk < BK / 16; ++kk) {
                        // a K = 16 slice further, in 16-byte units: M/N-major 16 rows of
                        // 128 bytes; K-major 32 bytes inside a box of four slices
                        constexpr int MN_STEP = 2048 >> 4;
                        const int k_off = (kk / 4) * (BOX_BYTES >> 4) + (kk % 4) * (32 >> 4);
                        tc_mma_f16_pair(d_tmem, da + (a_mn ? kk * MN_STEP : k_off), db + (b_mn ? kk * MN_STEP : k_off),
                                        idesc, (kb | kk) != 0 ? 1u : 0u);
                    }
                    tc_commit_pair_mc(bar_empty + 8 * stage, CLUSTER_MASK);
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
                if (!ok) break;
                tc_commit_pair_mc(bar_tfull + 8 * acc, CLUSTER_MASK);
                acc ^= 1u;
                if (acc == 0) aphase ^= 1u;
            }
            // Every MMA this thread issued has finished once this arrives.
            volatile int never = 0;
            tc_commit_pair(bar_drain);
            mbar_wait_bounded(bar_drain, 0, &never, DRAIN_LIMIT_NS);
        }
        __syncwarp();
    } else {
        // ===================== epilogue (warps 2..5, both CTAs) =====================
        const int quarter = warp & 3;                // TMEM lanes 32*quarter .. +31
        const uint32_t leader_tempty = mapa_shared(bar_tempty, 0);
        uint32_t acc = 0, aphase = 0;
        for (int32_t t = cluster_id; t < p.total_tiles; t += n_clusters) {
            const Tile ti = tile_at(p, t);
            const Problem& pr = p.pr[ti.q];
            const int64_t row0 = static_cast<int64_t>(ti.m) * (2 * BM) + static_cast<int64_t>(rank) * BM + quarter * 32;
            const int64_t left = pr.m - row0;
            const int32_t rows = left > 32 ? 32 : (left < 0 ? 0 : static_cast<int32_t>(left));
            const int32_t col0 = ti.n * p.tile_cols;
            const int64_t at = row0 * pr.n + col0;
            if (!mbar_wait_bounded(bar_tfull + 8 * acc, aphase, abort_flag, WAIT_LIMIT_NS)) break;
            tc_fence_after_sync();
            const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * BN;
            const int passes = rows > 0 ? (EPI == EPI_GATE_UP ? 2 : 4) : 0;    // of 64 output columns
#pragma unroll 1
            for (int c = 0; c < passes; ++c) {
                const int32_t cols = pr.n - col0 - c * 64;                      // columns left
                if (cols <= 0) break;
                if (EPI == EPI_STORE) {
                    uint4 el[8];
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        uint32_t v[32];
                        tmem_ld_32x32b_x32(taddr + c * 64 + hh * 32, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t w[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                w[j] = pack_16bit2<BF16>(__uint_as_float(v[8 * k + 2 * j]),
                                                         __uint_as_float(v[8 * k + 2 * j + 1]));
                            el[4 * hh + k] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                    store_rows_64(el, pr.dst + at + c * 64, pr.n, lane, rows, cols);
                } else if (EPI == EPI_GATE_UP) {
                    uint4 eh[8], eg[8], eu[8];
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        uint32_t g[32], u[32];
                        tmem_ld_32x32b_x32(taddr + c * 64 + hh * 32, g);
                        tmem_ld_32x32b_x32(taddr + 128 + c * 64 + hh * 32, u);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t w[4], wg[4], wu[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float g0 = __uint_as_float(g[8 * k + 2 * j]);
                                const float g1 = __uint_as_float(g[8 * k + 2 * j + 1]);
                                const float u0 = __uint_as_float(u[8 * k + 2 * j]);
                                const float u1 = __uint_as_float(u[8 * k + 2 * j + 1]);
                                w[j] = pack_16bit2<BF16>(__fdividef(g0, 1.0f + __expf(-g0)) * u0,
                                                         __fdividef(g1, 1.0f + __expf(-g1)) * u1);
                                wg[j] = pack_16bit2<BF16>(g0, g1);
                                wu[j] = pack_16bit2<BF16>(u0, u1);
                            }
                            eh[4 * hh + k] = make_uint4(w[0], w[1], w[2], w[3]);
                            eg[4 * hh + k] = make_uint4(wg[0], wg[1], wg[2], wg[3]);
                            eu[4 * hh + k] = make_uint4(wu[0], wu[1], wu[2], wu[3]);
                        }
                    }
                    store_rows_64(eh, pr.dst + at + c * 64, pr.n, lane, rows, cols);
                    if (p.dst_gate != nullptr) {
                        store_rows_64(eg, p.dst_gate + at + c * 64, pr.n, lane, rows, cols);
                        store_rows_64(eu, p.dst_up + at + c * 64, pr.n, lane, rows, cols);
                    }
                } else {
                    // eg and eu hold G and U, then d_G and d_U
                    uint4 eg[8], eu[8];
                    load_rows_64(eg, p.gate_in + at + c * 64, pr.n, lane, rows, cols);
                    load_rows_64(eu, p.up_in + at + c * 64, pr.n, lane, rows, cols);
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        uint32_t d[32];
                        tmem_ld_32x32b_x32(taddr + c * 64 + hh * 32, d);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t* pg = reinterpret_cast<uint32_t*>(&eg[4 * hh + k]);
                            uint32_t* pu = reinterpret_cast<uint32_t*>(&eu[4 * hh + k]);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float2 g = unpack_16bit2<BF16>(pg[j]);
                                const float2 u = unpack_16bit2<BF16>(pu[j]);
                                const float d0 = __uint_as_float(d[8 * k + 2 * j]);
                                const float d1 = __uint_as_float(d[8 * k + 2 * j + 1]);
                                const float s0 = __fdividef(1.0f, 1.0f + __expf(-g.x));
                                const float s1 = __fdividef(1.0f, 1.0f + __expf(-g.y));
                                pg[j] = pack_16bit2<BF16>(d0 * u.x * s0 * (1.0f + g.x * (1.0f - s0)),
                                                          d1 * u.y * s1 * (1.0f + g.y * (1.0f - s1)));
                                pu[j] = pack_16bit2<BF16>(d0 * g.x * s0, d1 * g.y * s1);
                            }
                        }
                    }
                    store_rows_64(eg, p.dst_gate + at + c * 64, pr.n, lane, rows, cols);
                    store_rows_64(eu, p.dst_up + at + c * 64, pr.n, lane, rows, cols);
                }
            }
            tc_fence_before_sync();
            // the accumulator may be reused once both CTAs have read their rows
            if (leader) mbar_arrive(bar_tempty + 8 * acc);
            else mbar_arrive_cluster(leader_tempty + 8 * acc);
            acc ^= 1u;
            if (acc == 0) aphase ^= 1u;
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    // Neither CTA leaves (or frees the pair's TMEM) while the other may still
    // write into its shared memory, arrive on its barriers or use the TMEM.
    cluster_sync_all();
    if (*abort_flag && tid == 0 && p.status) atomicOr(p.status, MOE_DEV_TIMEOUT);
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem_base, TMEM_COLS);
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// Clusters of two that fit on the device at once, after opting in to the
// kernel's shared memory (once per device and kernel).
template <int EPI, bool BF16>
cudaError_t resident_clusters(int* n) {
    static std::mutex mu;
    static std::map<int, int> cache;
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    std::lock_guard<std::mutex> lock(mu);
    auto it = cache.find(dev);
    if (it != cache.end()) {
        *n = it->second;
        return cudaSuccess;
    }
    err = cudaFuncSetAttribute(ffn_gemm_kernel<EPI, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (err != cudaSuccess) return err;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CLUSTER;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(CLUSTER * 64);
    cfg.blockDim = dim3(NUM_THREADS);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaOccupancyMaxActiveClusters(n, ffn_gemm_kernel<EPI, BF16>, &cfg);
    if (err != cudaSuccess) return err;
    if (*n <= 0) return cudaErrorNoDevice;
    cache[dev] = *n;
    return cudaSuccess;
}

template <int EPI, bool BF16>
cudaError_t launch(const Maps& maps, const Plan& p, cudaStream_t stream) {
    int nc = 0;
    cudaError_t err = resident_clusters<EPI, BF16>(&nc);
    if (err != cudaSuccess) return err;
    if (nc > p.total_tiles) nc = p.total_tiles;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CLUSTER;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(CLUSTER * nc));
    cfg.blockDim = dim3(NUM_THREADS);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, ffn_gemm_kernel<EPI, BF16>, maps, p);
}

template <int EPI>
cudaError_t launch(bool bf16, const Maps& maps, const Plan& p, cudaStream_t stream) {
    return bf16 ? launch<EPI, true>(maps, p, stream) : launch<EPI, false>(maps, p, stream);
}

int32_t ceil_div(int64_t a, int64_t b) { return static_cast<int32_t>((a + b - 1) / b); }

// Appends a problem; `cols` are the output columns of one tile.
Problem& add_problem(Plan& p, uint16_t* dst, int64_t m, int32_t n, int32_t cols) {
    Problem& pr = p.pr[p.n_problems++];
    pr.dst = dst;
    pr.m = m;
    pr.n = n;
    pr.m_tiles = ceil_div(m, 2 * BM);
    pr.n_tiles = ceil_div(n, cols);
    pr.first_tile = p.total_tiles;
    p.tile_cols = cols;
    p.total_tiles += pr.m_tiles * pr.n_tiles;
    return pr;
}

void set_operands(Problem& pr, int seg, int64_t k, int a, int b_even, int b_odd) {
    pr.steps[seg] = ceil_div(k, BK);
    pr.a_map[seg] = static_cast<int8_t>(a);
    pr.b_map[seg][0] = static_cast<int8_t>(b_even);
    pr.b_map[seg][1] = static_cast<int8_t>(b_odd);
}

// Boxes: 128 rows x 64 columns (K-major operand) or, of the same array read
// M/N-major, 128 rows of K x 64 columns of M/N: the same box either way.
bool box_map(Maps& maps, int i, const void* base, int64_t rows, int64_t cols) {
    return tensor_map_2d(&maps.m[i], base, static_cast<uint64_t>(rows), static_cast<uint64_t>(cols), 2, BM);
}

}  // namespace

cudaError_t launch_ffn_forward(const FfnForward& a, cudaStream_t stream) {
    if (a.n_tokens <= FFN_SMALL_TOKENS) return launch_ffn_forward_small(a, stream);
    if (!tensor_map_encoder()) return cudaErrorNotSupported;
    const int64_t T = a.n_tokens;
    const int32_t H = a.hidden, I = a.intermediate;
    Maps maps;
    Plan p{};
    if (!box_map(maps, 0, a.x, T, H) || !box_map(maps, 1, a.gate_w, I, H) || !box_map(maps, 2, a.up_w, I, H))
        return cudaErrorInvalidValue;
    Problem& gu = add_problem(p, a.up_logits, T, I, BM);
    set_operands(gu, 0, H, 0, 1, 2);
    p.dst_gate = a.gate;
    p.dst_up = a.up;
    p.status = a.status;
    cudaError_t err = launch<EPI_GATE_UP>(a.bf16, maps, p, stream);
    if (err != cudaSuccess) return err;

    Plan p2{};
    if (!box_map(maps, 0, a.up_logits, T, I) || !box_map(maps, 1, a.down_w, H, I)) return cudaErrorInvalidValue;
    Problem& dn = add_problem(p2, a.out, T, H, BN);
    set_operands(dn, 0, I, 0, 1, 1);
    p2.status = a.status;
    return launch<EPI_STORE>(a.bf16, maps, p2, stream);
}

cudaError_t launch_ffn_backward(const FfnBackward& a, cudaStream_t stream) {
    if (!tensor_map_encoder()) return cudaErrorNotSupported;
    const int64_t T = a.n_tokens;
    const int32_t H = a.hidden, I = a.intermediate;
    Maps maps;
    enum { DY, DOWN, DG, DU, GATE, UP, X, HG };
    if (!box_map(maps, DY, a.d_out, T, H) || !box_map(maps, DOWN, a.down_w, H, I) ||
        !box_map(maps, DG, a.d_gate, T, I) || !box_map(maps, DU, a.d_up, T, I) ||
        !box_map(maps, GATE, a.gate_w, I, H) || !box_map(maps, UP, a.up_w, I, H) || !box_map(maps, X, a.x, T, H) ||
        !box_map(maps, HG, a.up_logits, T, I))
        return cudaErrorInvalidValue;
    Plan p{};
    Problem& dh = add_problem(p, nullptr, T, I, BN);
    set_operands(dh, 0, H, DY, DOWN, DOWN);
    dh.b_mn = 1;
    p.gate_in = a.gate;
    p.up_in = a.up;
    p.dst_gate = a.d_gate;
    p.dst_up = a.d_up;
    p.status = a.status;
    cudaError_t err = launch<EPI_GRAD>(a.bf16, maps, p, stream);
    if (err != cudaSuccess) return err;

    Plan q{};
    q.status = a.status;
    Problem& dx = add_problem(q, a.d_x, T, H, BN);
    set_operands(dx, 0, I, DG, GATE, GATE);
    set_operands(dx, 1, I, DU, UP, UP);
    dx.b_mn = 1;
    struct { uint16_t* dst; int32_t m, n; int a, b; } w[3] = {
        {a.d_gate_w, I, H, DG, X}, {a.d_up_w, I, H, DU, X}, {a.d_down_w, H, I, DY, HG}};
    for (const auto& d : w) {
        Problem& pr = add_problem(q, d.dst, d.m, d.n, BN);
        set_operands(pr, 0, T, d.a, d.b, d.b);
        pr.a_mn = 1;
        pr.b_mn = 1;
    }
    return launch<EPI_STORE>(a.bf16, maps, q, stream);
}

}  // namespace moe
