// Matrix products of the dense gated feed-forward block and of its gradients.
//
// Forward, x [T, H], gate_w / up_w [I, H], down_w [H, I], all of one 16-bit type:
//     G = x·gate_wᵀ, U = x·up_wᵀ (fp32), h = G·sigmoid(G)·U      first launch
//     y = h·down_wᵀ                                              second launch
// Backward, from d_y and the stored G, U, h, with s = sigmoid(G):
//     d_h = d_y·down_w (fp32), d_U = d_h·G·s, d_G = d_h·U·s·(1 + G·(1 − s))   first launch
//     d_x = d_G·gate_w + d_U·up_w;  d_gate_w = d_Gᵀ·x;  d_up_w = d_Uᵀ·x        second launch
//     d_down_w = d_yᵀ·h             with whichever launch leaves pairs idle
//
// One kernel serves them all: C[m, n] = Σ_k A[m, k]·B[n, k] over up to four
// problems a launch, each with its own extents, operands and order of operands:
// an operand is K-major (K contiguous: x, h, d_y, d_G as A; the forward's
// weights as B) or M/N-major (M or N contiguous: the transposed ones), which
// the tensor cores read from shared memory as TMA leaves it, so nothing is ever
// transposed in memory.  d_x sums over two K segments (gate, then up) in one
// accumulator, and the products of the backward's second half share one
// launch, so that its last wave is one and not one each.
//
//  * Persistent clusters of two CTAs, one 2-SM MMA tile of M = 256 x N = 256 at
//    a time: each CTA holds 128 rows of A and 128 of B per stage (K = 64, 32 KB,
//    ring of six), warp 0 feeds the ring by TMA, warp 1 of the even CTA issues
//    the MMAs into one of two TMEM accumulators, and warps 2-9 of both CTAs turn
//    the other one into 16-bit rows meanwhile.  With 128 x 256 tiles on one SM
//    the operands' way into and out of shared memory, not the tensor core, is
//    the bound; the pair halves the bytes of B each SM moves.
//  * Launches with few tiles share a tile's K axis among two to four pairs of a
//    cluster: each pair computes its part, sends the columns that others finish
//    to them through distributed shared memory, and adds what it receives in
//    pair order.  300 tokens, 7168 / 2048: 59.7 -> 46.6 us when it came.
//  * Copies and MMAs are issued by converged warps (warp 0 and warp 1): from a
//    one-lane branch the copies alone held a stage up.
//  * Rows past T, columns past H or I and the end of K are zeros that TMA fills
//    in: no size needs padding, only whole 16-byte rows (H and I multiples of 8).
//  * First forward launch: a tile is 128 columns of gate (held by the even CTA)
//    and the same 128 of up (the odd one), so both projections and h come from
//    one pass over x, and h is formed in registers from the fp32 accumulators.
//  * First backward launch: d_h stays in TMEM; the epilogue reads G and U of the
//    tile and writes d_G and d_U.
//
// Measured (GPU time, bf16): forward of 8192 tokens, 7168 / 2048, 380 us = 1.90
// PFLOP/s, its gradients 780 us = 1.85 (calls back to back, under the power cap: 447 and
// 905); training forward of 4097 tokens, 2048 / 2816, 87.5 us = 1.6 (tensor pipe active
// 81% in gate and up, 75% in down); gradients of 301 tokens, 44.3 us.  Bound: the tensor pipe and close behind it the
// operands' way from L2 for many tokens (back to back, the power cap), the chain
// of fill, K loop, join and epilogue for few hundred.
//
// Roundings to 16 bits: h, y and every gradient once from fp32; G and U when the
// caller stores them for the backward (half the bytes of fp32 and the type the
// backward's products need); d_G and d_U, which are operands of products.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "../../include/moe_gb300.h"
#include "ffn_internal.h"
#include "moe_internal.h"
#include "sm103_products.cuh"
#include "tensor_map.h"
#include "tile_store.cuh"

namespace moe {
namespace {

constexpr int BM = 128;                        // rows of A (and of B) per CTA
constexpr int BN = 256;                        // columns of a tile
constexpr int BK = 64;                         // K per stage
constexpr int STAGES = 384 / BK;
constexpr int OP_BYTES = BM * BK * 2;          // one operand's stage
constexpr int K_BOX_BYTES = BM * 128;          // K-major: boxes of 64 along K x 128 rows
constexpr int MN_BOX_BYTES = BK * 128;         // M/N-major: two boxes of 64 along M/N x BK rows of K
constexpr int STAGE_BYTES = 2 * OP_BYTES;
constexpr int TMEM_COLS = 2 * BN;
constexpr int NUM_THREADS = 320;               // producer, MMA and eight epilogue warps
constexpr int NUM_EPI_WARPS = 8;
constexpr int PAIR = 2;                        // CTAs of one MMA tile
constexpr int MAX_SPLIT = 4;                   // pairs that may share a tile's K axis
constexpr int MIN_STEPS = 384 / BK;            // stages each of them keeps at least
constexpr int MIN_TILE_STEPS = 448 / BK;       // stages' worth of time that a tile takes at least (its epilogue)
constexpr float JOIN_STEPS = 512.0f / BK;             // time to join a shared tile (about 2.5 us), in stages
constexpr float JOIN_STEPS_AHEAD = 1536.0f / BK;      // the same ahead of unshared tiles, whose loads have to wait for it
constexpr float SHARED_STEPS = 1280.0f / BK;          // first data, join and epilogue of a shared tile
constexpr int GROUP_M = 8;                     // tile rows (of 256) that are walked together
constexpr uint64_t WAIT_LIMIT_NS = 2000000000ull;
constexpr uint64_t DRAIN_LIMIT_NS = 200000000ull;

constexpr int OFF_STAGING = STAGES * STAGE_BYTES;  // 4 KB per epilogue warp
constexpr int STAGING_BYTES = 32 * 128;
constexpr int OFF_BARS = OFF_STAGING + NUM_EPI_WARPS * STAGING_BYTES;
constexpr int NUM_BARS = 2 * STAGES + 2 + 2 + 1;   // full, empty, tfull, tempty, drain
constexpr int OFF_TMEM_SLOT = OFF_BARS + NUM_BARS * 8;
constexpr int OFF_ABORT = OFF_TMEM_SLOT + 4;
constexpr int SMEM_BYTES = 1024 + OFF_ABORT + 4;

constexpr int SMALL_ROWS = 32;                 // boxes of a K-major A that has no more rows
constexpr int MAX_MAPS = 12;
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
    int32_t split;                 // pairs per cluster
    int32_t split_tiles;           // the first so many tiles are shared by a cluster's pairs
    int32_t lead;                  // tiles a pair without a shared one does before the others join
    int32_t n_maps;
    int32_t early_weights;         // no B is a result of the launch before: see the producer
    int32_t a_box_bytes;           // of a K-major A
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

__device__ __forceinline__ void store_remote4(uint32_t cluster_addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// Adds the other pairs' partial sums of 32 columns (`at`: this row's first quad
// in the first pair's slot, quads 128 rows apart) in pair order.
__device__ __forceinline__ void add_partials(uint32_t (&v)[32], const uint8_t* at, int slots, uint32_t slot_bytes) {
    for (int s = 0; s < slots; ++s) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const float4 x = *reinterpret_cast<const float4*>(at + s * slot_bytes + q * (BM * 16));
            v[4 * q] = __float_as_uint(__uint_as_float(v[4 * q]) + x.x);
            v[4 * q + 1] = __float_as_uint(__uint_as_float(v[4 * q + 1]) + x.y);
            v[4 * q + 2] = __float_as_uint(__uint_as_float(v[4 * q + 2]) + x.z);
            v[4 * q + 3] = __float_as_uint(__uint_as_float(v[4 * q + 3]) + x.w);
        }
    }
}

template <int EPI, bool BF16, bool SPLIT>
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
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);     // known to be warp-uniform
    const int lane = tid & 31;
    const uint32_t cluster_rank = cluster_cta_rank();
    const uint32_t pair = SPLIT ? cluster_rank >> 1 : 0;         // of the cluster
    const uint32_t rank = cluster_rank & 1u;                     // inside the pair
    const bool leader = rank == 0;
    const uint16_t pair_mask = static_cast<uint16_t>(0x3u << (2 * pair));

    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar_full + 8 * s, 1);           // the even CTA's arrive.expect_tx
            mbar_init(bar_empty + 8 * s, 1);          // the MMAs' commit, multicast to both CTAs
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(bar_tfull + 8 * a, 1);
            mbar_init(bar_tempty + 8 * a, PAIR * NUM_EPI_WARPS);
        }
        mbar_init(bar_drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane < p.n_maps) tma_prefetch_map(&maps.m[lane]);
    if (warp == 1) {
        tmem_alloc_pair(sbase + OFF_TMEM_SLOT, TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    // Everything above overlaps the kernel before; every global access is below
    // (with early_weights the producer waits, after its first weights).  The next
    // kernel may start only now that this CTA holds its TMEM.
    if (!p.early_weights) {
        pdl_wait_prior_grid();
        pdl_launch_dependents();
    }
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    cluster_sync_all();            // both CTAs' barriers exist before copies and commits cross
    // No bounded wait runs while the launch before still works.  (Behind the cluster's
    // barrier, which the producer has to pass before its first weights.)
    if (p.early_weights && warp != 0) pdl_wait_prior_grid();

    const int32_t split = SPLIT ? p.split : 1;
    const int32_t cluster_id = static_cast<int32_t>(blockIdx.x) / (PAIR * split);
    const int32_t n_clusters = static_cast<int32_t>(gridDim.x) / (PAIR * split);
    const int32_t pair_id = static_cast<int32_t>(blockIdx.x) / PAIR;
    const int32_t n_pairs = static_cast<int32_t>(gridDim.x) / PAIR;

    // Pipeline state of whichever role this warp has.
    uint32_t stage = 0, phase = 0, acc = 0, aphase = 0;
    int64_t issued = 0;
    bool ok = true;
    const uint64_t policy = l2_policy_evict_normal();
    const uint32_t leader_full = mapa_shared(bar_full, 2 * pair);
    const uint32_t leader_tempty = mapa_shared(bar_tempty, 2 * pair);

    // TMA producer (warp 0 of both CTAs): stages [s0, s1) of a tile.
    const uint32_t issue = elect_one();
    const uint32_t leader_issue = leader ? issue : 0;
    bool early = p.early_weights != 0;
    auto produce = [&](const Tile& ti, int32_t s0, int32_t s1) {
        const Problem& pr = p.pr[ti.q];
        const int32_t arow = ti.m * 2 * BM + static_cast<int32_t>(rank) * BM;
        // gate and up side by side: both CTAs take the same 128 columns, of different weights
        const int32_t brow = EPI == EPI_GATE_UP ? ti.n * BM : ti.n * BN + static_cast<int32_t>(rank) * BM;
        const bool a_mn = pr.a_mn != 0, b_mn = pr.b_mn != 0;
        const int32_t steps0 = pr.steps[0];
        const uint32_t bytes = PAIR * (OP_BYTES + (a_mn ? OP_BYTES : static_cast<uint32_t>(p.a_box_bytes)));
        MOE_DCHECK(pr.a_map[0] < p.n_maps && pr.a_map[1] < p.n_maps && pr.b_map[0][rank] < p.n_maps &&
                       pr.b_map[1][rank] < p.n_maps,
                   p.status);
        MOE_DCHECK(s0 >= 0 && s0 < s1 && s1 <= pr.steps[0] + pr.steps[1], p.status);
        auto load = [&](const CUtensorMap* m, uint32_t dst, uint32_t fb, bool mn, int32_t row, int32_t k0) {
            if (mn) {
#pragma unroll
                for (int b = 0; b < 2; ++b) tma_load_2d_pair_if(issue, dst + b * MN_BOX_BYTES, m, fb, row + b * 64, k0, policy);
            } else {
#pragma unroll
                for (int b = 0; b < BK / 64; ++b)
                    tma_load_2d_pair_if(issue, dst + b * K_BOX_BYTES, m, fb, k0 + b * 64, row, policy);
            }
        };
        // The first tile of a launch right behind the one that makes its A: the
        // ring's first weights are on their way before that one has finished.
        // (It lets this launch start only after its own wait for everything
        // before it, and writes no weights.)
        int32_t have_b = 0;
        if (early) {
            have_b = s1 - s0 < STAGES ? s1 - s0 : STAGES;
            have_b = s0 + have_b <= steps0 ? have_b : (s0 < steps0 ? steps0 - s0 : 0);   // of the first K segment
            for (int32_t i = 0; i < have_b; ++i) {
                mbar_arrive_expect_tx_if(leader_issue, bar_full + 8 * i, bytes);
                load(&maps.m[pr.b_map[0][rank]], sbase + i * STAGE_BYTES + OP_BYTES, leader_full + 8 * i, b_mn, brow,
                     (s0 + i) * BK);
            }
            pdl_wait_prior_grid();
            pdl_launch_dependents();
            __syncwarp();
            early = false;
        }
#pragma unroll 1
        for (int seg = 0; seg < 2; ++seg) {
            const CUtensorMap* am = &maps.m[pr.a_map[seg]];
            const CUtensorMap* bm = &maps.m[pr.b_map[seg][rank]];
            int32_t k0 = ((seg == 0 ? s0 : (s0 > steps0 ? s0 : steps0)) - (seg == 0 ? 0 : steps0)) * BK;
            const int32_t k1 = (seg == 0 ? (s1 < steps0 ? s1 : steps0) : s1 - steps0) * BK;
            for (; k0 < k1; k0 += BK) {
                if (!mbar_wait_warp(bar_empty + 8 * stage, phase ^ 1u, abort_flag, WAIT_LIMIT_NS)) {
                    ok = false;
                    return;
                }
                const uint32_t fb = leader_full + 8 * stage;
                const uint32_t sa = sbase + stage * STAGE_BYTES;
                if (have_b == 0) {
                    mbar_arrive_expect_tx_if(leader_issue, bar_full + 8 * stage, bytes);
                    load(bm, sa + OP_BYTES, fb, b_mn, brow, k0);
                } else {
                    --have_b;
                }
                load(am, sa, fb, a_mn, arow, k0);
                ++issued;
                if (++stage == STAGES) { stage = 0; phase ^= 1u; }
            }
        }
    };

    // MMA issuer (warp 1 of the even CTA): the same stages into an accumulator.
    auto multiply = [&](const Tile& ti, int32_t s0, int32_t s1) {
        if (!mbar_wait_warp(bar_tempty + 8 * acc, aphase ^ 1u, abort_flag, WAIT_LIMIT_NS)) {
            ok = false;
            return;
        }
        tc_fence_after_sync();
        const Problem& pr = p.pr[ti.q];
        const uint32_t d_tmem = tmem_base + acc * BN;
        const bool a_mn = pr.a_mn != 0, b_mn = pr.b_mn != 0;
        const uint32_t idesc = idesc_16bit_f32acc(2 * BM, BN, BF16, a_mn, b_mn);
        for (int32_t st = s0; st < s1; ++st) {
            if (!mbar_wait_warp(bar_full + 8 * stage, phase, abort_flag, WAIT_LIMIT_NS)) {
                ok = false;
                return;
            }
            tc_fence_after_sync();
            const uint32_t sa = sbase + stage * STAGE_BYTES;
            const uint32_t sb = sa + OP_BYTES;
            const uint64_t da = a_mn ? smem_desc_mn_sw128(sa, MN_BOX_BYTES) : smem_desc_k_sw128(sa);
            const uint64_t db = b_mn ? smem_desc_mn_sw128(sb, MN_BOX_BYTES) : smem_desc_k_sw128(sb);
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk) {
                // a K = 16 slice further, in 16-byte units: M/N-major 16 rows of
                // 128 bytes; K-major 32 bytes inside a box of four slices
                constexpr int MN_STEP = 2048 >> 4;
                const int k_off = (kk / 4) * (K_BOX_BYTES >> 4) + (kk % 4) * (32 >> 4);
                tc_mma_f16_pair_if(issue, d_tmem, da + (a_mn ? kk * MN_STEP : k_off), db + (b_mn ? kk * MN_STEP : k_off),
                                   idesc, (st != s0 || kk != 0) ? 1u : 0u);
            }
            tc_commit_pair_mc_if(issue, bar_empty + 8 * stage, pair_mask);
            if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        tc_commit_pair_mc_if(issue, bar_tfull + 8 * acc, pair_mask);
        acc ^= 1u;
        if (acc == 0) aphase ^= 1u;
    };

    // Epilogue (warps 2-9, both CTAs): thread = row, 64 output columns a pass; of
    // the two warps with the same rows one takes the even passes, one the odd.
    const int quarter = warp & 3;                                // TMEM lanes 32*quarter .. +31
    const int odd = warp >= 6 ? 1 : 0;
    uint8_t* staging = smem + OFF_STAGING + (warp >= 2 ? warp - 2 : 0) * STAGING_BYTES;
    constexpr int PASSES = EPI == EPI_GATE_UP ? 2 : 4;
    const int row = quarter * 32 + lane;                         // of this CTA's 128
    struct Rows {
        int64_t at;            // first element of the warp's rows in C
        int32_t rows;          // of the warp's 32 that exist
    };
    auto rows_of = [&](const Tile& ti) {
        const Problem& pr = p.pr[ti.q];
        const int64_t row0 = static_cast<int64_t>(ti.m) * (2 * BM) + static_cast<int64_t>(rank) * BM + quarter * 32;
        const int64_t left = pr.m - row0;
        MOE_DCHECK(row0 >= 0 && left > -2 * BM && ti.n * p.tile_cols < pr.n, p.status);
        return Rows{row0 * pr.n + ti.n * p.tile_cols, left > 32 ? 32 : (left < 0 ? 0 : static_cast<int32_t>(left))};
    };
    // A shared tile: pass c belongs to pair c * split / PASSES.  The others'
    // partial sums wait in that pair's ring, a slot per pair.
    constexpr uint32_t PASS_BYTES = BM * BN * 4 / PASSES;
    const uint32_t slot_bytes = PASS_BYTES * static_cast<uint32_t>((PASSES + split - 1) / split);
    static_assert(PASS_BYTES * ((PASSES + 1) / 2) <= STAGES * STAGE_BYTES &&
                      PASS_BYTES * ((PASSES + 2) / 3) * 2 <= STAGES * STAGE_BYTES &&
                      PASS_BYTES * ((PASSES + 3) / 4) * 3 <= STAGES * STAGE_BYTES && MAX_SPLIT == 4,
                  "the slots fit in the ring for 2, 3 and 4 pairs");
    auto first_pass = [&](int owner) { return (owner * PASSES + split - 1) / split; };
    // EPI_GRAD: G and U of a warp's first pass are asked for before the tile is
    // finished, and turned from lines to rows when they are needed.
    uint4 eg[EPI == EPI_GRAD ? 8 : 1], eu[EPI == EPI_GRAD ? 8 : 1];
    auto ask_gate_up = [&](const Tile& ti, bool shared) {
        if constexpr (EPI == EPI_GRAD) {
            if (ti.q != 0) return;
            const Problem& pr = p.pr[ti.q];
            const Rows r = rows_of(ti);
            const int c = (SPLIT && shared ? first_pass(static_cast<int>(pair)) : 0) + odd;
            const int32_t cols = pr.n - ti.n * p.tile_cols - c * 64;
            load_lines_64(eg, p.gate_in + r.at + c * 64, pr.n, lane, r.rows, cols);
            load_lines_64(eu, p.up_in + r.at + c * 64, pr.n, lane, r.rows, cols);
        }
    };
    auto finish = [&](const Tile& ti, bool shared) {
        const Problem& pr = p.pr[ti.q];
        const Rows r = rows_of(ti);
        const int32_t rows = r.rows;
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * BN;
        const int c0 = SPLIT && shared ? first_pass(static_cast<int>(pair)) : 0;
        const int c1 = SPLIT && shared ? first_pass(static_cast<int>(pair) + 1) : PASSES;
#pragma unroll 1
        for (int c = c0 + odd; c < c1 && rows > 0; c += 2) {
            const int32_t cols = pr.n - ti.n * p.tile_cols - c * 64;             // columns left
            if (cols <= 0) break;
            const int64_t at = r.at + c * 64;
            MOE_DCHECK(c * 64 < p.tile_cols && cols % 8 == 0 && at >= 0 &&
                           at + static_cast<int64_t>(rows - 1) * pr.n + (cols < 64 ? cols : 64) <= pr.m * pr.n,
                       p.status);
            // this pass's first quad of the partial sums
            const uint8_t* part = smem + (c - c0) * PASS_BYTES + row * 16;
            if (EPI == EPI_STORE || (EPI == EPI_GRAD && ti.q != 0)) {
                uint4 el[8];
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(taddr + c * 64 + hh * 32, v);
                    tmem_ld_wait();
                    if (SPLIT && shared) add_partials(v, part + hh * 8 * BM * 16, split - 1, slot_bytes);
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
                store_staged_64(el, staging, pr.dst + at, pr.n, lane, rows, cols);
            } else if (EPI == EPI_GATE_UP) {
                // 32 columns of one projection (0 gate, 1 up)
                auto load32 = [&](uint32_t (&v)[32], int which, int hh) {
                    tmem_ld_32x32b_x32(taddr + which * 128 + c * 64 + hh * 32, v);
                    tmem_ld_wait();
                    if (SPLIT && shared)
                        add_partials(v, part + (which * 16 + hh * 8) * BM * 16, split - 1, slot_bytes);
                };
                uint4 el[8];
                auto round32 = [&](const uint32_t (&v)[32], int hh) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            w[j] = pack_16bit2<BF16>(__uint_as_float(v[8 * k + 2 * j]),
                                                     __uint_as_float(v[8 * k + 2 * j + 1]));
                        el[4 * hh + k] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                };
                if (p.dst_gate != nullptr) {
#pragma unroll 1
                    for (int which = 0; which < 2; ++which) {
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            uint32_t v[32];
                            load32(v, which, hh);
                            round32(v, hh);
                        }
                        store_staged_64(el, staging, (which ? p.dst_up : p.dst_gate) + at, pr.n, lane, rows, cols);
                    }
                }
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    uint32_t g[32], u[32];
                    load32(g, 0, hh);
                    load32(u, 1, hh);
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const float x = __uint_as_float(g[j]);
                        g[j] = __float_as_uint(x * sigmoid_approx(x) * __uint_as_float(u[j]));
                    }
                    round32(g, hh);
                }
                store_staged_64(el, staging, pr.dst + at, pr.n, lane, rows, cols);
            } else if constexpr (EPI == EPI_GRAD) {
                // eg and eu hold G and U, then d_G and d_U
                if (c != c0 + odd) {
                    load_lines_64(eg, p.gate_in + at, pr.n, lane, rows, cols);
                    load_lines_64(eu, p.up_in + at, pr.n, lane, rows, cols);
                }
                lines_to_rows(eg, staging, lane);
                lines_to_rows(eu, staging, lane);
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    uint32_t d[32];
                    tmem_ld_32x32b_x32(taddr + c * 64 + hh * 32, d);
                    tmem_ld_wait();
                    if (SPLIT && shared) add_partials(d, part + hh * 8 * BM * 16, split - 1, slot_bytes);
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
                            const float s0 = sigmoid_approx(g.x);
                            const float s1 = sigmoid_approx(g.y);
                            pg[j] = pack_16bit2<BF16>(d0 * u.x * s0 * (1.0f + g.x * (1.0f - s0)),
                                                      d1 * u.y * s1 * (1.0f + g.y * (1.0f - s1)));
                            pu[j] = pack_16bit2<BF16>(d0 * g.x * s0, d1 * g.y * s1);
                        }
                    }
                }
                store_staged_64(eg, staging, p.dst_gate + at, pr.n, lane, rows, cols);
                store_staged_64(eu, staging, p.dst_up + at, pr.n, lane, rows, cols);
            }
        }
        tc_fence_before_sync();
        // the accumulator may be reused once both CTAs have read their rows
        __syncwarp();
        if (lane == 0) {
            if (leader) mbar_arrive(bar_tempty + 8 * acc);
            else mbar_arrive_cluster_relaxed(leader_tempty + 8 * acc);
        }
        acc ^= 1u;
        if (acc == 0) aphase ^= 1u;
    };
    // Sends this CTA's sums of the passes that other pairs finish.
    auto push_partials = [&](const Tile& ti) {
        const Problem& pr = p.pr[ti.q];
        if (rows_of(ti).rows == 0) return;
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * BN;
#pragma unroll 1
        for (int c = odd; c < PASSES; c += 2) {
            const int owner = c * split / PASSES;
            if (owner == static_cast<int>(pair) || pr.n - ti.n * p.tile_cols - c * 64 <= 0) continue;
            const int slot = static_cast<int>(pair) - (static_cast<int>(pair) > owner ? 1 : 0);
            const int first = first_pass(owner);
            MOE_DCHECK(owner >= 0 && owner < split && slot >= 0 && slot < split - 1 && c >= first &&
                           slot * slot_bytes + (c - first + 1) * PASS_BYTES <= STAGES * STAGE_BYTES,
                       p.status);
            uint32_t dst = mapa_shared(sbase, static_cast<uint32_t>(owner) * 2 + rank) + slot * slot_bytes +
                           (c - first) * PASS_BYTES + row * 16;
#pragma unroll 1
            for (int hh = 0; hh < (EPI == EPI_GATE_UP ? 4 : 2); ++hh) {
                uint32_t v[32];
                // gate and up: 64 columns of gate, then the same of up
                tmem_ld_32x32b_x32(taddr + c * 64 + (hh & 1) * 32 + (hh >> 1) * 128, v);
                tmem_ld_wait();
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    store_remote4(dst + (hh * 8 + q) * (BM * 16), v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
            }
        }
    };

    // First the tiles that the cluster's pairs share, each with its part of the K
    // axis, then tiles of one pair each.  Nothing leaves the loop while there are
    // shared tiles: every thread meets every barrier.
    // (Pairs of clusters without a shared tile start on `lead` rounds of the others.)
    const int32_t busy = SPLIT && p.split_tiles < n_clusters ? p.split_tiles * split : n_pairs;
    const int32_t idle = n_pairs - busy;
    const int32_t joint = p.split_tiles + p.lead * idle;        // from here on the tiles go around all pairs
    int32_t t = SPLIT && cluster_id < p.split_tiles ? cluster_id
                : SPLIT && pair_id >= busy && p.lead > 0 ? p.split_tiles + pair_id - busy
                                                         : joint + pair_id;
    while (t < p.total_tiles && (ok || t < p.split_tiles)) {
        const bool shared = SPLIT && t < p.split_tiles;
        const Tile ti = tile_at(p, t);
        const int32_t steps = p.pr[ti.q].steps[0] + p.pr[ti.q].steps[1];
        MOE_DCHECK(ti.q < p.n_problems && ti.m >= 0 && ti.m < p.pr[ti.q].m_tiles && ti.n >= 0 &&
                       ti.n < p.pr[ti.q].n_tiles,
                   p.status);
        const int32_t s0 = shared ? steps * static_cast<int32_t>(pair) / split : 0;
        const int32_t s1 = shared ? steps * (static_cast<int32_t>(pair) + 1) / split : steps;
        if (warp == 0) {
            if (ok) produce(ti, s0, s1);
        } else if (warp == 1) {
            if (leader && ok) multiply(ti, s0, s1);
        } else if (ok) {
            ask_gate_up(ti, shared);
            // one answer for the whole warp, whose TMEM loads are collective
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar_tfull + 8 * acc, aphase, abort_flag, WAIT_LIMIT_NS));
            tc_fence_after_sync();
        }
        if (shared) {
            __syncwarp();
            cluster_sync_all();                    // every ring of the cluster is free
            if (warp >= 2 && ok) push_partials(ti);
            __syncwarp();
            cluster_sync_all();                    // the partial sums are there
        }
        if (warp >= 2 && ok) finish(ti, shared);
        if (shared) {
            // the ring's next writer is TMA
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncthreads();
            t += n_clusters;
            if (t >= p.split_tiles) t = joint + pair_id;
        } else if (t < joint) {
            t += idle;
            if (t >= joint) t = joint + pair_id;
        } else {
            t += n_pairs;
        }
    }
    if (warp == 1 && leader && issue) {
        // Every MMA this warp issued has finished once this arrives.
        volatile int never = 0;
        tc_commit_pair(bar_drain);
        mbar_wait_bounded(bar_drain, 0, &never, DRAIN_LIMIT_NS);
    }
    __syncwarp();

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 0 && lane == 0 && *abort_flag) {
        // Whichever role gave up: copies in flight land before the CTA exits.
        // (The odd CTA's report to the even CTA's barriers.)
        if (leader) drain_copies(bar_full, issued, STAGES, DRAIN_LIMIT_NS);
        else spin_ns(1000000ull);
    }
    __syncwarp();
    // No CTA leaves (or frees the pair's TMEM) while another may still write
    // into its shared memory, arrive on its barriers or use the TMEM.
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

// Clusters of 1 .. MAX_SPLIT pairs that fit on the device at once, after opting
// in to the kernels' shared memory; asked once per device.
struct Resident {
    std::once_flag once;
    cudaError_t err;
    int clusters[MAX_SPLIT + 1];
};

template <int EPI, bool BF16>
const Resident* resident() {
    constexpr int MAX_DEVICES = 16;
    static Resident table[MAX_DEVICES];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= MAX_DEVICES) return nullptr;
    Resident& r = table[dev];
    std::call_once(r.once, [&r] {
        for (int split = 1; split <= MAX_SPLIT; ++split) {
            const auto kernel = split > 1 ? ffn_gemm_kernel<EPI, BF16, true> : ffn_gemm_kernel<EPI, BF16, false>;
            r.err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
            if (r.err != cudaSuccess) return;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = static_cast<unsigned>(PAIR * split);
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(static_cast<unsigned>(PAIR * split * 64));
            cfg.blockDim = dim3(NUM_THREADS);
            cfg.dynamicSmemBytes = SMEM_BYTES;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            r.err = cudaOccupancyMaxActiveClusters(&r.clusters[split], kernel, &cfg);
            if (r.err == cudaSuccess && r.clusters[split] <= 0) r.err = cudaErrorNoDevice;
            if (r.err != cudaSuccess) return;
        }
    });
    return &r;
}

template <int EPI, bool BF16>
cudaError_t launch(const Maps& maps, Plan& p, cudaStream_t stream) {
    // How many pairs share a tile, and how many tiles are shared, goes by the time
    // of the launch in K steps: rounds of unshared tiles, plus rounds of shared
    // ones at steps / split each and JOIN_STEPS for joining them.  Of a launch of
    // one problem the tiles that do not fill a round are shared (all of them
    // where there is no full round); of several, the first problem's if they are
    // one round at most, while the pairs left over work on the other problems'.
    // Splitting also leaves SMs without a cluster: 144, 138 and 120 of 152 are in
    // one of 4, 6 and 8 CTAs.
    const int32_t tiles = p.pr[0].m_tiles * p.pr[0].n_tiles;
    const int32_t steps = p.pr[0].steps[0] + p.pr[0].steps[1];
    const Resident* r = resident<EPI, BF16>();
    if (!r) return cudaErrorNoDevice;
    if (r->err != cudaSuccess) return r->err;
    int nc = r->clusters[1];
    p.split = 1;
    p.split_tiles = 0;
    const bool several = p.n_problems > 1;
    const int32_t others = p.total_tiles - tiles;
    const int32_t own = several && p.pr[1].steps[0] > MIN_TILE_STEPS ? p.pr[1].steps[0] : MIN_TILE_STEPS;
    auto rounds = [](int32_t n, int32_t per_round) { return static_cast<float>((n + per_round - 1) / per_round); };
    float best = rounds(tiles, nc) * static_cast<float>(steps);
    if (several) {
        const float work = (static_cast<float>(tiles) * steps + static_cast<float>(others) * own) / nc;
        const float longest = 1.25f * static_cast<float>(steps);     // one pair's K loop beside the others' stores
        best = (work > longest ? work : longest) + SHARED_STEPS;
    }
    for (int split = 2; split <= MAX_SPLIT; ++split) {
        // Gate and up finish in two parts, so three pairs join no faster than two and only
        // the K loop gets shorter.  Measured with three allowed: 200 tokens 2048 / 2816 27.5
        // -> 28.8 us, 300 tokens 2048 / 1408 25.1 -> 26.5, 450 tokens 4104 / 1024 29.1 ->
        // 30.4; with the longest K alone it wins (200 tokens 7168 / 2048 39.8 -> 37.7).
        if (steps < MIN_STEPS * split || (EPI == EPI_GATE_UP && split == 3)) continue;
        const int n = r->clusters[split];
        const float part = static_cast<float>(steps) / static_cast<float>(split);
        const int32_t full = several ? 0 : tiles / (n * split);
        const int32_t rest = tiles - full * n * split;
        if (rest == 0 || (several && rest > n)) continue;
        float t = static_cast<float>(full * steps) + rounds(rest, n) * (part + (full > 0 ? JOIN_STEPS_AHEAD : JOIN_STEPS));
        int32_t lead = 0;
        if (several) {
            // meanwhile the other clusters' pairs are `lead` tiles ahead
            const int32_t idle = (n - rest) * split;
            lead = static_cast<int32_t>((part + SHARED_STEPS) / static_cast<float>(own));
            if (idle > 0 && lead > others / idle) lead = others / idle;
            t = part + SHARED_STEPS + rounds(others - lead * idle, n * split) * static_cast<float>(own);
        }
        if (t < best) {
            best = t;
            p.split = split;
            p.split_tiles = rest;
            p.lead = lead;
            nc = n;
        }
    }
    // clusters that have work: a shared tile each, or a tile for each of their pairs
    const int32_t unshared = (p.total_tiles - p.split_tiles + p.split - 1) / p.split;
    const int32_t want = unshared > p.split_tiles ? unshared : p.split_tiles;
    if (nc > want) nc = want;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(PAIR * p.split);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(PAIR * p.split * nc));
    cfg.blockDim = dim3(NUM_THREADS);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return p.split > 1 ? cudaLaunchKernelEx(&cfg, ffn_gemm_kernel<EPI, BF16, true>, maps, p)
                       : cudaLaunchKernelEx(&cfg, ffn_gemm_kernel<EPI, BF16, false>, maps, p);
}

template <int EPI>
cudaError_t launch(bool bf16, const Maps& maps, Plan& p, cudaStream_t stream) {
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

// Rows of a K-major A's boxes.  Of an array of few rows a box of 128 lies mostly
// outside, which TMA is slow at: gradients of one token, 2048 / 2816, 48.5 -> 33.5
// us, of 16 tokens 44 -> 34.  (The other rows' sums are never read.)  33 to 64 tokens
// take 34.8 to 35.1 us with boxes of 128, 32 tokens 33.4: no third size.
int a_box_rows(int64_t tokens) { return tokens <= SMALL_ROWS ? SMALL_ROWS : BM; }

// Boxes of 64 columns: 128 rows of a K-major operand, or BK rows of K of an
// M/N-major one.
bool box_map(Maps& maps, int i, const void* base, int64_t rows, int64_t cols, int box_rows = BM) {
    return tensor_map_2d(&maps.m[i], base, static_cast<uint64_t>(rows), static_cast<uint64_t>(cols), 2,
                         static_cast<uint32_t>(box_rows));
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
    p.n_maps = 3;
    p.a_box_bytes = BM * 128;
    p.dst_gate = a.gate;
    p.dst_up = a.up;
    p.status = a.status;
    cudaError_t err = launch<EPI_GATE_UP>(a.bf16, maps, p, stream);
    if (err != cudaSuccess) return err;

    Plan p2{};
    if (!box_map(maps, 0, a.up_logits, T, I) || !box_map(maps, 1, a.down_w, H, I)) return cudaErrorInvalidValue;
    Problem& dn = add_problem(p2, a.out, T, H, BN);
    set_operands(dn, 0, I, 0, 1, 1);
    p2.n_maps = 2;
    p2.a_box_bytes = BM * 128;
    p2.early_weights = 1;
    p2.status = a.status;
    return launch<EPI_STORE>(a.bf16, maps, p2, stream);
}

cudaError_t launch_ffn_backward(const FfnBackward& a, cudaStream_t stream) {
    if (!tensor_map_encoder()) return cudaErrorNotSupported;
    const int64_t T = a.n_tokens;
    const int32_t H = a.hidden, I = a.intermediate;
    Maps maps;
    // K-major operands, then M/N-major ones
    enum { DY, DG, DU, DOWN_T, GATE_T, UP_T, X_T, H_T, DY_T, DG_T, DU_T, MAPS };
    static_assert(MAPS <= MAX_MAPS, "maps fit");
    const int a_rows = a_box_rows(T);
    if (!box_map(maps, DY, a.d_out, T, H, a_rows) || !box_map(maps, DG, a.d_gate, T, I, a_rows) ||
        !box_map(maps, DU, a.d_up, T, I, a_rows) ||
        !box_map(maps, DOWN_T, a.down_w, H, I, BK) || !box_map(maps, GATE_T, a.gate_w, I, H, BK) ||
        !box_map(maps, UP_T, a.up_w, I, H, BK) || !box_map(maps, X_T, a.x, T, H, BK) ||
        !box_map(maps, H_T, a.up_logits, T, I, BK) || !box_map(maps, DY_T, a.d_out, T, H, BK) ||
        !box_map(maps, DG_T, a.d_gate, T, I, BK) || !box_map(maps, DU_T, a.d_up, T, I, BK))
        return cudaErrorInvalidValue;
    Plan p{};
    Problem& dh = add_problem(p, nullptr, T, I, BN);
    set_operands(dh, 0, H, DY, DOWN_T, DOWN_T);
    dh.b_mn = 1;
    // d_down needs nothing of either launch.  The first takes it where d_h has more
    // than a round of tiles, of which the last leaves pairs idle, and a tile of
    // d_down is neither shorter than its stores nor longer than one of d_h (2048 /
    // 2816: 1024 tokens 70.6 -> 66.2 us, 2048 tokens 109.8 -> 101.8).  Elsewhere the
    // second launch's first pairs start, with their weights, where d_h leaves room
    // (400 tokens, 768 / 2048: 31 us, 35 with d_down in the first; 1200: 42.6, 46.3;
    // 128 tokens, 4096 / 14336: 169, 177).
    const Resident* r = a.bf16 ? resident<EPI_GRAD, true>() : resident<EPI_GRAD, false>();
    if (!r) return cudaErrorNoDevice;
    if (r->err != cudaSuccess) return r->err;
    const int32_t dh_steps = dh.steps[0], dd_steps = ceil_div(T, BK);
    const bool down_first = dh.m_tiles * dh.n_tiles > r->clusters[2] && dd_steps >= MIN_TILE_STEPS &&
                            dd_steps <= dh_steps + dh_steps / 4;
    auto weight_gradient = [&](Plan& plan, uint16_t* dst, int32_t m, int32_t n, int a_map, int b_map) {
        Problem& pr = add_problem(plan, dst, m, n, BN);
        set_operands(pr, 0, T, a_map, b_map, b_map);
        pr.a_mn = 1;
        pr.b_mn = 1;
    };
    if (down_first) weight_gradient(p, a.d_down_w, H, I, DY_T, H_T);
    p.n_maps = MAPS;
    p.a_box_bytes = a_rows * 128;
    p.gate_in = a.gate;
    p.up_in = a.up;
    p.dst_gate = a.d_gate;
    p.dst_up = a.d_up;
    p.status = a.status;
    cudaError_t err = launch<EPI_GRAD>(a.bf16, maps, p, stream);
    if (err != cudaSuccess) return err;

    Plan q{};
    q.status = a.status;
    q.n_maps = MAPS;
    q.a_box_bytes = a_rows * 128;
    q.early_weights = 1;
    Problem& dx = add_problem(q, a.d_x, T, H, BN);
    set_operands(dx, 0, I, DG, GATE_T, GATE_T);
    set_operands(dx, 1, I, DU, UP_T, UP_T);
    dx.b_mn = 1;
    weight_gradient(q, a.d_gate_w, I, H, DG_T, X_T);
    weight_gradient(q, a.d_up_w, I, H, DU_T, X_T);
    if (!down_first) weight_gradient(q, a.d_down_w, H, I, DY_T, H_T);
    return launch<EPI_STORE>(a.bf16, maps, q, stream);
}

}  // namespace moe
