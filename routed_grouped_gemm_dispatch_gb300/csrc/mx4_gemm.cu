// Products of 4-bit microscaled operands: out[p, j] = Σ_k A[p, k]·B[e][j, k], sums in
// fp32, every product of two values and two power-of-two scales exact.
//
// Three forms over 128-row blocks of A:
//     matmul    rows as they come, one B
//     gate_up   rows grouped by expert: h = round16( G·sigmoid(G)·U ), G and U the
//               products with the expert's gate and up weights
//     down      rows grouped by expert: out = round16( C · routed weight of the row )
// A result is never rounded to 4 bits in here: that is a conversion of its own.
//
// The tensor cores take e2m1 operands with an e8m0 scale per 32 values along K
// directly (tcgen05.mma kind::mxf4): per K = 64 slice the bytes that move are
// those of a K = 16 slice of 16-bit operands, for four times the products.
//  * Persistent pairs of CTAs (one per SM) walk 2-SM tiles of M = 256 x N = 256: up to
//    two consecutive blocks of one expert (a unit), 128 rows in each CTA, against
//    256 columns, half of whose codes each CTA loads.  A 128 x 256 tile on one
//    SM moves 96 bytes per cycle out of and 100 into shared memory at the MMAs'
//    full rate, more than it has; the pair moves 64 and 68.  A lone block runs
//    with the other CTA's rows empty: nothing is loaded for them.
//  * The units are compacted first; tiles run slice by slice inside groups of
//    units (about an expert's), so that concurrent pairs share a weight slice in
//    L2.
//  * Per stage (K = 256) and CTA: 16 KB of A and 16 KB of B codes (128-byte
//    swizzle), and their scale tiles (512 bytes for 128 rows x 128 values: A's own,
//    all of B's), everything by TMA onto the even CTA's barrier.  The MMA thread
//    copies the scale tiles to TMEM, to columns of their stage, ahead of the
//    MMAs that read them.
//  * Copies and MMAs are issued by converged warps: one lane took 1021 cycles to
//    issue a stage whose MMAs take 512.
//  * TMEM: columns 0-255 accumulate, the stages' scales sit behind them; two
//    accumulators would leave no room for scales.  Instead the eight epilogue warps
//    take a finished tile into registers (128 values a thread) and hand the
//    accumulator back before they round and store.
//
// Measured (GPU time): 4096 x 7168 x 4096 40.0 us = 6.0 PFLOP/s; routed gate_up of
// 4096 tokens, top-6 of 64 experts, 2048 / 1408, 66.4 us = 4.3 PFLOP/s at 4.4 TB/s.  (The
// dense K = 96 form of the MMA, half as fast again, is not used.)  Bound:
// the operands' way from L2 (with one MMA in sixteen 35 and 61 us: 48 bytes a cycle
// and SM), under about 700 cycles a stage where the MMAs alone are 512, and 600
// between tiles while the accumulator changes hands.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "../../include/moe_gb300.h"
#include "moe_internal.h"
#include "mx4_internal.h"
#include "sm103_products.cuh"
#include "tensor_map.h"
#include "tile_store.cuh"

namespace moe {
namespace {

constexpr int BM = 128;                         // rows of A (and of B) per CTA
constexpr int BN = 256;                         // columns of B per tile
constexpr int BOX = 128;                        // bytes of codes of a row per stage (K = 256)
constexpr int OP_BYTES = BM * BOX;
constexpr int SCALE_TILE = 512;                 // scales of 128 rows x 128 values
constexpr int SFA_BYTES = 2 * SCALE_TILE;
constexpr int SFB_BYTES = 4 * SCALE_TILE;
constexpr int STAGE_BYTES = 2 * OP_BYTES + SFA_BYTES + SFB_BYTES;
constexpr int MAX_STAGES = 6;
constexpr int SMALL_ROWS = 32;                  // a block with at most this many rows loads a box of 32
constexpr int NUM_THREADS = 320;                // producer, MMA and eight epilogue warps
constexpr int NUM_EPI_WARPS = 8;
constexpr int PAIR = 2;
constexpr uint16_t PAIR_MASK = 0x3;
constexpr int MAX_GROUP = 8;                    // units walked together at most (2048 rows)
constexpr int TMEM_COLS = 512;
constexpr int TMEM_SCALES = 256;                // first scale column
constexpr int STAGE_SCALE_COLS = 2 * (4 + 8);   // per K = 128: 4 columns of A's, 8 of B's scales
// Average rows per expert up to which the few-rows kernel runs.  Pair kernel against
// few-rows kernel, us (experts, K / N):
//   gate_up  rows       64            96            128
//     128, 2048 / 768   47.1 / 44.2   47.6 / 46.8   48.9 / 50.9
//     64, 2048 / 1408   43.0 / 39.2   43.8 / 42.4   45.1 / 47.1
//     8, 4096 / 2048    21.2 / 20.8   21.5 / 20.6   21.9 / 20.7
//     32, 7168 / 2048   87.6 / 87.2   88.5 / 93.1   90.0 / 108
//     16, 1024 / 4096   22.6 / 19.7   22.8 / 21.3   23.6 / 24.7
//   down     rows       32            48            64
//     128, 768 / 2048   36.6 / 31.0   36.8 / 37.4   39.6 / 47.8
//     64, 1408 / 2048   27.1 / 25.0   27.8 / 28.0   28.4 / 33.0
//     32, 2048 / 7168   49.6 / 46.5   51.4 / 49.8   51.9 / 58.9
//     8, 2048 / 4096    13.5 / 10.5   14.1 / 11.3   14.5 / 14.5
//     16, 4096 / 1024   13.3 / 10.4   13.8 / 11.3   13.8 / 15.5
constexpr int64_t FEW_AVERAGE_GATE_UP = 64;
constexpr int64_t FEW_AVERAGE = 32;
constexpr int64_t FEW_MAX_BLOCKS = 4096;        // (its unit list stays small)
constexpr uint64_t WAIT_LIMIT_NS = 2000000000ull;
constexpr uint64_t DRAIN_LIMIT_NS = 200000000ull;

static_assert(STAGE_BYTES % 1024 == 0, "stages keep the swizzle's alignment");
static_assert(TMEM_SCALES + MAX_STAGES * STAGE_SCALE_COLS <= TMEM_COLS, "scales fit in TMEM");
static_assert(MOE_MAX_BLOCKS <= 1 << 16 && MOE_MAX_EXPERTS <= 1 << 16, "indices fit the unit list");

constexpr int OFF_BARS = 0;                     // full, empty [MAX_STAGES]; tfull, tempty, drain
constexpr int OFF_TMEM_SLOT = OFF_BARS + (2 * MAX_STAGES + 3) * 8;
constexpr int OFF_ABORT = OFF_TMEM_SLOT + 4;
constexpr int OFF_RUNS = OFF_ABORT + 4;
constexpr int OFF_WSUM = OFF_RUNS + 4;
constexpr int OFF_UNITS = (OFF_WSUM + (NUM_THREADS / 32) * 4 + 15) / 16 * 16;

struct Maps {
    CUtensorMap a, a_small, b, b2, sfa, sfb, sfb2;       // few rows: a has boxes of 64 rows
};

struct Params {
    const float* weights;
    const int32_t* sizes;
    const int32_t* offsets;
    const int32_t* padded;
    const int32_t* gidx;
    uint16_t* out;
    int32_t* status;
    int64_t rows;
    int64_t valid_total;
    int32_t num_blocks;
    int32_t n_experts;
    int32_t n;                                  // columns of out
    int32_t n_tiles;
    int32_t k_tiles;                            // K / 128
    int32_t stages;
    int32_t split;                              // few rows: CTAs that share a tile
};

// Rows of block bx that hold data, its expert and the row's place inside the
// expert.  Table entries that point outside their arrays make a block empty
// and raise MOE_DEV_BAD_TABLE.
template <int FORM>
__device__ __forceinline__ int32_t block_rows(const Params& p, int32_t bx, int32_t* e_out, int32_t* tok_out) {
    *e_out = -1;
    *tok_out = 0;
    if (FORM == MX4_MATMUL) {
        *e_out = 0;
        const int64_t left = p.rows - static_cast<int64_t>(bx) * BM;
        return left > BM ? BM : (left < 0 ? 0 : static_cast<int32_t>(left));
    }
    const int32_t e = __ldg(p.gidx + bx);
    bool bad = e < 0 || e >= p.n_experts;
    int64_t rows = 0, tok = 0;
    if (!bad) {
        tok = static_cast<int64_t>(bx) * BM - __ldg(p.padded + e);
        rows = static_cast<int64_t>(__ldg(p.sizes + e)) - tok;
        rows = rows > BM ? BM : (rows < 0 ? 0 : rows);
        if (rows > 0) {
            bad = tok < 0 || static_cast<int64_t>(bx) * BM + rows > p.rows;
            if (FORM == MX4_DOWN && !bad) {
                const int64_t c0 = static_cast<int64_t>(__ldg(p.offsets + e)) + tok;
                bad = c0 < 0 || c0 + rows > p.valid_total;
            }
        }
    }
    if (bad) {
        if (p.status) atomicOr(p.status, MOE_DEV_BAD_TABLE);
        return 0;
    }
    *e_out = e;
    *tok_out = static_cast<int32_t>(tok);
    return static_cast<int32_t>(rows);
}

// Rows of block bx + 1 if it goes on where block bx (of expert e, `tok` rows in)
// ends, else 0.
template <int FORM>
__device__ __forceinline__ int32_t rows_after(const Params& p, int32_t bx, int32_t e, int32_t tok) {
    if (bx + 1 >= p.num_blocks) return 0;
    int32_t e1, tok1;
    const int32_t rows = block_rows<FORM>(p, bx + 1, &e1, &tok1);
    return e1 == e && tok1 == tok + BM ? rows : 0;
}

// A value all lanes hold, known to the compiler as warp-uniform.
__device__ __forceinline__ int32_t uniform(int32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// A unit: one or two blocks of an expert.  The list keeps what every role needs
// to know of it, so that no tile starts with a chain of table loads.
struct Unit {
    int32_t bx, e;                              // first block, expert
    int32_t rows[2];                            // of the first and of the second block (0: there is none)
};

__device__ __forceinline__ uint2 pack_unit(int32_t bx, int32_t e, int32_t rows0, int32_t rows1) {
    return make_uint2(static_cast<uint32_t>(bx) | static_cast<uint32_t>(e) << 16,
                      static_cast<uint32_t>(rows0) | static_cast<uint32_t>(rows1) << 16);
}

struct Tile {
    Unit u;
    int32_t n;
};

// Groups of `group` units, slice by slice inside a group.
template <int FORM>
__device__ __forceinline__ Tile tile_at(const Params& p, int32_t t, const uint2* units, int32_t num_units, int32_t group) {
    const int32_t per_group = group * p.n_tiles;
    const int32_t g = t / per_group;
    const int32_t l = t - g * per_group;
    const int32_t left = num_units - g * group;
    const int32_t gs = left < group ? left : group;
    Tile ti;
    ti.n = l / gs;
    const int32_t u = g * group + (l - ti.n * gs);
    if (FORM == MX4_MATMUL) {
        int32_t e, tok;
        ti.u.bx = 2 * u;
        ti.u.e = 0;
        ti.u.rows[0] = block_rows<FORM>(p, 2 * u, &e, &tok);
        ti.u.rows[1] = block_rows<FORM>(p, 2 * u + 1, &e, &tok);
    } else {
        const uint2 v = units[u];
        ti.u.bx = static_cast<int32_t>(v.x & 0xffffu);
        ti.u.e = static_cast<int32_t>(v.x >> 16);
        ti.u.rows[0] = static_cast<int32_t>(v.y & 0xffffu);
        ti.u.rows[1] = static_cast<int32_t>(v.y >> 16);
    }
    MOE_DCHECK(u >= 0 && u < num_units && ti.n >= 0 && ti.n < p.n_tiles, p.status);
    MOE_DCHECK(ti.u.bx >= 0 && ti.u.bx < p.num_blocks && ti.u.e >= 0 && ti.u.e < p.n_experts, p.status);
    MOE_DCHECK(ti.u.rows[0] > 0 && ti.u.rows[0] <= BM && ti.u.rows[1] >= 0 && ti.u.rows[1] <= BM, p.status);
    MOE_DCHECK(static_cast<int64_t>(ti.u.bx) * BM + (ti.u.rows[1] > 0 ? BM + ti.u.rows[1] : ti.u.rows[0]) <= p.rows,
               p.status);
    return ti;
}

template <int FORM, bool BF16>
__global__ void __launch_bounds__(NUM_THREADS, 1)
mx4_gemm_kernel(const __grid_constant__ Maps maps, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem =
        reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* ctl = smem + p.stages * STAGE_BYTES;
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar_full = smem_u32(ctl) + OFF_BARS;          // (used in the even CTA)
    const uint32_t bar_empty = bar_full + 8 * MAX_STAGES;
    const uint32_t bar_tfull = bar_empty + 8 * MAX_STAGES;
    const uint32_t bar_tempty = bar_tfull + 8;                   // (used in the even CTA)
    const uint32_t bar_drain = bar_tempty + 8;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(ctl + OFF_TMEM_SLOT);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(ctl + OFF_ABORT);
    int32_t* wsum = reinterpret_cast<int32_t*>(ctl + OFF_WSUM);
    int32_t* runs = reinterpret_cast<int32_t*>(ctl + OFF_RUNS);
    uint2* units = reinterpret_cast<uint2*>(ctl + OFF_UNITS);

    const int tid = threadIdx.x;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);     // known to be warp-uniform
    const int lane = tid & 31;
    const uint32_t rank = cluster_cta_rank();
    const bool leader = rank == 0;
    const uint32_t stages = static_cast<uint32_t>(p.stages);

    if (tid == 0) {
        for (int s = 0; s < MAX_STAGES; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 1);
        }
        mbar_init(bar_tfull, 1);
        mbar_init(bar_tempty, PAIR * NUM_EPI_WARPS);
        mbar_init(bar_drain, 1);
        *abort_flag = 0;
        *runs = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(ctl) + OFF_TMEM_SLOT, TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    // The next kernel may start only now that this CTA holds its TMEM.
    pdl_wait_prior_grid();
    pdl_launch_dependents();

    // ---- units, in block order, and the number of experts they belong to ----
    int32_t num_units = 0;
    if (FORM == MX4_MATMUL) {
        num_units = (p.num_blocks + 1) / 2;
    } else {
        for (int32_t base = 0; base < p.num_blocks; base += NUM_THREADS) {
            const int32_t bx = base + tid;
            int32_t starts = 0, e = 0, tok = 0, rows1 = 0;
            const int32_t rows0 = bx < p.num_blocks ? block_rows<FORM>(p, bx, &e, &tok) : 0;
            if (rows0 > 0) {
                // an expert's blocks pair up from its first; a block is a unit's
                // second if it is an odd one and the block before it leads up to it
                starts = 1;
                if ((tok / BM) & 1) {
                    int32_t e0, tok0;
                    if (bx > 0 && block_rows<FORM>(p, bx - 1, &e0, &tok0) > 0 && e0 == e && tok0 == tok - BM) starts = 0;
                } else {
                    rows1 = rows_after<FORM>(p, bx, e, tok);
                }
            }
            const uint32_t ballot = __ballot_sync(0xffffffffu, starts);
            const uint32_t first = __ballot_sync(0xffffffffu, starts && tok == 0);
            if (lane == 0) {
                wsum[warp] = __popc(ballot);
                if (first) atomicAdd(runs, __popc(first));
            }
            __syncthreads();
            int32_t before = 0, total = 0;
#pragma unroll
            for (int w = 0; w < NUM_THREADS / 32; ++w) {
                const int32_t c = wsum[w];
                before += (w < warp) ? c : 0;
                total += c;
            }
            if (starts) units[num_units + before + __popc(ballot & ((1u << lane) - 1u))] = pack_unit(bx, e, rows0, rows1);
            num_units += total;
            __syncthreads();
        }
    }
    int32_t group = FORM == MX4_MATMUL ? MAX_GROUP : (*runs > 0 ? (num_units + *runs - 1) / *runs : 1);
    group = group > MAX_GROUP ? MAX_GROUP : group;
    const int32_t total_tiles = num_units * p.n_tiles;
    const int32_t k_steps = (p.k_tiles + 1) / 2;
    const int32_t pair_id = static_cast<int32_t>(blockIdx.x) / PAIR;
    const int32_t n_pairs = static_cast<int32_t>(gridDim.x) / PAIR;
    cluster_sync_all();            // both CTAs' barriers exist before copies and commits cross

    int64_t issued = 0;            // stages fed, by warp 0
    if (warp == 0) {
        // ===================== producer (both CTAs) =====================
        const uint32_t issue = elect_one();
        const uint32_t leader_issue = leader ? issue : 0;
        const uint64_t policy = l2_policy_evict_normal();
        const uint32_t leader_full = mapa_shared(bar_full, 0);
        uint32_t stage = 0, phase = 0;
        bool ok = true;
        const int32_t my_tiles = __shfl_sync(0xffffffffu, total_tiles, 0);
        for (int32_t t = pair_id; t < my_tiles && ok; t += n_pairs) {
            const Tile ti = tile_at<FORM>(p, t, units, num_units, group);
            const int32_t e = uniform(ti.u.e), rows0 = uniform(ti.u.rows[0]), rows1 = uniform(ti.u.rows[1]);
            const int32_t bx = uniform(ti.u.bx) + static_cast<int32_t>(rank), slice = uniform(ti.n);
            // a block's codes: 128 rows, 32 where it has no more, none where it has none
            const uint32_t a0 = rows0 > SMALL_ROWS ? OP_BYTES : SMALL_ROWS * BOX;
            const uint32_t a1 = rows1 > SMALL_ROWS ? OP_BYTES : (rows1 > 0 ? SMALL_ROWS * BOX : 0);
            const int32_t rows = leader ? rows0 : rows1;
            const uint32_t bytes = a0 + SFA_BYTES + (rows1 > 0 ? a1 + SFA_BYTES : 0) + 2 * (OP_BYTES + SFB_BYTES);
            const CUtensorMap* am = rows > SMALL_ROWS ? &maps.a : &maps.a_small;
            // weight rows: the same 128 of gate (even CTA) and up (odd), or this CTA's half of 256
            const int32_t tile_row = e * p.n + slice * (FORM == MX4_GATE_UP ? BM : BN);
            const CUtensorMap* bm = FORM == MX4_GATE_UP && !leader ? &maps.b2 : &maps.b;
            const int32_t brow = tile_row + (FORM == MX4_GATE_UP ? 0 : static_cast<int32_t>(rank) * BM);
            for (int32_t kb = 0; kb < k_steps; ++kb) {
                if (!mbar_wait_warp(bar_empty + 8 * stage, phase ^ 1u, abort_flag, WAIT_LIMIT_NS)) {
                    ok = false;
                    break;
                }
                const uint32_t fb = leader_full + 8 * stage;
                const uint32_t sa = sbase + stage * STAGE_BYTES;
                const uint32_t sb = sa + OP_BYTES;
                const uint32_t ss = sb + OP_BYTES;
                mbar_arrive_expect_tx_if(leader_issue, bar_full + 8 * stage, bytes);
                tma_load_2d_pair_if(issue, sb, bm, fb, kb * BOX, brow, policy);
                if (rows > 0) {
                    tma_load_2d_pair_if(issue, sa, am, fb, kb * BOX, bx * BM, policy);
                    tma_load_2d_pair_if(issue, ss, &maps.sfa, fb, kb * 256, bx, policy);
                }
                // every CTA needs the scales of all of B's rows
                tma_load_2d_pair_if(issue, ss + SFA_BYTES, &maps.sfb, fb, kb * 256, tile_row / BM, policy);
                if (FORM == MX4_GATE_UP)
                    tma_load_2d_pair_if(issue, ss + SFA_BYTES + SFB_BYTES / 2, &maps.sfb2, fb, kb * 256, tile_row / BM, policy);
                ++issued;
                if (++stage == stages) { stage = 0; phase ^= 1u; }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ===================== MMA issuer (even CTA only) =====================
        if (leader) {
            const uint32_t issue = elect_one();
            const int32_t my_tiles = __shfl_sync(0xffffffffu, total_tiles, 0);
            uint32_t stage = 0, phase = 0, aphase = 0;
            bool ok = true;
            for (int32_t t = pair_id; t < my_tiles && ok; t += n_pairs) {
                for (int32_t kb = 0; kb < k_steps; ++kb) {
                    if (!mbar_wait_warp(bar_full + 8 * stage, phase, abort_flag, WAIT_LIMIT_NS)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint32_t sa = sbase + stage * STAGE_BYTES;
                    // this stage's scale columns: free since the stage's last MMAs finished
                    const uint32_t tsc = tmem_base + TMEM_SCALES + stage * STAGE_SCALE_COLS;
                    const uint64_t da = smem_desc_k_sw128(sa), db = smem_desc_k_sw128(sa + OP_BYTES);
                    const uint64_t ds = smem_desc_scales(sa + 2 * OP_BYTES);
                    constexpr uint32_t TILE16 = SCALE_TILE >> 4;
                    // (the second K = 128 of a last odd stage is zeros that TMA filled in)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {                                // K = 128 each
                        tc_cp_scales_pair(issue, tsc + i * 12, ds + i * TILE16);
                        tc_cp_scales_pair(issue, tsc + i * 12 + 4, ds + (SFA_BYTES >> 4) + i * TILE16);
                        tc_cp_scales_pair(issue, tsc + i * 12 + 8, ds + (SFA_BYTES >> 4) + (2 + i) * TILE16);
                    }
                    if (kb == 0) {
                        // the scales do not have to wait for the accumulator
                        if (!mbar_wait_warp(bar_tempty, aphase ^ 1u, abort_flag, WAIT_LIMIT_NS)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after_sync();
                    }
                    const bool both = p.k_tiles - 2 * kb >= 2;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {                                // K = 64 each
                        if (i == 2 && !both) break;
                        tc_mma_mxf4_pair(issue, tmem_base, da + i * 2, db + i * 2, idesc_mxf4(2 * BM, BN, i & 1),
                                         tsc + (i >> 1) * 12, tsc + (i >> 1) * 12 + 4, (kb | i) != 0 ? 1u : 0u);
                    }
                    tc_commit_pair_mc_if(issue, bar_empty + 8 * stage, PAIR_MASK);
                    if (++stage == stages) { stage = 0; phase ^= 1u; }
                }
                if (!ok) break;
                tc_commit_pair_mc_if(issue, bar_tfull, PAIR_MASK);
                aphase ^= 1u;
            }
            // Every MMA issued here has finished once this arrives.
            volatile int never = 0;
            if (issue) {
                tc_commit_pair(bar_drain);
                mbar_wait_bounded(bar_drain, 0, &never, DRAIN_LIMIT_NS);
            }
        }
        __syncwarp();
    } else {
        // ===================== epilogue (warps 2..9, both CTAs) =====================
        const int quarter = warp & 3;                            // TMEM lanes 32*quarter .. +31
        const int half = warp >= 6 ? 1 : 0;                      // of the tile's columns
        const uint32_t leader_tempty = mapa_shared(bar_tempty, 0);
        uint32_t aphase = 0;
        for (int32_t t = pair_id; t < total_tiles; t += n_pairs) {
            const Tile ti = tile_at<FORM>(p, t, units, num_units, group);
            const int32_t bx = ti.u.bx + static_cast<int32_t>(rank);
            const int32_t rows = (leader ? ti.u.rows[0] : ti.u.rows[1]) - quarter * 32;   // of this warp
            const int64_t row0 = static_cast<int64_t>(bx) * BM + quarter * 32;
            // 64 output columns of gate and up, or 128 plain ones
            const int32_t col0 = FORM == MX4_GATE_UP ? ti.n * BM + half * 64 : ti.n * BN + half * 128;
            float w = 1.0f;
            if (FORM == MX4_DOWN && lane < rows) {
                const int64_t c = static_cast<int64_t>(__ldg(p.offsets + ti.u.e)) + row0 - __ldg(p.padded + ti.u.e) + lane;
                MOE_DCHECK(c >= 0 && c < p.valid_total, p.status);
                w = __ldg(p.weights + c);
            }
            // one answer for the whole warp, whose TMEM loads are collective
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar_tfull, aphase, abort_flag, WAIT_LIMIT_NS))) break;
            tc_fence_after_sync();
            const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
            const bool any = rows > 0 && col0 < p.n;
            MOE_DCHECK(!any || row0 + (rows < 32 ? rows : 32) <= p.rows, p.status);
            MOE_DCHECK(FORM != MX4_GATE_UP || col0 + 64 <= p.n, p.status);
            uint16_t* dst = p.out + row0 * p.n + col0;
            auto release = [&]() {
                // one arrival a warp: 512 single ones, half of them from the other
                // SM, would take longer than the loads before them
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if (leader) mbar_arrive(bar_tempty);
                    else mbar_arrive_cluster_relaxed(leader_tempty);
                }
                aphase ^= 1u;
            };
            if (!any) {
                release();
                continue;
            }
            // eight columns as one 16-byte piece
            auto piece = [](const uint32_t* x) {
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    o[j] = pack_16bit2<BF16>(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1]));
                return make_uint4(o[0], o[1], o[2], o[3]);
            };
            if (FORM == MX4_GATE_UP) {
                // the activation takes longer than the loads: hand the accumulator back first
                uint32_t g[2][32], u[2][32];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    tmem_ld_32x32b_x32(taddr + half * 64 + i * 32, g[i]);
                    tmem_ld_32x32b_x32(taddr + 128 + half * 64 + i * 32, u[i]);
                }
                tmem_ld_wait();
                release();
                uint4 el[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    uint32_t x[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float f = __uint_as_float(g[k >> 2][8 * (k & 3) + j]);
                        x[j] = __float_as_uint(f * sigmoid_approx(f) *
                                               __uint_as_float(u[k >> 2][8 * (k & 3) + j]));
                    }
                    el[k] = piece(x);
                }
                store_rows_64(el, dst, p.n, lane, rows, 64);
            } else {
                uint4 el[2][8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(taddr + half * 128 + i * 32, v);
                    tmem_ld_wait();
                    if (FORM == MX4_DOWN) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * w);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) el[i >> 1][4 * (i & 1) + k] = piece(v + 8 * k);
                }
                release();
#pragma unroll
                for (int c = 0; c < 2; ++c) store_rows_64(el[c], dst + c * 64, p.n, lane, rows, p.n - col0 - c * 64);
            }
        }
        __syncwarp();
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 0 && lane == 0 && *abort_flag) {
        // Whichever role gave up: copies in flight land before the CTA exits.
        // (The odd CTA's report to the even CTA's barriers.)
        if (leader) drain_copies(bar_full, issued, p.stages, DRAIN_LIMIT_NS);
        else spin_ns(1000000ull);
    }
    __syncwarp();
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
// few rows per block
// ---------------------------------------------------------------------------

// With a handful of rows per expert the weights' bytes bound the product, and a
// tile that spends its MMA time on 256 rows of A would not keep up with them.
// Here the weights are the M side: a CTA takes 128 weight rows (gate_up: 128 of
// gate and the same 128 of up, two accumulators) against the N side of at most 64
// rows of a block, rounded up to 16.  MMA time goes with the rows that are there;
// what is left is the stream of weights through the ring.  The results lie
// transposed in TMEM (a lane is an output column), so a warp writes 64
// consecutive bytes of a row at a time.  32 tokens, top-8 of 128 experts, 2048 / 768:
// 33.6 us on the pair kernel, 23 here (116 MB from memory; the unit list and the
// first fill take about 4 of them).
//
// SPLIT (a plain product with fewer tiles than SMs): a cluster of CTAs shares a
// tile, each with its part of the K axis.  They exchange fp32 sums through
// distributed shared memory, in the rings that the MMAs have emptied; groups of
// 16 rows go around the CTAs, and an owner adds the parts in rank order.  The
// join costs about 1 us: one row, K 7168 / N 1408 8.9 -> 5.5 us, 7168 / 4096 9.6 ->
// 8.3, 4096 / 2048 6.0 -> 5.0, but K 2048 / N 4096 4.5 -> 5.1: from K = 4096 on.
constexpr int FEW_ROWS = 64;                    // rows of a block per unit
constexpr int FEW_THREADS = 320;                // producer, MMA and eight epilogue warps
constexpr int FEW_MAX_STAGES = 8;
constexpr int FEW_MAX_SPLIT = 4;                // CTAs that share a tile
constexpr int FEW_SPLIT_STEPS = 16;             // K / 256 from which they do
constexpr int FEW_OFF_TMEM_SLOT = (2 * FEW_MAX_STAGES + 5) * 8;   // full, empty; tfull, tempty [2]; drain
constexpr int FEW_OFF_ABORT = FEW_OFF_TMEM_SLOT + 4;
constexpr int FEW_OFF_WSUM = FEW_OFF_ABORT + 4;
constexpr int FEW_OFF_UNITS = (FEW_OFF_WSUM + (FEW_THREADS / 32) * 4 + 15) / 16 * 16;

template <int FORM>
struct Few {
    static constexpr int ACCS = FORM == MX4_GATE_UP ? 2 : 1;
    static constexpr int W_BYTES = ACCS * BM * BOX;
    static constexpr int X_BYTES = FEW_ROWS * BOX;
    static constexpr int STAGE = W_BYTES + X_BYTES + (ACCS + 1) * 2 * SCALE_TILE;
    static constexpr int SCALE_COLS = 2 * 4 * (ACCS + 1);            // of a stage
    static constexpr int TMEM_SCALE0 = 2 * ACCS * FEW_ROWS;          // behind two sets of accumulators
    static_assert(STAGE % 1024 == 0, "stages keep the swizzle's alignment");
    static_assert(TMEM_SCALE0 + FEW_MAX_STAGES * SCALE_COLS <= TMEM_COLS, "scales fit in TMEM");
};

__device__ __forceinline__ void store_remote(uint32_t cluster_addr, uint32_t v) {
    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}

template <int FORM, bool BF16, bool SPLIT>
__global__ void __launch_bounds__(FEW_THREADS, 1)
mx4_few_rows_kernel(const __grid_constant__ Maps maps, const Params p) {
    using F = Few<FORM>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem =
        reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* ctl = smem + p.stages * F::STAGE;
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar_full = smem_u32(ctl);
    const uint32_t bar_empty = bar_full + 8 * FEW_MAX_STAGES;
    const uint32_t bar_tfull = bar_empty + 8 * FEW_MAX_STAGES;   // [2]
    const uint32_t bar_tempty = bar_tfull + 16;                  // [2]
    const uint32_t bar_drain = bar_tempty + 16;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(ctl + FEW_OFF_TMEM_SLOT);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(ctl + FEW_OFF_ABORT);
    int32_t* wsum = reinterpret_cast<int32_t*>(ctl + FEW_OFF_WSUM);
    uint2* units = reinterpret_cast<uint2*>(ctl + FEW_OFF_UNITS);

    const int tid = threadIdx.x;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int lane = tid & 31;
    const uint32_t stages = static_cast<uint32_t>(p.stages);
    if (tid == 0) {
        for (int s = 0; s < FEW_MAX_STAGES; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(bar_tfull + 8 * a, 1);
            mbar_init(bar_tempty + 8 * a, FEW_THREADS / 32 - 2);
        }
        mbar_init(bar_drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(ctl) + FEW_OFF_TMEM_SLOT, TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    // The next kernel may start only now that this CTA holds its TMEM.
    pdl_wait_prior_grid();
    pdl_launch_dependents();

    // ---- units: the active blocks, a second entry for rows 64 and up ----
    int32_t num_units = 0;
    for (int32_t base = 0; base < p.num_blocks; base += FEW_THREADS) {
        const int32_t bx = base + tid;
        int32_t e = 0, tok = 0;
        const int32_t rows = bx < p.num_blocks ? block_rows<FORM>(p, bx, &e, &tok) : 0;
        const int32_t mine = rows > FEW_ROWS ? 2 : (rows > 0 ? 1 : 0);
        const uint32_t one = __ballot_sync(0xffffffffu, mine > 0), two = __ballot_sync(0xffffffffu, mine > 1);
        if (lane == 0) wsum[warp] = __popc(one) + __popc(two);
        __syncthreads();
        int32_t before = 0, total = 0;
#pragma unroll
        for (int w = 0; w < FEW_THREADS / 32; ++w) {
            const int32_t c = wsum[w];
            before += (w < warp) ? c : 0;
            total += c;
        }
        const uint32_t below = (1u << lane) - 1u;
        const int32_t at = num_units + before + __popc(one & below) + __popc(two & below);
        if (mine > 0) units[at] = pack_unit(bx, e, rows > FEW_ROWS ? FEW_ROWS : rows, 0);
        if (mine > 1) units[at + 1] = pack_unit(bx, e, rows - FEW_ROWS, 1);
        num_units += total;
        __syncthreads();
    }
    const int32_t total_tiles = __shfl_sync(0xffffffffu, num_units * p.n_tiles, 0);
    const int32_t k_steps = (p.k_tiles + 1) / 2;
    // this CTA's tiles and its part of their K axis (SPLIT: one tile per cluster)
    const int32_t split = SPLIT ? p.split : 1;
    const int32_t crank = SPLIT ? static_cast<int32_t>(cluster_cta_rank()) : 0;
    const int32_t kb0 = k_steps * crank / split, kb1 = k_steps * (crank + 1) / split;
    const int32_t t0 = static_cast<int32_t>(blockIdx.x) / split;
    const int32_t t_step = static_cast<int32_t>(gridDim.x) / split;

    // A unit's weight slices follow one another, so its few rows stay in L2.
    struct FewTile {
        int32_t bx, n, first, rows, e;           // first: of the block's rows
    };
    auto tile = [&](int32_t t) {
        FewTile ti;
        const int32_t u = t / p.n_tiles;
        const uint2 v = units[u];
        ti.n = t - u * p.n_tiles;
        ti.bx = static_cast<int32_t>(v.x & 0xffffu);
        ti.e = static_cast<int32_t>(v.x >> 16);
        ti.rows = static_cast<int32_t>(v.y & 0xffffu);
        ti.first = static_cast<int32_t>(v.y >> 16) * FEW_ROWS;
        MOE_DCHECK(u >= 0 && u < num_units && ti.bx < p.num_blocks && ti.e < p.n_experts, p.status);
        MOE_DCHECK(ti.rows > 0 && ti.rows <= FEW_ROWS && ti.first <= FEW_ROWS &&
                       static_cast<int64_t>(ti.bx) * BM + ti.first + ti.rows <= p.rows,
                   p.status);
        return ti;
    };

    int64_t issued = 0;            // stages fed, by warp 0
    if (warp == 0) {
        // ===================== producer =====================
        const uint32_t issue = elect_one();
        const uint64_t policy = l2_policy_evict_normal();
        uint32_t stage = 0, phase = 0;
        bool ok = true;
        for (int32_t t = t0; t < total_tiles && ok; t += t_step) {
            const FewTile ti = tile(t);
            const int32_t wrow = uniform(ti.e) * p.n + uniform(ti.n) * BM;
            const int32_t xrow = uniform(ti.bx) * BM + uniform(ti.first), bx = uniform(ti.bx);
            const bool small = uniform(ti.rows) <= SMALL_ROWS;
            const uint32_t bytes = F::W_BYTES + (small ? SMALL_ROWS : FEW_ROWS) * BOX + (F::ACCS + 1) * 2 * SCALE_TILE;
            for (int32_t kb = kb0; kb < kb1; ++kb) {
                if (!mbar_wait_warp(bar_empty + 8 * stage, phase ^ 1u, abort_flag, WAIT_LIMIT_NS)) {
                    ok = false;
                    break;
                }
                const uint32_t fb = bar_full + 8 * stage;
                const uint32_t sw = sbase + stage * F::STAGE;
                const uint32_t sx = sw + F::W_BYTES;
                const uint32_t ss = sx + F::X_BYTES;
                mbar_arrive_expect_tx_if(issue, fb, bytes);
                tma_load_2d_if(issue, sw, &maps.b, fb, kb * BOX, wrow, policy);
                tma_load_2d_if(issue, ss + 2 * SCALE_TILE, &maps.sfb, fb, kb * 256, wrow / BM, policy);
                if (FORM == MX4_GATE_UP) {
                    tma_load_2d_if(issue, sw + BM * BOX, &maps.b2, fb, kb * BOX, wrow, policy);
                    tma_load_2d_if(issue, ss + 4 * SCALE_TILE, &maps.sfb2, fb, kb * 256, wrow / BM, policy);
                }
                tma_load_2d_if(issue, sx, small ? &maps.a_small : &maps.a, fb, kb * BOX, xrow, policy);
                tma_load_2d_if(issue, ss, &maps.sfa, fb, kb * 256, bx, policy);
                ++issued;
                if (++stage == stages) { stage = 0; phase ^= 1u; }
            }
        }
        __syncwarp();
        if (SPLIT) {
            cluster_sync_all();
            cluster_sync_all();
        }
    } else if (warp == 1) {
        // ===================== MMA issuer =====================
        const uint32_t issue = elect_one();
        uint32_t stage = 0, phase = 0, acc = 0, aphase = 0;
        bool ok = true;
        for (int32_t t = t0; t < total_tiles && ok; t += t_step) {
            const FewTile ti = tile(t);
            const uint32_t n = __shfl_sync(0xffffffffu, static_cast<uint32_t>((ti.rows + 15) & ~15), 0);
            const uint32_t first = __shfl_sync(0xffffffffu, static_cast<uint32_t>(ti.first), 0);
            if (!mbar_wait_warp(bar_tempty + 8 * acc, aphase ^ 1u, abort_flag, WAIT_LIMIT_NS)) break;
            tc_fence_after_sync();
            const uint32_t d = tmem_base + acc * F::ACCS * FEW_ROWS;
            for (int32_t kb = kb0; kb < kb1; ++kb) {
                if (!mbar_wait_warp(bar_full + 8 * stage, phase, abort_flag, WAIT_LIMIT_NS)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t sw = sbase + stage * F::STAGE;
                const uint64_t dw = smem_desc_k_sw128(sw), dx = smem_desc_k_sw128(sw + F::W_BYTES);
                const uint64_t ds = smem_desc_scales(sw + F::W_BYTES + F::X_BYTES);
                // this stage's scale columns: free since the stage's last MMAs finished
                const uint32_t tsc = tmem_base + F::TMEM_SCALE0 + stage * F::SCALE_COLS;
                const bool both = p.k_tiles - 2 * kb >= 2;
#pragma unroll
                for (int i = 0; i < 2; ++i) {                                    // K = 128 each
                    if (i == 1 && !both) break;
                    constexpr uint32_t TILE16 = SCALE_TILE >> 4;
                    const uint32_t ts = tsc + i * 4 * (F::ACCS + 1);             // rows', then the weights' scales
#pragma unroll
                    for (int a = 0; a <= F::ACCS; ++a) tc_cp_scales(issue, ts + 4 * a, ds + (2 * a + i) * TILE16);
#pragma unroll
                    for (int j = 0; j < 2; ++j)                                  // K = 64 each
#pragma unroll
                        for (int a = 0; a < F::ACCS; ++a)
                            tc_mma_mxf4(issue, d + a * FEW_ROWS, dw + a * (BM * BOX >> 4) + (2 * i + j) * 2,
                                        dx + (2 * i + j) * 2, idesc_mxf4(BM, n, j), ts + 4 * (a + 1), ts + first / 32,
                                        ((kb - kb0) | i | j) != 0 ? 1u : 0u);
                }
                tc_commit_if(issue, bar_empty + 8 * stage);
                if (++stage == stages) { stage = 0; phase ^= 1u; }
            }
            if (!ok) break;
            tc_commit_if(issue, bar_tfull + 8 * acc);
            acc ^= 1u;
            if (acc == 0) aphase ^= 1u;
        }
        // Every MMA issued here has finished once this arrives.
        volatile int never = 0;
        if (issue) {
            tc_commit(bar_drain);
            mbar_wait_bounded(bar_drain, 0, &never, DRAIN_LIMIT_NS);
        }
        __syncwarp();
        if (SPLIT) {
            cluster_sync_all();
            cluster_sync_all();
        }
    } else {
        // ===================== epilogue (warps 2..9) =====================
        // of the two warps with the same columns one takes the even groups of
        // eight rows, one the odd
        const int quarter = warp & 3;
        const int odd = warp >= 6 ? 1 : 0;
        uint32_t acc = 0, aphase = 0;
        for (int32_t t = t0; t < total_tiles; t += t_step) {
            const FewTile ti = tile(t);
            const uint32_t taddr =
                tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * F::ACCS * FEW_ROWS;
            const int32_t col = ti.n * BM + quarter * 32 + lane;
            const int64_t row0 = static_cast<int64_t>(ti.bx) * BM + ti.first;
            uint16_t* dst = p.out + row0 * p.n + col;
            const float* rw = nullptr;
            if (FORM == MX4_DOWN) rw = p.weights + (static_cast<int64_t>(__ldg(p.offsets + ti.e)) + row0 - __ldg(p.padded + ti.e));
            const bool done =
                __all_sync(0xffffffffu, mbar_wait_bounded(bar_tfull + 8 * acc, aphase, abort_flag, WAIT_LIMIT_NS)) != 0;
            tc_fence_after_sync();
            if (SPLIT) {
                // [rank that sends][row][column of 128] in the owner's ring
                __syncwarp();
                cluster_sync_all();                    // every ring of the cluster is free
                const uint32_t slot = sbase + (crank * FEW_ROWS * BM + quarter * 32 + lane) * 4;
#pragma unroll 1
                for (int32_t r0 = odd * 8; r0 < ti.rows && done; r0 += 16) {
                    const int32_t owner = (r0 >> 4) % split;
                    if (owner == crank) continue;
                    MOE_DCHECK(r0 + 8 <= FEW_ROWS && split * FEW_ROWS * BM * 4 <= p.stages * F::STAGE, p.status);
                    uint32_t v[8];
                    tmem_ld_32x32b_x8(taddr + r0, v);
                    tmem_ld_wait();
                    const uint32_t at = mapa_shared(slot + r0 * BM * 4, static_cast<uint32_t>(owner));
#pragma unroll
                    for (int j = 0; j < 8; ++j) store_remote(at + j * BM * 4, v[j]);
                }
                __syncwarp();
                cluster_sync_all();                    // the partial sums are there
            }
            if (!done) break;
#pragma unroll 1
            for (int32_t r0 = odd * 8; r0 < ti.rows; r0 += 16) {
                if (SPLIT && (r0 >> 4) % split != crank) continue;
                uint32_t v[8], u[8];
                tmem_ld_32x32b_x8(taddr + r0, v);
                if (FORM == MX4_GATE_UP) tmem_ld_32x32b_x8(taddr + FEW_ROWS + r0, u);
                tmem_ld_wait();
                if (SPLIT) {
                    float sum[8] = {};
                    for (int32_t c = 0; c < split; ++c) {
                        const float* from = reinterpret_cast<const float*>(smem) + (c * FEW_ROWS + r0) * BM + quarter * 32 + lane;
#pragma unroll
                        for (int j = 0; j < 8; ++j) sum[j] += c == crank ? __uint_as_float(v[j]) : from[j * BM];
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = __float_as_uint(sum[j]);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (r0 + j >= ti.rows) break;
                    float x = __uint_as_float(v[j]);
                    if (FORM == MX4_GATE_UP) x = x * sigmoid_approx(x) * __uint_as_float(u[j]);
                    MOE_DCHECK(row0 + r0 + j < p.rows && col < p.n, p.status);
                    MOE_DCHECK(FORM != MX4_DOWN || (rw + r0 + j >= p.weights && rw + r0 + j < p.weights + p.valid_total),
                               p.status);
                    if (FORM == MX4_DOWN) x *= __ldg(rw + r0 + j);
                    dst[static_cast<int64_t>(r0 + j) * p.n] = static_cast<uint16_t>(pack_16bit2<BF16>(x, 0.0f) & 0xffffu);
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_tempty + 8 * acc);
            acc ^= 1u;
            if (acc == 0) aphase ^= 1u;
        }
        __syncwarp();
    }

    tc_fence_before_sync();
    __syncthreads();
    // Whichever role gave up: copies in flight land before the CTA exits.
    if (warp == 0 && lane == 0 && *abort_flag) drain_copies(bar_full, issued, p.stages, DRAIN_LIMIT_NS);
    __syncwarp();
    if (*abort_flag && tid == 0 && p.status) atomicOr(p.status, MOE_DEV_TIMEOUT);
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

template <int FORM, bool BF16>
cudaError_t launch(const Maps& maps, Params& p, cudaStream_t stream) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    constexpr int MAX_DEVICES = 16;
    if (dev >= MAX_DEVICES) return cudaErrorNoDevice;
    // Once per device: the most shared memory, and the pairs that fit at once.
    struct Limits {
        std::once_flag once;
        cudaError_t err;
        int smem, pairs;
    };
    static Limits limits[MAX_DEVICES];
    Limits& lim = limits[dev];
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = PAIR;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(NUM_THREADS);
    cfg.attrs = attr;
    std::call_once(lim.once, [&] {
        lim.err = cudaDeviceGetAttribute(&lim.smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
        if (lim.err == cudaSuccess)
            lim.err = cudaFuncSetAttribute(mx4_gemm_kernel<FORM, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           lim.smem);
        cfg.gridDim = dim3(PAIR * 64);
        cfg.dynamicSmemBytes = static_cast<size_t>(lim.smem);
        cfg.numAttrs = 1;
        if (lim.err == cudaSuccess) lim.err = cudaOccupancyMaxActiveClusters(&lim.pairs, mx4_gemm_kernel<FORM, BF16>, &cfg);
        if (lim.err == cudaSuccess && lim.pairs <= 0) lim.err = cudaErrorNoDevice;
    });
    if (lim.err != cudaSuccess) return lim.err;
    // (a plain product's units need no list: with one, 2 M rows would leave two stages of six)
    const int control = 1024 + OFF_UNITS + (FORM == MX4_MATMUL ? 0 : 8 * p.num_blocks);
    p.stages = (lim.smem - control) / STAGE_BYTES;
    if (p.stages > MAX_STAGES) p.stages = MAX_STAGES;
    // a unit has one block at least (two, but for the last, in a plain product)
    const int64_t units = FORM == MX4_MATMUL ? (p.num_blocks + 1) / 2 : p.num_blocks;
    const int64_t tiles = units * p.n_tiles;
    cfg.gridDim = dim3(static_cast<unsigned>(PAIR * (tiles < lim.pairs ? tiles : lim.pairs)));
    cfg.dynamicSmemBytes = static_cast<size_t>(control + p.stages * STAGE_BYTES);
    cfg.stream = stream;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, mx4_gemm_kernel<FORM, BF16>, maps, p);
}

template <int FORM, bool BF16>
cudaError_t launch_few_rows(const Maps& maps, Params& p, cudaStream_t stream) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    constexpr int MAX_DEVICES = 16;
    if (dev >= MAX_DEVICES) return cudaErrorNoDevice;
    struct Limits {
        std::once_flag once;
        cudaError_t err;
        int smem, sms;
        int clusters[FEW_MAX_SPLIT + 1];       // that fit at once, by CTAs of one
    };
    static Limits limits[MAX_DEVICES];
    Limits& lim = limits[dev];
    std::call_once(lim.once, [&] {
        lim.err = cudaDeviceGetAttribute(&lim.smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
        if (lim.err == cudaSuccess) lim.err = cudaDeviceGetAttribute(&lim.sms, cudaDevAttrMultiProcessorCount, dev);
        if (lim.err == cudaSuccess)
            lim.err = cudaFuncSetAttribute(mx4_few_rows_kernel<FORM, BF16, false>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, lim.smem);
        if (FORM == MX4_MATMUL && lim.err == cudaSuccess) {
            lim.err = cudaFuncSetAttribute(mx4_few_rows_kernel<FORM, BF16, FORM == MX4_MATMUL>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, lim.smem);
            for (int split = 2; split <= FEW_MAX_SPLIT && lim.err == cudaSuccess; split *= 2) {
                cudaLaunchAttribute size[1];
                size[0].id = cudaLaunchAttributeClusterDimension;
                size[0].val.clusterDim.x = static_cast<unsigned>(split);
                size[0].val.clusterDim.y = 1;
                size[0].val.clusterDim.z = 1;
                cudaLaunchConfig_t probe{};
                probe.gridDim = dim3(static_cast<unsigned>(split * 64));
                probe.blockDim = dim3(FEW_THREADS);
                probe.dynamicSmemBytes = static_cast<size_t>(lim.smem);
                probe.attrs = size;
                probe.numAttrs = 1;
                lim.err = cudaOccupancyMaxActiveClusters(
                    &lim.clusters[split], mx4_few_rows_kernel<FORM, BF16, FORM == MX4_MATMUL>, &probe);
            }
        }
    });
    if (lim.err != cudaSuccess) return lim.err;
    p.n_tiles = p.n / BM;
    const int control = 1024 + FEW_OFF_UNITS + 16 * p.num_blocks;
    p.stages = (lim.smem - control) / Few<FORM>::STAGE;
    if (p.stages > FEW_MAX_STAGES) p.stages = FEW_MAX_STAGES;
    const int64_t tiles = 2 * static_cast<int64_t>(p.num_blocks) * p.n_tiles;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles < lim.sms ? tiles : lim.sms));
    cfg.blockDim = dim3(FEW_THREADS);
    cfg.dynamicSmemBytes = static_cast<size_t>(control + p.stages * Few<FORM>::STAGE);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    p.split = 1;
    if constexpr (FORM == MX4_MATMUL) {
        // a plain product's tiles are known here (one block, 64 rows a unit)
        const int32_t k_steps = (p.k_tiles + 1) / 2;
        const int64_t exact = p.num_blocks == 1 ? (p.rows > FEW_ROWS ? 2 : 1) * static_cast<int64_t>(p.n_tiles) : tiles;
        for (int split = 2; split <= FEW_MAX_SPLIT; split *= 2)
            if (exact <= lim.clusters[split] && k_steps >= FEW_SPLIT_STEPS &&
                p.stages * Few<FORM>::STAGE >= split * FEW_ROWS * BM * 4)
                p.split = split;
        if (p.split > 1) {
            attr[1].id = cudaLaunchAttributeClusterDimension;
            attr[1].val.clusterDim.x = static_cast<unsigned>(p.split);
            attr[1].val.clusterDim.y = 1;
            attr[1].val.clusterDim.z = 1;
            cfg.numAttrs = 2;
            cfg.gridDim = dim3(static_cast<unsigned>(exact * p.split));
            return cudaLaunchKernelEx(&cfg, mx4_few_rows_kernel<FORM, BF16, true>, maps, p);
        }
    }
    return cudaLaunchKernelEx(&cfg, mx4_few_rows_kernel<FORM, BF16, false>, maps, p);
}

template <int FORM>
cudaError_t launch(bool bf16, bool few, const Maps& maps, Params& p, cudaStream_t stream) {
    if (few) return bf16 ? launch_few_rows<FORM, true>(maps, p, stream) : launch_few_rows<FORM, false>(maps, p, stream);
    return bf16 ? launch<FORM, true>(maps, p, stream) : launch<FORM, false>(maps, p, stream);
}

}  // namespace

cudaError_t launch_mx4_product(const Mx4Product& a, cudaStream_t stream) {
    if (!tensor_map_encoder()) return cudaErrorNotSupported;
    Maps maps;
    const bool gate_up = a.form == MX4_GATE_UP;
    // Rows per expert are on the device; num_blocks_m (a block per 128 pairs and one
    // per expert) bounds the pairs, and so the average.
    const int64_t pair_blocks = a.form == MX4_MATMUL ? a.num_blocks : a.num_blocks - a.n_experts;
    const int64_t average = gate_up ? FEW_AVERAGE_GATE_UP : FEW_AVERAGE;
    const bool few = (pair_blocks <= 1 || pair_blocks * BM <= average * a.n_experts) &&
                     a.num_blocks <= FEW_MAX_BLOCKS;
    const uint64_t rows = static_cast<uint64_t>(a.rows), kb = static_cast<uint64_t>(a.k) / 2,
                   kt = static_cast<uint64_t>(a.k) / 128;
    const uint64_t brows = static_cast<uint64_t>(a.n_experts) * static_cast<uint64_t>(a.n);
    bool made = tensor_map_2d(&maps.a, a.a, rows, kb, 1, few ? FEW_ROWS : BM) &&
                tensor_map_2d(&maps.a_small, a.a, rows, kb, 1, SMALL_ROWS) &&
                tensor_map_2d(&maps.b, a.b, brows, kb, 1, BM) &&
                tensor_map_scales(&maps.sfa, a.a_scales, (rows + BM - 1) / BM, kt, 1) &&
                tensor_map_scales(&maps.sfb, a.b_scales, brows / BM, kt, few || gate_up ? 1 : 2);
    if (gate_up)
        made = made && tensor_map_2d(&maps.b2, a.b2, brows, kb, 1, BM) &&
               tensor_map_scales(&maps.sfb2, a.b2_scales, brows / BM, kt, 1);
    if (!made) return cudaErrorInvalidValue;
    Params p{};
    p.weights = a.weights;
    p.sizes = a.sizes;
    p.offsets = a.offsets;
    p.padded = a.padded;
    p.gidx = a.gidx;
    p.out = a.out;
    p.status = a.status;
    p.rows = a.rows;
    p.valid_total = a.valid_total;
    p.num_blocks = static_cast<int32_t>(a.num_blocks);
    p.n_experts = a.n_experts;
    p.n = a.n;
    p.n_tiles = gate_up ? a.n / BM : (a.n + BN - 1) / BN;
    p.k_tiles = a.k / 128;
    switch (a.form) {
        case MX4_MATMUL: return launch<MX4_MATMUL>(a.bf16, few, maps, p, stream);
        case MX4_GATE_UP: return launch<MX4_GATE_UP>(a.bf16, few, maps, p, stream);
        default: return launch<MX4_DOWN>(a.bf16, few, maps, p, stream);
    }
}

}  // namespace moe
