// Products on tiles of a CTA pair, for the router's gradients and the orthogonalised
// updates: C[m, n] = Σ_k A[m, k]·B[n, k] over a list of tiles that an operation
// describes, with what becomes of the sums left to the operation too.
//
//  * Persistent clusters of two CTAs, one 2-SM MMA tile of M = 256 x N = 128 or 256 (at most
//    Op::BN) at a time: each CTA holds 128 rows of A and half of the tile's rows of B per stage
//    (K = 64).  Warp 0 feeds the ring by TMA, warp 1 of the even CTA issues the MMAs
//    into one of two TMEM accumulators, warps 2-9 of both CTAs finish the other one
//    meanwhile.
//  * Operands are K-major (K contiguous) or M/N-major (M or N contiguous), as they lie in
//    memory.  All are 3-D arrays [batch, rows, columns] with 16-byte rows; rows
//    and columns past the end are zeros that TMA fills in.
//  * Copies and MMAs are issued by converged warps, waits are bounded, and a wait that
//    runs out ends the launch as in the other products.
//
// An operation `Op` has
//     BN, BF16, MASKABLE       most columns of a tile, operand type, see below
//     QUEUE                    see below
//     Params                   with int32_t total_tiles, n_maps, *status
//     Code, code(p, t)         what all roles need to know of tile t: four or eight bytes
//     tile(p, code)            what it multiplies (nothing where it has no steps)
//     Finish(p, smem, ...)     per epilogue warp: before(code) ahead of the sums (false where
//                              there are none), width_of() its columns, pass(c, taddr)
//                              for 64 of them, of the warp's 32 rows
//
// QUEUE: pairs take tiles from a counter in memory (Params::queue, zero at the start) in the order of
// their numbers instead of every n-th one, and a tile may need results of lower ones:
// Op::wait(p, code, abort) returns once they are there, Op::publish(p, code) says that this CTA's part
// of a tile is.  Whoever holds the lowest unfinished tile never waits for one that no running
// pair holds, so this needs no pair to be resident beside another.  The even CTA's warp 11 takes a
// tile as soon as the one before is being copied, waits for what it reads, and hands its code to all
// roles of both CTAs through a ring: all that costs some 3 us, which nobody waits for while there is
// work.  Publishing waits for stores to arrive, which takes microseconds too where all SMs
// store: warp 10 of either CTA does it.
//
// MASKABLE: where Op::dirty(p) says so, rows of an M/N-major B (rows of K) whose bit
// Op::valid64 gives as 0 are set to zero in shared memory before they are multiplied, so
// that what stands there, a NaN say, meets nothing.  Each CTA then has its own "full"
// barriers, its warp 1 clears the rows, and the odd CTA's reports its half to the even one's.
// (That hop doubles the time of a launch, so it is taken only if there is something to remove.)
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "../../include/moe_gb300.h"
#include "moe_internal.h"
#include "sm103_products.cuh"
#include "tensor_map.h"
#include "tile_store.cuh"

namespace moe {
namespace pairs {

constexpr int BM = 128;                        // rows of A per CTA
constexpr int BK = 64;                         // K per stage
constexpr int THREADS = 320;                   // producer, MMA and eight epilogue warps
constexpr int THREADS_QUEUE = 384;             // with a queue: and one that publishes, one that takes tiles
constexpr int EPI_WARPS = 8;
constexpr int MAX_MAPS = 10;
constexpr int QUEUE = 8;                       // tiles that the roles of a pair may be apart
constexpr int A_BYTES = BM * BK * 2;
constexpr int BOX_BYTES = BK * 128;            // an M/N-major box: 64 along M/N x BK rows of K
constexpr int STAGING_BYTES = 32 * 128;        // per epilogue warp
constexpr uint64_t WAIT_LIMIT_NS = 2000000000ull;
constexpr uint64_t DRAIN_LIMIT_NS = 200000000ull;

struct Maps {
    CUtensorMap m[MAX_MAPS];
};

// What a tile multiplies: rows a_row .. + 255 of A by rows b_row .. + width - 1 of B
// (coordinates in their own arrays), K steps k0 .. k0 + steps of 64; with two terms, each step twice,
// by A's next matrix the second time (`steps` counts both).
struct Tile {
    int32_t a_map, b_map;
    bool a_mn, b_mn;
    int32_t a_row, b_row, batch;
    int32_t k0, steps;
    int32_t width;                 // 128 or 256 columns
    int32_t two;                   // 1: two terms
};

template <int BN>
struct Layout {
    static constexpr int B_BYTES = BN / 2 * BK * 2;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int STAGES = 196608 / STAGE_BYTES;          // (a tile of 128 columns in stages for 256 leaves a quarter free)
    static constexpr int OFF_STAGING = STAGES * STAGE_BYTES;
    static constexpr int OFF_BARS = OFF_STAGING + EPI_WARPS * STAGING_BYTES;
    static constexpr int NUM_BARS = 3 * STAGES + 2 + 2 + 1 + 3 * QUEUE + 1;   // full, empty, peer, tfull, tempty, drain, queue, stored, taken
    static constexpr int OFF_QUEUE = OFF_BARS + NUM_BARS * 8;
    static constexpr int OFF_TMEM_SLOT = OFF_QUEUE + 8 * QUEUE;
    static constexpr int OFF_ABORT = OFF_TMEM_SLOT + 4;
    static constexpr int SMEM_BYTES = 1024 + OFF_ABORT + 4;
    static constexpr int TMEM_COLS = 2 * BN;
    static_assert(SMEM_BYTES <= 227 * 1024, "the ring fits");
};

__device__ __forceinline__ void tma_load_3d_pair_if(uint32_t issue, uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                                    int32_t c0, int32_t c1, int32_t c2, uint64_t policy) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.b32 e, %7, 0;\n\t"
        "@e cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;\n\t}"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy), "r"(issue)
        : "memory");
}

template <class Op>
__global__ void __launch_bounds__(Op::QUEUE ? THREADS_QUEUE : THREADS, 1)
pair_kernel(const __grid_constant__ Maps maps, const __grid_constant__ typename Op::Params p) {
    constexpr int BN = Op::BN;
    using L = Layout<BN>;
    constexpr int STAGES = L::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem =
        reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar_full = sbase + L::OFF_BARS;               // [STAGES]
    const uint32_t bar_empty = bar_full + 8 * STAGES;            // [STAGES]
    const uint32_t bar_peer = bar_empty + 8 * STAGES;            // [STAGES] masked: the odd CTA's half is there
    const uint32_t bar_tfull = bar_peer + 8 * STAGES;            // [2]
    const uint32_t bar_tempty = bar_tfull + 16;                  // [2] (used in the even CTA)
    const uint32_t bar_drain = bar_tempty + 16;                  // [1]
    const uint32_t bar_qfull = bar_drain + 8;                    // [QUEUE]
    const uint32_t bar_qempty = bar_qfull + 8 * QUEUE;           // [QUEUE] (used in the even CTA)
    const uint32_t bar_stored = bar_qempty + 8 * QUEUE;          // [QUEUE] a tile's rows are stored by this CTA's warps
    const uint32_t bar_taken = bar_stored + 8 * QUEUE;           // [1] (used in the even CTA) a tile is being copied
    using Code = typename Op::Code;
    static_assert(sizeof(Code) <= 8, "an entry of the queue");
    volatile int2* queue = reinterpret_cast<volatile int2*>(smem + L::OFF_QUEUE);      // x: end of the list, y and x: a code
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + L::OFF_TMEM_SLOT);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_ABORT);

    const int tid = threadIdx.x;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);      // known to be warp-uniform
    const int lane = tid & 31;
    const uint32_t rank = cluster_cta_rank();
    const bool leader = rank == 0;

    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar_full + 8 * s, 1);           // arrive.expect_tx
            mbar_init(bar_empty + 8 * s, 1);          // the MMAs' commit, multicast to both CTAs
            mbar_init(bar_peer + 8 * s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(bar_tfull + 8 * a, 1);
            mbar_init(bar_tempty + 8 * a, 2 * EPI_WARPS);
        }
        mbar_init(bar_drain, 1);
        for (int q = 0; q < QUEUE; ++q) {
            mbar_init(bar_qfull + 8 * q, 1);
            mbar_init(bar_qempty + 8 * q, 2 * EPI_WARPS + 5);    // producers, MMA issuer, epilogues, publishers
            mbar_init(bar_stored + 8 * q, EPI_WARPS);
        }
        mbar_init(bar_taken, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane < p.n_maps) tma_prefetch_map(&maps.m[lane]);
    if (warp == 1) {
        tmem_alloc_pair(sbase + L::OFF_TMEM_SLOT, L::TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    // Everything above overlaps the kernel before; every global access is below.  The
    // next kernel may start only now that this CTA holds its TMEM.
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const bool masked = Op::MASKABLE && __syncthreads_or(Op::dirty(p)) != 0;       // the same in all CTAs
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    cluster_sync_all();            // both CTAs' barriers exist before copies and commits cross

    const int32_t pair = static_cast<int32_t>(blockIdx.x) / 2;
    const int32_t n_pairs = static_cast<int32_t>(gridDim.x) / 2;
    const uint32_t issue = elect_one();
    int64_t issued = 0;            // stages that warp 0 has filled

    // The next tile of this warp's role: its code, or false past the last one.
    uint32_t qslot = 0, qphase = 0;
    int32_t t_static = pair;
    const uint32_t leader_qempty = mapa_shared(bar_qempty, 0);
    auto next_slot = [&]() {
        if (++qslot == QUEUE) { qslot = 0; qphase ^= 1u; }
    };
    auto free_slot = [&]() {
        // (relaxed: the entry is in registers, and a release would wait for this thread's stores in flight)
        if (lane == 0) mbar_arrive_cluster_relaxed(leader_qempty + 8 * qslot);
        next_slot();
    };
    auto next_tile = [&](Code& code, bool keep_slot = false) -> bool {
        if constexpr (!Op::QUEUE) {
            const int32_t t = t_static;
            t_static += n_pairs;
            code = Op::code(p, t);
            return t < p.total_tiles;
        } else {
            const bool there = mbar_wait_bounded<true>(bar_qfull + 8 * qslot, qphase, abort_flag, WAIT_LIMIT_NS);
            if (!__all_sync(0xffffffffu, there)) return false;
            const int32_t x = __shfl_sync(0xffffffffu, queue[qslot].x, 0), y = __shfl_sync(0xffffffffu, queue[qslot].y, 0);
            if (!keep_slot) free_slot();
            code = Op::unpack(x, y);
            return x >= 0;
        }
    };

    if (warp == 0) {
        // ---- TMA producer, both CTAs
        const uint64_t policy = l2_policy_evict_normal();
        const uint32_t full0 = mapa_shared(bar_full, masked ? rank : 0u);
        const uint32_t expect = masked || leader ? issue : 0;
        uint32_t stage = 0, phase = 0;
        bool ok = true;
        Code code;
        while (ok && next_tile(code)) {
            const Tile ti = Op::tile(p, code);
            if constexpr (Op::QUEUE) {
                if (leader && lane == 0) mbar_arrive(bar_taken);
                // what generic stores wrote is read by TMA from here on
                asm volatile("fence.proxy.async.global;" ::: "memory");
            }
            if (ti.steps == 0) continue;
            const int32_t arow = ti.a_row + static_cast<int32_t>(rank) * BM;
            const int32_t brow = ti.b_row + static_cast<int32_t>(rank) * (ti.width / 2);
            const uint32_t bytes = static_cast<uint32_t>(masked ? 1 : 2) * (A_BYTES + static_cast<uint32_t>(ti.width) * BK);
            const bool wide = BN == 256 && ti.width == 256;
            const CUtensorMap* am = &maps.m[ti.a_map];
            const CUtensorMap* bm = &maps.m[ti.b_map];
            MOE_DCHECK(ti.a_map >= 0 && ti.a_map < p.n_maps && ti.b_map >= 0 && ti.b_map < p.n_maps && ti.steps > 0 &&
                           ti.k0 >= 0 && arow >= 0 && brow >= 0 && ti.batch >= 0,
                       p.status);
            for (int32_t st = 0; st < ti.steps; ++st) {
                if (!mbar_wait_warp(bar_empty + 8 * stage, phase ^ 1u, abort_flag, WAIT_LIMIT_NS)) {
                    ok = false;
                    break;
                }
                const uint32_t fb = full0 + 8 * stage;
                const uint32_t sa = sbase + stage * L::STAGE_BYTES;
                const uint32_t sb = sa + A_BYTES;
                const int32_t k = (ti.k0 + (st >> ti.two)) * BK;
                const int32_t a_batch = ti.batch + (st & ti.two);
                mbar_arrive_expect_tx_if(expect, bar_full + 8 * stage, bytes);
                if (ti.a_mn) {
#pragma unroll
                    for (int b = 0; b < BM / 64; ++b)
                        tma_load_3d_pair_if(issue, sa + b * BOX_BYTES, am, fb, arow + b * 64, k, a_batch, policy);
                } else {
                    tma_load_3d_pair_if(issue, sa, am, fb, k, arow, a_batch, policy);
                }
                if (ti.b_mn) {
                    tma_load_3d_pair_if(issue, sb, bm, fb, brow, k, ti.batch, policy);
                    if (wide) tma_load_3d_pair_if(issue, sb + BOX_BYTES, bm, fb, brow + 64, k, ti.batch, policy);
                } else {
                    tma_load_3d_pair_if(issue, sb, bm, fb, k, brow, ti.batch, policy);
                }
                ++issued;
                if (++stage == STAGES) { stage = 0; phase ^= 1u; }
            }
        }
    } else if (warp == 1) {
        // ---- MMA issuer: warp 1 of the even CTA (masked: the odd CTA's clears its rows)
        const uint32_t leader_peer = mapa_shared(bar_peer, 0);
        uint32_t stage = 0, phase = 0, acc = 0, aphase = 0;
        bool ok = true;
        Code code;
        while (ok && (leader || masked) && next_tile(code)) {
            const Tile ti = Op::tile(p, code);
            if (ti.steps == 0) continue;
            if (leader) {
                if (!mbar_wait_warp(bar_tempty + 8 * acc, aphase ^ 1u, abort_flag, WAIT_LIMIT_NS)) break;
                tc_fence_after_sync();
            }
            const uint32_t d_tmem = tmem_base + acc * BN;
            const uint32_t idesc = idesc_16bit_f32acc(2 * BM, static_cast<uint32_t>(ti.width), Op::BF16, ti.a_mn, ti.b_mn);
            uint32_t w0 = 0xffffffffu, w1 = 0xffffffffu;         // the stage's 64 valid bits
            if constexpr (Op::MASKABLE) {
                if (masked && Op::maskable(ti)) Op::valid64(p, ti.k0, w0, w1);
            }
            for (int32_t st = 0; st < ti.steps; ++st) {
                uint32_t n0 = 0xffffffffu, n1 = 0xffffffffu;
                if constexpr (Op::MASKABLE) {
                    if (masked && st + 1 < ti.steps && Op::maskable(ti)) Op::valid64(p, ti.k0 + ((st + 1) >> ti.two), n0, n1);
                }
                if (!mbar_wait_warp(bar_full + 8 * stage, phase, abort_flag, WAIT_LIMIT_NS)) {
                    ok = false;
                    break;
                }
                const uint32_t sa = sbase + stage * L::STAGE_BYTES;
                const uint32_t sb = sa + A_BYTES;
                if (Op::MASKABLE && masked) {
                    if ((w0 & w1) != 0xffffffffu) {
                        // K rows are whole 128-byte lines of each box
                        uint8_t* b0 = smem + stage * L::STAGE_BYTES + A_BYTES;
                        for (int half = 0; half < 2; ++half) {
                            for (uint32_t bad = ~(half ? w1 : w0); bad != 0; bad &= bad - 1) {
                                const int r = 32 * half + __ffs(static_cast<int>(bad)) - 1;
                                if (lane < 8 * (BN / 128))
                                    *reinterpret_cast<uint4*>(b0 + (lane >> 3) * BOX_BYTES + r * 128 + (lane & 7) * 16) =
                                        make_uint4(0, 0, 0, 0);
                            }
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    }
                    __syncwarp();
                    w0 = n0;
                    w1 = n1;
                    if (!leader) {
                        if (lane == 0) mbar_arrive_cluster(leader_peer + 8 * stage);
                        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                        continue;
                    }
                    const bool there = mbar_wait_bounded<true>(bar_peer + 8 * stage, phase, abort_flag, WAIT_LIMIT_NS);
                    if (!__all_sync(0xffffffffu, there)) {
                        ok = false;
                        break;
                    }
                }
                tc_fence_after_sync();
                const uint64_t da = ti.a_mn ? smem_desc_mn_sw128(sa, BOX_BYTES) : smem_desc_k_sw128(sa);
                const uint64_t db = ti.b_mn ? smem_desc_mn_sw128(sb, BOX_BYTES) : smem_desc_k_sw128(sb);
                const uint32_t a_step = ti.a_mn ? 2048 >> 4 : 32 >> 4, b_step = ti.b_mn ? 2048 >> 4 : 32 >> 4;
#pragma unroll
                for (int kk = 0; kk < BK / 16; ++kk)
                    tc_mma_f16_pair_if(issue, d_tmem, da + kk * a_step, db + kk * b_step, idesc,
                                       (st != 0 || kk != 0) ? 1u : 0u);
                tc_commit_pair_mc_if(issue, bar_empty + 8 * stage, 0x3);
                if (++stage == STAGES) { stage = 0; phase ^= 1u; }
            }
            if (!ok) break;
            if (leader) tc_commit_pair_mc_if(issue, bar_tfull + 8 * acc, 0x3);
            acc ^= 1u;
            if (acc == 0) aphase ^= 1u;
        }
        if (leader && issue) {
            // every MMA this warp issued has finished once this arrives
            volatile int never = 0;
            tc_commit_pair(bar_drain);
            mbar_wait_bounded(bar_drain, 0, &never, DRAIN_LIMIT_NS);
        }
        __syncwarp();
    } else if (warp < 2 + EPI_WARPS) {
        // ---- epilogue: a warp has 32 of the CTA's rows, and every other 64 columns
        const int quarter = warp & 3;
        const int odd = warp >= 6 ? 1 : 0;
        uint8_t* staging = smem + L::OFF_STAGING + (warp - 2) * STAGING_BYTES;
        const uint32_t leader_tempty = mapa_shared(bar_tempty, 0);
        typename Op::Finish fin(p, staging, static_cast<int32_t>(rank) * BM + quarter * 32, odd, lane);
        uint32_t acc = 0, aphase = 0;
        Code code;
        while (true) {
            const uint32_t slot = qslot;
            if (!next_tile(code)) break;
            if (!fin.before(code)) continue;
            // one answer for the whole warp, whose TMEM loads are collective
            if (!mbar_wait_warp(bar_tfull + 8 * acc, aphase, abort_flag, WAIT_LIMIT_NS)) break;
            tc_fence_after_sync();
            const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * BN;
#pragma unroll 1
            for (int c = odd; c < fin.width_of() / 64; c += 2) fin.pass(c, taddr + c * 64);
            tc_fence_before_sync();
            // the accumulator may be reused once both CTAs have read their rows
            __syncwarp();
            if (lane == 0) {
                if (leader) mbar_arrive(bar_tempty + 8 * acc);
                else mbar_arrive_cluster_relaxed(leader_tempty + 8 * acc);
            }
            if constexpr (Op::QUEUE) {
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_stored + 8 * slot);
            }
            acc ^= 1u;
            if (acc == 0) aphase ^= 1u;
        }
    } else if constexpr (Op::QUEUE) {
        if (warp == 2 + EPI_WARPS) {
            // ---- publisher
            Code code;
            while (next_tile(code, true)) {
                // (a slot's next tile may come only when this phase of its barrier has been seen)
                if (!mbar_wait_warp(bar_stored + 8 * qslot, qphase, abort_flag, WAIT_LIMIT_NS)) break;
                free_slot();
                if (lane == 0) Op::publish(p, code);
                __syncwarp();
            }
        } else if (leader) {
            // ---- takes tiles, in whole-warp steps; lane 0 holds the number
            uint32_t tphase = 0;
            while (true) {
                int32_t t = lane == 0 ? atomicAdd(p.queue, 1) : 0;
                t = __shfl_sync(0xffffffffu, t, 0);
                const bool end = t >= p.total_tiles;
                Code code = Op::code(p, end ? 0 : t);
                if (!end && !Op::wait(p, code, abort_flag)) break;
                asm volatile("fence.proxy.async.global;" ::: "memory");
                if (!mbar_wait_warp(bar_qempty + 8 * qslot, qphase ^ 1u, abort_flag, WAIT_LIMIT_NS)) break;
                if (lane < 2) {
                    // lane 0 for this CTA, lane 1 for the other
                    int32_t x, y;
                    Op::pack(code, x, y);
                    if (end) x = -1;
                    const uint32_t at = mapa_shared(sbase + L::OFF_QUEUE + 8 * qslot, static_cast<uint32_t>(lane));
                    asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(x), "r"(y) : "memory");
                    mbar_arrive_cluster(mapa_shared(bar_qfull + 8 * qslot, static_cast<uint32_t>(lane)));
                }
                __syncwarp();
                next_slot();
                if (end) break;
                // the next one when this one is being copied, not before: another pair may be free
                if (!mbar_wait_warp(bar_taken, tphase, abort_flag, WAIT_LIMIT_NS)) break;
                tphase ^= 1u;
            }
        }
    }
    __syncwarp();

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 0 && lane == 0 && *abort_flag) {
        // Whichever role gave up: copies in flight land before the CTA exits.
        // (The odd CTA's report to the even CTA's barriers, unless each has its own.)
        if (leader || masked) drain_copies(bar_full, issued, STAGES, DRAIN_LIMIT_NS);
        else spin_ns(1000000ull);
    }
    __syncwarp();
    // No CTA leaves (or frees the pair's TMEM) while the other may still copy into its
    // shared memory, arrive on its barriers or use the TMEM.
    cluster_sync_all();
    if (*abort_flag && tid == 0 && p.status) atomicOr(p.status, MOE_DEV_TIMEOUT);
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem_base, L::TMEM_COLS);
    }
}

// Pairs that fit on the device at once, after opting in to the kernel's shared memory; asked
// once per device.  0 on an error.
template <class Op>
int resident_pairs() {
    struct Entry {
        std::once_flag once;
        int pairs = 0;
    };
    constexpr int MAX_DEVICES = 16;
    static Entry table[MAX_DEVICES];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= MAX_DEVICES) return 0;
    Entry& r = table[dev];
    std::call_once(r.once, [&r] {
        constexpr int SMEM = Layout<Op::BN>::SMEM_BYTES;
        if (cudaFuncSetAttribute(pair_kernel<Op>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) != cudaSuccess)
            return;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(128);
        cfg.blockDim = dim3(Op::QUEUE ? THREADS_QUEUE : THREADS);
        cfg.dynamicSmemBytes = SMEM;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, pair_kernel<Op>, &cfg) == cudaSuccess && n > 0) r.pairs = n;
    });
    return r.pairs;
}

// `most` pairs, or as many as fit on the device and have a tile.
template <class Op>
cudaError_t launch(const Maps& maps, const typename Op::Params& p, cudaStream_t stream, int most = 1 << 20) {
    int pairs = resident_pairs<Op>();
    if (pairs == 0) return cudaErrorNoDevice;
    if (pairs > most) pairs = most;
    if (pairs > p.total_tiles) pairs = p.total_tiles;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
    cfg.blockDim = dim3(Op::QUEUE ? THREADS_QUEUE : THREADS);
    cfg.dynamicSmemBytes = Layout<Op::BN>::SMEM_BYTES;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, pair_kernel<Op>, maps, p);
}

// [batch, rows, cols] of 16-bit elements with rows `stride` elements apart (a multiple of 8), box of
// 64 columns x box_rows, 128-byte swizzle, zeros outside.
inline bool map_3d(CUtensorMap* m, const void* base, int64_t batch, int64_t rows, int64_t cols, int64_t stride,
                   int box_rows) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(batch)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(stride) * 2, static_cast<cuuint64_t>(rows * stride) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return tensor_map_encoder()(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline int32_t ceil_div(int64_t a, int64_t b) { return static_cast<int32_t>((a + b - 1) / b); }

}  // namespace pairs
}  // namespace moe
