// Forward of the dense gated feed-forward block for few tokens.
//
// With T tokens at hand every weight is used T times, so for small T the block is
// the time to read gate_w, up_w and down_w once; what counts is that all of the
// chip reads, from the first microsecond.  The products are therefore turned
// around: a CTA takes 128 weight rows as the M side of the MMA and the tokens as
// its N side (T rounded up to 16), so no tile is spent on tokens that are not
// there, and the K axis is split over a cluster of S CTAs, S chosen so that
// about two CTAs per SM stream.
//  * Gate and up: 64 rows of gate_w and the same 64 of up_w make one tile, so both
//    projections of a column meet in one CTA's results and h is formed there.
//  * A ring of 64-wide K slices (weights 16 KB, tokens T·128 bytes) fed by TMA with
//    128-byte swizzle; one warp feeds, one issues MMAs, four join and store.
//  * Joining: each CTA leaves its fp32 partial sums in its own shared memory; after
//    a cluster barrier the S CTAs divide the outputs and add the S partial sums
//    in rank order, read over distributed shared memory.  The order is fixed, so
//    results do not change from run to run, and nothing goes through memory.
//  * Copies and MMAs are issued by converged warps: the first stages are on their
//    way a microsecond earlier than from one lane (one token, 2048 / 2816: 14.3 ->
//    12.3 us).
//  * The down product is launched with programmatic dependent launch and fills its
//    ring with weights before it waits for h.
//
// Measured (GPU time): one token 7168 / 2048 20.5 us for 88 MB of weights (the
// streams themselves run at 6.5 TB/s; the rest is two joins of about 2 us and 2.5 us
// from one grid's end to the next one's start), 37 tokens 2048 / 2816 14.5 us.
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

constexpr int BM = 128;                        // weight rows per tile
constexpr int BK = 64;                         // K per stage: one 128-byte swizzle row
constexpr int W_BYTES = BM * BK * 2;
constexpr int MAX_STAGES = 8;
constexpr int MAX_CLUSTER = 8;
constexpr int MAX_NP = static_cast<int>((FFN_SMALL_TOKENS + 15) / 16 * 16);
constexpr int NUM_THREADS = 192;
constexpr int NUM_EPI_THREADS = 128;
constexpr int SMEM_LIMIT = 112 * 1024;         // two CTAs per SM
// Launches of at most so many weight bytes ask L2 for all of them ahead of the wait.  Up
// to there it saves 0.2 to 1.3 us a forward (hidden / intermediate 2048 / 1408, 64 tokens
// 14.8 -> 14.4; 2048 / 2816 17.3 -> 16.1; one token of 2048 / 1024 alone loses 0.2).
// Gate and up of 32 to 48 MB go either way (4096 / 2816, one token 17.2 -> 17.7; 2048 /
// 4096, 64 tokens 19.1 -> 18.3; 6144 / 2048 27.8 -> 27.2), and above 56 MB the lines asked
// for hold up the stages' own loads (7168 / 2048 24.7 -> 26.9; 4096 / 8192 40.8 -> 46.6).
constexpr int64_t PREFETCH_BYTES = 24ll << 20;
constexpr uint64_t WAIT_LIMIT_NS = 2000000000ull;
constexpr uint64_t DRAIN_LIMIT_NS = 200000000ull;

constexpr int OFF_BARS = 0;                    // full, empty [MAX_STAGES]; done
constexpr int OFF_TMEM_SLOT = (2 * MAX_STAGES + 1) * 8;
constexpr int OFF_ABORT = OFF_TMEM_SLOT + 4;
constexpr int CTL_BYTES = 256;
static_assert(OFF_ABORT + 4 <= CTL_BYTES, "control area");

struct Params {
    uint16_t* dst;             // h (gate and up) or out, [tokens, n]
    uint16_t* dst_gate;        // nullable
    uint16_t* dst_up;
    int32_t* status;
    int32_t tokens;
    int32_t n;                 // columns of dst
    int32_t chunks;            // K slices of 64 in all
    int32_t np;                // tokens rounded up to 16
    int32_t stages;
    int32_t tmem_cols;
    int32_t prefetch;          // ask for the weights ahead of the wait
};

__device__ __forceinline__ float4 load_remote4(uint32_t cluster_addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(cluster_addr) : "memory");
    return v;
}

template <bool GATE_UP, bool BF16>
__global__ void __launch_bounds__(NUM_THREADS)
ffn_small_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                 const __grid_constant__ CUtensorMap map_w2, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem =
        reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t x_bytes = static_cast<uint32_t>(p.np) * BK * 2;
    const uint32_t stage_bytes = W_BYTES + x_bytes;
    uint8_t* ctl = smem + p.stages * stage_bytes;
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar_full = smem_u32(ctl) + OFF_BARS;
    const uint32_t bar_empty = bar_full + 8 * MAX_STAGES;
    const uint32_t bar_done = bar_empty + 8 * MAX_STAGES;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(ctl + OFF_TMEM_SLOT);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(ctl + OFF_ABORT);

    const int tid = threadIdx.x;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);     // known to be warp-uniform
    const int lane = tid & 31;
    const uint32_t rank = cluster_cta_rank();
    uint32_t nranks;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(nranks));
    const int32_t tile = static_cast<int32_t>(blockIdx.x / nranks);
    // this CTA's K slices
    const int32_t c0 = static_cast<int32_t>(static_cast<int64_t>(p.chunks) * rank / nranks);
    const int32_t c1 = static_cast<int32_t>(static_cast<int64_t>(p.chunks) * (rank + 1) / nranks);
    const int32_t stages = p.stages;
    MOE_DCHECK(c0 < c1 && c1 <= p.chunks && tile * (GATE_UP ? BM / 2 : BM) < p.n && nranks <= MAX_CLUSTER, p.status);
    MOE_DCHECK(p.tokens <= p.np && p.np * BM * 4 <= stages * static_cast<int32_t>(stage_bytes) && p.np <= p.tmem_cols,
               p.status);

    if (tid == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 1);
        }
        mbar_init(bar_done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(ctl) + OFF_TMEM_SLOT, static_cast<uint32_t>(p.tmem_cols));
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);

    int32_t issued = 0;            // stages fed, by warp 0
    if (warp == 0) {
        // ===================== producer =====================
        const uint32_t issue = elect_one();
        const uint64_t policy = l2_policy_evict_normal();
        auto load_w = [&](int32_t c, int32_t s) {
            const uint32_t fb = bar_full + 8 * s, dst = sbase + s * stage_bytes;
            mbar_arrive_expect_tx_if(issue, fb, stage_bytes);
            if (GATE_UP) {
                tma_load_2d_if(issue, dst, &map_w, fb, c * BK, tile * (BM / 2), policy);
                tma_load_2d_if(issue, dst + W_BYTES / 2, &map_w2, fb, c * BK, tile * (BM / 2), policy);
            } else {
                tma_load_2d_if(issue, dst, &map_w, fb, c * BK, tile * BM, policy);
            }
        };
        auto load_x = [&](int32_t c, int32_t s) {
            tma_load_2d_if(issue, sbase + s * stage_bytes + W_BYTES, &map_x, bar_full + 8 * s, c * BK, 0, policy);
        };
        const int32_t first = c1 - c0 < stages ? c1 - c0 : stages;
        // Weight lines on their way into L2 while the grid before still works.
        for (int32_t c = c0 + (GATE_UP ? 0 : first); p.prefetch && c < c1; ++c) {
            if (!issue) break;
            if (GATE_UP) {
                tma_prefetch_2d(&map_w, c * BK, tile * (BM / 2));
                tma_prefetch_2d(&map_w2, c * BK, tile * (BM / 2));
            } else {
                tma_prefetch_2d(&map_w, c * BK, tile * BM);
            }
        }
        __syncwarp();
        if (GATE_UP) pdl_wait_prior_grid();
        // Behind the gate and up launch of the same call the weights may be
        // read at once: that launch lets this one start only after its own
        // wait for everything before it, and writes no weights.
        for (int32_t i = 0; i < first; ++i) load_w(c0 + i, i);
        if (!GATE_UP) pdl_wait_prior_grid();
        for (int32_t i = 0; i < first; ++i) load_x(c0 + i, i);
        int32_t stage = first == stages ? 0 : first;
        uint32_t phase = first == stages ? 1u : 0u;
        int32_t c = c0 + first;
        for (; c < c1; ++c) {
            if (!mbar_wait_warp(bar_empty + 8 * stage, phase ^ 1u, abort_flag, WAIT_LIMIT_NS)) break;
            load_w(c, stage);
            load_x(c, stage);
            if (++stage == stages) { stage = 0; phase ^= 1u; }
        }
        issued = c - c0;
        __syncwarp();
    } else if (warp == 1) {
        // ===================== MMA issuer =====================
        pdl_wait_prior_grid();     // no bounded wait runs while the launch before still works
        const uint32_t issue = elect_one();
        const uint32_t idesc = idesc_16bit_f32acc(BM, static_cast<uint32_t>(p.np), BF16, false, false);
        int32_t stage = 0;
        uint32_t phase = 0;
        for (int32_t c = c0; c < c1; ++c) {
            if (!mbar_wait_warp(bar_full + 8 * stage, phase, abort_flag, WAIT_LIMIT_NS)) break;
            tc_fence_after_sync();
            const uint64_t dw = smem_desc_k_sw128(sbase + stage * stage_bytes);
            const uint64_t dx = smem_desc_k_sw128(sbase + stage * stage_bytes + W_BYTES);
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
                tc_mma_f16_if(issue, tmem_base, dw + kk * 2, dx + kk * 2, idesc, (c != c0 || kk != 0) ? 1u : 0u);
            tc_commit_if(issue, bar_empty + 8 * stage);
            if (++stage == stages) { stage = 0; phase ^= 1u; }
        }
        tc_commit_if(issue, bar_done);
        __syncwarp();
    } else {
        // ===================== partial sums to shared memory =====================
        // after the last MMA the ring is free: [token][weight row] in fp32
        pdl_wait_prior_grid();
        // one answer for the whole warp, whose TMEM loads are collective
        if (mbar_wait_warp(bar_done, 0, abort_flag, WAIT_LIMIT_NS)) {
            tc_fence_after_sync();
            const int row = (warp & 3) * 32 + lane;
            const uint32_t taddr = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16);
            float* part = reinterpret_cast<float*>(smem);
#pragma unroll 1
            for (int t0 = 0; t0 < p.tokens; t0 += 16) {
                uint32_t v[8], w[8];
                tmem_ld_32x32b_x8(taddr + t0, v);
                tmem_ld_32x32b_x8(taddr + t0 + 8, w);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    part[(t0 + j) * BM + row] = __uint_as_float(v[j]);
                    part[(t0 + 8 + j) * BM + row] = __uint_as_float(w[j]);
                }
            }
            tc_fence_before_sync();
        }
    }
    // The next launch may start: everything this one reads from memory is on its way.
    pdl_launch_dependents();
    __syncwarp();
    cluster_sync_all();
    // Whichever role gave up: copies in flight land before the CTA exits.
    if (warp == 0 && lane == 0 && *abort_flag) drain_copies(bar_full, issued, stages, DRAIN_LIMIT_NS);

    // ===================== join and store =====================
    if (warp >= 2 && !*abort_flag) {
        constexpr int QUADS = (GATE_UP ? BM / 2 : BM) / 4;      // groups of 4 columns of a token
        const int32_t col0 = tile * (GATE_UP ? BM / 2 : BM);
        const int32_t total = p.tokens * QUADS;
        const uint32_t mine = sbase;
        for (int32_t i = static_cast<int32_t>(rank) * NUM_EPI_THREADS + tid - 64; i < total;
             i += static_cast<int32_t>(nranks) * NUM_EPI_THREADS) {
            const int32_t t = i / QUADS, q = i - t * QUADS;
            const uint32_t at = mine + static_cast<uint32_t>((t * BM + q * 4) * 4);
            // all ranks' loads in flight together, then added in rank order
            float4 v[MAX_CLUSTER], u[GATE_UP ? MAX_CLUSTER : 1];
#pragma unroll
            for (uint32_t r = 0; r < MAX_CLUSTER; ++r) {
                if (r >= nranks) break;
                const uint32_t src = mapa_shared(at, r);
                v[r] = load_remote4(src);
                if (GATE_UP) u[r] = load_remote4(src + BM / 2 * 4);
            }
            float4 a = v[0], b = u[0];
#pragma unroll
            for (uint32_t r = 1; r < MAX_CLUSTER; ++r) {
                if (r >= nranks) break;
                a.x += v[r].x; a.y += v[r].y; a.z += v[r].z; a.w += v[r].w;
                if (GATE_UP) { b.x += u[r].x; b.y += u[r].y; b.z += u[r].z; b.w += u[r].w; }
            }
            const int32_t col = col0 + q * 4;
            if (col >= p.n) continue;
            const int64_t o = static_cast<int64_t>(t) * p.n + col;
            MOE_DCHECK(t >= 0 && t < p.tokens && col >= 0 && col + 4 <= p.n, p.status);
            auto put = [&](uint16_t* d, const float4& v) {
                *reinterpret_cast<uint2*>(d + o) = make_uint2(pack_16bit2<BF16>(v.x, v.y), pack_16bit2<BF16>(v.z, v.w));
            };
            if (GATE_UP) {
                if (p.dst_gate != nullptr) {
                    put(p.dst_gate, a);
                    put(p.dst_up, b);
                }
                a.x *= sigmoid_approx(a.x) * b.x;
                a.y *= sigmoid_approx(a.y) * b.y;
                a.z *= sigmoid_approx(a.z) * b.z;
                a.w *= sigmoid_approx(a.w) * b.w;
            }
            put(p.dst, a);
        }
    }
    __syncwarp();
    cluster_sync_all();            // no CTA's partial sums leave before all have read them
    if (*abort_flag && tid == 0 && p.status) atomicOr(p.status, MOE_DEV_TIMEOUT);
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, static_cast<uint32_t>(p.tmem_cols));
    }
}

template <bool GATE_UP, bool BF16>
cudaError_t launch(const CUtensorMap& mx, const CUtensorMap& mw, const CUtensorMap& mw2, Params& p, int32_t k,
                   cudaStream_t stream) {
    static std::once_flag once[16];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev >= 16) return cudaErrorNoDevice;
    std::call_once(once[dev], [&] {
        err = cudaFuncSetAttribute(ffn_small_kernel<GATE_UP, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   SMEM_LIMIT);
    });
    if (err != cudaSuccess) return err;
    const int stage_bytes = W_BYTES + p.np * BK * 2;
    p.chunks = (k + BK - 1) / BK;
    p.stages = (SMEM_LIMIT - 1024 - CTL_BYTES) / stage_bytes;
    if (p.stages > MAX_STAGES) p.stages = MAX_STAGES;
    p.tmem_cols = p.np <= 32 ? 32 : (p.np <= 64 ? 64 : 128);
    const int32_t cols = GATE_UP ? BM / 2 : BM;
    const int32_t tiles = (p.n + cols - 1) / cols;
    // K split: up to two CTAs per SM, each with a slice of its own
    const int sms = device_sm_count();
    int32_t s = 2 * sms / tiles;
    if (s > MAX_CLUSTER) s = MAX_CLUSTER;
    if (s > p.chunks) s = p.chunks;
    if (s < 1) s = 1;
    const int64_t weights = static_cast<int64_t>(p.n) * k * 2 * (GATE_UP ? 2 : 1);
    p.prefetch = weights <= PREFETCH_BYTES ? 1 : 0;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(s);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(s * tiles));
    cfg.blockDim = dim3(NUM_THREADS);
    // the ring, which later holds the partial sums
    static_assert(3 * (W_BYTES + MAX_NP * BK * 2) >= MAX_NP * BM * 4 &&
                      1024 + CTL_BYTES + 3 * (W_BYTES + MAX_NP * BK * 2) <= SMEM_LIMIT,
                  "three stages fit and hold the partial sums of the widest tile");
    cfg.dynamicSmemBytes = static_cast<size_t>(1024 + CTL_BYTES + p.stages * stage_bytes);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, ffn_small_kernel<GATE_UP, BF16>, mx, mw, mw2, p);
}

}  // namespace

cudaError_t launch_ffn_forward_small(const FfnForward& a, cudaStream_t stream) {
    if (!tensor_map_encoder()) return cudaErrorNotSupported;
    const uint64_t T = static_cast<uint64_t>(a.n_tokens), H = static_cast<uint64_t>(a.hidden),
                   I = static_cast<uint64_t>(a.intermediate);
    Params p{};
    p.status = a.status;
    p.tokens = static_cast<int32_t>(T);
    p.np = static_cast<int32_t>((T + 15) / 16 * 16);
    CUtensorMap mx, mw, mw2;
    const uint32_t np = static_cast<uint32_t>(p.np);
    if (!tensor_map_2d(&mx, a.x, T, H, 2, np) || !tensor_map_2d(&mw, a.gate_w, I, H, 2, BM / 2) ||
        !tensor_map_2d(&mw2, a.up_w, I, H, 2, BM / 2))
        return cudaErrorInvalidValue;
    p.dst = a.up_logits;
    p.dst_gate = a.gate;
    p.dst_up = a.up;
    p.n = a.intermediate;
    cudaError_t err = a.bf16 ? launch<true, true>(mx, mw, mw2, p, a.hidden, stream)
                             : launch<true, false>(mx, mw, mw2, p, a.hidden, stream);
    if (err != cudaSuccess) return err;
    if (!tensor_map_2d(&mx, a.up_logits, T, I, 2, np) || !tensor_map_2d(&mw, a.down_w, H, I, 2, BM))
        return cudaErrorInvalidValue;
    p.dst = a.out;
    p.dst_gate = p.dst_up = nullptr;
    p.n = a.hidden;
    return a.bf16 ? launch<false, true>(mx, mw, mw, p, a.intermediate, stream)
                  : launch<false, false>(mx, mw, mw, p, a.intermediate, stream);
}

}  // namespace moe
