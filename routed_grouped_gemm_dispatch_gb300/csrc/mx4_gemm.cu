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
//  * A persistent CTA per SM walks 128 x 256 tiles: the active blocks (rows of
//    some expert) are compacted first, and tiles run slice by slice inside
//    groups of blocks, so that concurrent CTAs share a weight slice in L2.
//  * Per stage (K = 256): 16 KB of A and 32 KB of B codes by TMA (128-byte swizzle),
//    and their scale tiles (512 bytes for 128 rows x 128 values) by plain bulk
//    copies.  The MMA warp copies the scale tiles into TMEM (tcgen05.cp,
//    in order with the MMAs that read them).
//  * TMEM: columns 0-255 accumulate, the stages' scales sit behind them.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <map>
#include <mutex>

#include "../../include/moe_gb300.h"
#include "moe_internal.h"
#include "mx4_internal.h"
#include "sm103_ptx.cuh"
#include "tensor_map.h"
#include "tile_store.cuh"

namespace moe {
namespace {

constexpr int BM = 128;
constexpr int BN = 256;                         // columns of B per tile
constexpr int BOX = 128;                        // bytes of codes of a row per stage (K = 256)
constexpr int A_BYTES = BM * BOX;
constexpr int B_BYTES = BN * BOX;
constexpr int SCALE_TILE = 512;                 // scales of 128 rows x 128 values
constexpr int STAGE_BYTES = A_BYTES + B_BYTES + 2 * SCALE_TILE + 4 * SCALE_TILE;
constexpr int MAX_STAGES = 4;
constexpr int NUM_THREADS = 192;
constexpr int NUM_EPI_THREADS = 128;
constexpr int TMEM_COLS = 512;
constexpr int TMEM_SCALES = 256;                // first scale column
constexpr int STAGE_SCALE_COLS = 2 * (4 + 8);   // per K = 128: 4 columns of A's, 8 of B's scales
constexpr uint64_t WAIT_LIMIT_NS = 2000000000ull;
constexpr uint64_t DRAIN_LIMIT_NS = 200000000ull;

constexpr int OFF_BARS = 0;                     // full, empty [MAX_STAGES]; tfull, tempty, drain
constexpr int OFF_TMEM_SLOT = OFF_BARS + (2 * MAX_STAGES + 3) * 8;
constexpr int OFF_ABORT = OFF_TMEM_SLOT + 4;
constexpr int OFF_WSUM = OFF_ABORT + 4;
constexpr int OFF_RUNS = OFF_WSUM + (NUM_THREADS / 32) * 4;
constexpr int OFF_BLOCKS = (OFF_RUNS + 4 + 15) / 16 * 16;

struct Params {
    const uint8_t* a_scales;
    const uint8_t* b_scales;
    const uint8_t* b2_scales;
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
};

// Rows of block bx that hold data, its expert and the row's place inside the
// expert.  Table entries that point outside their arrays make a block empty
// and raise MOE_DEV_BAD_TABLE.
template <int FORM>
__device__ __forceinline__ int32_t block_rows(const Params& p, int32_t bx, int32_t* e_out, int32_t* tok_out) {
    if (FORM == MX4_MATMUL) {
        *e_out = 0;
        *tok_out = 0;
        const int64_t left = p.rows - static_cast<int64_t>(bx) * BM;
        return left > BM ? BM : static_cast<int32_t>(left);
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

struct Tile {
    int32_t bx, n;
};

// Groups of `group` active blocks, slice by slice inside a group.
__device__ __forceinline__ Tile tile_at(int32_t t, const uint16_t* blocks, int32_t nact, int32_t n_tiles,
                                        int32_t group) {
    const int32_t per_group = group * n_tiles;
    const int32_t g = t / per_group;
    const int32_t l = t - g * per_group;
    const int32_t left = nact - g * group;
    const int32_t gs = left < group ? left : group;
    Tile ti;
    ti.n = l / gs;
    ti.bx = blocks[g * group + (l - ti.n * gs)];
    return ti;
}

template <int FORM, bool BF16>
__global__ void __launch_bounds__(NUM_THREADS, 1)
mx4_gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                const __grid_constant__ CUtensorMap map_b2, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem =
        reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* ctl = smem + p.stages * STAGE_BYTES;
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar_full = smem_u32(ctl) + OFF_BARS;
    const uint32_t bar_empty = bar_full + 8 * MAX_STAGES;
    const uint32_t bar_tfull = bar_empty + 8 * MAX_STAGES;
    const uint32_t bar_tempty = bar_tfull + 8;
    const uint32_t bar_drain = bar_tempty + 8;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(ctl + OFF_TMEM_SLOT);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(ctl + OFF_ABORT);
    int32_t* wsum = reinterpret_cast<int32_t*>(ctl + OFF_WSUM);
    int32_t* runs = reinterpret_cast<int32_t*>(ctl + OFF_RUNS);
    uint16_t* blocks = reinterpret_cast<uint16_t*>(ctl + OFF_BLOCKS);

    const int tid = threadIdx.x;
    const int warp = tid >> 5;
    const int lane = tid & 31;
    const uint32_t stages = static_cast<uint32_t>(p.stages);

    if (tid == 0) {
        for (int s = 0; s < MAX_STAGES; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 1);
        }
        mbar_init(bar_tfull, 1);
        mbar_init(bar_tempty, NUM_EPI_THREADS);
        mbar_init(bar_drain, 1);
        *abort_flag = 0;
        *runs = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(ctl) + OFF_TMEM_SLOT, TMEM_COLS);
        tmem_relinquish();
    }
    __syncthreads();
    pdl_wait_prior_grid();
    pdl_launch_dependents();

    // ---- active blocks, in order, and the number of experts they belong to ----
    int32_t nact = 0;
    if (FORM == MX4_MATMUL) {
        nact = p.num_blocks;
        for (int32_t b = tid; b < nact; b += NUM_THREADS) blocks[b] = static_cast<uint16_t>(b);
    } else {
        for (int32_t base = 0; base < p.num_blocks; base += NUM_THREADS) {
            const int32_t bx = base + tid;
            int32_t flag = 0, e = 0, tok = 0;
            if (bx < p.num_blocks) flag = block_rows<FORM>(p, bx, &e, &tok) > 0;
            const uint32_t ballot = __ballot_sync(0xffffffffu, flag);
            const uint32_t first = __ballot_sync(0xffffffffu, flag && tok == 0);
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
            if (flag) blocks[nact + before + __popc(ballot & ((1u << lane) - 1u))] = static_cast<uint16_t>(bx);
            nact += total;
            __syncthreads();
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    // blocks walked together: about an expert's, at most 16 (2048 rows)
    int32_t group = FORM == MX4_MATMUL ? 16 : (*runs > 0 ? (nact + *runs - 1) / *runs : 1);
    group = group > 16 ? 16 : group;
    const int32_t total_tiles = nact * p.n_tiles;
    const int32_t k_steps = (p.k_tiles + 1) / 2;

    if (warp == 0) {
        // ===================== producer =====================
        if (lane == 0) {
            const uint64_t policy = l2_policy_evict_normal();
            uint32_t stage = 0, phase = 0;
            int64_t issued = 0;
            bool ok = true;
            for (int32_t t = blockIdx.x; t < total_tiles && ok; t += gridDim.x) {
                const Tile ti = tile_at(t, blocks, nact, p.n_tiles, group);
                const int32_t e = FORM == MX4_MATMUL ? 0 : __ldg(p.gidx + ti.bx);
                // first weight row of the tile (of gate and of up: 128 rows each)
                const int32_t brow = e * p.n + ti.n * (FORM == MX4_GATE_UP ? 128 : BN);
                // the last slice of a matrix may be half a tile: its second scale tile is another matrix's or none
                const bool two = FORM == MX4_GATE_UP || ti.n * BN + 128 < p.n;
                const uint8_t* as = p.a_scales + static_cast<int64_t>(ti.bx) * p.k_tiles * SCALE_TILE;
                const uint8_t* bs = p.b_scales + static_cast<int64_t>(brow / 128) * p.k_tiles * SCALE_TILE;
                const uint8_t* bs2 = FORM == MX4_GATE_UP
                                         ? p.b2_scales + static_cast<int64_t>(brow / 128) * p.k_tiles * SCALE_TILE
                                         : bs + static_cast<int64_t>(p.k_tiles) * SCALE_TILE;
                for (int32_t kb = 0; kb < k_steps; ++kb) {
                    if (!mbar_wait_bounded(bar_empty + 8 * stage, phase ^ 1u, abort_flag, WAIT_LIMIT_NS)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = bar_full + 8 * stage;
                    const uint32_t sa = sbase + stage * STAGE_BYTES;
                    const uint32_t sb = sa + A_BYTES;
                    const uint32_t ss = sb + B_BYTES;
                    const uint32_t kt = p.k_tiles - 2 * kb >= 2 ? 2 : 1;       // scale tiles along K
                    const uint32_t sbytes = kt * SCALE_TILE;
                    mbar_arrive_expect_tx(fb, A_BYTES + B_BYTES + sbytes * (two ? 3 : 2));
                    tma_load_2d(sa, &map_a, fb, kb * BOX, ti.bx * BM, policy);
                    tma_load_2d(sb, &map_b, fb, kb * BOX, brow, policy);
                    tma_load_2d(sb + B_BYTES / 2, FORM == MX4_GATE_UP ? &map_b2 : &map_b, fb, kb * BOX,
                                FORM == MX4_GATE_UP ? brow : brow + 128, policy);
                    bulk_load(ss, as + kb * 2 * SCALE_TILE, sbytes, fb);
                    bulk_load(ss + 2 * SCALE_TILE, bs + kb * 2 * SCALE_TILE, sbytes, fb);
                    if (two) bulk_load(ss + 4 * SCALE_TILE, bs2 + kb * 2 * SCALE_TILE, sbytes, fb);
                    ++issued;
                    if (++stage == stages) { stage = 0; phase ^= 1u; }
                }
            }
            if (!ok) {
                // Let the copies already in flight land before the CTA exits.
                volatile int never = 0;
                const int64_t n = issued < stages ? issued : stages;
                for (int64_t i = 0; i < n; ++i) {
                    const int64_t idx = issued - 1 - i;
                    mbar_wait_bounded(bar_full + 8 * static_cast<uint32_t>(idx % stages),
                                      static_cast<uint32_t>((idx / stages) & 1), &never, DRAIN_LIMIT_NS);
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ===================== MMA issuer =====================
        if (lane == 0) {
            uint32_t stage = 0, phase = 0, aphase = 0;
            bool ok = true;
            for (int32_t t = blockIdx.x; t < total_tiles && ok; t += gridDim.x) {
                if (!mbar_wait_bounded(bar_tempty, aphase ^ 1u, abort_flag, WAIT_LIMIT_NS)) break;
                tc_fence_after_sync();
                for (int32_t kb = 0; kb < k_steps; ++kb) {
                    if (!mbar_wait_bounded(bar_full + 8 * stage, phase, abort_flag, WAIT_LIMIT_NS)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint32_t sa = sbase + stage * STAGE_BYTES;
                    const uint32_t sb = sa + A_BYTES;
                    const uint32_t ss = sb + B_BYTES;
                    const uint32_t tsc = tmem_base + TMEM_SCALES + stage * STAGE_SCALE_COLS;
                    const int kt = p.k_tiles - 2 * kb >= 2 ? 2 : 1;
                    for (int i = 0; i < kt; ++i) {
                        tc_cp_scales(tsc + i * 12, smem_desc_scales(ss + i * SCALE_TILE));
                        tc_cp_scales(tsc + i * 12 + 4, smem_desc_scales(ss + (2 + i) * SCALE_TILE));
                        tc_cp_scales(tsc + i * 12 + 8, smem_desc_scales(ss + (4 + i) * SCALE_TILE));
                    }
                    const uint64_t da = smem_desc_k_sw128(sa), db = smem_desc_k_sw128(sb);
                    for (int i = 0; i < 2 * kt; ++i)                             // K = 64 each
                        tc_mma_mxf4(tmem_base, da + i * 2, db + i * 2, idesc_mxf4(BM, BN, i & 1), tsc + (i >> 1) * 12,
                                    tsc + (i >> 1) * 12 + 4, (kb | i) != 0 ? 1u : 0u);
                    tc_commit(bar_empty + 8 * stage);
                    if (++stage == stages) { stage = 0; phase ^= 1u; }
                }
                if (!ok) break;
                tc_commit(bar_tfull);
                aphase ^= 1u;
            }
            volatile int never = 0;
            tc_commit(bar_drain);
            mbar_wait_bounded(bar_drain, 0, &never, DRAIN_LIMIT_NS);
        }
        __syncwarp();
    } else {
        // ===================== epilogue (warps 2..5) =====================
        const int quarter = warp & 3;
        uint32_t aphase = 0;
        for (int32_t t = blockIdx.x; t < total_tiles; t += gridDim.x) {
            const Tile ti = tile_at(t, blocks, nact, p.n_tiles, group);
            int32_t e = 0, tok = 0;
            const int32_t rows = block_rows<FORM>(p, ti.bx, &e, &tok) - quarter * 32;   // of this warp
            const int64_t row0 = static_cast<int64_t>(ti.bx) * BM + quarter * 32;
            const int32_t col0 = ti.n * (FORM == MX4_GATE_UP ? 128 : BN);
            uint16_t* dst = p.out + row0 * p.n + col0;
            float w = 1.0f;
            if (FORM == MX4_DOWN && lane < rows) w = __ldg(p.weights + (__ldg(p.offsets + e) + tok + quarter * 32 + lane));
            if (!mbar_wait_bounded(bar_tfull, aphase, abort_flag, WAIT_LIMIT_NS)) break;
            tc_fence_after_sync();
            const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
            const int passes = rows > 0 ? (FORM == MX4_GATE_UP ? 2 : 4) : 0;
#pragma unroll 1
            for (int c = 0; c < passes; ++c) {
                const int32_t cols = p.n - col0 - c * 64;
                if (cols <= 0) break;
                uint4 el[8];
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(taddr + c * 64 + hh * 32, v);
                    if (FORM == MX4_GATE_UP) {
                        uint32_t u[32];
                        tmem_ld_32x32b_x32(taddr + 128 + c * 64 + hh * 32, u);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const float g = __uint_as_float(v[j]);
                            v[j] = __float_as_uint(__fdividef(g, 1.0f + __expf(-g)) * __uint_as_float(u[j]));
                        }
                    } else {
                        tmem_ld_wait();
                        if (FORM == MX4_DOWN) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * w);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t o[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            o[j] = pack_16bit2<BF16>(__uint_as_float(v[8 * k + 2 * j]), __uint_as_float(v[8 * k + 2 * j + 1]));
                        el[4 * hh + k] = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                }
                store_rows_64(el, dst + c * 64, p.n, lane, rows, cols);
            }
            tc_fence_before_sync();
            mbar_arrive(bar_tempty);
            aphase ^= 1u;
        }
    }

    tc_fence_before_sync();
    __syncthreads();
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
cudaError_t launch(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mb2, Params& p, cudaStream_t stream) {
    int dev = 0, max_smem = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(&max_smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (err != cudaSuccess) return err;
    const int control = 1024 + OFF_BLOCKS + (2 * p.num_blocks + 15) / 16 * 16;
    p.stages = (max_smem - control) / STAGE_BYTES;
    if (p.stages > MAX_STAGES) p.stages = MAX_STAGES;
    const int smem = control + p.stages * STAGE_BYTES;
    // the attribute only ever grows to the device's limit: set it once
    static std::once_flag once[16];
    if (dev >= 16) return cudaErrorNoDevice;
    std::call_once(once[dev], [&] {
        err = cudaFuncSetAttribute(mx4_gemm_kernel<FORM, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, max_smem);
    });
    if (err != cudaSuccess) return err;
    const int64_t tiles = static_cast<int64_t>(p.num_blocks) * p.n_tiles;
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorNoDevice;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles < sms ? tiles : sms));
    cfg.blockDim = dim3(NUM_THREADS);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, mx4_gemm_kernel<FORM, BF16>, ma, mb, mb2, p);
}

template <int FORM>
cudaError_t launch(bool bf16, const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mb2, Params& p,
                   cudaStream_t stream) {
    return bf16 ? launch<FORM, true>(ma, mb, mb2, p, stream) : launch<FORM, false>(ma, mb, mb2, p, stream);
}

}  // namespace

cudaError_t launch_mx4_product(const Mx4Product& a, cudaStream_t stream) {
    if (!tensor_map_encoder()) return cudaErrorNotSupported;
    CUtensorMap ma, mb, mb2;
    const uint64_t kb = static_cast<uint64_t>(a.k) / 2;
    const uint64_t brows = static_cast<uint64_t>(a.n_experts) * static_cast<uint64_t>(a.n);
    if (!tensor_map_2d(&ma, a.a, static_cast<uint64_t>(a.rows), kb, 1, BM) || !tensor_map_2d(&mb, a.b, brows, kb, 1, 128) ||
        !tensor_map_2d(&mb2, a.form == MX4_GATE_UP ? a.b2 : a.b, brows, kb, 1, 128))
        return cudaErrorInvalidValue;
    Params p{};
    p.a_scales = a.a_scales;
    p.b_scales = a.b_scales;
    p.b2_scales = a.b2_scales;
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
    p.n_tiles = a.form == MX4_GATE_UP ? a.n / 128 : (a.n + BN - 1) / BN;
    p.k_tiles = a.k / 128;
    switch (a.form) {
        case MX4_MATMUL: return launch<MX4_MATMUL>(a.bf16, ma, mb, mb2, p, stream);
        case MX4_GATE_UP: return launch<MX4_GATE_UP>(a.bf16, ma, mb, mb2, p, stream);
        default: return launch<MX4_DOWN>(a.bf16, ma, mb, mb2, p, stream);
    }
}

}  // namespace moe
