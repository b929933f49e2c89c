// The router's gradients: from those of the logits (router_loss.cu), rounded to 16 bits,
//     d_x = d_z·W_g       [T, H]     K = experts
//     d_W = d_zᵀ·x        [E, H]     K = tokens
// in one launch of tiles of 256 x 256 (pair_tiles.cuh), and a second that adds up the parts of
// d_W where it has any.  x is read once, d_x written once; d_z and W_g stay in L2.
//
//  * d_W has few tiles (DeepSeek-V3-shaped: 28) and a long K, so K is split into as many parts as
//    pairs allow, whose sums go to fp32 slots and are added in their order.  Pairs that
//    run at the same time have neighbouring columns of the same tokens, so DRAM is read in whole rows.
//  * The pairs of every other part do their share of d_x first, so that x is read while d_x is
//    written, and pairs without a part do more of it.
//  * Operands are read as they lie: d_z by token rows for d_x, transposed for d_W.
//  * Rows of x whose token does not count are multiplied by a d_z of zero.  If one of them holds an
//    infinity or a NaN, which the pass over the logits looks for, they are cleared in shared
//    memory first.
//
// Bound: no single unit.  16384 x 256 x 7168 moves 467 MB in these products (255 read, 212 written; 69 us at the rate of a
// copy) in a launch of 104 us (cold, by itself), with DRAM at 56% of its peak, L2 at 44% (1142 MB go to the SMs: W_g's and
// d_z's tiles again for every tile), the tensor pipe at 51% and the SMs active for 89% of the time; which waits keep
// all of them below their limits has not been taken apart.  The whole call takes 123 to 125 as a graph.
// 4097 x 64 x 2048 takes 23.7 (bytes 5.2) and 32 x 128 x 2048 12.1 (0.2): the chain of launches, fill, K loop and stores.
//
// Rounding: d_x and d_W once from fp32.  d_z, an operand of 16-bit products, once too where there are many
// tokens: over thousands of them its roundings add half as much again as that of the result to the
// mean square (the root mean square error of either output is √2 of a single rounding's, 2.4e-3 in bf16).
// Over few tokens the same few roundings are in all of an output, so up to TWO_TERM_TOKENS d_z is two
// 16-bit terms, its rounding and what that left, and every K step is taken with both.  (With two
// terms throughout the products of 16384 x 256 x 7168 would be bound by the tensor pipe, at 124 us.)
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/moe_gb300.h"
#include "moe_internal.h"
#include "pair_tiles.cuh"
#include "train_internal.h"

namespace moe {
namespace {

using pairs::Tile;

constexpr int TILE = 256;
constexpr int MIN_PART = 8;          // K steps of a part of d_W at least
constexpr int64_t TWO_TERM_TOKENS = 2048;

struct GradProducts {
    int32_t total_tiles, n_maps;
    int32_t* status;
    int64_t n_tokens;
    int32_t n_experts, hidden;
    int32_t n_pairs;                 // of the launch
    int32_t two;                     // 1: d_z is two terms
    int32_t tiles_n;                 // column tiles, of both products
    int32_t w_tiles, w_parts;        // tiles of d_W, and parts of each along K
    int32_t w_steps;                 // K steps of a tile
    int32_t w_items;                 // parts that a pair has at most
    int32_t x_tiles;                 // of d_x
    int32_t x_items, x_lead;         // those of a pair with w_items parts, and how many more the others have
    uint16_t* d_x;
    uint16_t* d_w;                   // where tiles are not split (otherwise null)
    float* slots;                    // [w_parts][w_tiles][256][256]
    const float* scale;              // [1]: what undoes the power of two in d_z
    const uint32_t* valid;           // a bit per token; null: all count
    const int32_t* dirty;            // [n_dirty] is there something to remove from x
    int32_t n_dirty;
};

template <bool BF16_>
struct GradOp {
    static constexpr int BN = TILE;
    static constexpr bool BF16 = BF16_;
    static constexpr bool MASKABLE = true;
    static constexpr bool QUEUE = false;
    using Params = GradProducts;
    // Part `part` of tile `tile` of d_W, or tile `tile` of d_x (part < 0); nothing where tile < 0.
    struct Code {
        int32_t tile, part;
    };
    static __device__ __forceinline__ Code code(const Params& p, int32_t t) {
        const int32_t pair = t % p.n_pairs;
        int32_t k = t / p.n_pairs;
        const int32_t pieces = p.w_tiles * p.w_parts;
        const int32_t busy = pieces - (p.w_items - 1) * p.n_pairs;       // pairs with w_items parts; the others have one less
        const int32_t x_most = p.x_items + p.x_lead;
        // every other part last
        if (pair / p.w_tiles & 1) k = k < x_most ? k + p.w_items : k - x_most;
        if (k < p.w_items) {
            const int32_t piece = k * p.n_pairs + pair;
            if (piece >= pieces) return Code{-1, 0};
            const int32_t part = piece / p.w_tiles;
            return Code{piece - part * p.w_tiles, part};
        }
        k -= p.w_items;
        if (k >= p.x_items && pair < busy) return Code{-1, 0};
        const int32_t x = k < p.x_items ? k * p.n_pairs + pair
                                        : p.x_items * p.n_pairs + (k - p.x_items) * (p.n_pairs - busy) + pair - busy;
        return Code{x < p.x_tiles ? x : -1, -1};
    }
    enum { DZ, W_T, DZ_T, X_T, MAPS };

    static __device__ __forceinline__ Tile tile(const Params& p, const Code& c) {
        Tile ti{};
        ti.width = TILE;
        if (c.tile < 0) return ti;
        ti.two = p.two;
        const int32_t m = c.tile / p.tiles_n;
        ti.a_row = m * TILE;
        ti.b_row = (c.tile - m * p.tiles_n) * TILE;
        if (c.part >= 0) {
            ti.a_map = DZ_T;
            ti.b_map = X_T;
            ti.a_mn = ti.b_mn = true;
            ti.k0 = static_cast<int32_t>(static_cast<int64_t>(p.w_steps) * c.part / p.w_parts);
            ti.steps = (static_cast<int32_t>(static_cast<int64_t>(p.w_steps) * (c.part + 1) / p.w_parts) - ti.k0) << p.two;
        } else {
            ti.a_map = DZ;
            ti.b_map = W_T;
            ti.b_mn = true;
            ti.steps = (p.n_experts + pairs::BK - 1) / pairs::BK << p.two;
        }
        return ti;
    }
    static __device__ __forceinline__ bool dirty(const Params& p) {
        bool any = false;
        for (int32_t i = threadIdx.x; i < p.n_dirty; i += pairs::THREADS) any |= p.dirty[i] != 0;
        return any;
    }
    static __device__ __forceinline__ bool maskable(const Tile& ti) { return ti.b_map == X_T; }
    static __device__ __forceinline__ void valid64(const Params& p, int32_t step, uint32_t& w0, uint32_t& w1) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p.valid) + step);
        w0 = v.x;
        w1 = v.y;
    }

    struct Finish {
        const Params& p;
        uint8_t* staging;
        int32_t row, lane;           // first of the warp's rows inside the tile
        float inv;
        bool part;                   // a part of d_W for the slots
        uint16_t* dst;               // otherwise d_x or d_W
        int64_t at;                  // of the warp's first row there
        int32_t rows, cols;

        __device__ __forceinline__ Finish(const Params& p_, uint8_t* staging_, int32_t row_, int, int lane_)
            : p(p_), staging(staging_), row(row_), lane(lane_) {
            inv = __ldg(p.scale + 1);
        }
        __device__ __forceinline__ int width_of() const { return TILE; }
        __device__ __forceinline__ bool before(const Code& c) {
            if (c.tile < 0) return false;
            part = c.part >= 0 && p.d_w == nullptr;
            if (part) {
                at = ((static_cast<int64_t>(c.part) * p.w_tiles + c.tile) * TILE + row) * TILE;
                rows = 32;
                cols = TILE;
                MOE_DCHECK(c.part < p.w_parts && c.tile < p.w_tiles, p.status);
                return true;
            }
            const int32_t m = c.tile / p.tiles_n;
            const int32_t col = (c.tile - m * p.tiles_n) * TILE;
            const int64_t first = static_cast<int64_t>(m) * TILE + row;
            const int64_t left = (c.part >= 0 ? p.n_experts : p.n_tokens) - first;
            rows = left > 32 ? 32 : (left < 0 ? 0 : static_cast<int32_t>(left));
            cols = p.hidden - col;
            at = first * p.hidden + col;
            dst = c.part >= 0 ? p.d_w : p.d_x;
            return true;
        }
        __device__ __forceinline__ void pass(int c, uint32_t taddr) {
            if (rows <= 0 || c * 64 >= cols) return;
            uint4 el[8];
            if (part) {
#pragma unroll 1
                for (int hh = 0; hh < 2; ++hh) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(taddr + hh * 32, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 8; ++i) el[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    // 32 fp32 columns are a line of 64 16-bit ones
                    store_staged_64(el, staging, reinterpret_cast<uint16_t*>(p.slots + at + c * 64 + hh * 32), 2 * TILE,
                                    lane, 32, 64);
                }
                return;
            }
            MOE_DCHECK(at >= 0 && at + static_cast<int64_t>(rows - 1) * p.hidden + c * 64 +
                                      (cols - c * 64 < 64 ? cols - c * 64 : 64) <=
                                  (dst == p.d_x ? p.n_tokens : p.n_experts) * static_cast<int64_t>(p.hidden),
                       p.status);
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(taddr + hh * 32, v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        w[j] = pack_16bit2<BF16>(__uint_as_float(v[8 * i + 2 * j]) * inv,
                                                 __uint_as_float(v[8 * i + 2 * j + 1]) * inv);
                    el[4 * hh + i] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            store_staged_64(el, staging, dst + at + c * 64, p.hidden, lane, rows, cols - c * 64);
        }
    };
};

// d_W from its parts, in their order: a block has 4 rows of a tile, a thread four columns of one.
template <bool BF16>
__global__ void __launch_bounds__(256) join_parts_kernel(const GradProducts p, uint16_t* d_w) {
    const int32_t tile = static_cast<int32_t>(blockIdx.x) >> 6;
    const int32_t m = tile / p.tiles_n;
    const int32_t row = (static_cast<int32_t>(blockIdx.x) & 63) * 4 + (static_cast<int32_t>(threadIdx.x) >> 6);
    const int32_t e = m * TILE + row, h = (tile - m * p.tiles_n) * TILE + (static_cast<int32_t>(threadIdx.x) & 63) * 4;
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    if (e >= p.n_experts || h >= p.hidden) return;
    const float inv = __ldg(p.scale + 1);
    const float4* src = reinterpret_cast<const float4*>(p.slots + (static_cast<int64_t>(tile) * TILE + row) * TILE) +
                        (threadIdx.x & 63);
    const int64_t next = static_cast<int64_t>(p.w_tiles) * (TILE * TILE / 4);
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int32_t i = 0; i < p.w_parts; ++i) {
        const float4 x = __ldg(src + i * next);
        v.x += x.x;
        v.y += x.y;
        v.z += x.z;
        v.w += x.w;
    }
    *reinterpret_cast<uint2*>(d_w + static_cast<int64_t>(e) * p.hidden + h) =
        make_uint2(pack_16bit2<BF16>(v.x * inv, v.y * inv), pack_16bit2<BF16>(v.z * inv, v.w * inv));
}

struct GradLayout {
    int32_t ld;
    int64_t dz, d_logits, scale, block_max, block_dirty, valid, slots, bytes;
};

int64_t round256(int64_t n) { return (n + 255) / 256 * 256; }

int32_t weight_tiles(int32_t n_experts, int32_t hidden) {
    return pairs::ceil_div(n_experts, TILE) * pairs::ceil_div(hidden, TILE);
}

// Parts of a tile of d_W along K: as many as there are pairs for, of MIN_PART steps at least.
constexpr int32_t MAX_PAIRS = 76;
int32_t weight_parts(int64_t n_tokens, int32_t tiles, int32_t pairs_) {
    int64_t n = pairs_ / tiles;
    const int64_t most = pairs::ceil_div(n_tokens, pairs::BK) / MIN_PART;
    if (n > most) n = most;
    return n > 1 ? static_cast<int32_t>(n) : 1;
}

GradLayout grad_layout(int64_t n_tokens, int32_t n_experts, int32_t hidden) {
    GradLayout l;
    l.ld = (n_experts + 7) / 8 * 8;
    int64_t at = 0;
    auto take = [&at](int64_t n) {
        const int64_t r = at;
        at += round256(n);
        return r;
    };
    l.dz = take(n_tokens * l.ld * 2 * (n_tokens <= TWO_TERM_TOKENS ? 2 : 1));
    l.d_logits = take(n_tokens * n_experts * 4);
    l.scale = take(8);
    l.block_max = take(int64_t{4} * router_grad_blocks(n_tokens));
    l.block_dirty = take(int64_t{4} * router_grad_blocks(n_tokens));
    l.valid = take((n_tokens + 63) / 64 * 8);
    const int32_t tiles = weight_tiles(n_experts, hidden);
    const int32_t parts = weight_parts(n_tokens, tiles, MAX_PAIRS);
    l.slots = take(parts > 1 ? static_cast<int64_t>(parts) * tiles * TILE * TILE * 4 : 0);
    l.bytes = at;
    return l;
}

template <bool BF16>
cudaError_t launch_products(const RouterBackward& a, const LogitGradients& g, float* slots, cudaStream_t stream) {
    using Op = GradOp<BF16>;
    if (!tensor_map_encoder()) return cudaErrorNotSupported;
    const int64_t T = a.r.n_tokens;
    const int32_t E = a.r.n_experts, H = a.hidden;
    pairs::Maps maps;
    const int terms = g.two ? 2 : 1;
    if (!pairs::map_3d(&maps.m[Op::DZ], g.dz, terms, T, E, g.ld, pairs::BM) ||
        !pairs::map_3d(&maps.m[Op::W_T], a.router_w, 1, E, H, H, pairs::BK) ||
        !pairs::map_3d(&maps.m[Op::DZ_T], g.dz, terms, T, E, g.ld, pairs::BK) ||
        !pairs::map_3d(&maps.m[Op::X_T], a.x, 1, T, H, H, pairs::BK))
        return cudaErrorInvalidValue;
    int n_pairs = pairs::resident_pairs<Op>();
    if (n_pairs == 0) return cudaErrorNoDevice;
    if (n_pairs > MAX_PAIRS) n_pairs = MAX_PAIRS;
    GradProducts p{};
    p.n_maps = Op::MAPS;
    p.status = a.status;
    p.n_tokens = T;
    p.n_experts = E;
    p.hidden = H;
    p.two = g.two ? 1 : 0;
    p.tiles_n = pairs::ceil_div(H, TILE);
    p.w_tiles = weight_tiles(E, H);
    p.w_steps = pairs::ceil_div(T, pairs::BK);
    p.w_parts = weight_parts(T, p.w_tiles, n_pairs);
    p.x_tiles = pairs::ceil_div(T, TILE) * p.tiles_n;
    // as many pairs as there is work for: a part or a tile each
    const int32_t pieces = p.w_tiles * p.w_parts, items = pieces + p.x_tiles;
    p.n_pairs = items < n_pairs ? items : n_pairs;
    p.w_items = (pieces + p.n_pairs - 1) / p.n_pairs;
    // pairs with one part less do more tiles of d_x meanwhile (us: a step of a part 0.36; a tile of d_x its
    // steps and 0.4, its stores 1.7)
    const int32_t free_pairs = p.w_items * p.n_pairs - pieces;
    const float part = 0.36f * static_cast<float>(p.w_steps) / static_cast<float>(p.w_parts);
    const float x_mma = 0.36f * static_cast<float>(pairs::ceil_div(E, pairs::BK)) + 0.4f;
    p.x_lead = free_pairs > 0 ? static_cast<int32_t>(part / (x_mma > 1.7f ? x_mma : 1.7f)) : 0;
    int64_t rest = p.x_tiles - static_cast<int64_t>(p.x_lead) * free_pairs;
    if (rest < 0) {
        p.x_lead = (p.x_tiles + free_pairs - 1) / free_pairs;
        rest = 0;
    }
    p.x_items = static_cast<int32_t>((rest + p.n_pairs - 1) / p.n_pairs);
    p.total_tiles = p.n_pairs * (p.w_items + p.x_items + p.x_lead);
    p.d_x = a.d_x;
    p.d_w = p.w_parts == 1 ? a.d_router_w : nullptr;
    p.slots = slots;
    p.scale = g.scale;
    p.valid = g.valid;
    p.dirty = g.block_dirty;
    p.n_dirty = g.valid ? router_grad_blocks(T) : 0;
    cudaError_t err = pairs::launch<Op>(maps, p, stream, p.n_pairs);
    if (err != cudaSuccess || p.d_w) return err;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.w_tiles) * 64);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_parts_kernel<BF16>, p, a.d_router_w);
}

}  // namespace

int64_t router_backward_workspace_bytes(int64_t n_tokens, int32_t n_experts, int32_t hidden) {
    return grad_layout(n_tokens, n_experts, hidden).bytes;
}

cudaError_t launch_router_backward(const RouterBackward& a, cudaStream_t stream) {
    if (a.r.n_tokens == 0)
        return cudaMemsetAsync(a.d_router_w, 0, static_cast<size_t>(a.r.n_experts) * a.hidden * 2, stream);
    const GradLayout l = grad_layout(a.r.n_tokens, a.r.n_experts, a.hidden);
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    LogitGradients g;
    g.dz = reinterpret_cast<uint16_t*>(ws + l.dz);
    g.ld = l.ld;
    g.two = a.r.n_tokens <= TWO_TERM_TOKENS;
    g.d_logits = reinterpret_cast<float*>(ws + l.d_logits);
    g.scale = reinterpret_cast<float*>(ws + l.scale);
    g.block_max = reinterpret_cast<float*>(ws + l.block_max);
    const bool some = a.r.token_mask != nullptr || a.r.seq_offsets != nullptr;
    g.valid = some ? reinterpret_cast<uint32_t*>(ws + l.valid) : nullptr;
    g.block_dirty = some ? reinterpret_cast<int32_t*>(ws + l.block_dirty) : nullptr;
    const cudaError_t err = launch_logit_gradients(a, g, stream);
    if (err != cudaSuccess) return err;
    float* slots = reinterpret_cast<float*>(ws + l.slots);
    return a.bf16 ? launch_products<true>(a, g, slots, stream) : launch_products<false>(a, g, slots, stream);
}

}  // namespace moe
