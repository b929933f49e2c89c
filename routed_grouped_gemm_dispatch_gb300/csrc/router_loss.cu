// The router's losses with its per-expert counts, and the gradients of its logits.
//
// With z the logits, p = softmax(z), T valid tokens, T_s of them in sequence s:
//     counts[s, e] = pairs of sequence s whose id is e
//     losses[0] = E / (k T) · Σ_s 1/T_s · Σ_e counts[s, e] · Σ_t∈s p[t, e]
//     losses[1] = 1/T · Σ_t logsumexp(z[t])²
//     g[t, e] = d_losses[0]·E / (k T T_s)·counts[s, e] + Σ_j [id[t, j] = e]·d_w[t, j]
//     d_z = p ⊙ (g − Σ_e p g) + d_losses[1]·2/T·logsumexp(z)·p
//
// A group of 4 to 16 lanes has a token, 16 logits a lane (32 lanes and up to 32 logits above 256
// experts), and a lane has the same experts of every token, so that column sums over a warp's tokens stay in
// registers until the end of a piece.  All is read once.  Sums over tokens are fp32 over the
// tokens of a warp and of a block and pairs of fp32 (Sum) beyond, always in the same
// order.  (FP64 is slow here: with it the second launch took 16 us, by itself, for 32 tokens.)
//
// Bound: latency.  The losses of 16384 x 256 (17 MB, 2.6 us of HBM) take 15.5 to 17 us in two launches: a block's 64
// tokens are two rounds of loads, exponentials and sums over lanes, then come its warps' sums, and a
// second launch that waits for the first, reads the parts and counts its blocks.  (No unit is busy: 21% of the SMs' issue
// rate in the first launch.)  One cluster needs no second
// launch: 4097 x 64 in five sequences 9.4 us, 32 x 128 3.9.  The gradients of 16384 x 256 logits take
// 15 us cold (34 MB), their rounding 8.5.
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>
#include <type_traits>

#include "../../include/moe_gb300.h"
#include "moe_internal.h"
#include "sm103_ptx.cuh"
#include "tile_store.cuh"
#include "train_internal.h"

namespace moe {
namespace {

constexpr int WARPS = 16;
constexpr int THREADS = 32 * WARPS;
constexpr int REDUCE_WARPS = 32;
constexpr int HALF = WARPS / 2;
constexpr int MAX_CLUSTER = 16;

// Value i of lane l of a token's L lanes is expert `expert(l, i)`.  VEC: E is a multiple of 4 and rows
// are whole 16-byte pieces.
template <int L, bool VEC>
__device__ __forceinline__ int expert(int l, int i) {
    return VEC ? (i >> 3) * 8 * L + 8 * l + (i & 7) : l + L * i;
}

template <int L, int PER, bool VEC>
__device__ __forceinline__ void load_row(float (&z)[PER], const float* row, int l, int32_t n_experts) {
    if (VEC) {
#pragma unroll
        for (int i = 0; i < PER; i += 4) {
            const int e = expert<L, VEC>(l, i);
            float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (e < n_experts) v = __ldg(reinterpret_cast<const float4*>(row + e));
            z[i] = v.x;
            z[i + 1] = v.y;
            z[i + 2] = v.z;
            z[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = expert<L, VEC>(l, i);
            z[i] = e < n_experts ? __ldg(row + e) : -INFINITY;
        }
    }
}

// Over a token's lanes; all lanes of the warp take part.
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// The row becomes its softmax; returns its logsumexp.  (A row of minus infinities has no probability anywhere: all
// zeros, and 0.)  An exponential is 2^((z - top) log2 e) by ex2.approx (2^-22).  The difference, the constant and the
// product are rounded by 2^-24 each, which is an absolute error of the exponent: at a distance D from the row's maximum
// the exponential is off by 3·2^-24·D of itself besides, and below 2^-126 it is 0.
template <int L, int PER>
__device__ __forceinline__ float softmax_row(float (&z)[PER]) {
    float top = z[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) top = fmaxf(top, z[i]);
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    constexpr float LOG2E = 1.4426950408889634f;
    if (top == -INFINITY) top = 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(z[i]) : "f"((z[i] - top) * LOG2E));
        sum += z[i];
    }
    sum = lanes_sum<L>(sum);
    const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;            // (NaN stays NaN)
#pragma unroll
    for (int i = 0; i < PER; ++i) z[i] *= inv;
    return sum != 0.0f ? top + logf(sum) : 0.0f;
}

// Sequence bounds, held inside [0, n_tokens] whatever the array says.
struct Seqs {
    const int32_t* offsets;
    int32_t n;
    int64_t n_tokens;

    __device__ __forceinline__ int64_t bound(int32_t i) const {
        if (offsets == nullptr) return i == 0 ? 0 : n_tokens;
        const int64_t v = __ldg(offsets + i);
        return v < 0 ? 0 : (v > n_tokens ? n_tokens : v);
    }
    // the last sequence that starts at or before token t (-1: none); by a whole warp, 32 bounds at a time
    __device__ __forceinline__ int32_t find(int64_t t) const {
        if (offsets == nullptr) return 0;
        int32_t lo = 0, hi = n;                  // the first bound past t is in [lo, hi]
        while (lo < hi) {
            const int32_t step = (hi - lo + 31) / 32;
            const int32_t i = lo + static_cast<int32_t>(threadIdx.x & 31) * step;
            const int c = __popc(__ballot_sync(0xffffffffu, i < hi && bound(i) <= t));
            if (c == 0) {
                hi = lo;
            } else {
                hi = lo + c * step < hi ? lo + c * step : hi;
                lo += (c - 1) * step + 1;
            }
        }
        return lo - 1;
    }
};

// An fp32 sum with what its additions lost (an exact sum of two, and of a product).  What an infinite one lost is NaN,
// and not part of its value.
struct Sum {
    float hi = 0.0f, lo = 0.0f;
    __device__ __forceinline__ void add(float x) {
        const float s = __fadd_rn(hi, x);
        const float b = __fsub_rn(s, hi);
        lo += __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b));
        hi = s;
    }
    __device__ __forceinline__ void add(const Sum& o) {
        add(o.hi);
        lo += o.lo;
    }
    __device__ __forceinline__ float value() const { return fabsf(hi) == INFINITY ? hi : hi + lo; }
    __device__ __forceinline__ Sum times(float f) const {
        Sum r;
        r.hi = __fmul_rn(hi, f);
        r.lo = __fmaf_rn(hi, f, -r.hi) + lo * f;
        return r;
    }
    __device__ __forceinline__ void add_lanes() {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            Sum o;
            o.hi = __shfl_xor_sync(0xffffffffu, hi, d);
            o.lo = __shfl_xor_sync(0xffffffffu, lo, d);
            add(o);
        }
    }
};

__device__ __forceinline__ bool counts_token(const uint8_t* mask, int64_t t) { return mask == nullptr || mask[t] != 0; }

struct BalanceParams {
    Routing r;
    int32_t chunk;                // tokens of a block
    int32_t n_slots;
    float2* part;                 // [n_slots, E] Σ p of a block's tokens of one sequence, and (as an int) their pairs
    float2* tokens;               // [n_slots] Σ logsumexp², and (as an int) the tokens that count
    Sum* dots;                    // [n_seqs, expert blocks] Σ_e counts·Σ p
    Sum* zsum;                    // [n_seqs]
    unsigned* done;
    float* losses;
    int32_t* counts;
    int32_t* seq_tokens;
    int32_t* status;
};

// From Σ_s 1/T_s·Σ_e counts·Σ p, Σ logsumexp² and the tokens that count.
__device__ __forceinline__ void store_losses(const BalanceParams& p, const Sum& balance, const Sum& z, int32_t n) {
    const float tokens = static_cast<float>(n > 0 ? n : 1);
    p.losses[0] = balance.value() * static_cast<float>(p.r.n_experts) / (static_cast<float>(p.r.top_k) * tokens);
    p.losses[1] = z.value() / tokens;
    p.seq_tokens[p.r.n_seqs] = n;
}

// Tokens first .. last - 1 of a block, one sequence after the other: store(s, e, Σ p, pairs) by a
// thread for each expert, store(s, Σ logsumexp², tokens that count) by one.  shared: [HALF][E] floats, then
// [E] counts, which are zero (a barrier may be still to come).  Ends with a barrier.
template <int L, int PER, bool VEC, class Store>
__device__ __forceinline__ void add_tokens(const BalanceParams& p, int64_t first, int64_t last, float* sums, const Store& store) {
    __shared__ float zpart[WARPS];
    __shared__ int npart[WARPS];
    constexpr int PACK = 32 / L;                                  // tokens a warp has at a time
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane & (L - 1);
    const int32_t E = p.r.n_experts, k = p.r.top_k;
    int32_t* hist = reinterpret_cast<int32_t*>(sums + HALF * E);
    const Seqs seqs{p.r.seq_offsets, p.r.n_seqs, p.r.n_tokens};
    int32_t s = seqs.find(first);
    if (s < 0) s = 0;
    int64_t t0 = first > seqs.bound(0) ? first : seqs.bound(0);
    while (t0 < last && s < p.r.n_seqs) {
        const int64_t end = seqs.bound(s + 1);
        const int64_t t1 = end < last ? end : last;
        if (t1 <= t0) {
            ++s;
            continue;
        }
        const float* row = p.r.logits + (t0 + warp * PACK + lane / L) * E;
        int32_t left = static_cast<int32_t>(t1 - t0) - warp * PACK - lane / L;      // tokens from this lane's on
        const uint8_t* mask = p.r.token_mask ? p.r.token_mask + (t1 - left) : nullptr;
        float z[PER];
        bool live = false;
        auto ask = [&]() {
            live = left > 0 && (mask == nullptr || *mask != 0);
#pragma unroll
            for (int i = 0; i < PER; ++i) z[i] = 0.0f;
            if (live) load_row<L, PER, VEC>(z, row, l, E);
        };
        ask();                                                    // on its way while the pairs are counted
        __syncthreads();                                          // the counts are zero
        // pairs of the tokens that count
        const int32_t pairs = static_cast<int32_t>(t1 - t0) * k;
        for (int32_t i = threadIdx.x; i < pairs; i += THREADS) {
            if (p.r.token_mask && p.r.token_mask[t0 + i / k] == 0) continue;
            const int32_t id = __ldg(p.r.topk_ids + t0 * k + i);
            if (id >= 0 && id < E) atomicAdd(&hist[id], 1);
            else if (id >= E && p.status) atomicOr(p.status, MOE_DEV_BAD_EXPERT_ID);
        }
        float acc[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] = 0.0f;
        float zz = 0.0f;
        int n = 0;
        for (int32_t i0 = warp * PACK; i0 < static_cast<int32_t>(t1 - t0); i0 += WARPS * PACK) {
            const float lse = softmax_row<L, PER>(z);
            if (live) {
#pragma unroll
                for (int i = 0; i < PER; ++i) acc[i] += z[i];
                if (l == 0) {
                    zz += lse * lse;
                    ++n;
                }
            }
            row += static_cast<int64_t>(WARPS * PACK) * E;
            left -= WARPS * PACK;
            if (mask) mask += WARPS * PACK;
            ask();
        }
        // a warp's tokens, then the block's warps
#pragma unroll
        for (int d = L; d < 32; d <<= 1) {
#pragma unroll
            for (int i = 0; i < PER; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], d);
            zz += __shfl_xor_sync(0xffffffffu, zz, d);
            n += __shfl_xor_sync(0xffffffffu, n, d);
        }
        if (lane == 0) {
            zpart[warp] = zz;
            npart[warp] = n;
        }
        if (warp >= HALF && lane < L) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = expert<L, VEC>(l, i);
                if (e < E) sums[(warp - HALF) * E + e] = acc[i];
            }
        }
        __syncthreads();
        if (warp < HALF && lane < L) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = expert<L, VEC>(l, i);
                if (e < E) sums[warp * E + e] += acc[i];
            }
        }
        __syncthreads();
        MOE_DCHECK(t0 >= 0 && t1 <= p.r.n_tokens && s >= 0 && s < p.r.n_seqs, p.status);
        for (int e = threadIdx.x; e < E; e += THREADS) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < HALF; ++w) v += sums[w * E + e];
            store(s, e, v, hist[e]);
            hist[e] = 0;
        }
        if (threadIdx.x == 0) {
            float zt = 0.0f;
            int nt = 0;
            for (int w = 0; w < WARPS; ++w) {
                zt += zpart[w];
                nt += npart[w];
            }
            store(s, zt, nt);
        }
        __syncthreads();
        t0 = t1;
        ++s;
    }
}

// One block per `chunk` tokens.  The part of sequence s in block b goes to slot b + s:
// from one part to the next either b or s grows, so no two share a slot.
struct StoreSlot {
    const BalanceParams& p;
    __device__ __forceinline__ int64_t slot(int32_t s) const {
        const int64_t i = static_cast<int64_t>(blockIdx.x) + s;
        MOE_DCHECK(i < p.n_slots, p.status);
        return i;
    }
    __device__ __forceinline__ void operator()(int32_t s, int32_t e, float v, int32_t n) const {
        p.part[slot(s) * p.r.n_experts + e] = make_float2(v, __int_as_float(n));
    }
    __device__ __forceinline__ void operator()(int32_t s, float z, int32_t n) const {
        p.tokens[slot(s)] = make_float2(z, __int_as_float(n));
    }
};

template <int L, int PER, bool VEC>
__global__ void __launch_bounds__(THREADS, PER <= 16 ? 2 : 1) balance_kernel(const BalanceParams p) {
    extern __shared__ float sums[];                               // [HALF][E], then int [E]
    for (int e = threadIdx.x; e < p.r.n_experts; e += THREADS) sums[HALF * p.r.n_experts + e] = 0.0f;
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.done = 0;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * p.chunk;
    add_tokens<L, PER, VEC>(p, first, first + p.chunk < p.r.n_tokens ? first + p.chunk : p.r.n_tokens, sums, StoreSlot{p});
}

// Few tokens: all of it by one cluster, whose CTAs have `chunk` tokens each.  Their parts stay in shared memory;
// CTA i of C adds up the parts of sequences i, i + C, ... and the first CTA the sequences.
struct StoreShared {
    float2* part;                 // [n_seqs, E], as in the slots
    float2* tokens;               // [n_seqs]
    int32_t E;
    __device__ __forceinline__ void operator()(int32_t s, int32_t e, float v, int32_t n) const {
        part[s * E + e] = make_float2(v, __int_as_float(n));
    }
    __device__ __forceinline__ void operator()(int32_t s, float z, int32_t n) const {
        tokens[s] = make_float2(z, __int_as_float(n));
    }
};

__device__ __forceinline__ float2 load_cluster2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

template <int L, int PER, bool VEC>
__global__ void __launch_bounds__(THREADS, PER <= 16 ? 2 : 1) balance_cluster_kernel(const BalanceParams p) {
    extern __shared__ float sums[];                               // [HALF][E], int [E], then StoreShared's
    __shared__ Sum dots[WARPS];
    __shared__ float2 final_sums[MAX_CLUSTER][2];                 // of the first CTA: Σ 1/T_s·Σ counts·Σ p, Σ logsumexp²
    __shared__ int32_t final_tokens[MAX_CLUSTER];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t E = p.r.n_experts, S = p.r.n_seqs;
    const int32_t rank = static_cast<int32_t>(blockIdx.x), C = static_cast<int32_t>(gridDim.x);
    float2* part = reinterpret_cast<float2*>(sums + (HALF + 1) * E + (E & 1));
    const StoreShared store{part, part + S * E, E};
    for (int e = threadIdx.x; e < E; e += THREADS) sums[HALF * E + e] = 0.0f;
    for (int i = threadIdx.x; i < S * E + S; i += THREADS) part[i] = make_float2(0.0f, 0.0f);
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    if (p.r.seq_offsets && rank == 0 && static_cast<int32_t>(threadIdx.x) < S && p.status) {
        const int32_t a = p.r.seq_offsets[threadIdx.x], b = p.r.seq_offsets[threadIdx.x + 1];
        if (a > b || a < 0 || b > p.r.n_tokens) atomicOr(p.status, MOE_DEV_BAD_TABLE);
    }
    const int64_t first = static_cast<int64_t>(rank) * p.chunk;
    add_tokens<L, PER, VEC>(p, first, first + p.chunk < p.r.n_tokens ? first + p.chunk : p.r.n_tokens, sums, store);
    auto sync_all = [C] {
        if (C > 1) cluster_sync_all();
        else __syncthreads();
    };
    sync_all();
    Sum bal, z;                                                   // of this CTA's sequences, by its first thread
    int32_t n = 0;
    for (int32_t s = rank; s < S; s += C) {
        Sum dot;
        for (int32_t e = threadIdx.x; e < E; e += THREADS) {
            const uint32_t at = smem_u32(part + s * E + e);
            Sum v;
            int32_t c = 0;
#pragma unroll 8
            for (int32_t r = 0; r < C; ++r) {
                const float2 x = load_cluster2(mapa_shared(at, static_cast<uint32_t>(r)));
                v.add(x.x);
                c += __float_as_int(x.y);
            }
            p.counts[static_cast<int64_t>(s) * E + e] = c;
            dot.add(v.times(static_cast<float>(c)));
        }
        dot.add_lanes();
        if (lane == 0) dots[warp] = dot;
        __syncthreads();
        if (warp == 0) {
            float2 x = make_float2(0.0f, 0.0f);
            if (lane < C) x = load_cluster2(mapa_shared(smem_u32(store.tokens + s), static_cast<uint32_t>(lane)));
            Sum zs, d;
            int32_t ns = __float_as_int(x.y);
            zs.add(x.x);
            zs.add_lanes();
            if (lane < WARPS) d = dots[lane];
            d.add_lanes();
#pragma unroll
            for (int i = 16; i > 0; i >>= 1) ns += __shfl_xor_sync(0xffffffffu, ns, i);
            if (ns > 0) bal.add(d.times(1.0f / static_cast<float>(ns)));
            z.add(zs);
            n += ns;
            if (lane == 0) p.seq_tokens[s] = ns;
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        const uint32_t to = mapa_shared(smem_u32(&final_sums[rank][0]), 0), n_to = mapa_shared(smem_u32(&final_tokens[rank]), 0);
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(bal.hi), "f"(bal.lo) : "memory");
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to + 8), "f"(z.hi), "f"(z.lo) : "memory");
        asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(n_to), "r"(n) : "memory");
    }
    sync_all();
    if (rank == 0 && warp == 0) {
        Sum b, y;
        int32_t m = 0;
        if (lane < C) {
            b.hi = final_sums[lane][0].x;
            b.lo = final_sums[lane][0].y;
            y.hi = final_sums[lane][1].x;
            y.lo = final_sums[lane][1].y;
            m = final_tokens[lane];
        }
        b.add_lanes();
        y.add_lanes();
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) m += __shfl_xor_sync(0xffffffffu, m, i);
        if (lane == 0) store_losses(p, b, y, m);
    }
}

// Grid: 32 experts of a sequence per block.  The last block to finish adds the sequences up.
__global__ void __launch_bounds__(32 * REDUCE_WARPS) balance_reduce_kernel(const BalanceParams p) {
    __shared__ Sum sum[REDUCE_WARPS][33];
    __shared__ int32_t cnt[REDUCE_WARPS][33];
    __shared__ bool final_block;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t E = p.r.n_experts, S = p.r.n_seqs;
    const int32_t s = blockIdx.y, e = blockIdx.x * 32 + lane;
    const Seqs seqs{p.r.seq_offsets, S, p.r.n_tokens};
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int64_t t0 = seqs.bound(s), t1 = seqs.bound(s + 1);
    if (threadIdx.x == 0 && blockIdx.x == 0 && p.r.seq_offsets && p.status &&
        (t1 < t0 || t0 != p.r.seq_offsets[s] || t1 != p.r.seq_offsets[s + 1]))
        atomicOr(p.status, MOE_DEV_BAD_TABLE);
    const bool any = t1 > t0;
    const int32_t b0 = any ? static_cast<int32_t>(t0 / p.chunk) + s : 0;
    const int32_t b1 = any ? static_cast<int32_t>((t1 - 1) / p.chunk) + s : -1;
    Sum v;
    int32_t c = 0;
    if (e < E) {
#pragma unroll 4
        for (int32_t b = b0 + warp; b <= b1; b += REDUCE_WARPS) {
            const float2 x = p.part[static_cast<int64_t>(b) * E + e];
            v.add(x.x);
            c += __float_as_int(x.y);
        }
    }
    sum[warp][lane] = v;
    cnt[warp][lane] = c;
    // the tokens of the sequence: another warp than the one that goes on with the experts
    if (blockIdx.x == 0 && warp == 1) {
        Sum z;
        int32_t n = 0;
        for (int32_t b = b0 + lane; b <= b1; b += 32) {
            const float2 x = p.tokens[b];
            z.add(x.x);
            n += __float_as_int(x.y);
        }
        z.add_lanes();
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) n += __shfl_xor_sync(0xffffffffu, n, d);
        if (lane == 0) {
            p.zsum[s] = z;
            p.seq_tokens[s] = n;
            __threadfence();
        }
    }
    __syncthreads();
    // a warp has an expert, a lane one of the parts
    static_assert(REDUCE_WARPS == 32, "as many warps as experts and as lanes");
    v = sum[lane][warp];
    c = cnt[lane][warp];
    v.add_lanes();
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) c += __shfl_xor_sync(0xffffffffu, c, d);
    __syncthreads();
    const int32_t ew = blockIdx.x * 32 + warp;
    if (lane == 0) {
        if (ew < E) p.counts[static_cast<int64_t>(s) * E + ew] = c;
        sum[0][warp] = ew < E ? v.times(static_cast<float>(c)) : Sum();
    }
    __syncthreads();
    if (warp == 0) {
        v = sum[0][lane];
        v.add_lanes();
        if (lane == 0) {
            p.dots[static_cast<int64_t>(s) * gridDim.x + blockIdx.x] = v;
            __threadfence();
            final_block = atomicAdd(p.done, 1u) == gridDim.x * gridDim.y - 1;
        }
    }
    __syncthreads();
    if (!final_block) return;
    __threadfence();
    // every warp its sequences in order, a lane each of their parts; then the warps in a tree
    static_assert(MOE_MAX_EXPERTS <= 32 * 32, "a lane for every block of experts");
    Sum bal, z;
    int32_t n = 0;
    for (int32_t i = warp; i < S; i += REDUCE_WARPS) {
        float2 x = make_float2(0.0f, 0.0f);
        if (lane < static_cast<int>(gridDim.x))
            x = __ldcg(reinterpret_cast<const float2*>(p.dots + static_cast<int64_t>(i) * gridDim.x + lane));
        const float2 y = __ldcg(reinterpret_cast<const float2*>(p.zsum + i));
        const int32_t ni = __ldcg(p.seq_tokens + i);
        Sum d, one;
        d.hi = x.x;
        d.lo = x.y;
        d.add_lanes();
        if (ni > 0) bal.add(d.times(1.0f / static_cast<float>(ni)));
        one.hi = y.x;
        one.lo = y.y;
        z.add(one);
        n += ni;
    }
    if (lane == 0) {
        sum[0][warp] = bal;
        sum[1][warp] = z;
        cnt[0][warp] = n;
    }
    __syncthreads();
    if (warp == 0) {
        bal = sum[0][lane];
        z = sum[1][lane];
        n = cnt[0][lane];
        bal.add_lanes();
        z.add_lanes();
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) n += __shfl_xor_sync(0xffffffffu, n, d);
        if (lane == 0) {
            store_losses(p, bal, z, n);
        }
    }
}

// ---------------------------------------------------------------------------
// gradients of the logits
// ---------------------------------------------------------------------------

struct GradParams {
    Routing r;
    int32_t chunk;                // tokens of a block, a multiple of 64
    const float* d_weights;
    const float* d_losses;
    const int32_t* counts;
    const int32_t* seq_tokens;
    uint16_t* dz;                 // [n_tokens, ld], in bf16 by the first pass, in fp16 by the second
    uint16_t* rest;               // [n_tokens, ld], nullable: what the rounding left
    int32_t ld;
    float* d_logits;              // [n_tokens, E]; nullable in bf16
    float* scale;
    float* block_max;             // [blocks of the first pass]
    int32_t n_blocks;
    uint32_t* valid;              // nullable, as is what follows: all tokens count
    int32_t* block_dirty;
    const uint16_t* x;
    int32_t hidden;
    int32_t* status;
};

// 2^s that brings a largest magnitude m into [2^13, 2^14): fp16 then holds values down to
// 2^-27 of it with all their bits, and sums of products stay far inside fp32.
__device__ __forceinline__ float grad_scale(float m) {
    if (!(m > 0.0f)) return 1.0f;
    int x;
    frexpf(m, &x);
    const int s = 14 - x;
    return ldexpf(1.0f, s > 120 ? 120 : (s < -120 ? -120 : s));
}

// Is one of the 8 values in 16 bytes infinite or NaN.
template <bool BF16>
__device__ __forceinline__ uint32_t not_finite(const uint4& v) {
    // all exponent bits set: adding one of them to the magnitude reaches the sign's place
    constexpr uint32_t ONE = BF16 ? 0x00800080u : 0x04000400u;
    return (((v.x & 0x7fff7fffu) + ONE) | ((v.y & 0x7fff7fffu) + ONE) | ((v.z & 0x7fff7fffu) + ONE) |
            ((v.w & 0x7fff7fffu) + ONE)) & 0x80008000u;
}

// Eight values rounded, and what that left.
template <bool BF16>
__device__ __forceinline__ void store_eight(uint16_t* at, uint16_t* rest, const float (&v)[8]) {
    uint32_t w[4], r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        w[j] = pack_16bit2<BF16>(v[2 * j], v[2 * j + 1]);
        const float2 f = unpack_16bit2<BF16>(w[j]);
        r[j] = pack_16bit2<BF16>(v[2 * j] - f.x, v[2 * j + 1] - f.y);
    }
    *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
    if (rest) *reinterpret_cast<uint4*>(rest) = make_uint4(r[0], r[1], r[2], r[3]);
}

// fp16 operands from fp32 gradients, times the power of two that their largest magnitude asks for: pieces
// first, first + step, ...
__device__ __forceinline__ void round_values(const GradParams& p, float largest, int64_t first, int64_t step) {
    const float scale = grad_scale(largest);
    if (first == 0) {
        p.scale[0] = scale;
        p.scale[1] = 1.0f / scale;
    }
    const int32_t E = p.r.n_experts, pieces = p.ld / 8;
    const int64_t all = p.r.n_tokens * pieces;
    for (int64_t i = first; i < all; i += step) {
        float v[8];
        if ((E & 7) == 0) {
            // rows one after the other in both arrays
            const float4* src = reinterpret_cast<const float4*>(p.d_logits) + 2 * i;
            const float4 a = src[0], b = src[1];
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
            const int64_t t = i / pieces;
            const int32_t e = static_cast<int32_t>(i - t * pieces) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = e + j < E ? p.d_logits[t * E + e + j] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= scale;
        store_eight<false>(p.dz + 8 * i, p.rest ? p.rest + 8 * i : nullptr, v);
    }
}

// d_z, and of the tokens that do not count whether x holds something that a product with zero does not
// remove.  bf16 operands are rounded here.  fp16 would lose gradients of a mean over tokens, so its
// operands are d_z times a power of two that the largest of all sets: round_kernel, from the
// fp32 values and the blocks' largest magnitudes that are left here (one block does it itself).  (Computing d_z twice instead, once
// for its maximum, took 8 us more for 16384 x 256.)
template <int L, int PER, bool VEC, bool BF16>
__global__ void __launch_bounds__(THREADS, PER <= 16 ? 2 : 1) logit_gradient_kernel(const GradParams p) {
    __shared__ float smax[WARPS];
    constexpr int PACK = 32 / L;
    constexpr int ROW = L * PER + 4;
    // per token that the block has at a time: the counts' part of g, by expert, to which the routed
    // gradients are added and taken off again
    extern __shared__ float rows[];                               // [WARPS * PACK][ROW]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane & (L - 1);
    const int32_t E = p.r.n_experts, k = p.r.top_k;
    float* mine = rows + (warp * PACK + lane / L) * ROW;
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    if (BF16 && blockIdx.x == 0 && threadIdx.x == 0) p.scale[0] = p.scale[1] = 1.0f;
    const Seqs seqs{p.r.seq_offsets, p.r.n_seqs, p.r.n_tokens};
    const int64_t first = static_cast<int64_t>(blockIdx.x) * p.chunk;
    const int64_t last = first + p.chunk < p.r.n_tokens ? first + p.chunk : p.r.n_tokens;
    const int64_t begin = seqs.bound(0), finish = seqs.bound(p.r.n_seqs);
    float cb = 0.0f, cz = 0.0f;
    if (p.d_losses) {
        const float n = static_cast<float>(p.seq_tokens[p.r.n_seqs]);
        if (n > 0.0f) {
            cb = p.d_losses[0] * static_cast<float>(E) / (static_cast<float>(k) * n);
            cz = p.d_losses[1] * 2.0f / n;
        }
    }
    int64_t t = first + warp * PACK + lane / L;
    int32_t s = seqs.find(first + warp * PACK);
    int64_t s_end = seqs.bound(s + 1);           // (of s = -1: where the first one starts)
    int32_t base_of = -1;                        // the sequence whose counts are in `mine`
    for (int i = l; i < L * PER; i += L) mine[i] = 0.0f;
    __syncwarp();
    float largest = 0.0f;
    for (int64_t tw = first + warp * PACK; tw < last; tw += WARPS * PACK, t += WARPS * PACK) {
        const bool live = t < last && t >= begin && t < finish && counts_token(p.r.token_mask, t);
        float z[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) z[i] = 0.0f;
        int32_t id = -1;
        float dw = 0.0f;
        if (live) {
            load_row<L, PER, VEC>(z, p.r.logits + t * E, l, E);
            if (p.d_weights && l < k) {
                id = __ldg(p.r.topk_ids + t * k + l);
                dw = __ldg(p.d_weights + t * k + l);
            }
        }
        if (cb != 0.0f) {
            while (t >= s_end && s + 1 < p.r.n_seqs) {
                ++s;
                s_end = seqs.bound(s + 1);
            }
            if (live && s != base_of && s >= 0) {
                base_of = s;
                const float per_count = cb / static_cast<float>(max(p.seq_tokens[s], 1));
                const int32_t* row = p.counts + static_cast<int64_t>(s) * E;
                for (int e = l; e < E; e += L) mine[e] = per_count * static_cast<float>(__ldg(row + e));
            }
            __syncwarp();
        }
        float base = 0.0f;
        if (p.d_weights) {
            if (id >= E) {
                if (p.status) atomicOr(p.status, MOE_DEV_BAD_EXPERT_ID);
                id = -1;
            }
            // an expert named twice gets both, in their order, from either lane
            const uint32_t same = __match_any_sync(0xffffffffu, id < 0 ? -1 - lane : id * 32 + lane / L);
            if (__any_sync(0xffffffffu, (same & (same - 1)) != 0)) {
                float w = 0.0f;
                for (int q = 0; q < k; ++q) {
                    const int from = (lane & ~(L - 1)) + q;
                    const float wq = __shfl_sync(0xffffffffu, dw, from);
                    if (same >> from & 1u) w += wq;
                }
                dw = w;
            }
            if (id >= 0) base = mine[id];
            __syncwarp();
            if (id >= 0) mine[id] = base + dw;
            __syncwarp();
        }
        float d[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) d[i] = mine[expert<L, VEC>(l, i)];
        if (p.d_weights) {
            __syncwarp();
            if (id >= 0) mine[id] = base;
            __syncwarp();                                         // before the next token's lanes read or replace it
        }
        const float lse = softmax_row<L, PER>(z);
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) dot += z[i] * d[i];
        const float shift = cz * lse - lanes_sum<L>(dot);
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            d[i] = live ? z[i] * (d[i] + shift) : 0.0f;
            if (!BF16 && expert<L, VEC>(l, i) < E) top = fmaxf(top, fabsf(d[i]));
        }
        // (an infinity, beside which nothing of the token is finite, is one at any scale, and the others keep theirs)
        if (!BF16 && top < INFINITY) largest = fmaxf(largest, top);
        if (t >= last) continue;
        if (VEC) {
#pragma unroll
            for (int i = 0; i < PER; i += 8) {
                const int e = expert<L, VEC>(l, i);
                if (BF16 && e < p.ld) {                  // (columns E .. ld - 1 are not read)
                    const float v[8] = {d[i], d[i + 1], d[i + 2], d[i + 3], d[i + 4], d[i + 5], d[i + 6], d[i + 7]};
                    store_eight<true>(p.dz + t * p.ld + e, p.rest ? p.rest + t * p.ld + e : nullptr, v);
                }
                if (p.d_logits && e < E)
                    *reinterpret_cast<float4*>(p.d_logits + t * E + e) = make_float4(d[i], d[i + 1], d[i + 2], d[i + 3]);
                if (p.d_logits && e + 4 < E)
                    *reinterpret_cast<float4*>(p.d_logits + t * E + e + 4) =
                        make_float4(d[i + 4], d[i + 5], d[i + 6], d[i + 7]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = expert<L, VEC>(l, i);
                if (BF16 && e < p.ld) {
                    const uint32_t w = pack_16bit2<true>(d[i], 0.0f) & 0xffffu;
                    p.dz[t * p.ld + e] = static_cast<uint16_t>(w);
                    if (p.rest) p.rest[t * p.ld + e] = static_cast<uint16_t>(pack_16bit2<true>(d[i] - unpack_16bit2<true>(w).x, 0.0f) & 0xffffu);
                }
                if (p.d_logits && e < E) p.d_logits[t * E + e] = d[i];
            }
        }
    }
    if (p.r.seq_offsets && p.status) {
        for (int32_t i = static_cast<int32_t>(blockIdx.x) * THREADS + static_cast<int32_t>(threadIdx.x); i < p.r.n_seqs;
             i += static_cast<int32_t>(gridDim.x) * THREADS) {
            const int32_t lo = __ldg(p.r.seq_offsets + i), hi = __ldg(p.r.seq_offsets + i + 1);
            if (lo > hi || lo < 0 || hi > p.r.n_tokens) atomicOr(p.status, MOE_DEV_BAD_TABLE);
        }
    }
    if (p.valid) {
        // a bit per token that counts; whole steps of 64, zero past the end
        uint32_t bad = 0;
        for (int64_t tv = first + 32 * warp; tv < first + p.chunk && tv < (p.r.n_tokens + 63) / 64 * 64; tv += THREADS) {
            const int64_t ti = tv + lane;
            const bool v = ti < p.r.n_tokens && ti >= begin && ti < finish && counts_token(p.r.token_mask, ti);
            const uint32_t bits = __ballot_sync(0xffffffffu, v);
            if (lane == 0) p.valid[tv >> 5] = bits;
            for (uint32_t out = ~bits; out != 0; out &= out - 1) {
                const int64_t to = tv + __ffs(static_cast<int>(out)) - 1;
                if (to >= p.r.n_tokens) break;
                const uint4* row = reinterpret_cast<const uint4*>(p.x + to * p.hidden);
#pragma unroll 4
                for (int32_t i = lane; i < p.hidden / 8; i += 32) bad |= not_finite<BF16>(__ldg(row + i));
            }
        }
        const int any = __syncthreads_or(bad != 0);
        if (threadIdx.x == 0) p.block_dirty[blockIdx.x] = any;
    }
    if (!BF16) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) largest = fmaxf(largest, __shfl_xor_sync(0xffffffffu, largest, d));
        if (lane == 0) smax[warp] = largest;
        __syncthreads();
        for (int w = 0; w < WARPS; ++w) largest = fmaxf(largest, smax[w]);
        if (gridDim.x == 1) round_values(p, largest, threadIdx.x, THREADS);       // nobody else's to wait for
        else if (threadIdx.x == 0) p.block_max[blockIdx.x] = largest;
    }
}

// The same for many blocks.
__global__ void __launch_bounds__(256) round_kernel(const GradParams p) {
    __shared__ float smax[8];
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    float m = 0.0f;
    for (int i = threadIdx.x; i < p.n_blocks; i += 256) m = fmaxf(m, p.block_max[i]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((threadIdx.x & 31) == 0) smax[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = fmaxf(m, smax[w]);
    round_values(p, m, static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, static_cast<int64_t>(gridDim.x) * 256);
}

int64_t round256(int64_t n) { return (n + 255) / 256 * 256; }

// Tokens of a block: about two blocks an SM, a multiple of `step`.
int32_t chunk_tokens(int64_t n_tokens, int step) {
    const int64_t blocks = 2 * 152;
    const int64_t c = (n_tokens + blocks - 1) / blocks;
    return static_cast<int32_t>((c + step - 1) / step * step);
}

template <class Params>
cudaError_t launch_pdl(void (*kernel)(Params), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                       const std::remove_const_t<Params>& p, int cluster = 1) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Lanes of a token, for its logits.
int balance_lanes(int32_t n_experts) {
    return n_experts > 256 ? 32 : n_experts % 4 != 0 || n_experts > 128 ? 16 : n_experts > 64 ? 8 : 4;
}

// CTAs of the cluster that does it all in one launch without a workspace; 0: too much for it.  As measured (us), one
// launch and two: 64 tokens of 64 experts 4.3 and 8.8, 4097 in 5 sequences 8.5 and 13.8, 16384 13.4 and 10.5; a round
// of all warps of 16 CTAs takes 0.8 to 1.1, and every sequence of a CTA is a round of its own.
constexpr int32_t CLUSTER_ROUNDS = 4;
constexpr int32_t CLUSTER_SEQS = 32;
constexpr int64_t CLUSTER_SHARED_BYTES = 47 * 1024;
int64_t cluster_shared_bytes(int32_t n_experts, int32_t n_seqs) {
    return int64_t{4} * (HALF + 1) * n_experts + 8 + int64_t{8} * n_seqs * (n_experts + 1);
}
int32_t balance_cluster(int64_t n_tokens, int32_t n_experts, int32_t n_seqs) {
    const int64_t round = WARPS * 32 / balance_lanes(n_experts);          // tokens that a CTA has at a time
    if (n_tokens > CLUSTER_ROUNDS * MAX_CLUSTER * round || n_seqs > CLUSTER_SEQS ||
        cluster_shared_bytes(n_experts, n_seqs) > CLUSTER_SHARED_BYTES)
        return 0;
    int32_t c = 1;
    while (c < MAX_CLUSTER && (n_tokens > 2 * c * round || n_seqs > 2 * c)) c *= 2;
    return c;
}

struct BalanceLayout {
    int32_t cluster, chunk, chunks, slots, expert_blocks;
    int64_t part, tokens, dots, zsum, done, bytes;
};

BalanceLayout balance_layout(int64_t n_tokens, int32_t n_experts, int32_t n_seqs) {
    BalanceLayout l;
    l.cluster = balance_cluster(n_tokens, n_experts, n_seqs);
    l.chunk = l.cluster ? static_cast<int32_t>((n_tokens + l.cluster - 1) / l.cluster) : chunk_tokens(n_tokens, n_tokens < int64_t{WARPS} * n_seqs ? 4 : WARPS);   // (short sequences are rounds, too)
    if (l.chunk == 0) l.chunk = WARPS;
    l.chunks = l.cluster ? l.cluster : static_cast<int32_t>((n_tokens + l.chunk - 1) / l.chunk);
    if (l.chunks == 0) l.chunks = 1;
    l.slots = l.chunks + n_seqs;
    l.expert_blocks = (n_experts + 31) / 32;
    int64_t at = 0;
    auto take = [&at](int64_t n) {
        const int64_t r = at;
        at += round256(n);
        return r;
    };
    l.part = take(int64_t{8} * l.slots * n_experts);
    l.tokens = take(int64_t{8} * l.slots);
    l.dots = take(int64_t{8} * n_seqs * l.expert_blocks);
    l.zsum = take(int64_t{8} * n_seqs);
    l.done = take(4);
    l.bytes = l.cluster ? 0 : at;
    return l;
}

// The largest cluster, a power of two, that the current device can place of any variant, asked once per device (more
// than 8 CTAs have to be allowed, and a part of a device may not have room for them); 0 on an error.
int32_t placeable_cluster() {
    struct Entry {
        std::once_flag once;
        int32_t ctas = 0;
    };
    constexpr int MAX_DEVICES = 16;
    static Entry table[MAX_DEVICES];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= MAX_DEVICES) return 0;
    Entry& r = table[dev];
    std::call_once(r.once, [&r] {
        int32_t all = MAX_CLUSTER;
        for (auto kernel : {balance_cluster_kernel<32, 32, true>, balance_cluster_kernel<32, 32, false>,
                            balance_cluster_kernel<16, 16, false>, balance_cluster_kernel<16, 16, true>,
                            balance_cluster_kernel<8, 16, true>, balance_cluster_kernel<4, 16, true>}) {
            cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            for (; all > 0; all /= 2) {
                cudaLaunchAttribute attr[1];
                attr[0].id = cudaLaunchAttributeClusterDimension;
                attr[0].val.clusterDim.x = static_cast<unsigned>(all);
                attr[0].val.clusterDim.y = 1;
                attr[0].val.clusterDim.z = 1;
                cudaLaunchConfig_t cfg{};
                cfg.gridDim = dim3(static_cast<unsigned>(all));
                cfg.blockDim = dim3(THREADS);
                cfg.dynamicSmemBytes = CLUSTER_SHARED_BYTES;
                cfg.attrs = attr;
                cfg.numAttrs = 1;
                int n = 0;
                if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n > 0) break;
            }
        }
        cudaGetLastError();
        r.ctas = all;
    });
    return r.ctas;
}

}  // namespace

int64_t router_balance_workspace_bytes(int64_t n_tokens, int32_t n_experts, int32_t n_seqs) {
    return balance_layout(n_tokens, n_experts, n_seqs).bytes;
}

cudaError_t launch_router_balance(const RouterBalance& a, cudaStream_t stream) {
    const BalanceLayout l = balance_layout(a.r.n_tokens, a.r.n_experts, a.r.n_seqs);
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    BalanceParams p{};
    p.r = a.r;
    p.chunk = l.chunk;
    p.n_slots = l.slots;
    p.part = reinterpret_cast<float2*>(ws + l.part);
    p.tokens = reinterpret_cast<float2*>(ws + l.tokens);
    p.dots = reinterpret_cast<Sum*>(ws + l.dots);
    p.zsum = reinterpret_cast<Sum*>(ws + l.zsum);
    p.done = reinterpret_cast<unsigned*>(ws + l.done);
    p.losses = a.losses;
    p.counts = a.counts;
    p.seq_tokens = a.seq_tokens;
    p.status = a.status;
    const int32_t E = a.r.n_experts;
    const bool vec = E % 4 == 0;
    const int lanes = balance_lanes(E);
    if (l.cluster) {
        // (any number of CTAs will do, with more tokens each; there is no workspace for the two launches)
        const int32_t most = placeable_cluster();
        if (most == 0) return cudaErrorNoDevice;
        const int32_t ctas = l.cluster < most ? l.cluster : most;
        if (ctas < l.cluster) p.chunk = static_cast<int32_t>((a.r.n_tokens + ctas - 1) / ctas);
        auto kernel = lanes == 32   ? (vec ? balance_cluster_kernel<32, 32, true> : balance_cluster_kernel<32, 32, false>)
                      : !vec        ? balance_cluster_kernel<16, 16, false>
                      : lanes == 16 ? balance_cluster_kernel<16, 16, true>
                      : lanes == 8  ? balance_cluster_kernel<8, 16, true>
                                    : balance_cluster_kernel<4, 16, true>;
        return launch_pdl(kernel, dim3(static_cast<unsigned>(ctas)), THREADS,
                          static_cast<size_t>(cluster_shared_bytes(E, a.r.n_seqs)), stream, p, ctas);
    }
    const size_t smem = static_cast<size_t>(HALF + 1) * E * 4;
    auto kernel = lanes == 32   ? (vec ? balance_kernel<32, 32, true> : balance_kernel<32, 32, false>)
                  : !vec        ? balance_kernel<16, 16, false>
                  : lanes == 16 ? balance_kernel<16, 16, true>
                  : lanes == 8  ? balance_kernel<8, 16, true>
                                : balance_kernel<4, 16, true>;
    const cudaError_t err = launch_pdl(kernel, dim3(static_cast<unsigned>(l.chunks)), THREADS, smem, stream, p);
    if (err != cudaSuccess) return err;
    return launch_pdl(balance_reduce_kernel, dim3(static_cast<unsigned>(l.expert_blocks), static_cast<unsigned>(a.r.n_seqs)),
                      32 * REDUCE_WARPS, 0, stream, p);
}

int router_grad_blocks(int64_t n_tokens) {
    const int32_t c = chunk_tokens(n_tokens, 64);
    return static_cast<int>((n_tokens + c - 1) / c);
}

template <bool BF16>
static cudaError_t launch_gradient_pass(const GradParams& p, cudaStream_t stream) {
    const int32_t E = p.r.n_experts;
    const bool vec = E % 4 == 0;
    // 16 logits a lane, and a lane for each of a token's ids
    const int k = p.r.top_k;
    const int lanes = E > 256 ? 32 : !vec || E > 128 || k > 8 ? 16 : E > 64 || k > 4 ? 8 : 4;
    const int per = E > 256 ? 32 : 16;
    auto kernel = per == 32     ? (vec ? logit_gradient_kernel<32, 32, true, BF16> : logit_gradient_kernel<32, 32, false, BF16>)
                : !vec          ? logit_gradient_kernel<16, 16, false, BF16>
                : lanes == 16   ? logit_gradient_kernel<16, 16, true, BF16>
                : lanes == 8    ? logit_gradient_kernel<8, 16, true, BF16>
                                : logit_gradient_kernel<4, 16, true, BF16>;
    const size_t smem = static_cast<size_t>(WARPS) * (32 / lanes) * (lanes * per + 4) * 4;
    if (smem > 48 * 1024) {
        const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (err != cudaSuccess) return err;
    }
    return launch_pdl(kernel, dim3(static_cast<unsigned>(p.n_blocks)), THREADS, smem, stream, p);
}

cudaError_t launch_logit_gradients(const RouterBackward& a, const LogitGradients& g, cudaStream_t stream) {
    GradParams p{};
    p.r = a.r;
    p.chunk = chunk_tokens(a.r.n_tokens, 64);
    p.n_blocks = router_grad_blocks(a.r.n_tokens);
    p.d_weights = a.d_topk_weights;
    p.d_losses = a.d_losses;
    p.counts = a.counts;
    p.seq_tokens = a.seq_tokens;
    p.dz = g.dz;
    p.rest = g.two ? g.dz + a.r.n_tokens * g.ld : nullptr;
    p.ld = g.ld;
    p.d_logits = a.d_logits || a.bf16 ? a.d_logits : g.d_logits;
    p.scale = g.scale;
    p.block_max = g.block_max;
    p.valid = g.valid;
    p.block_dirty = g.block_dirty;
    p.x = a.x;
    p.hidden = a.hidden;
    p.status = a.status;
    if (a.bf16) return launch_gradient_pass<true>(p, stream);
    const cudaError_t err = launch_gradient_pass<false>(p, stream);
    if (err != cudaSuccess || p.n_blocks == 1) return err;
    const int64_t blocks = (a.r.n_tokens * (g.ld / 8) + 255) / 256, most = 8 * 152;
    return launch_pdl(round_kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), 256, 0, stream, p);
}

}  // namespace moe
