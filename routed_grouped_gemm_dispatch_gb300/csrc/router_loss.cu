// The router's losses with its per-expert counts, and the gradients of its logits.
//
// With z the logits, p = softmax(z), T valid tokens, T_s of them in sequence s:
//     counts[s, e] = pairs of sequence s whose id is e
//     losses[0] = E / (k T) · Σ_s 1/T_s · Σ_e counts[s, e] · Σ_t∈s p[t, e]
//     losses[1] = 1/T · Σ_t logsumexp(z[t])²
//     g[t, e] = d_losses[0]·E / (k T T_s)·counts[s, e] + Σ_j [id[t, j] = e]·d_w[t, j]
//     d_z = p ⊙ (g − Σ_e p g) + d_losses[1]·2/T·logsumexp(z)·p
//
// A warp has a token: its lanes hold the token's logits in registers, lane for
// lane the same experts, so that column sums over a warp's tokens stay in
// registers until the end of a piece.  All is read once; sums over tokens are fp32 over the
// tokens of a warp and of a block, fp64 beyond, always in the same order.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/moe_gb300.h"
#include "moe_internal.h"
#include "sm103_ptx.cuh"
#include "tile_store.cuh"
#include "train_internal.h"

namespace moe {
namespace {

constexpr int WARPS = 16;
constexpr int THREADS = 32 * WARPS;
constexpr int REDUCE_WARPS = 8;
constexpr int HALF = WARPS / 2;

// A token's logits in the lanes of a warp: value i of a lane is expert
// `expert(i)`.  VEC: E is a multiple of 4 and rows are whole 16-byte pieces.
template <int PER, bool VEC>
__device__ __forceinline__ int expert(int lane, int i) {
    return VEC ? 4 * lane + 128 * (i >> 2) + (i & 3) : lane + 32 * i;
}

template <int PER, bool VEC>
__device__ __forceinline__ void load_row(float (&z)[PER], const float* row, int lane, int32_t n_experts) {
    if (VEC) {
#pragma unroll
        for (int i = 0; i < PER; i += 4) {
            const int e = expert<PER, VEC>(lane, i);
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
            const int e = expert<PER, VEC>(lane, i);
            z[i] = e < n_experts ? __ldg(row + e) : -INFINITY;
        }
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// The row becomes its softmax; returns its logsumexp.
template <int PER>
__device__ __forceinline__ float softmax_row(float (&z)[PER]) {
    float top = z[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) top = fmaxf(top, z[i]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        z[i] = expf(z[i] - top);
        sum += z[i];
    }
    sum = warp_sum(sum);
    const float inv = 1.0f / sum;
#pragma unroll
    for (int i = 0; i < PER; ++i) z[i] *= inv;
    return top + logf(sum);
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
    // the last sequence that starts at or before token t (-1: none)
    __device__ __forceinline__ int32_t find(int64_t t) const {
        int32_t lo = 0, hi = n;
        while (lo < hi) {
            const int32_t mid = (lo + hi) >> 1;
            if (bound(mid) <= t) lo = mid + 1;
            else hi = mid;
        }
        return lo - 1;
    }
};

__device__ __forceinline__ bool counts_token(const uint8_t* mask, int64_t t) { return mask == nullptr || mask[t] != 0; }

struct BalanceParams {
    Routing r;
    int32_t chunk;                // tokens of a block
    int32_t n_slots;
    float* psum;                  // [n_slots, E] Σ p of a block's tokens of one sequence
    int32_t* pcount;              // [n_slots, E]
    float* pz;                    // [n_slots] Σ logsumexp²
    int32_t* pn;                  // [n_slots] valid tokens
    double* dots;                 // [n_seqs, expert blocks] Σ_e counts·Σ p
    double* zsum;                 // [n_seqs]
    unsigned* done;
    float* losses;
    int32_t* counts;
    int32_t* seq_tokens;
    int32_t* status;
};

// One block per `chunk` tokens.  The part of sequence s in block b goes to slot b + s:
// from one part to the next either b or s grows, so no two share a slot.
template <int PER, bool VEC>
__global__ void __launch_bounds__(THREADS, PER <= 8 ? 2 : 1) balance_kernel(const BalanceParams p) {
    extern __shared__ float sums[];                               // [HALF][E], then int [E]
    __shared__ float zpart[WARPS];
    __shared__ int npart[WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t E = p.r.n_experts, k = p.r.top_k;
    int32_t* hist = reinterpret_cast<int32_t*>(sums + HALF * E);
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.done = 0;
    const Seqs seqs{p.r.seq_offsets, p.r.n_seqs, p.r.n_tokens};
    const int64_t first = static_cast<int64_t>(blockIdx.x) * p.chunk;
    const int64_t last = first + p.chunk < p.r.n_tokens ? first + p.chunk : p.r.n_tokens;
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
        for (int e = threadIdx.x; e < E; e += THREADS) hist[e] = 0;
        __syncthreads();
        float acc[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] = 0.0f;
        float zz = 0.0f;
        int n = 0;
        // the next token's row is on its way while this one is reduced
        float z[PER], next[PER];
        int64_t t = t0 + warp;
        bool live = t < t1 && counts_token(p.r.token_mask, t);
        if (live) load_row<PER, VEC>(z, p.r.logits + t * E, lane, E);
        while (t < t1) {
            const int64_t tn = t + WARPS;
            const bool live_next = tn < t1 && counts_token(p.r.token_mask, tn);
            if (live_next) load_row<PER, VEC>(next, p.r.logits + tn * E, lane, E);
            if (live) {
                if (lane < k) {
                    const int32_t id = p.r.topk_ids[t * k + lane];
                    if (id >= 0 && id < E) atomicAdd(&hist[id], 1);
                    else if (id >= E && p.status) atomicOr(p.status, MOE_DEV_BAD_EXPERT_ID);
                }
                const float lse = softmax_row<PER>(z);
#pragma unroll
                for (int i = 0; i < PER; ++i) acc[i] += z[i];
                zz += lse * lse;
                ++n;
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) z[i] = next[i];
            live = live_next;
            t = tn;
        }
        if (lane == 0) {
            zpart[warp] = zz;
            npart[warp] = n;
        }
        if (warp >= HALF) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = expert<PER, VEC>(lane, i);
                if (e < E) sums[(warp - HALF) * E + e] = acc[i];
            }
        }
        __syncthreads();
        if (warp < HALF) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = expert<PER, VEC>(lane, i);
                if (e < E) sums[warp * E + e] += acc[i];
            }
        }
        __syncthreads();
        const int64_t slot = static_cast<int64_t>(blockIdx.x) + s;
        MOE_DCHECK(slot < p.n_slots && t0 >= 0 && t1 <= p.r.n_tokens, p.status);
        for (int e = threadIdx.x; e < E; e += THREADS) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < HALF; ++w) v += sums[w * E + e];
            p.psum[slot * E + e] = v;
            p.pcount[slot * E + e] = hist[e];
        }
        if (threadIdx.x == 0) {
            float zt = 0.0f;
            int nt = 0;
            for (int w = 0; w < WARPS; ++w) {
                zt += zpart[w];
                nt += npart[w];
            }
            p.pz[slot] = zt;
            p.pn[slot] = nt;
        }
        __syncthreads();
        t0 = t1;
        ++s;
    }
}

// Grid: 32 experts of a sequence per block.  The last block to finish adds the sequences up.
__global__ void __launch_bounds__(32 * REDUCE_WARPS) balance_reduce_kernel(const BalanceParams p) {
    __shared__ double sum[REDUCE_WARPS][32];
    __shared__ int32_t cnt[REDUCE_WARPS][32];
    __shared__ double zs[REDUCE_WARPS];
    __shared__ int32_t ns[REDUCE_WARPS];
    __shared__ bool final_block;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t E = p.r.n_experts, S = p.r.n_seqs;
    const int32_t s = blockIdx.y, e = blockIdx.x * 32 + lane;
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const Seqs seqs{p.r.seq_offsets, S, p.r.n_tokens};
    const int64_t t0 = seqs.bound(s), t1 = seqs.bound(s + 1);
    if (threadIdx.x == 0 && blockIdx.x == 0 && p.r.seq_offsets && p.status &&
        (t1 < t0 || t0 != p.r.seq_offsets[s] || t1 != p.r.seq_offsets[s + 1]))
        atomicOr(p.status, MOE_DEV_BAD_TABLE);
    double v = 0.0, z = 0.0;
    int32_t c = 0, n = 0;
    if (t1 > t0) {
        const int64_t b0 = t0 / p.chunk + s, b1 = (t1 - 1) / p.chunk + s;
        if (e < E) {
#pragma unroll 8
            for (int64_t b = b0 + warp; b <= b1; b += REDUCE_WARPS) {
                v += p.psum[b * E + e];
                c += p.pcount[b * E + e];
            }
        }
        if (blockIdx.x == 0) {
            for (int64_t b = b0 + threadIdx.x; b <= b1; b += 32 * REDUCE_WARPS) {
                z += p.pz[b];
                n += p.pn[b];
            }
        }
    }
    sum[warp][lane] = v;
    cnt[warp][lane] = c;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        z += __shfl_xor_sync(0xffffffffu, z, d);
        n += __shfl_xor_sync(0xffffffffu, n, d);
    }
    if (lane == 0) {
        zs[warp] = z;
        ns[warp] = n;
    }
    __syncthreads();
    if (warp == 0) {
        v = 0.0;
        c = 0;
        for (int w = 0; w < REDUCE_WARPS; ++w) {
            v += sum[w][lane];
            c += cnt[w][lane];
        }
        if (e < E) p.counts[static_cast<int64_t>(s) * E + e] = c;
        v *= c;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        if (lane == 0) {
            p.dots[static_cast<int64_t>(s) * gridDim.x + blockIdx.x] = v;
            if (blockIdx.x == 0) {
                z = 0.0;
                n = 0;
                for (int w = 0; w < REDUCE_WARPS; ++w) {
                    z += zs[w];
                    n += ns[w];
                }
                p.zsum[s] = z;
                p.seq_tokens[s] = n;
            }
            __threadfence();
            final_block = atomicAdd(p.done, 1u) == gridDim.x * gridDim.y - 1;
        }
    }
    __syncthreads();
    if (!final_block) return;
    __threadfence();
    // every thread its sequences in order, then the threads in order
    v = 0.0;
    z = 0.0;
    n = 0;
    for (int32_t i = threadIdx.x; i < S; i += 32 * REDUCE_WARPS) {
        const int32_t ni = __ldcg(p.seq_tokens + i);
        double d = 0.0;
        for (unsigned b = 0; b < gridDim.x; ++b) d += __ldcg(p.dots + static_cast<int64_t>(i) * gridDim.x + b);
        if (ni > 0) v += d / ni;
        z += __ldcg(p.zsum + i);
        n += ni;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        v += __shfl_xor_sync(0xffffffffu, v, d);
        z += __shfl_xor_sync(0xffffffffu, z, d);
        n += __shfl_xor_sync(0xffffffffu, n, d);
    }
    __syncthreads();
    if (lane == 0) {
        sum[warp][0] = v;
        cnt[warp][0] = n;
        zs[warp] = z;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        v = 0.0;
        z = 0.0;
        n = 0;
        for (int w = 0; w < REDUCE_WARPS; ++w) {
            v += sum[w][0];
            z += zs[w];
            n += cnt[w][0];
        }
        const double tokens = n > 0 ? n : 1;
        p.losses[0] = static_cast<float>(v * E / (p.r.top_k * tokens));
        p.losses[1] = static_cast<float>(z / tokens);
        p.seq_tokens[S] = n;
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
    uint16_t* dz;
    int32_t ld;
    float* d_logits;
    float* scale;
    float* block_max;
    uint32_t* valid;
    int32_t* status;
};

// 2^s that brings a largest magnitude m into [2^13, 2^14): fp16 then holds values down to
// 2^-27 of it with all their bits, and sums of products stay far inside fp32.
__device__ __forceinline__ float grad_scale(float m) {
    if (!(m > 0.0f) || m > 3.0e38f) return 1.0f;
    int x;
    frexpf(m, &x);
    const int s = 14 - x;
    return ldexpf(1.0f, s > 120 ? 120 : (s < -120 ? -120 : s));
}

// MAX: only the largest |d_z| of each block, which sets the power of two that
// the values are stored times (fp16 would lose gradients of a mean over tokens
// otherwise; bf16 has fp32's range and needs none).  Otherwise the values.
template <int PER, bool VEC, bool BF16, bool MAX>
__global__ void __launch_bounds__(THREADS, PER <= 8 ? 2 : 1) logit_gradient_kernel(const GradParams p) {
    __shared__ float smax[WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t E = p.r.n_experts, k = p.r.top_k;
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    float scale = 1.0f;
    if (!MAX && !BF16) {
        float m = 0.0f;
        for (unsigned i = threadIdx.x; i < gridDim.x; i += THREADS) m = fmaxf(m, p.block_max[i]);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        if (lane == 0) smax[warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WARPS; ++w) m = fmaxf(m, smax[w]);
        scale = grad_scale(m);
    }
    if (!MAX && blockIdx.x == 0 && threadIdx.x == 0) {
        p.scale[0] = scale;
        p.scale[1] = 1.0f / scale;
    }
    const Seqs seqs{p.r.seq_offsets, p.r.n_seqs, p.r.n_tokens};
    const int64_t first = static_cast<int64_t>(blockIdx.x) * p.chunk;
    const int64_t last = first + p.chunk < p.r.n_tokens ? first + p.chunk : p.r.n_tokens;
    const int64_t begin = seqs.bound(0), finish = seqs.bound(p.r.n_seqs);
    if (!MAX) {
        // a bit per token that counts; whole steps of 64, zero past the end
        for (int64_t t = first + 32 * warp; t < first + p.chunk && t < (p.r.n_tokens + 63) / 64 * 64; t += THREADS) {
            const int64_t ti = t + lane;
            const bool v = ti < p.r.n_tokens && ti >= begin && ti < finish && counts_token(p.r.token_mask, ti);
            const uint32_t bits = __ballot_sync(0xffffffffu, v);
            if (lane == 0) p.valid[t >> 5] = bits;
        }
    }
    float cb = 0.0f, cz = 0.0f;
    if (p.d_losses) {
        const float n = static_cast<float>(p.seq_tokens[p.r.n_seqs]);
        if (n > 0.0f) {
            cb = p.d_losses[0] * static_cast<float>(E) / (static_cast<float>(k) * n);
            cz = p.d_losses[1] * 2.0f / n;
        }
    }
    int32_t s = seqs.find(first + warp);
    float largest = 0.0f;
    for (int64_t t = first + warp; t < last; t += WARPS) {
        while (s + 1 < p.r.n_seqs && seqs.bound(s + 1) <= t) ++s;
        const bool live = t >= begin && t < finish && s >= 0 && counts_token(p.r.token_mask, t);
        float d[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) d[i] = 0.0f;
        if (live) {
            float z[PER];
            load_row<PER, VEC>(z, p.r.logits + t * E, lane, E);
            const float per_count = cb != 0.0f ? cb / static_cast<float>(max(p.seq_tokens[s], 1)) : 0.0f;
            if (cb != 0.0f) {
                const int32_t* row = p.counts + static_cast<int64_t>(s) * E;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int e = expert<PER, VEC>(lane, i);
                    if (e < E) d[i] = per_count * static_cast<float>(__ldg(row + e));
                }
            }
            if (p.d_weights) {
                int32_t id = -1;
                float dw = 0.0f;
                if (lane < k) {
                    id = p.r.topk_ids[t * k + lane];
                    dw = p.d_weights[t * k + lane];
                    if (id >= E) {
                        if (p.status) atomicOr(p.status, MOE_DEV_BAD_EXPERT_ID);
                        id = -1;
                    }
                }
                for (int j = 0; j < k; ++j) {
                    const int32_t ej = __shfl_sync(0xffffffffu, id, j);
                    const float wj = __shfl_sync(0xffffffffu, dw, j);
#pragma unroll
                    for (int i = 0; i < PER; ++i)
                        if (ej >= 0 && expert<PER, VEC>(lane, i) == ej) d[i] += wj;
                }
            }
            const float lse = softmax_row<PER>(z);
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i) dot += z[i] * d[i];
            const float shift = cz * lse - warp_sum(dot);
#pragma unroll
            for (int i = 0; i < PER; ++i) d[i] = z[i] * (d[i] + shift);
        }
        if (MAX) {
#pragma unroll
            for (int i = 0; i < PER; ++i) largest = fmaxf(largest, fabsf(d[i]));
        } else {
            uint16_t* out = p.dz + t * p.ld;
            if (VEC) {
#pragma unroll
                for (int i = 0; i < PER; i += 4) {
                    const int e = expert<PER, VEC>(lane, i);
                    if (e < p.ld)                        // columns E .. ld - 1 are zeros
                        *reinterpret_cast<uint2*>(out + e) =
                            make_uint2(pack_16bit2<BF16>(d[i] * scale, d[i + 1] * scale),
                                       pack_16bit2<BF16>(d[i + 2] * scale, d[i + 3] * scale));
                    if (p.d_logits && e < E)
                        *reinterpret_cast<float4*>(p.d_logits + t * E + e) = make_float4(d[i], d[i + 1], d[i + 2], d[i + 3]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int e = expert<PER, VEC>(lane, i);
                    if (e < p.ld) out[e] = static_cast<uint16_t>(pack_16bit2<BF16>(d[i] * scale, 0.0f) & 0xffffu);
                    if (p.d_logits && e < E) p.d_logits[t * E + e] = d[i];
                }
            }
        }
    }
    if (MAX) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) largest = fmaxf(largest, __shfl_xor_sync(0xffffffffu, largest, d));
        if (lane == 0) smax[warp] = largest;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 0; w < WARPS; ++w) largest = fmaxf(largest, smax[w]);
            p.block_max[blockIdx.x] = largest;
        }
    }
}

int64_t round256(int64_t n) { return (n + 255) / 256 * 256; }

// Tokens of a block: about two blocks an SM, a multiple of `step`.
int32_t chunk_tokens(int64_t n_tokens, int step) {
    const int64_t blocks = 2 * 152;
    const int64_t c = (n_tokens + blocks - 1) / blocks;
    return static_cast<int32_t>((c + step - 1) / step * step);
}

template <class... Args>
cudaError_t launch_pdl(void (*kernel)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t stream, Args... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

struct BalanceLayout {
    int32_t chunk, chunks, slots, expert_blocks;
    int64_t psum, pcount, pz, pn, dots, zsum, done, bytes;
};

BalanceLayout balance_layout(int64_t n_tokens, int32_t n_experts, int32_t n_seqs) {
    BalanceLayout l;
    l.chunk = n_tokens > 0 ? chunk_tokens(n_tokens, WARPS) : WARPS;
    l.chunks = static_cast<int32_t>((n_tokens + l.chunk - 1) / l.chunk);
    if (l.chunks == 0) l.chunks = 1;
    l.slots = l.chunks + n_seqs;
    l.expert_blocks = (n_experts + 31) / 32;
    int64_t at = 0;
    auto take = [&at](int64_t n) {
        const int64_t r = at;
        at += round256(n);
        return r;
    };
    l.psum = take(int64_t{4} * l.slots * n_experts);
    l.pcount = take(int64_t{4} * l.slots * n_experts);
    l.pz = take(int64_t{4} * l.slots);
    l.pn = take(int64_t{4} * l.slots);
    l.dots = take(int64_t{8} * n_seqs * l.expert_blocks);
    l.zsum = take(int64_t{8} * n_seqs);
    l.done = take(4);
    l.bytes = at;
    return l;
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
    p.psum = reinterpret_cast<float*>(ws + l.psum);
    p.pcount = reinterpret_cast<int32_t*>(ws + l.pcount);
    p.pz = reinterpret_cast<float*>(ws + l.pz);
    p.pn = reinterpret_cast<int32_t*>(ws + l.pn);
    p.dots = reinterpret_cast<double*>(ws + l.dots);
    p.zsum = reinterpret_cast<double*>(ws + l.zsum);
    p.done = reinterpret_cast<unsigned*>(ws + l.done);
    p.losses = a.losses;
    p.counts = a.counts;
    p.seq_tokens = a.seq_tokens;
    p.status = a.status;
    const int32_t E = a.r.n_experts;
    const bool vec = E % 4 == 0;
    const size_t smem = static_cast<size_t>(HALF + 1) * E * 4;
    auto kernel = E <= 128 ? (vec ? balance_kernel<4, true> : balance_kernel<4, false>)
                : E <= 256 ? (vec ? balance_kernel<8, true> : balance_kernel<8, false>)
                           : (vec ? balance_kernel<32, true> : balance_kernel<32, false>);
    cudaError_t err = launch_pdl(kernel, dim3(static_cast<unsigned>(l.chunks)), THREADS, smem, stream, p);
    if (err != cudaSuccess) return err;
    return launch_pdl(balance_reduce_kernel, dim3(static_cast<unsigned>(l.expert_blocks), static_cast<unsigned>(a.r.n_seqs)),
                      32 * REDUCE_WARPS, 0, stream, p);
}

int router_grad_blocks(int64_t n_tokens) {
    const int32_t c = chunk_tokens(n_tokens, 64);
    return static_cast<int>((n_tokens + c - 1) / c);
}

template <bool BF16, bool MAX>
static cudaError_t launch_gradient_pass(const GradParams& p, int blocks, cudaStream_t stream) {
    const int32_t E = p.r.n_experts;
    const bool vec = E % 4 == 0;
    auto kernel = E <= 128 ? (vec ? logit_gradient_kernel<4, true, BF16, MAX> : logit_gradient_kernel<4, false, BF16, MAX>)
                : E <= 256 ? (vec ? logit_gradient_kernel<8, true, BF16, MAX> : logit_gradient_kernel<8, false, BF16, MAX>)
                           : (vec ? logit_gradient_kernel<32, true, BF16, MAX>
                                  : logit_gradient_kernel<32, false, BF16, MAX>);
    return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), THREADS, 0, stream, p);
}

cudaError_t launch_logit_gradients(const RouterBackward& a, const LogitGradients& g, cudaStream_t stream) {
    GradParams p{};
    p.r = a.r;
    p.chunk = chunk_tokens(a.r.n_tokens, 64);
    p.d_weights = a.d_topk_weights;
    p.d_losses = a.d_losses;
    p.counts = a.counts;
    p.seq_tokens = a.seq_tokens;
    p.dz = g.dz;
    p.ld = g.ld;
    p.d_logits = a.d_logits;
    p.scale = g.scale;
    p.block_max = g.block_max;
    p.valid = g.valid;
    p.status = a.status;
    const int blocks = router_grad_blocks(a.r.n_tokens);
    if (a.bf16) return launch_gradient_pass<true, false>(p, blocks, stream);
    const cudaError_t err = launch_gradient_pass<false, true>(p, blocks, stream);
    if (err != cudaSuccess) return err;
    return launch_gradient_pass<false, false>(p, blocks, stream);
}

}  // namespace moe
