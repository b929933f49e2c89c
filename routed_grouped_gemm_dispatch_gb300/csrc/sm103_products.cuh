// Inline-PTX building blocks of the feed-forward and 4-bit products, beside those
// of sm103_ptx.cuh: warp-uniform issue, M/N-major operands, block-scaled MMAs.
#pragma once

#include "sm103_ptx.cuh"

namespace moe {

// ---------------------------------------------------------------------------
// waits, arrivals, hints
// ---------------------------------------------------------------------------

// mbar_wait_bounded for a whole warp: one answer for all lanes, which the
// compiler knows to be warp-uniform.
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, abort, limit_ns)) != 0;
}

// For one thread, once every role of the CTA has stopped: waits, at most `limit_ns`
// each, until the copies of the last `stages` of `issued` ring stages have landed.
__device__ __forceinline__ void drain_copies(uint32_t bar_full, int64_t issued, int32_t stages, uint64_t limit_ns) {
    volatile int never = 0;
    const int64_t n = issued < stages ? issued : stages;
    for (int64_t i = 0; i < n; ++i) {
        const int64_t idx = issued - 1 - i;
        mbar_wait_bounded(bar_full + 8 * static_cast<uint32_t>(idx % stages), static_cast<uint32_t>((idx / stages) & 1),
                          &never, limit_ns);
    }
}

__device__ __forceinline__ void spin_ns(uint64_t ns) {
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < ns) { }
}

// True in one lane of a converged warp.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e;
}

// mbar_arrive_cluster without ordering this thread's earlier memory operations, for handing
// back TMEM that tcgen05.wait::ld has already emptied: the release form would
// first wait for the thread's global stores in flight (about 3000 cycles).
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// 1 / (1 + 2^(-x log2 e)) by two approximate instructions that flush subnormals, which
// spares the compiler's range handling around each (4-bit gate_up of 4096 tokens, top-6
// of 64: 69.2 -> 67.3 us; gradients of 2048 tokens: 109.5 -> 107.0).  The relative error is
// below 2^-21 + 2^-23.7 |x|: the rounding of x log2 e before the power is an absolute
// error of the exponent, so it grows with |x| (2^-16 at x = -87, where the result is
// next rounded to 8 or 11 bits).  Below about x = -87.3 the result, less than 2^-126, is 0.
__device__ __forceinline__ float sigmoid_approx(float x) {
    float e, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
    return s;
}

// Ask for a box's lines to be brought into L2.  A hint that moves no data to the
// SM: safe before the kernels that may still write the array have finished.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int32_t c0, int32_t c1) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1) : "memory");
}

// ---------------------------------------------------------------------------
// warp-uniform issue
// ---------------------------------------------------------------------------

// The `_if` forms of copies, MMAs and commits are executed by a converged warp and
// issued by the lane with `issue` set.  With the operands computed by the whole
// warp the compiler keeps addresses, coordinates and descriptors in uniform
// registers, where these instructions want them; computed inside a one-lane
// branch each has to be moved there first, about 90 cycles an instruction, which
// is longer than a 4-bit MMA takes and leaves a ring of copies short of work.
__device__ __forceinline__ void mbar_arrive_expect_tx_if(uint32_t issue, uint32_t bar, uint32_t bytes) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.b32 e, %2, 0;\n\t"
        "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar), "r"(bytes), "r"(issue)
        : "memory");
}

__device__ __forceinline__ void tma_load_2d_if(uint32_t issue, uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                               int32_t c0, int32_t c1, uint64_t policy) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.b32 e, %6, 0;\n\t"
        "@e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3}], [%4], %5;\n\t}"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar), "l"(policy), "r"(issue)
        : "memory");
}

__device__ __forceinline__ void tma_load_2d_pair_if(uint32_t issue, uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                                    int32_t c0, int32_t c1, uint64_t policy) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.b32 e, %6, 0;\n\t"
        "@e cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %3}], [%4], %5;\n\t}"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar), "l"(policy), "r"(issue)
        : "memory");
}

// ---------------------------------------------------------------------------
// 16-bit operands
// ---------------------------------------------------------------------------

__device__ __forceinline__ void tc_mma_f16_pair_if(uint32_t issue, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                                   uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(issue)
        : "memory");
}

__device__ __forceinline__ void tc_mma_f16_if(uint32_t issue, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(issue)
        : "memory");
}

__device__ __forceinline__ void tc_commit_pair_mc_if(uint32_t issue, uint32_t bar, uint16_t cta_mask) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.b32 e, %2, 0;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}"
        ::"r"(bar), "h"(cta_mask), "r"(issue) : "memory");
}

// Descriptor for an M/N-major operand (M or N contiguous) in 128-byte swizzled
// atoms of 64 elements (16-bit) along M/N by 8 along K, as TMA boxes 64 wide
// leave it: K rows of 128 bytes, so 1024 bytes between 8-row groups along K
// (the stride-dimension offset) and `mn_stride` bytes between 64-element
// chunks along M/N (the leading-dimension offset).  K = 16 further is 2048
// bytes further.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr, uint32_t mn_stride) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(mn_stride >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

// idesc_f16_f32acc for either 16-bit type (A and B alike) and either major-ness.
__host__ __device__ constexpr uint32_t idesc_16bit_f32acc(uint32_t m, uint32_t n, bool bf16, bool a_mn, bool b_mn) {
    return idesc_f16_f32acc(m, n) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (a_mn ? 1u << 15 : 0u) |
           (b_mn ? 1u << 16 : 0u);
}

// ---------------------------------------------------------------------------
// 4-bit operands with a scale per 32 values along K (kind::mxf4)
// ---------------------------------------------------------------------------

// Copy 32 rows of 16 bytes (512 contiguous bytes at the descriptor's address)
// into four TMEM columns of lanes 0-31, repeated in the other three lane
// quarters: the layout in which the block-scaled MMA reads the scales of 128
// rows x 4 blocks, row r in lane r % 32, column r / 32, a byte per block.  Issued
// by the even CTA of a pair; each CTA's TMEM is filled from its own shared memory.
// Executed by a converged warp; the lane with `issue` set issues it.
__device__ __forceinline__ void tc_cp_scales_pair(uint32_t issue, uint32_t taddr, uint64_t desc) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.b32 e, %2, 0;\n\t"
        "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr), "l"(desc), "r"(issue) : "memory");
}

// The same for one CTA.
__device__ __forceinline__ void tc_cp_scales(uint32_t issue, uint32_t taddr, uint64_t desc) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.b32 e, %2, 0;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr), "l"(desc), "r"(issue) : "memory");
}

// Descriptor of such a 512-byte tile: no swizzle, 8-row groups of 128 bytes.
__device__ __forceinline__ uint64_t smem_desc_scales(uint32_t saddr) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | static_cast<uint64_t>(128u >> 4) << 32 |
           static_cast<uint64_t>(1u) << 46;
}

// D[tmem] (+)= (A ⊙ scales)·(B ⊙ scales)ᵀ for one K = 64 slice of e2m1 values, on a
// CTA pair (operands as in tc_mma_f16_pair).  Each CTA's TMEM holds the scales
// of its own rows of A and of all rows of B.
__device__ __forceinline__ void tc_mma_mxf4_pair(uint32_t issue, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                                 uint32_t idesc, uint32_t a_scales, uint32_t b_scales,
                                                 uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "setp.ne.b32 e, %7, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(a_scales), "r"(b_scales), "r"(accumulate), "r"(issue)
        : "memory");
}

// The same for one CTA.
__device__ __forceinline__ void tc_mma_mxf4(uint32_t issue, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t a_scales, uint32_t b_scales, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "setp.ne.b32 e, %7, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(a_scales), "r"(b_scales), "r"(accumulate), "r"(issue)
        : "memory");
}

__device__ __forceinline__ void tc_commit_if(uint32_t issue, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.b32 e, %1, 0;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(issue)
        : "memory");
}

// Instruction descriptor of kind::mxf4, K = 64: e2m1 A and B (format 1, bits
// 7-9 and 10-11), both K-major, e8m0 scales (bit 23), N >> 3 in bits 17-22,
// M >> 4 in bits 24-28.  `half` picks the scale bytes inside each 32-bit TMEM
// word: 0 the first two blocks of 32, 1 the last two (data id 0 or 2, bits 4-5
// for B and 29-30 for A).
__host__ __device__ constexpr uint32_t idesc_mxf4(uint32_t m, uint32_t n, uint32_t half) {
    return (1u << 7) | (1u << 10) | ((n >> 3) << 17) | (1u << 23) | ((m >> 4) << 24) | ((2u * half) << 4) |
           ((2u * half) << 29);
}

}  // namespace moe
