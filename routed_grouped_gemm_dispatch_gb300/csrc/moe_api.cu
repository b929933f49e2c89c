// C ABI of the library: argument validation and dispatch to the launchers.
// Every check here runs on the host before anything is enqueued; a failed
// check returns a MOE_ERR_* code and launches nothing.
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/moe_gb300.h"
#include "ffn_internal.h"
#include "moe_internal.h"
#include "mx4_internal.h"

namespace {

constexpr int32_t ABI_VERSION = 1;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

moe_status_t check_device() {
    int dev = 0, major = 0, minor = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_DEVICE;
    // A device's architecture is asked for once.
    static std::atomic<bool> usable[64];
    const bool kept = dev >= 0 && dev < 64;
    if (kept && usable[dev].load(std::memory_order_relaxed)) return MOE_OK;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
        return MOE_ERR_DEVICE;
    // The library is compiled for sm_103a only.
    if (major != 10 || minor != 3) return MOE_ERR_DEVICE;
    if (kept) usable[dev].store(true, std::memory_order_relaxed);
    return MOE_OK;
}

moe_status_t from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return MOE_OK;
    if (e == cudaErrorNotSupported || e == cudaErrorNoDevice) return MOE_ERR_DEVICE;
    return MOE_ERR_LAUNCH;
}

}  // namespace

extern "C" {

int32_t moe_abi_version(void) { return ABI_VERSION; }

const char* moe_status_string(moe_status_t s) {
    switch (s) {
        case MOE_OK: return "MOE_OK";
        case MOE_ERR_NULL: return "MOE_ERR_NULL: a required pointer is NULL";
        case MOE_ERR_SHAPE: return "MOE_ERR_SHAPE: a size is negative, inconsistent or not the multiple asked for";
        case MOE_ERR_ALIGN: return "MOE_ERR_ALIGN: a pointer is not 16-byte aligned";
        case MOE_ERR_BLOCK: return "MOE_ERR_BLOCK: block_token must be 128";
        case MOE_ERR_DEVICE: return "MOE_ERR_DEVICE: no usable sm_103 device or driver entry point";
        case MOE_ERR_LAUNCH: return "MOE_ERR_LAUNCH: a kernel launch failed";
        case MOE_ERR_LIMIT: return "MOE_ERR_LIMIT: n_experts or num_blocks_m above the library limits";
        case MOE_ERR_WORKSPACE: return "MOE_ERR_WORKSPACE: workspace missing or too small";
        case MOE_ERR_STATIC_WORKSPACE:
            return "MOE_ERR_STATIC_WORKSPACE: total_padded_tokens * intermediate * 2 bytes exceeds the "
                   "library's fixed workspace (MOE_STATIC_WORKSPACE_BYTES)";
        default: return "unknown moe status";
    }
}

int64_t moe_num_blocks(int64_t pairs, int32_t n_experts, int32_t block_token) {
    if (pairs < 0 || n_experts < 0 || block_token <= 0) return -1;
    return (pairs + block_token - 1) / block_token + n_experts;
}

moe_status_t moe_build_dispatch(const int32_t* topk_ids, int64_t n_tokens, int32_t top_k,
                                int32_t n_experts, int32_t block_token, int32_t* group_sizes,
                                int32_t* group_offsets, int32_t* group_padded_offsets,
                                int32_t* group_idx_for_bx, int64_t num_blocks_m, int32_t* status_dev,
                                void* stream) {
    if (n_tokens < 0 || top_k <= 0) return MOE_ERR_SHAPE;
    if (block_token != MOE_BLOCK_TOKEN) return MOE_ERR_BLOCK;
    if (n_experts <= 0 || n_experts > MOE_MAX_EXPERTS) return MOE_ERR_LIMIT;
    const int64_t pairs = n_tokens * static_cast<int64_t>(top_k);
    if (num_blocks_m != moe_num_blocks(pairs, n_experts, block_token)) return MOE_ERR_SHAPE;
    if (num_blocks_m > MOE_MAX_BLOCKS) return MOE_ERR_LIMIT;
    if ((pairs > 0 && !topk_ids) || !group_sizes || !group_offsets || !group_padded_offsets ||
        !group_idx_for_bx)
        return MOE_ERR_NULL;
    if (moe_status_t s = check_device()) return s;
    return from_cuda(moe::launch_build_dispatch(topk_ids, pairs, n_experts, block_token, group_sizes,
                                                group_offsets, group_padded_offsets, group_idx_for_bx,
                                                num_blocks_m, status_dev,
                                                static_cast<cudaStream_t>(stream)));
}

int64_t moe_pack_workspace_bytes(int64_t pairs, int32_t n_experts) {
    if (pairs < 0 || n_experts <= 0) return -1;
    return moe::pack_workspace_bytes(pairs, n_experts);
}

moe_status_t moe_pack_routed(const int32_t* topk_ids, const float* topk_weights, int64_t n_tokens, int32_t top_k,
                             int32_t n_experts, const uint16_t* x_tokens, int32_t hidden,
                             const int32_t* group_offsets, const int32_t* group_padded_offsets,
                             int64_t total_padded_tokens, uint16_t* stacked_expert_tokens,
                             float* routed_expert_weights, int32_t* pair_padded_rows, void* workspace,
                             size_t workspace_bytes, int32_t* status_dev, void* stream) {
    if (n_tokens < 0 || top_k <= 0 || hidden <= 0 || hidden % 128 != 0 || total_padded_tokens < 0)
        return MOE_ERR_SHAPE;
    if (n_experts <= 0 || n_experts > MOE_MAX_EXPERTS) return MOE_ERR_LIMIT;
    const int64_t pairs = n_tokens * static_cast<int64_t>(top_k);
    if (pairs == 0) return MOE_OK;
    if (!topk_ids || !group_offsets || !group_padded_offsets || !pair_padded_rows) return MOE_ERR_NULL;
    if (stacked_expert_tokens && !x_tokens) return MOE_ERR_NULL;
    if (routed_expert_weights && !topk_weights) return MOE_ERR_NULL;
    if ((stacked_expert_tokens && (!aligned16(stacked_expert_tokens) || !aligned16(x_tokens))))
        return MOE_ERR_ALIGN;
    if (!workspace || static_cast<int64_t>(workspace_bytes) < moe::pack_workspace_bytes(pairs, n_experts))
        return MOE_ERR_WORKSPACE;
    if (moe_status_t s = check_device()) return s;
    return from_cuda(moe::launch_pack(topk_ids, topk_weights, n_tokens, top_k, n_experts, x_tokens, hidden,
                                      group_offsets, group_padded_offsets, total_padded_tokens, pairs,
                                      stacked_expert_tokens, routed_expert_weights, pair_padded_rows, workspace,
                                      status_dev, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_combine_routed(const uint16_t* out, int64_t total_padded_tokens, int32_t hidden,
                                const int32_t* pair_padded_rows, int64_t n_tokens, int32_t top_k, uint16_t* y,
                                void* stream) {
    if (n_tokens < 0 || top_k <= 0 || hidden <= 0 || hidden % 128 != 0 || total_padded_tokens < 0)
        return MOE_ERR_SHAPE;
    if (n_tokens == 0) return MOE_OK;
    if (!out || !pair_padded_rows || !y) return MOE_ERR_NULL;
    if (!aligned16(out) || !aligned16(y)) return MOE_ERR_ALIGN;
    if (moe_status_t s = check_device()) return s;
    return from_cuda(moe::launch_combine(out, total_padded_tokens, hidden, pair_padded_rows, n_tokens, top_k, y,
                                         static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_router_topk(const uint16_t* x_tokens, int64_t n_tokens, int32_t hidden,
                             const uint16_t* router_w, int32_t n_experts, int32_t top_k, int32_t* topk_ids,
                             float* topk_weights, int32_t* status_dev, void* stream) {
    if (n_tokens < 0 || hidden <= 0 || hidden % 128 != 0) return MOE_ERR_SHAPE;
    if (n_experts <= 0 || n_experts > MOE_ROUTER_MAX_EXPERTS) return MOE_ERR_LIMIT;
    if (top_k <= 0 || top_k > n_experts || top_k > MOE_ROUTER_MAX_TOPK) return MOE_ERR_LIMIT;
    if (n_tokens == 0) return MOE_OK;
    if (!x_tokens || !router_w || !topk_ids || !topk_weights) return MOE_ERR_NULL;
    if (!aligned16(x_tokens) || !aligned16(router_w)) return MOE_ERR_ALIGN;
    if (moe_status_t s = check_device()) return s;
    return from_cuda(moe::launch_router(x_tokens, n_tokens, hidden, router_w, n_experts, top_k, topk_ids,
                                        topk_weights, status_dev, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace moe {

int32_t check_forward_args(const ForwardArgs& a, bool check_up_logits) {
    if (!a.x || !a.gate_w || !a.up_w || !a.down_w || (a.valid_total > 0 && !a.rw) || !a.sizes || !a.offsets ||
        !a.padded || !a.gidx || (check_up_logits && !a.up_logits) || !a.out)
        return MOE_ERR_NULL;
    if (a.hidden <= 0 || a.intermediate <= 0 || a.hidden % 128 != 0 || a.intermediate % 128 != 0)
        return MOE_ERR_SHAPE;
    if (a.rows_total < 0 || a.valid_total < 0 || a.num_blocks_m < 0) return MOE_ERR_SHAPE;
    if (a.n_experts <= 0 || a.n_experts > MOE_MAX_EXPERTS) return MOE_ERR_LIMIT;
    if (a.num_blocks_m > MOE_MAX_BLOCKS) return MOE_ERR_LIMIT;
    if (a.rows_total < a.num_blocks_m * MOE_BLOCK_TOKEN) return MOE_ERR_SHAPE;
    if (!aligned16(a.x) || !aligned16(a.gate_w) || !aligned16(a.up_w) || !aligned16(a.down_w) ||
        (check_up_logits && !aligned16(a.up_logits)) || !aligned16(a.out))
        return MOE_ERR_ALIGN;
    return MOE_OK;
}

}  // namespace moe

namespace {

moe_status_t forward_impl(const uint16_t* stacked_expert_tokens, int64_t total_padded_tokens, int32_t hidden,
                          const uint16_t* gate_w, const uint16_t* up_w, const uint16_t* down_w, int32_t n_experts,
                          int32_t intermediate, const float* routed_expert_weights, int64_t total_valid_tokens,
                          const int32_t* group_sizes, const int32_t* group_offsets,
                          const int32_t* group_padded_offsets, const int32_t* group_idx_for_bx,
                          int64_t num_blocks_m, uint16_t* up_logits, uint16_t* out, int32_t* status_dev,
                          void* stream, uint32_t flags, void* ready_ws) {
    const uint32_t phases = flags & (MOE_RUN_PHASE1 | MOE_RUN_PHASE2);
    if (phases == 0 || (flags & ~(MOE_RUN_PHASE1 | MOE_RUN_PHASE2 | MOE_NO_PDL | MOE_TEST_DROP_SIGNAL)) != 0)
        return MOE_ERR_SHAPE;
    moe::ForwardArgs a{};
    a.x = stacked_expert_tokens;
    a.rows_total = total_padded_tokens;
    a.hidden = hidden;
    a.gate_w = gate_w;
    a.up_w = up_w;
    a.down_w = down_w;
    a.n_experts = n_experts;
    a.intermediate = intermediate;
    a.rw = routed_expert_weights;
    a.valid_total = total_valid_tokens;
    a.sizes = group_sizes;
    a.offsets = group_offsets;
    a.padded = group_padded_offsets;
    a.gidx = group_idx_for_bx;
    a.num_blocks_m = num_blocks_m;
    a.up_logits = up_logits;
    a.out = out;
    a.status = status_dev;
    if (moe_status_t s = moe::check_forward_args(a, true)) return s;
    if (moe_status_t s = check_device()) return s;
    if (num_blocks_m == 0) return MOE_OK;
    return from_cuda(moe::launch_fused_forward(a, flags, static_cast<cudaStream_t>(stream), ready_ws));
}

}  // namespace

extern "C" {

moe_status_t moe_fused_forward_ex(const uint16_t* stacked_expert_tokens, int64_t total_padded_tokens,
                                  int32_t hidden, const uint16_t* gate_w, const uint16_t* up_w,
                                  const uint16_t* down_w, int32_t n_experts, int32_t intermediate,
                                  const float* routed_expert_weights, int64_t total_valid_tokens,
                                  const int32_t* group_sizes, const int32_t* group_offsets,
                                  const int32_t* group_padded_offsets, const int32_t* group_idx_for_bx,
                                  int64_t num_blocks_m, uint16_t* up_logits, uint16_t* out,
                                  int32_t* status_dev, void* stream, uint32_t flags) {
    return forward_impl(stacked_expert_tokens, total_padded_tokens, hidden, gate_w, up_w, down_w, n_experts,
                        intermediate, routed_expert_weights, total_valid_tokens, group_sizes, group_offsets,
                        group_padded_offsets, group_idx_for_bx, num_blocks_m, up_logits, out, status_dev, stream,
                        flags, nullptr);
}

int64_t moe_single_launch_workspace_bytes(int64_t num_blocks_m) {
    if (num_blocks_m < 0) return -1;
    return moe::single_launch_workspace_bytes(num_blocks_m);
}

moe_status_t moe_fused_forward_single_launch(
    const uint16_t* stacked_expert_tokens, int64_t total_padded_tokens, int32_t hidden, const uint16_t* gate_w,
    const uint16_t* up_w, const uint16_t* down_w, int32_t n_experts, int32_t intermediate,
    const float* routed_expert_weights, int64_t total_valid_tokens, const int32_t* group_sizes,
    const int32_t* group_offsets, const int32_t* group_padded_offsets, const int32_t* group_idx_for_bx,
    int64_t num_blocks_m, uint16_t* up_logits, uint16_t* out, void* workspace, size_t workspace_bytes,
    int32_t* status_dev, void* stream) {
    if (num_blocks_m < 0) return MOE_ERR_SHAPE;
    if (!workspace || static_cast<int64_t>(workspace_bytes) < moe::single_launch_workspace_bytes(num_blocks_m))
        return MOE_ERR_WORKSPACE;
    return forward_impl(stacked_expert_tokens, total_padded_tokens, hidden, gate_w, up_w, down_w, n_experts,
                        intermediate, routed_expert_weights, total_valid_tokens, group_sizes, group_offsets,
                        group_padded_offsets, group_idx_for_bx, num_blocks_m, up_logits, out, status_dev, stream,
                        MOE_RUN_PHASE1 | MOE_RUN_PHASE2, workspace);
}

moe_status_t moe_fused_forward(const uint16_t* stacked_expert_tokens, int64_t total_padded_tokens,
                               int32_t hidden, const uint16_t* gate_w, const uint16_t* up_w,
                               const uint16_t* down_w, int32_t n_experts, int32_t intermediate,
                               const float* routed_expert_weights, int64_t total_valid_tokens,
                               const int32_t* group_sizes, const int32_t* group_offsets,
                               const int32_t* group_padded_offsets, const int32_t* group_idx_for_bx,
                               int64_t num_blocks_m, uint16_t* up_logits, uint16_t* out,
                               int32_t* status_dev, void* stream) {
    return moe_fused_forward_ex(stacked_expert_tokens, total_padded_tokens, hidden, gate_w, up_w, down_w,
                                n_experts, intermediate, routed_expert_weights, total_valid_tokens,
                                group_sizes, group_offsets, group_padded_offsets, group_idx_for_bx,
                                num_blocks_m, up_logits, out, status_dev, stream,
                                MOE_RUN_PHASE1 | MOE_RUN_PHASE2);
}

}  // extern "C"

// ---------------------------------------------------------------------------
// dense gated feed-forward block
// ---------------------------------------------------------------------------

namespace {

moe_status_t check_ffn_sizes(int32_t dtype, int64_t n_tokens, int32_t hidden, int32_t intermediate) {
    if (dtype != MOE_DTYPE_F16 && dtype != MOE_DTYPE_BF16) return MOE_ERR_SHAPE;
    if (n_tokens < 0 || hidden <= 0 || intermediate <= 0 || hidden % 8 != 0 || intermediate % 8 != 0)
        return MOE_ERR_SHAPE;
    if (n_tokens > MOE_FFN_MAX_TOKENS || hidden > MOE_FFN_MAX_WIDTH || intermediate > MOE_FFN_MAX_WIDTH)
        return MOE_ERR_LIMIT;
    return MOE_OK;
}

// Bytes of one [n_tokens, intermediate] array of the backward's workspace.
int64_t ffn_grad_bytes(int64_t n_tokens, int32_t intermediate) {
    return (n_tokens * intermediate * 2 + 255) / 256 * 256;
}

}  // namespace

extern "C" {

moe_status_t moe_ffn_forward(int32_t dtype, const uint16_t* x, int64_t n_tokens, int32_t hidden,
                             const uint16_t* gate_w, const uint16_t* up_w, const uint16_t* down_w,
                             int32_t intermediate, uint16_t* gate, uint16_t* up, uint16_t* up_logits, uint16_t* out,
                             int32_t* status_dev, void* stream) {
    if (moe_status_t s = check_ffn_sizes(dtype, n_tokens, hidden, intermediate)) return s;
    if (n_tokens == 0) return MOE_OK;
    if (!x || !gate_w || !up_w || !down_w || !up_logits || !out || !gate != !up) return MOE_ERR_NULL;
    if (!aligned16(x) || !aligned16(gate_w) || !aligned16(up_w) || !aligned16(down_w) || !aligned16(gate) ||
        !aligned16(up) || !aligned16(up_logits) || !aligned16(out))
        return MOE_ERR_ALIGN;
    if (moe_status_t s = check_device()) return s;
    moe::FfnForward a{};
    a.bf16 = dtype == MOE_DTYPE_BF16;
    a.x = x;
    a.n_tokens = n_tokens;
    a.hidden = hidden;
    a.gate_w = gate_w;
    a.up_w = up_w;
    a.down_w = down_w;
    a.intermediate = intermediate;
    a.gate = gate;
    a.up = up;
    a.up_logits = up_logits;
    a.out = out;
    a.status = status_dev;
    return from_cuda(moe::launch_ffn_forward(a, static_cast<cudaStream_t>(stream)));
}

int64_t moe_ffn_backward_workspace_bytes(int64_t n_tokens, int32_t intermediate) {
    if (n_tokens < 0 || intermediate < 0) return -1;
    return 2 * ffn_grad_bytes(n_tokens, intermediate);
}

moe_status_t moe_ffn_backward(int32_t dtype, const uint16_t* d_out, const uint16_t* x, int64_t n_tokens,
                              int32_t hidden, const uint16_t* gate_w, const uint16_t* up_w, const uint16_t* down_w,
                              int32_t intermediate, const uint16_t* gate, const uint16_t* up,
                              const uint16_t* up_logits, void* workspace, size_t workspace_bytes, uint16_t* d_x,
                              uint16_t* d_gate_w, uint16_t* d_up_w, uint16_t* d_down_w, int32_t* status_dev,
                              void* stream) {
    if (moe_status_t s = check_ffn_sizes(dtype, n_tokens, hidden, intermediate)) return s;
    if (!d_gate_w || !d_up_w || !d_down_w) return MOE_ERR_NULL;
    if (!aligned16(d_gate_w) || !aligned16(d_up_w) || !aligned16(d_down_w)) return MOE_ERR_ALIGN;
    if (n_tokens == 0) {
        // a sum over no tokens
        if (moe_status_t s = check_device()) return s;
        const size_t bytes = static_cast<size_t>(hidden) * static_cast<size_t>(intermediate) * 2;
        for (uint16_t* d : {d_gate_w, d_up_w, d_down_w})
            if (cudaMemsetAsync(d, 0, bytes, static_cast<cudaStream_t>(stream)) != cudaSuccess) return MOE_ERR_LAUNCH;
        return MOE_OK;
    }
    if (!d_out || !x || !gate_w || !up_w || !down_w || !gate || !up || !up_logits || !d_x) return MOE_ERR_NULL;
    if (!aligned16(d_out) || !aligned16(x) || !aligned16(gate_w) || !aligned16(up_w) || !aligned16(down_w) ||
        !aligned16(gate) || !aligned16(up) || !aligned16(up_logits) || !aligned16(d_x) || !aligned16(workspace))
        return MOE_ERR_ALIGN;
    if (!workspace || static_cast<int64_t>(workspace_bytes) < moe_ffn_backward_workspace_bytes(n_tokens, intermediate))
        return MOE_ERR_WORKSPACE;
    if (moe_status_t s = check_device()) return s;
    moe::FfnBackward a{};
    a.bf16 = dtype == MOE_DTYPE_BF16;
    a.d_out = d_out;
    a.x = x;
    a.n_tokens = n_tokens;
    a.hidden = hidden;
    a.gate_w = gate_w;
    a.up_w = up_w;
    a.down_w = down_w;
    a.intermediate = intermediate;
    a.gate = gate;
    a.up = up;
    a.up_logits = up_logits;
    a.d_gate = static_cast<uint16_t*>(workspace);
    a.d_up = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(workspace) + ffn_grad_bytes(n_tokens, intermediate));
    a.d_x = d_x;
    a.d_gate_w = d_gate_w;
    a.d_up_w = d_up_w;
    a.d_down_w = d_down_w;
    a.status = status_dev;
    return from_cuda(moe::launch_ffn_backward(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

// ---------------------------------------------------------------------------
// 4-bit microscaled values
// ---------------------------------------------------------------------------

namespace {

moe_status_t check_mx4_array(int64_t rows, int32_t cols) {
    if (rows < 0 || cols <= 0 || cols % 128 != 0) return MOE_ERR_SHAPE;
    if (rows > MOE_MX4_MAX_ROWS || cols > MOE_MX4_MAX_COLS) return MOE_ERR_LIMIT;
    return MOE_OK;
}

moe_status_t check_16bit(int32_t dtype) {
    return dtype == MOE_DTYPE_F16 || dtype == MOE_DTYPE_BF16 ? MOE_OK : MOE_ERR_SHAPE;
}

// Sizes, limits, pointers and alignment of a product, in that order.
moe_status_t check_mx4_product(const moe::Mx4Product& a, bool grouped) {
    if (moe_status_t s = check_mx4_array(a.rows, a.k)) return s;
    if (a.n <= 0 || a.n % 128 != 0 || a.num_blocks < 0 || a.valid_total < 0) return MOE_ERR_SHAPE;
    if (a.n_experts <= 0 || a.n_experts > MOE_MAX_EXPERTS || a.n > MOE_MX4_MAX_COLS ||
        static_cast<int64_t>(a.n_experts) * a.n > MOE_MX4_MAX_ROWS || a.num_blocks > MOE_MAX_BLOCKS)
        return MOE_ERR_LIMIT;
    if (grouped && a.rows < a.num_blocks * MOE_BLOCK_TOKEN) return MOE_ERR_SHAPE;
    if (a.num_blocks == 0) return MOE_OK;
    const bool gate_up = a.form == moe::MX4_GATE_UP;
    if (!a.a || !a.a_scales || !a.b || !a.b_scales || (gate_up && (!a.b2 || !a.b2_scales)) || !a.out)
        return MOE_ERR_NULL;
    if (grouped && (!a.sizes || !a.padded || !a.gidx)) return MOE_ERR_NULL;
    if (a.form == moe::MX4_DOWN && (!a.offsets || (a.valid_total > 0 && !a.weights))) return MOE_ERR_NULL;
    if (!aligned16(a.a) || !aligned16(a.a_scales) || !aligned16(a.b) || !aligned16(a.b_scales) ||
        !aligned16(a.b2) || !aligned16(a.b2_scales) || !aligned16(a.out))
        return MOE_ERR_ALIGN;
    return check_device();
}

moe_status_t run_mx4_product(const moe::Mx4Product& a, bool grouped, void* stream) {
    if (moe_status_t s = check_mx4_product(a, grouped)) return s;
    if (a.num_blocks == 0) return MOE_OK;
    return from_cuda(moe::launch_mx4_product(a, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int64_t moe_mx4_scale_bytes(int64_t rows, int32_t cols) {
    if (check_mx4_array(rows, cols) != MOE_OK) return -1;
    return (rows + 127) / 128 * (cols / 128) * 512;
}

moe_status_t moe_mx4_quantize(int32_t dtype, const void* x, int64_t n_src_rows, int32_t cols, const int32_t* src_rows,
                              int64_t n_rows, const int32_t* dest_rows, int32_t copies, int64_t n_dest_rows,
                              uint8_t* codes, uint8_t* scales, int32_t* status_dev, void* stream) {
    if (dtype != MOE_DTYPE_F32)
        if (moe_status_t s = check_16bit(dtype)) return s;
    if (copies < 1 || n_rows < 0 || (!src_rows && n_rows != n_src_rows) ||
        (!dest_rows && (copies != 1 || n_dest_rows != n_rows)))
        return MOE_ERR_SHAPE;
    if (moe_status_t s = check_mx4_array(n_src_rows, cols)) return s;
    if (moe_status_t s = check_mx4_array(n_dest_rows, cols)) return s;
    if (n_rows > MOE_MX4_MAX_ROWS) return MOE_ERR_LIMIT;
    if (n_rows == 0) return MOE_OK;
    if (!x || !codes || !scales) return MOE_ERR_NULL;
    if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return MOE_ERR_ALIGN;
    if (moe_status_t s = check_device()) return s;
    moe::Mx4Quantize a{};
    a.dtype = dtype;
    a.x = x;
    a.n_src = n_src_rows;
    a.n_rows = n_rows;
    a.cols = cols;
    a.src_rows = src_rows;
    a.dest_rows = dest_rows;
    a.copies = copies;
    a.n_dest = n_dest_rows;
    a.codes = codes;
    a.scales = scales;
    a.status = status_dev;
    return from_cuda(moe::launch_mx4_quantize(a, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t cols, int32_t dtype,
                                void* out, void* stream) {
    if (dtype != MOE_DTYPE_F32)
        if (moe_status_t s = check_16bit(dtype)) return s;
    if (moe_status_t s = check_mx4_array(rows, cols)) return s;
    if (rows == 0) return MOE_OK;
    if (!codes || !scales || !out) return MOE_ERR_NULL;
    if (!aligned16(codes) || !aligned16(scales) || !aligned16(out)) return MOE_ERR_ALIGN;
    if (moe_status_t s = check_device()) return s;
    return from_cuda(
        moe::launch_mx4_dequantize(codes, scales, rows, cols, dtype, out, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_mx4_matmul(const uint8_t* a, const uint8_t* a_scales, int64_t rows, int32_t k, const uint8_t* b,
                            const uint8_t* b_scales, int32_t n, int32_t dtype, uint16_t* out, int32_t* status_dev,
                            void* stream) {
    if (moe_status_t s = check_16bit(dtype)) return s;
    moe::Mx4Product m{};
    m.form = moe::MX4_MATMUL;
    m.bf16 = dtype == MOE_DTYPE_BF16;
    m.a = a;
    m.a_scales = a_scales;
    m.rows = rows;
    m.k = k;
    m.b = b;
    m.b_scales = b_scales;
    m.n_experts = 1;
    m.n = n;
    m.num_blocks = rows < 0 ? 0 : (rows + MOE_BLOCK_TOKEN - 1) / MOE_BLOCK_TOKEN;
    m.out = out;
    m.status = status_dev;
    return run_mx4_product(m, false, stream);
}

moe_status_t moe_mx4_gate_up(const uint8_t* x, const uint8_t* x_scales, int64_t total_padded_tokens, int32_t hidden,
                             const uint8_t* gate, const uint8_t* gate_scales, const uint8_t* up,
                             const uint8_t* up_scales, int32_t n_experts, int32_t intermediate,
                             const int32_t* group_sizes, const int32_t* group_padded_offsets,
                             const int32_t* group_idx_for_bx, int64_t num_blocks_m, int32_t dtype,
                             uint16_t* up_logits, int32_t* status_dev, void* stream) {
    if (moe_status_t s = check_16bit(dtype)) return s;
    moe::Mx4Product m{};
    m.form = moe::MX4_GATE_UP;
    m.bf16 = dtype == MOE_DTYPE_BF16;
    m.a = x;
    m.a_scales = x_scales;
    m.rows = total_padded_tokens;
    m.k = hidden;
    m.b = gate;
    m.b_scales = gate_scales;
    m.b2 = up;
    m.b2_scales = up_scales;
    m.n_experts = n_experts;
    m.n = intermediate;
    m.sizes = group_sizes;
    m.padded = group_padded_offsets;
    m.gidx = group_idx_for_bx;
    m.num_blocks = num_blocks_m;
    m.out = up_logits;
    m.status = status_dev;
    return run_mx4_product(m, true, stream);
}

moe_status_t moe_mx4_down(const uint8_t* h, const uint8_t* h_scales, int64_t total_padded_tokens, int32_t intermediate,
                          const uint8_t* down, const uint8_t* down_scales, int32_t n_experts, int32_t hidden,
                          const float* routed_expert_weights, int64_t total_valid_tokens, const int32_t* group_sizes,
                          const int32_t* group_offsets, const int32_t* group_padded_offsets,
                          const int32_t* group_idx_for_bx, int64_t num_blocks_m, int32_t dtype, uint16_t* out,
                          int32_t* status_dev, void* stream) {
    if (moe_status_t s = check_16bit(dtype)) return s;
    moe::Mx4Product m{};
    m.form = moe::MX4_DOWN;
    m.bf16 = dtype == MOE_DTYPE_BF16;
    m.a = h;
    m.a_scales = h_scales;
    m.rows = total_padded_tokens;
    m.k = intermediate;
    m.b = down;
    m.b_scales = down_scales;
    m.n_experts = n_experts;
    m.n = hidden;
    m.weights = routed_expert_weights;
    m.valid_total = total_valid_tokens;
    m.sizes = group_sizes;
    m.offsets = group_offsets;
    m.padded = group_padded_offsets;
    m.gidx = group_idx_for_bx;
    m.num_blocks = num_blocks_m;
    m.out = out;
    m.status = status_dev;
    return run_mx4_product(m, true, stream);
}

}  // extern "C"
