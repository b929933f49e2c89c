// Operators that train a routed layer: arguments of their launchers (host side).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace moe {

// What the router's loss and its gradients know of the tokens.
struct Routing {
    const float* logits;          // [n_tokens, n_experts]
    const int32_t* topk_ids;      // [n_tokens, top_k]
    int64_t n_tokens;
    int32_t n_experts;
    int32_t top_k;
    const uint8_t* token_mask;    // [n_tokens], nullable
    const int32_t* seq_offsets;   // [n_seqs + 1], nullable with n_seqs = 1
    int32_t n_seqs;
};

struct RouterBalance {
    Routing r;
    float* losses;                // [2]
    int32_t* counts;              // [n_seqs, n_experts]
    int32_t* seq_tokens;          // [n_seqs + 1]
    void* workspace;
    int32_t* status;
};

struct RouterBackward {
    Routing r;
    bool bf16;
    const uint16_t* x;            // [n_tokens, hidden]
    int32_t hidden;
    const uint16_t* router_w;     // [n_experts, hidden]
    const float* d_topk_weights;  // [n_tokens, top_k], nullable
    const float* d_losses;        // [2], nullable
    const int32_t* counts;        // [n_seqs, n_experts], with d_losses
    const int32_t* seq_tokens;    // [n_seqs + 1], with d_losses
    uint16_t* d_x;                // [n_tokens, hidden]
    uint16_t* d_router_w;         // [n_experts, hidden]
    float* d_logits;              // [n_tokens, n_experts], nullable
    void* workspace;
    int32_t* status;
};

int64_t router_balance_workspace_bytes(int64_t n_tokens, int32_t n_experts, int32_t n_seqs);
int64_t router_backward_workspace_bytes(int64_t n_tokens, int32_t n_experts, int32_t hidden);

// Arguments already validated.
cudaError_t launch_router_balance(const RouterBalance& a, cudaStream_t stream);
cudaError_t launch_router_backward(const RouterBackward& a, cudaStream_t stream);

// Gradients of the logits (router_loss.cu) as an operand of the products: 16-bit
// [n_tokens, ld], times the power of two in scale[0] (its inverse in scale[1]).  Where some tokens may not
// count, a bit per token in `valid` (1: it counts), whole 64-token steps, zero past the end, and per
// block whether x holds an infinity or a NaN in one that does not; otherwise both are null.
struct LogitGradients {
    uint16_t* dz;                 // [n_tokens, ld], and with `two` the same again of what its rounding left
    int32_t ld;
    bool two;
    float* d_logits;              // [n_tokens, n_experts], fp16 only: d_z where the caller keeps none
    float* scale;                 // [2]
    float* block_max;             // [router_grad_blocks()]
    uint32_t* valid;
    int32_t* block_dirty;         // [router_grad_blocks()]
};
int router_grad_blocks(int64_t n_tokens);
cudaError_t launch_logit_gradients(const RouterBackward& a, const LogitGradients& g, cudaStream_t stream);

struct Orthogonalize {
    int32_t dtype;                // of update: MOE_DTYPE_*
    const void* update;           // [batch, rows, cols]
    int64_t batch;
    int32_t rows, cols;
    int32_t steps;
    float a, b, c;
    float least_norm;             // what a norm is taken as at least: eps, or ORTHO_LEAST_VALUE in every entry
    uint16_t* out;                // [batch, rows, cols], bf16
    void* workspace;
    int32_t* status;
};

constexpr float ORTHO_MAX_SHIFT = 1024.0f;         // |b / 2c|, where c is not 0
// 2^-69: squares of smaller values have fewer than 11 bits in fp32 (its steps are 2^-149), and a norm of theirs
// means nothing; one that is too small would let X₀ overflow.
constexpr float ORTHO_LEAST_VALUE = 1.6940658945086007e-21f;
int64_t orthogonalize_workspace_bytes(int64_t batch, int32_t rows, int32_t cols);
// Matrices of at most 128 rows or columns, by a cluster each; cudaErrorNotSupported where the device
// cannot place one.
bool orthogonalize_is_small(int32_t rows, int32_t cols);
cudaError_t launch_orthogonalize_small(const Orthogonalize& a, cudaStream_t stream);
cudaError_t launch_orthogonalize(const Orthogonalize& a, cudaStream_t stream);

}  // namespace moe
