// Dense gated feed-forward block: arguments of its launchers (host side).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace moe {

struct FfnForward {
    bool bf16;
    const uint16_t* x;          // [n_tokens, hidden]
    int64_t n_tokens;
    int32_t hidden;
    const uint16_t* gate_w;     // [intermediate, hidden]
    const uint16_t* up_w;
    const uint16_t* down_w;     // [hidden, intermediate]
    int32_t intermediate;
    uint16_t* gate;             // [n_tokens, intermediate], both or neither
    uint16_t* up;
    uint16_t* up_logits;        // [n_tokens, intermediate]
    uint16_t* out;              // [n_tokens, hidden]
    int32_t* status;
};

struct FfnBackward {
    bool bf16;
    const uint16_t* d_out;      // [n_tokens, hidden]
    const uint16_t* x;
    int64_t n_tokens;
    int32_t hidden;
    const uint16_t* gate_w;
    const uint16_t* up_w;
    const uint16_t* down_w;
    int32_t intermediate;
    const uint16_t* gate;       // stored by the forward
    const uint16_t* up;
    const uint16_t* up_logits;
    uint16_t* d_gate;           // workspace [n_tokens, intermediate]
    uint16_t* d_up;
    uint16_t* d_x;              // [n_tokens, hidden]
    uint16_t* d_gate_w;         // [intermediate, hidden]
    uint16_t* d_up_w;
    uint16_t* d_down_w;         // [hidden, intermediate]
    int32_t* status;
};

// Arguments already validated, n_tokens > 0.
cudaError_t launch_ffn_forward(const FfnForward& a, cudaStream_t stream);
// The forward for at most FFN_SMALL_TOKENS tokens, by weight rows instead of token
// tiles: 128 tokens of 7168 / 2048 take 31 us, 129 on the tiles 39.5 us; beyond, a
// second tile of tokens was slower than they were (512 tokens 64 against 50 us).
constexpr int64_t FFN_SMALL_TOKENS = 128;
cudaError_t launch_ffn_forward_small(const FfnForward& a, cudaStream_t stream);
cudaError_t launch_ffn_backward(const FfnBackward& a, cudaStream_t stream);

}  // namespace moe
