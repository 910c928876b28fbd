// ep_router_launch.h -- launch interfaces of the router kernels (ep_router.cu),
// called by the C-ABI layer (ep_api.cu), which has checked the arguments.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "ep_router.h"

namespace ep {

constexpr int kRouterMaxExperts = 1024; // 32 logits a lane
constexpr int kRouterMaxTopk = 32;      // one slot a lane
constexpr int kRouterMaxGroups = 32;
constexpr int kRouterMaxTokens = 1 << 30; // a token past the last, and a chunk more, is still an int

struct RouterTopkLaunch {
    ep_router_desc_t r;
    const void* logits;
    const float* bias;
    const uint8_t* token_mask;
    int64_t* topk_idx;
    float* topk_weights;
};
cudaError_t launch_router_topk(const RouterTopkLaunch& a, cudaStream_t stream);

struct BalanceLaunch {
    ep_router_desc_t r;
    const void* logits;
    const int64_t* topk_idx;
    const uint8_t* token_mask;
    const int32_t* seq_offsets; // nullptr: one sequence of all tokens
    int32_t num_seqs;
    float* losses;
    int32_t* counts;
    int32_t* seq_tokens;
    float* mean_scores; // or nullptr
    void* workspace;
};
size_t balance_workspace_bytes(int64_t T, int64_t E, int64_t S);
cudaError_t launch_balance_loss(const BalanceLaunch& a, cudaStream_t stream);

struct RouterBackwardLaunch {
    ep_router_desc_t r;
    const void* logits;
    const int64_t* topk_idx;
    const uint8_t* token_mask;
    const float* d_topk_weights; // or nullptr
    const int32_t* seq_offsets;  // nullptr: one sequence of all tokens
    int32_t num_seqs;
    const int32_t* counts;
    const int32_t* seq_tokens;
    const float* d_losses; // or nullptr
    void* d_logits;
};
cudaError_t launch_router_backward(const RouterBackwardLaunch& a, cudaStream_t stream);

} // namespace ep
