// ep_lora_launch.h -- launch interfaces of the low-rank adapter kernels
// (ep_lora.cu), called by the C-ABI layer, which has checked the arguments.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "ep_internal.h"
#include "ep_lora.h"

namespace ep {

constexpr int kLoraMaxRank = 128;
constexpr int kLoraMaxAdapters = 1024;
constexpr int64_t kLoraMaxRows = (int64_t{1} << 31) - 1024; // a row a few tiles past the last is still an int

// The rows of every adapter, and where a row's data is.
struct LoraRows {
    const int32_t* offsets; // COMPACT: [E + 1]
    const int32_t* counts;  // PADDED: [E]
    int32_t mode, max_tokens, E;
    int32_t num_rows;
    int32_t pairs;            // T * K: no routing fills more rows
    const int32_t* row_token; // [num_rows], or nullptr: row i is at row i
    int32_t T;                // with row_token: rows of x, base and out
    uint32_t* err;
};

struct RowTokensLaunch {
    TcRows rows;
    int32_t T;
    int32_t* row_token;
    uint32_t* err;
};
cudaError_t launch_row_tokens(const RowTokensLaunch& a, cudaStream_t stream);

// u[row, j] = scales[e] * sum over k of x[row, k] * w_e(j, k); w_e is [rank, K]
// (transposed 0) or [K, rank] (1).
struct LoraShrinkLaunch {
    LoraRows rows;
    const void* x;
    const void* w;
    const float* scales; // or nullptr
    int32_t K, rank, transposed;
    float* u;
    int32_t trigger_dependents; // the kernel launched next is one of the same call
};
cudaError_t launch_lora_shrink(const LoraShrinkLaunch& a, cudaStream_t stream);

// out[row, n] = base[row, n] + sum over j of u[row, j] * w_e(n, j); w_e is
// [N, rank] (transposed 0) or [rank, N] (1).
struct LoraExpandLaunch {
    LoraRows rows;
    const float* u;
    const void* w;
    const void* base; // or nullptr
    void* out;
    int32_t N, rank, transposed;
    const int32_t* slot; // [T]: copy base to out for tokens with slot -1; or nullptr
    // 0: the kernel before may have written anything; 1: it is the one that
    // writes u; 2: u was complete before that one let its dependents start
    int32_t after_u;
};
cudaError_t launch_lora_expand(const LoraExpandLaunch& a, cudaStream_t stream);

// Both products of a forward call in one kernel, for few rows an adapter
// (lora_few): u as LoraShrinkLaunch gives it with w = a [rank, K], out as
// LoraExpandLaunch does with w = b [N, rank].
struct LoraFewLaunch {
    LoraRows rows;
    const void* x;
    const void* a;
    const void* b;
    const float* scales; // or nullptr
    const void* base;    // or nullptr
    void* out;
    float* u;
    int32_t K, N, rank;
    const int32_t* slot; // as for LoraExpandLaunch
};
bool lora_few(const LoraRows& rows, int rank);
cudaError_t launch_lora_few(const LoraFewLaunch& a, cudaStream_t stream);

// da[e][j, n] = sum over e's rows of dh[row, j] * x[row, n]  and
// db[e][n, j] = sum over e's rows of dy[row, n] * h[row, j]
struct LoraOuterLaunch {
    LoraRows rows;
    const void* x;
    const float* dh;
    void* da;
    const void* dy;
    const float* h;
    void* db;
    int32_t hidden_in, hidden_out, rank;
    int32_t trigger_dependents; // as for LoraShrinkLaunch
};
cudaError_t launch_lora_outer(const LoraOuterLaunch& a, cudaStream_t stream);

} // namespace ep
