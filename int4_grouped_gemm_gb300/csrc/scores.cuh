// Log probabilities, entropy and top alternatives of an output head's scores:
// arguments and launch entry.
#pragma once

#include "common.cuh"
#include "layout.cuh"

namespace moe {

constexpr int kMaxTop = 32;  // alternatives a row: a lane each

struct ScoresArgs {
    const void *x;           // [T][V] fp32 or bf16, row stride `stride`
    int64_t stride;
    const int *targets;      // [T] or NULL
    float *logprob;          // [T] or NULL
    float *entropy;          // [T] or NULL
    int *top_ids;            // [T][n_top]
    float *top_logprobs;     // [T][n_top]
    int *status;             // may be NULL
    int T, V, n_top, fp32;
    int fill;                // padding rows' results become NaN and -1 (0: stay as they are)
    // filled in by the launch
    int parts;               // of a row, each a block
    int part_batches;        // batches of 256 scores of a part
    float4 *part_sums;       // [T][parts]: reference, sum, weighted sum
    unsigned long long *part_top;  // [T][parts][32]
};

// (max_sms: for any GPU of up to so many)
size_t scores_workspace_bytes(int T, int V, int n_top, int max_sms);
cudaError_t launch_scores(ScoresArgs &a, void *ws, int num_sms, cudaStream_t s);

}  // namespace moe
