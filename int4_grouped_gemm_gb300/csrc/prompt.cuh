// Attention of packed prompts over the paged cache: arguments and launch entry.
#pragma once

#include "paged.cuh"

namespace moe {

struct PromptArgs {
    Pages c;
    const __nv_bfloat16 *q;          // [T][Hq][D], row stride q_stride
    __nv_bfloat16 *out;              // [T][Hq][D], row stride out_stride
    int64_t q_stride, out_stride;
    const int *q_start;              // [n_seq + 1]: first row of each sequence
    const int *prefix_pages, *table, *seq_len;
    int *status;                     // may be NULL
    int T, Hq, group, n_seq, prefix_len, table_ld;
    float scale;
    long long wait_limit;
};

// (max_sms: for any GPU of up to so many)
size_t prompt_workspace_bytes(int T, int n_seq, int Hq, int Hkv, int D, int max_sms);
cudaError_t launch_prompt(PromptArgs &a, const CUtensorMap *maps, void *ws, int num_sms, cudaStream_t s);

}  // namespace moe
