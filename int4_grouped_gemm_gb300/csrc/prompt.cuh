// Attention of packed prompts over the paged cache: arguments and launch entry.
#pragma once

#include "paged.cuh"

namespace moe {

// What the combine kernel needs of a block of rows that a cut between two pieces
// runs through; pieces: how many it lies in (0: nothing to join at this cut).
struct PromptCut {
    int pieces, kv, row0, ntok;
    int pos0, pad[3];
};

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
    // filled in by the launch
    int tq;                          // tokens of a sub-tile of 128 rows
    int ncta;                        // pieces
    int negate;                      // scale < 0: the queries are taken with their signs flipped
    float scale_log2;                // |scale| log2(e)
    PromptCut *cuts;                 // [ncta]: at a piece's beginning
    float2 *part_ml;                 // [piece][its block began before, it ends later][sub-tile][128 rows]
    float *part_o;                   // same, [D / 4][128 rows][4]
};

// (max_sms: for any GPU of up to so many)
size_t prompt_workspace_bytes(int D, int max_sms);
// maps: queries (boxes of 64 x group x tq in (D, Hq, T)), keys, values.
inline int prompt_tokens(int group) { return 128 / group; }  // of a sub-tile
cudaError_t launch_prompt(PromptArgs &a, const CUtensorMap *maps, void *ws, int num_sms, cudaStream_t s);

}  // namespace moe
