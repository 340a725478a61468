// Attention of packed prompts over the paged cache: arguments and launch entry.
#pragma once

#include "paged.cuh"

namespace moe {

// A block of rows of one sequence: up to 2 x tq tokens (tq = 128 / group) with all
// heads of a key-value head each.
struct PromptBlock {
    int seq, row0;   // sequence, first row of q
    int pos0, ntok;  // own position of that token (negative: none), tokens
};

// What the plan kernel leaves for the others.
struct PromptPlan {
    int64_t tiles;   // of all blocks of one key-value head
    int64_t per;     // tiles of a piece
    int nblocks;
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
    int max_blocks;                  // that the workspace has room for
    int negate, zero_q;              // scale < 0: the queries' signs are flipped instead; 0: zero queries, scale_log2 = 1
    float scale_log2;                // |scale| log2(e)
    PromptPlan *plan;
    int *seq_blocks;                 // [n_seq + 1]: blocks of the sequences before
    int64_t *start;                  // [blocks + 1]: tiles of the blocks before (of one key-value head)
    PromptBlock *blocks;
    int *piece_block;                // [ncta]: block of a piece's first tile
    float2 *part_ml;                 // [piece][it began before, it ends later][sub-tile][128 rows]
    float *part_o;                   // same, [D / 4][128 rows][4]
};

// (max_sms: for any GPU of up to so many)
size_t prompt_workspace_bytes(int T, int n_seq, int Hq, int Hkv, int D, int max_sms);
cudaError_t launch_prompt(PromptArgs &a, const CUtensorMap *maps, void *ws, int num_sms, cudaStream_t s);

}  // namespace moe
