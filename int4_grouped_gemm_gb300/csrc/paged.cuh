// The paged key-value cache: appending to it and attending over it.  Argument
// bundles and launch entries, shared by the kernels and the C ABI.
#pragma once

#include <stddef.h>

#include "common.cuh"
#include "layout.cuh"

namespace moe {

// Element (page, head, position in the page, dimension) of a pool is at
// page * page_stride + head * head_stride + pos * pos_stride + dimension.
struct Pages {
    __nv_bfloat16 *k, *v;
    int64_t page_stride, head_stride, pos_stride;
    int n_pages, page_shift, Hkv, D;
};

struct AppendArgs {
    Pages c;
    const __nv_bfloat16 *q, *k, *v;  // [T][heads][D] with row strides (q NULL: none)
    __nv_bfloat16 *q_out;
    int64_t q_stride, k_stride, v_stride, qo_stride;
    const int *seq, *index, *table;
    const float *inv_freq;
    int *status;                     // may be NULL
    int T, Hq, n_seq, table_ld, pos_offset, rot, interleaved;
};

// A part's reference m (log2 units) is never below this, so that a part with
// positions differs from one without (-inf): scores of -inf weigh nothing, and
// NaN, which a maximum passes over, stays in the sums.
constexpr float kLeastRef = -3.402823466e38f;

// Partial results of the attention, merged by the combine kernel.  A list of
// tiles is cut into pieces of `per` tiles; piece c and item i of the list (a
// row's key-value head, or a block of rows of the prefix) that meet have
// partial slot c + i, which no other pair has (both only grow along the list).
struct PagedArgs {
    Pages c;
    const __nv_bfloat16 *q;          // [B][Hq][D], row stride q_stride
    __nv_bfloat16 *out;              // [B][Hq][D], row stride out_stride
    int64_t q_stride, out_stride;
    const int *prefix_pages, *table, *seq_len;
    int *status;
    int64_t *starts;                 // [B + 1]: 16-position tiles of the rows before b; [B + 1] tiles of a piece
    float2 *prefix_ml;               // [2 slot + sub][128 rows]: as own_ml
    float *prefix_o;                 // [2 slot + sub][D / 4][128 rows][4]
    float2 *own_ml;                  // [slot][8 heads]: running maximum (log2) and sum
    float *own_o;                    // [slot][D / 4][8 heads][4]: unnormalised output
    int *pieces;                     // behind a prefix kernel: pieces to be taken from the counter + 1 (0: not known
                                     // yet), and the counter
    int B, Hq, group, prefix_len, table_ld;
    int join;                        // the prefix is read as the start of every row
    int ncta;                        // blocks of the own-position kernel
    int own_first;                   // of them, those that find a SM while the prefix kernel runs
    int prefix_two, prefix_blocks;   // prefix: 256-row blocks (else one of 128), blocks a key-value head
    int prefix_tiles, prefix_per;    // 128-position tiles of the prefix, tiles of a piece
    int prefix_ncta;                 // pieces and blocks of the prefix kernel, 0 without one
    int negate;                      // scale < 0: the queries' signs are flipped instead
    int zero_q;                      // scale = 0: the queries are taken as zeros, with scale_log2 = 1
    long long wait_limit;
    float scale_log2;                // |scale| log2(e)
};

cudaError_t launch_append(const AppendArgs &a, int num_sms, cudaStream_t s);
cudaError_t launch_prefix(const CUtensorMap &k, const CUtensorMap &v, const PagedArgs &a, cudaStream_t s);
bool paged_joins(int B, int prefix_len);  // the prefix is read per row instead of by the prefix kernel
size_t paged_workspace_bytes(int B, int Hq, int Hkv, int D, int prefix_len, int num_sms);
cudaError_t launch_paged(PagedArgs &a, const CUtensorMap *maps, float scale, void *ws, int num_sms, cudaStream_t s);

}  // namespace moe
