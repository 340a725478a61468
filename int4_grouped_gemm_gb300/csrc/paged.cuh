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

struct PagedArgs {
    Pages c;
    const __nv_bfloat16 *q;          // [B][Hq][D], row stride q_stride
    __nv_bfloat16 *out;              // [B][Hq][D], row stride out_stride
    int64_t q_stride, out_stride;
    const int *prefix_pages, *table, *seq_len;
    int *status;
    int B, Hq, group, prefix_len, table_ld;
    float scale;
};

cudaError_t launch_append(const AppendArgs &a, int num_sms, cudaStream_t s);
size_t paged_workspace_bytes(int B, int Hq, int Hkv, int D, int prefix_len, int num_sms);
cudaError_t launch_paged(const PagedArgs &a, void *ws, int num_sms, cudaStream_t s);

}  // namespace moe
