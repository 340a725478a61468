// Matrix-vector products with int4 weights (the projections either side of
// the attention): argument bundle and launch entry, shared by the kernels and
// the C ABI.
#pragma once

#include <stddef.h>

#include "common.cuh"

namespace moe {

constexpr int kLinearMaxB = 64;      // tokens of one call
constexpr int kLinearMaxK = 32768;
constexpr int kFewTokens = 8;        // up to here launch_linear_few

struct LinearArgs {
    const uint32_t *q;         // [N][K/8]
    const uint16_t *s, *b;     // [N][ldg] bf16 bits
    const __nv_bfloat16 *x;    // [B][x_stride]
    void *y;                   // [B][y_stride] bf16 or fp32
    int64_t x_stride, y_stride;
    int N, K, G, ldg, B;
    int y_fp32;
    // filled in by launch_linear: blocks of a cluster (they split K), units of
    // 128 k in a chunk of tokens, buffers for chunks
    int split, chunk_units, x_buffers;

    __device__ __forceinline__ int rank_of(int block) const { return block % split; }
    __device__ __forceinline__ void store(int t, int n, float v) const {
        if (y_fp32)
            static_cast<float *>(y)[t * y_stride + n] = v;
        else
            static_cast<__nv_bfloat16 *>(y)[t * y_stride + n] = __float2bfloat16_rn(v);
    }
};

cudaError_t launch_linear_few(const LinearArgs &a, int num_sms, cudaStream_t s);
cudaError_t launch_linear(const LinearArgs &a, int num_sms, cudaStream_t s);

}  // namespace moe
