// Matrix-vector products with int4 weights (the projections either side of
// the attention): argument bundle and launch entry, shared by the kernels and
// the C ABI.
#pragma once

#include <stddef.h>

#include "common.cuh"

namespace moe {

constexpr int kLinearMaxB = 64;      // tokens of one call
constexpr int kLinearMaxK = 32768;

struct LinearArgs {
    const uint32_t *q;         // [N][K/8]
    const uint16_t *s, *b;     // [N][ldg] bf16 bits
    const __nv_bfloat16 *x;    // [B][x_stride]
    void *y;                   // [B][y_stride] bf16 or fp32
    int64_t x_stride, y_stride;
    int N, K, G, ldg, B;
    int y_fp32;
};

cudaError_t launch_linear(const LinearArgs &a, int num_sms, cudaStream_t s);

}  // namespace moe
