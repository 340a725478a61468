// y[t][n] = sum_k x[t][k] (s[n][k/G] q[n][k] + z[n][k/G]) for any number of tokens.
//
// Simple form: tiles of 16 x 16 results, 32 k at a time through shared memory,
// weights unpacked to fp32.
#include "linear.cuh"

namespace moe {

__global__ void __launch_bounds__(256) linear_prompt_kernel(const __grid_constant__ LinearArgs a) {
    __shared__ float sx[16][33], sw[16][33];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int n0 = blockIdx.x * 16, t0 = blockIdx.y * 16;
    float acc = 0.f;
    for (int k0 = 0; k0 < a.K; k0 += 32) {
        for (int i = threadIdx.x; i < 16 * 32; i += 256) {
            const int r = i / 32, k = k0 + i % 32, t = t0 + r, n = n0 + r;
            sx[r][i % 32] = t < a.B ? __bfloat162float(a.x[t * a.x_stride + k]) : 0.f;
            float w = 0.f;
            if (n < a.N) {
                const uint32_t word = a.q[static_cast<int64_t>(n) * (a.K / 8) + k / 8];
                const int64_t g = static_cast<int64_t>(n) * a.ldg + k / a.G;
                w = bf16_bits_to_float(a.s[g]) * ((word >> (4 * (k % 8 / 2 + k % 2 * 4))) & 15u) + bf16_bits_to_float(a.b[g]);
            }
            sw[r][i % 32] = w;
        }
        __syncthreads();
        float part = 0.f;
        for (int k = 0; k < 32; ++k) part += sx[ty][k] * sw[tx][k];
        acc += part;
        __syncthreads();
    }
    const int t = t0 + ty, n = n0 + tx;
    if (t < a.B && n < a.N) {
        if (a.y_fp32)
            static_cast<float *>(a.y)[t * a.y_stride + n] = acc;
        else
            static_cast<__nv_bfloat16 *>(a.y)[t * a.y_stride + n] = __float2bfloat16_rn(acc);
    }
}

size_t linear_prompt_workspace_bytes(int, int, int, int) { return kCtrlBytes; }

cudaError_t launch_linear_prompt(const LinearArgs &a, void *, int, cudaStream_t s) {
    linear_prompt_kernel<<<dim3((a.N + 15) / 16, (a.B + 15) / 16), 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
