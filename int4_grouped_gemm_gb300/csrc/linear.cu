// y[b][n] = sum_k x[b][k] (s[n][k/G] q[n][k] + z[n][k/G]) for 1 to 64 tokens,
// the weights in the int4 format of pack_int4.  One warp per weight row: its
// lanes take the row's words in turn, eight tokens at a time.
#include "linear.cuh"

namespace moe {

constexpr int kLinWarps = 8;

__global__ void __launch_bounds__(kLinWarps * 32) int4_linear_kernel(const LinearArgs a) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n = blockIdx.x * kLinWarps + warp;
    if (n >= a.N) return;
    const int words = a.K / 8;
    const uint32_t *q = a.q + static_cast<int64_t>(n) * words;
    const uint16_t *s = a.s + static_cast<int64_t>(n) * a.ldg, *z = a.b + static_cast<int64_t>(n) * a.ldg;
    for (int t0 = 0; t0 < a.B; t0 += 8) {
        const int nt = a.B - t0 < 8 ? a.B - t0 : 8;
        float acc[8] = {};
        for (int w = lane; w < words; w += 32) {
            const uint32_t word = q[w];
            const float sc = bf16_bits_to_float(s[w * 8 / a.G]), bi = bf16_bits_to_float(z[w * 8 / a.G]);
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = fmaf(sc, static_cast<float>((word >> (4 * (e / 2 + 4 * (e % 2)))) & 15u), bi);
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                if (t < nt) {
                    const uint4 xv = *reinterpret_cast<const uint4 *>(a.x + (t0 + t) * a.x_stride + w * 8);
                    const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        acc[t] = fmaf(v[2 * j], __uint_as_float(xw[j] << 16), acc[t]);
                        acc[t] = fmaf(v[2 * j + 1], __uint_as_float(xw[j] & 0xFFFF0000u), acc[t]);
                    }
                }
            }
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) {
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], off);
            if (lane == 0 && t < nt) {
                const int64_t o = (t0 + t) * a.y_stride + n;
                if (a.y_fp32)
                    static_cast<float *>(a.y)[o] = acc[t];
                else
                    static_cast<__nv_bfloat16 *>(a.y)[o] = __float2bfloat16_rn(acc[t]);
            }
        }
    }
}

cudaError_t launch_linear(const LinearArgs &a, int, cudaStream_t s) {
    int4_linear_kernel<<<(a.N + kLinWarps - 1) / kLinWarps, kLinWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
