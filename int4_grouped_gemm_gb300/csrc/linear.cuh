// Matrix-vector products with int4 weights (the projections either side of
// the attention): argument bundle and launch entry, shared by the kernels and
// the C ABI.
#pragma once

#include <stddef.h>

#include "common.cuh"
#include "layout.cuh"

namespace moe {

constexpr int kLinearMaxB = 64;      // tokens of one call
constexpr int kLinearMaxK = 32768;
constexpr int kLinearPromptMaxT = 1 << 20;
constexpr int kFewTokens = 8;        // up to here launch_linear_few

struct LinearArgs {
    const uint32_t *q;         // [N][K/8]
    const uint16_t *s, *b;     // [N][ldg] bf16 bits
    const __nv_bfloat16 *x;    // [B][x_stride]
    void *y;                   // [B][y_stride] bf16 or fp32
    int64_t x_stride, y_stride;
    int N, K, G, ldg, B;
    int y_fp32;
    int *status;               // may be NULL
    long long wait_limit;
    // filled in by the launches: blocks of a cluster (they share K); few tokens:
    // units of k in a chunk of tokens
    int split, chunk_units;

    __device__ __forceinline__ int rank_of(int block) const { return block % split; }
    __device__ __forceinline__ void store(int t, int n, float v) const {
        if (y_fp32)
            static_cast<float *>(y)[t * y_stride + n] = v;
        else
            static_cast<__nv_bfloat16 *>(y)[t * y_stride + n] = __float2bfloat16_rn(v);
    }
};

// (w & mask) | set in one instruction (written plainly, with two immediates, it
// becomes two)
__device__ __forceinline__ uint32_t mask_set(uint32_t w, uint32_t mask, uint32_t set) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(set));
    return r;
}

// A float of another block of the cluster, at this block's own address of it.
__device__ __forceinline__ float dsmem_ld(uint32_t addr, uint32_t rank) {
    uint32_t remote;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
    return v;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// 1 to 8 tokens.
cudaError_t launch_linear_few(const LinearArgs &a, int num_sms, cudaStream_t s);
// 9 to 64 tokens; maps: codes (u32, boxes of linear_code_words(G, B) x 128 rows,
// swizzled over their width), scales, biases (u16, 16 x 128 rows), tokens (bf16,
// 64 x linear_token_rows(B), 128-byte swizzle).
int linear_token_rows(int B);
int linear_code_words(int G, int B);
cudaError_t launch_linear_many(const CUtensorMap *maps, const LinearArgs &a, int num_sms, cudaStream_t s);
// Many tokens; encode: the map of a row-major matrix of fp16 (half; 128-byte swizzle) or 32-bit words
// (32-byte swizzle) in boxes of box_inner x box_rows (false: none can be made).
using LinearMap = bool (*)(CUtensorMap *map, const void *ptr, bool half, int inner, int rows, int box_inner, int box_rows);
size_t linear_prompt_workspace_bytes(int N, int K, int G, int T);
cudaError_t launch_linear_prompt(const LinearArgs &a, LinearMap encode, void *ws, int num_sms, cudaStream_t s);

}  // namespace moe
