// Log probabilities of given tokens, the entropy and the most probable tokens of
// rows of scores.
//
// Simple form: one block per row; a pass for the maximum, one for the sums, and
// one for each alternative.
#include "scores.cuh"

namespace moe {

// A score's place in the order of alternatives: larger scores first, NaN before
// all, equal ones (zeros of both signs too) by lower id.
__device__ __forceinline__ unsigned long long rank_key(float x, int id) {
    const uint32_t u = x != x ? 0x7FFFFFFFu : __float_as_uint(x + 0.f);
    const uint32_t up = u & 0x80000000u ? ~u : u | 0x80000000u;
    return static_cast<unsigned long long>(up) << 32 | ~static_cast<uint32_t>(id);
}

__device__ __forceinline__ float score_at(const ScoresArgs &a, int64_t i) {
    return a.fp32 ? static_cast<const float *>(a.x)[i] : __bfloat162float(static_cast<const __nv_bfloat16 *>(a.x)[i]);
}

__global__ void __launch_bounds__(256) scores_kernel(const __grid_constant__ ScoresArgs a) {
    __shared__ float red[256];
    __shared__ unsigned long long best[256];
    const int t = blockIdx.x, tid = threadIdx.x;
    const int target = a.targets ? a.targets[t] : 0;
    if (target < 0) return;
    const int64_t row = t * a.stride;
    float m = -INFINITY;
    bool nan = false;
    for (int i = tid; i < a.V; i += 256) {
        const float x = score_at(a, row + i);
        nan |= x != x;
        m = fmaxf(m, x);
    }
    nan = __syncthreads_or(nan);
    red[tid] = m;
    __syncthreads();
    for (int s = 128; s; s >>= 1) {
        if (tid < s) red[tid] = fmaxf(red[tid], red[tid + s]);
        __syncthreads();
    }
    m = red[0];
    __syncthreads();
    float sum = 0.f, dot = 0.f;
    for (int i = tid; i < a.V; i += 256) {
        const float d = score_at(a, row + i) - m, e = expf(d);
        sum += e;
        dot += e > 0.f ? e * d : 0.f;
    }
    red[tid] = sum;
    __syncthreads();
    for (int s = 128; s; s >>= 1) {
        if (tid < s) red[tid] += red[tid + s];
        __syncthreads();
    }
    sum = red[0];
    __syncthreads();
    red[tid] = dot;
    __syncthreads();
    for (int s = 128; s; s >>= 1) {
        if (tid < s) red[tid] += red[tid + s];
        __syncthreads();
    }
    dot = red[0];
    // a NaN, an infinity above, or no score at all: no distribution
    const bool none = nan || !(m > -INFINITY) || m == INFINITY;
    const float lse = none ? NAN : logf(sum);
    if (tid == 0) {
        if (a.logprob) {
            const bool in = target < a.V;
            if (!in) record_status(a.status, MOE_ERR_TOKEN_ID);
            a.logprob[t] = in ? score_at(a, row + target) - m - lse : NAN;
        }
        if (a.entropy) a.entropy[t] = lse - dot / sum;
    }
    unsigned long long last = ~0ull;
    for (int n = 0; n < a.n_top; ++n) {
        unsigned long long mine = 0;
        for (int i = tid; i < a.V; i += 256) {
            const unsigned long long k = rank_key(score_at(a, row + i), i);
            if (k < last && k > mine) mine = k;
        }
        __syncthreads();
        best[tid] = mine;
        __syncthreads();
        for (int s = 128; s; s >>= 1) {
            if (tid < s && best[tid + s] > best[tid]) best[tid] = best[tid + s];
            __syncthreads();
        }
        last = best[0];
        if (tid == 0) {
            const int id = static_cast<int>(~static_cast<uint32_t>(last));
            a.top_ids[static_cast<int64_t>(t) * a.n_top + n] = id;
            a.top_logprobs[static_cast<int64_t>(t) * a.n_top + n] = score_at(a, row + id) - m - lse;
        }
    }
}

size_t scores_workspace_bytes(int, int, int, int) { return kCtrlBytes; }

cudaError_t launch_scores(ScoresArgs &a, void *, int, cudaStream_t s) {
    scores_kernel<<<a.T, 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
