// Causal attention of packed sequences of query tokens over the paged cache.
//
// Simple form: one warp per (token, query head), 32 positions at a time with an
// online softmax; a lane scores one position, then holds D / 32 dimensions of
// the output.
#include "prompt.cuh"

namespace moe {

template <int D>
__global__ void __launch_bounds__(128) prompt_kernel(const __grid_constant__ PromptArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (item >= static_cast<int64_t>(a.T) * a.Hq) return;
    const int t = static_cast<int>(item / a.Hq), h = static_cast<int>(item % a.Hq), kv = h / a.group;
    // the token's sequence
    int b = -1, r0 = 0, r1 = 0;
    for (int i = 0; i < a.n_seq; ++i) {
        r0 = a.q_start[i];
        r1 = a.q_start[i + 1];
        if (r0 < 0 || r1 < r0 || r1 > a.T) {
            record_status(a.status, MOE_ERR_PAGE);
            continue;
        }
        if (t >= r0 && t < r1) {
            b = i;
            break;
        }
    }
    if (b < 0) return;
    const int len = a.seq_len[b];
    if (len < 0) return;
    if (len > static_cast<int64_t>(a.table_ld) << a.c.page_shift) {
        record_status(a.status, MOE_ERR_PAGE);
        return;
    }
    const int pos = len - (r1 - r0) + (t - r0);
    const int n = a.prefix_len + (pos < 0 ? 0 : pos + 1);
    auto row = [&](int p) -> int64_t {  // element offset of position p, or -1
        const bool pre = p < a.prefix_len;
        const int o = pre ? p : p - a.prefix_len;
        const int page = (pre ? a.prefix_pages : a.table + static_cast<int64_t>(b) * a.table_ld)[o >> a.c.page_shift];
        if (page < 0 || page >= a.c.n_pages) {
            record_status(a.status, MOE_ERR_PAGE);
            return -1;
        }
        return page * a.c.page_stride + kv * a.c.head_stride + (o & ((1 << a.c.page_shift) - 1)) * a.c.pos_stride;
    };
    const __nv_bfloat16 *q = a.q + t * a.q_stride + static_cast<int64_t>(h) * D;
    float m = kLeastRef, l = 0.f, o[D / 32] = {};
    for (int p0 = 0; p0 < n; p0 += 32) {
        float s = -INFINITY;
        const int64_t at = p0 + lane < n ? row(p0 + lane) : -1;
        if (p0 + lane < n) {
            s = 0.f;
            if (at >= 0)
                for (int d = 0; d < D; ++d) s += __bfloat162float(q[d]) * __bfloat162float(a.c.k[at + d]);
            s *= a.scale;
        }
        float mx = s;
        for (int i = 16; i; i >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, i));
        const float mn = fmaxf(m, mx), corr = expf(m - mn), w = expf(s - mn);
        m = mn;
        l = l * corr + w;
        for (int i = 0; i < D / 32; ++i) o[i] *= corr;
        for (int j = 0; j < 32 && p0 + j < n; ++j) {
            const float wj = __shfl_sync(0xffffffffu, w, j);
            const int64_t vj = __shfl_sync(0xffffffffu, at, j);
            if (vj >= 0)
                for (int i = 0; i < D / 32; ++i) o[i] += wj * __bfloat162float(a.c.v[vj + i * 32 + lane]);
        }
    }
    for (int i = 16; i; i >>= 1) l += __shfl_xor_sync(0xffffffffu, l, i);
    for (int i = 0; i < D / 32; ++i)
        a.out[t * a.out_stride + static_cast<int64_t>(h) * D + i * 32 + lane] = __float2bfloat16_rn(n ? o[i] / l : 0.f);
}

size_t prompt_workspace_bytes(int, int, int, int, int, int) { return kCtrlBytes; }

cudaError_t launch_prompt(PromptArgs &a, const CUtensorMap *, void *, int, cudaStream_t s) {
    const int64_t blocks = (static_cast<int64_t>(a.T) * a.Hq + 3) / 4;
    if (a.c.D == 64)
        prompt_kernel<64><<<static_cast<unsigned>(blocks), 128, 0, s>>>(a);
    else
        prompt_kernel<128><<<static_cast<unsigned>(blocks), 128, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
