// Appending to a paged key-value cache and attending over it.
#include "paged.cuh"

namespace moe {

// The rotation angle pos * f as the cosine and sine of its fraction of a
// turn.  The turns are taken in fp64 (pos up to 2^31 times f / 2 pi leaves
// 2^-52 * 2^28 = 2^-24 of a turn at most), only the fraction in fp32.
__device__ __forceinline__ float2 angle_cs(int64_t pos, float f) {
    const double turns = static_cast<double>(pos) * (static_cast<double>(f) * 0.15915494309189533577);
    const float frac = static_cast<float>(turns - rint(turns));
    float2 r;
    sincospif(2.0f * frac, &r.y, &r.x);
    return r;
}

// One block per token: keys (and queries) rotated pair by pair, values copied.
__global__ void __launch_bounds__(256) append_kernel(const AppendArgs a) {
    const int t = blockIdx.x;
    const int seq = a.seq[t], idx = a.index[t];
    if (seq < 0 || idx < 0) return;  // padding
    const int ps = a.c.page_shift, D = a.c.D;
    const bool in_table = seq < a.n_seq && (idx >> ps) < a.table_ld;
    const int page = in_table ? a.table[static_cast<int64_t>(seq) * a.table_ld + (idx >> ps)] : -1;
    if (page < 0 || page >= a.c.n_pages) {
        if (threadIdx.x == 0) record_status(a.status, MOE_ERR_PAGE);
        return;
    }
    const int64_t slot = page * a.c.page_stride + (idx & ((1 << ps) - 1)) * a.c.pos_stride;
    const int Hq = a.q ? a.Hq : 0, half = D / 2;
    for (int i = threadIdx.x; i < (Hq + a.c.Hkv) * half; i += blockDim.x) {
        const int h = i / half, p = i % half;  // pair p of head h
        const __nv_bfloat16 *src = h < Hq ? a.q + t * a.q_stride + h * D : a.k + t * a.k_stride + (h - Hq) * D;
        __nv_bfloat16 *dst =
            h < Hq ? a.q_out + t * a.qo_stride + h * D : a.c.k + slot + (h - Hq) * a.c.head_stride;
        int i0 = 2 * p, i1 = 2 * p + 1;
        const bool turn = p < a.rot / 2;
        if (turn && !a.interleaved) {
            i0 = p;
            i1 = p + a.rot / 2;
        }
        const __nv_bfloat16 x0 = src[i0], x1 = src[i1];
        if (turn) {
            const float2 cs = angle_cs(static_cast<int64_t>(idx) + a.pos_offset, a.inv_freq[p]);
            const float f0 = __bfloat162float(x0), f1 = __bfloat162float(x1);
            dst[i0] = __float2bfloat16_rn(f0 * cs.x - f1 * cs.y);
            dst[i1] = __float2bfloat16_rn(f1 * cs.x + f0 * cs.y);
        } else {
            dst[i0] = x0;
            dst[i1] = x1;
        }
    }
    for (int i = threadIdx.x; i < a.c.Hkv * D; i += blockDim.x) {
        const int h = i / D, d = i % D;
        a.c.v[slot + h * a.c.head_stride + d] = a.v[t * a.v_stride + i];
    }
}

cudaError_t launch_append(const AppendArgs &a, int, cudaStream_t s) {
    append_kernel<<<a.T, 256, 0, s>>>(a);
    return cudaGetLastError();
}

// One warp per (row, query head), lane l holding dimensions l, l + 32, ...:
// the prefix, then the row's own positions, with an online softmax.
template <int D>
__global__ void __launch_bounds__(256) paged_attention_kernel(const PagedArgs a) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (row >= static_cast<int64_t>(a.B) * a.Hq) return;
    const int b = static_cast<int>(row / a.Hq), h = static_cast<int>(row % a.Hq), kv = h / a.group;
    const int ps = a.c.page_shift;
    int n = a.seq_len[b];
    if (n < 0) return;  // padding
    if (static_cast<int64_t>(n) > (static_cast<int64_t>(a.table_ld) << ps)) {
        if (lane == 0) record_status(a.status, MOE_ERR_PAGE);
        n = a.table_ld << ps;
    }
    float q[E], o[E] = {};
    for (int e = 0; e < E; ++e) q[e] = __bfloat162float(a.q[b * a.q_stride + h * D + lane + 32 * e]);
    float m = -INFINITY, l = 0.f;
    for (int part = 0; part < 2; ++part) {
        const int *pages = part == 0 ? a.prefix_pages : a.table + static_cast<int64_t>(b) * a.table_ld;
        const int count = part == 0 ? a.prefix_len : n;
        for (int t = 0; t < count; ++t) {
            const int page = pages[t >> ps];
            if (page < 0 || page >= a.c.n_pages) {
                if (lane == 0) record_status(a.status, MOE_ERR_PAGE);
                continue;
            }
            const int64_t at = page * a.c.page_stride + kv * a.c.head_stride + (t & ((1 << ps) - 1)) * a.c.pos_stride;
            float s = 0.f;
            for (int e = 0; e < E; ++e) s += q[e] * __bfloat162float(a.c.k[at + lane + 32 * e]);
            for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
            s *= a.scale;
            const float mn = fmaxf(m, s);
            const float c = expf(m - mn), p = expf(s - mn);
            l = l * c + p;
            for (int e = 0; e < E; ++e) o[e] = o[e] * c + p * __bfloat162float(a.c.v[at + lane + 32 * e]);
            m = mn;
        }
    }
    for (int e = 0; e < E; ++e)
        a.out[b * a.out_stride + h * D + lane + 32 * e] = __float2bfloat16_rn(l > 0.f ? o[e] / l : 0.f);
}

size_t paged_workspace_bytes(int, int, int, int, int, int) { return kCtrlBytes; }

cudaError_t launch_paged(const PagedArgs &a, void *, int, cudaStream_t s) {
    const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(a.B) * a.Hq + 7) / 8);
    if (a.c.D == 64)
        paged_attention_kernel<64><<<blocks, 256, 0, s>>>(a);
    else
        paged_attention_kernel<128><<<blocks, 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
