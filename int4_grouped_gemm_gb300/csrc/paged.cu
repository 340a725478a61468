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

// ------------------------------------------------------------- attention
//
// Row b, query head h, key-value head g = h / group: o = softmax(scale q . K) V
// over the prefix and the row's own positions, by the online softmax: over any
// part of the positions a running maximum m, sum l = sum 2^(s - m) and output
// O = sum 2^(s - m) v (scores in units of log2), and parts merge as
// m = max m_i, l = sum 2^(m_i - m) l_i, O likewise.
//
// paged_own_kernel: every key and value is read once for the (at most 8) query
// heads that share it, so the work is bound by those bytes.  The rows' positions
// are cut into tiles of 16 (never across a page), all tiles of all rows and
// key-value heads form one list, and each of the (one per SM) blocks takes an
// even piece of it, whatever the lengths: a batch of one long and many short
// rows fills the GPU like one row does.  Within a block, warp w takes tiles w,
// w + 8, ... of the piece through its own ring of cp.async stages (24 KB), which
// runs on across the items of the piece; at an item's end the warps' (m, l, O)
// are merged in shared memory and written as one partial.
//   scores   mma.sync m16n8k16, the heads as M, 16 positions as N
//   output   O += P V, P from the score registers, rounded to bf16; l sums the
//            rounded values, so that a weight's rounding cancels where one
//            position dominates
constexpr int kOwnWarps = 8;
constexpr int kOwnThreads = kOwnWarps * 32;
constexpr int kPosTile = 16;
constexpr int kOwnMinTiles = kOwnWarps;  // tiles a block takes at least: one per warp

__host__ __device__ constexpr int own_stages(int D) { return D == 128 ? 3 : 6; }
__host__ __device__ constexpr int own_stage_bytes(int D) { return 2 * kPosTile * D * 2; }
__host__ __device__ constexpr int own_ring_bytes(int D) { return kOwnWarps * own_stages(D) * own_stage_bytes(D); }
__host__ __device__ constexpr int merge_pitch(int D) { return D + 8; }
__host__ __device__ constexpr int own_merge_bytes(int D) { return kOwnWarps / 2 * 8 * merge_pitch(D) * 4; }
constexpr int kMaxRows = 1024;
__host__ __device__ constexpr int own_smem_bytes(int D) {
    return own_ring_bytes(D) + own_merge_bytes(D) + 2 * kOwnWarps * 8 * 4 + kOwnWarps * own_stages(D) * 4 +
           (kMaxRows + 1) * 8;
}
static_assert(own_smem_bytes(128) <= 227 * 1024 && own_smem_bytes(64) <= 227 * 1024, "one block per SM");

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

// 16 bytes from global to shared memory, or zeros (the source is then not read).
__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const void *src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    return bf162_as_u32(__floats2bfloat162_rn(lo, hi));
}

__host__ __device__ __forceinline__ int tiles16(int n) { return (n + kPosTile - 1) / kPosTile; }

// Row b's own positions: none for a padding row, the table's room at most.
__device__ __forceinline__ int own_len(const PagedArgs &a, int b, bool &over) {
    const int n = a.seq_len[b];
    const int64_t room = static_cast<int64_t>(a.table_ld) << a.c.page_shift;
    over = n > room;
    return n < 0 ? 0 : over ? static_cast<int>(room) : n;
}

// First tile of piece c of W tiles cut into n pieces, and the piece of tile f.
__device__ __forceinline__ int64_t piece_start(int64_t W, int n, int c) { return W * c / n; }
__device__ __forceinline__ int piece_of(int64_t W, int n, int64_t f) {
    return static_cast<int>(((f + 1) * n - 1) / W);
}
__device__ __forceinline__ int own_pieces(int64_t W, int ncta) {
    const int64_t most = (W + kOwnMinTiles - 1) / kOwnMinTiles;
    return most < ncta ? static_cast<int>(most) : ncta;
}

template <int D>
__global__ void __launch_bounds__(kOwnThreads, 1) paged_own_kernel(const __grid_constant__ PagedArgs a) {
    constexpr int KD = D / 16;          // MMA k-steps of the scores
    constexpr int NT = D / 8;           // 8-dimension MMA tiles of the output
    constexpr int CH = D * 2 / 16;      // 16-byte chunks of a row
    constexpr int ROW = D * 2;
    constexpr int NS = own_stages(D), STAGE = own_stage_bytes(D), MP = merge_pitch(D);
    extern __shared__ __align__(128) uint8_t smem[];
    float *mo = reinterpret_cast<float *>(smem + own_ring_bytes(D));          // [4 warps][8 heads][MP]
    float *mm = reinterpret_cast<float *>(smem + own_ring_bytes(D) + own_merge_bytes(D));  // [warp][head]
    float *ml = mm + kOwnWarps * 8;
    int *s_valid = reinterpret_cast<int *>(ml + kOwnWarps * 8);               // [warp][stage]
    int64_t *s_start = reinterpret_cast<int64_t *>(s_valid + kOwnWarps * NS);  // [B + 1]
    __shared__ int64_t s_warp[kOwnWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g8 = lane >> 2, c = lane & 3;
    pdl_trigger();
    const int Hkv = a.c.Hkv, ps = a.c.page_shift;
    const int ntp = a.join ? tiles16(a.prefix_len) : 0;

    // tiles of the rows before each row (four rows a thread, then a scan)
    {
        int64_t n[4], sum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int b = tid * 4 + i;
            n[i] = 0;
            if (b < a.B) {
                bool over;
                const int len = own_len(a, b, over);
                n[i] = a.seq_len[b] < 0 ? 0 : ntp + tiles16(len);
                if (over && blockIdx.x == 0) record_status(a.status, MOE_ERR_PAGE);
            }
            sum += n[i];
        }
        int64_t scan = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, scan, off);
            if (lane >= off) scan += v;
        }
        if (lane == 31) s_warp[warp] = scan;
        __syncthreads();
        scan -= sum;
        for (int w = 0; w < warp; ++w) scan += s_warp[w];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int b = tid * 4 + i;
            if (b <= a.B) {
                s_start[b] = scan;
                if (blockIdx.x == 0) a.starts[b] = scan;
            }
            scan += n[i];
        }
        if (tid == kOwnThreads - 1 && a.B == kMaxRows) {
            s_start[kMaxRows] = scan;
            if (blockIdx.x == 0) a.starts[kMaxRows] = scan;
        }
        __syncthreads();
    }
    const int64_t W = s_start[a.B] * Hkv;
    const int np = own_pieces(W, a.ncta);
    if (static_cast<int>(blockIdx.x) >= np) {
        pdl_wait();
        return;
    }
    const int64_t f0 = piece_start(W, np, blockIdx.x), f1 = piece_start(W, np, blockIdx.x + 1);

    // the row of tile f: the last one that starts at or before it
    auto row_of = [&](int64_t f) {
        int lo = 0, hi = a.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_start[mid] * Hkv <= f)
                lo = mid;
            else
                hi = mid - 1;
        }
        return lo;
    };

    // this warp's i-th tile is f0 + warp + 8 i; lane j describes tile 32 k + j:
    // where its first key is, and how many positions it has (none if the page
    // is outside the pool)
    const int my_n = f1 - f0 > warp ? static_cast<int>((f1 - f0 - warp + kOwnWarps - 1) / kOwnWarps) : 0;
    int64_t d_at = 0;
    int d_valid = 0;
    auto describe = [&](int i) {
        d_valid = 0;
        if (i >= my_n) return;
        const int64_t f = f0 + warp + static_cast<int64_t>(kOwnWarps) * i;
        const int b = row_of(f);
        const int64_t nt = s_start[b + 1] - s_start[b];
        const int64_t in_row = f - s_start[b] * Hkv;
        const int kv = static_cast<int>(in_row / nt);
        int t = static_cast<int>(in_row - kv * nt);
        const int *pages = a.table + static_cast<int64_t>(b) * a.table_ld;
        bool over;
        int n = own_len(a, b, over);
        if (t < ntp) {
            pages = a.prefix_pages;
            n = a.prefix_len;
        } else {
            t -= ntp;
        }
        const int p0 = t * kPosTile;
        const int page = pages[p0 >> ps];
        if (page < 0 || page >= a.c.n_pages) {
            record_status(a.status, MOE_ERR_PAGE);
            return;
        }
        d_at = page * a.c.page_stride + kv * a.c.head_stride + (p0 & ((1 << ps) - 1)) * a.c.pos_stride;
        d_valid = n - p0 < kPosTile ? n - p0 : kPosTile;
    };
    const uint32_t ring = smem_u32(smem) + warp * NS * STAGE;
    // tile i into stage i % NS: keys then values, chunk ch of row r at
    // ch ^ (r & 7); rows past the last position are zeros
    auto issue = [&](int i) {
        if ((i & 31) == 0) describe(i + lane);
        const int64_t at = __shfl_sync(0xffffffffu, d_at, i & 31);
        const int valid = __shfl_sync(0xffffffffu, d_valid, i & 31);
        const uint32_t st = ring + (i % NS) * STAGE;
        if (lane == 0) s_valid[warp * NS + i % NS] = valid;
#pragma unroll
        for (int j = lane; j < kPosTile * CH; j += 32) {
            const int r = j / CH, ch = j % CH;
            const bool ok = r < valid;
            const int64_t src = ok ? at + r * a.c.pos_stride + ch * 8 : 0;
            const uint32_t dst = st + r * ROW + ((ch ^ (r & 7)) << 4);
            cp16_or_zero(dst, a.c.k + src, ok);
            cp16_or_zero(dst + kPosTile * ROW, a.c.v + src, ok);
        }
    };
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        if (i < my_n) issue(i);
        cp_async_commit();
    }

    // ldmatrix lane roles: matrix mi = lane / 8, row rr = lane % 8
    const int mi = lane >> 3, rr = lane & 7;
    const int kpos = (mi >> 1) * 8 + rr, kch = mi & 1;
    const int vpos = (mi & 1) * 8 + rr, vch = mi >> 1;
    const uint32_t flip = a.negate ? 0x80008000u : 0u, keep = a.zero_q ? 0u : 0xFFFFFFFFu;

    int i = 0;
    for (int64_t f = f0; f < f1;) {
        const int b = row_of(f);
        const int64_t nt = s_start[b + 1] - s_start[b];
        const int kv = static_cast<int>((f - s_start[b] * Hkv) / nt);
        const int64_t item_end = s_start[b] * Hkv + (kv + 1) * nt;
        const int64_t end = item_end < f1 ? item_end : f1;

        // the group's queries as the A operand: thread (g8, c) holds
        // q[g8][16 kd + 2c, +1] and [16 kd + 2c + 8, +9]
        uint32_t qa[KD][2];
        {
            const bool real = g8 < a.group;
            const uint32_t *qrow = reinterpret_cast<const uint32_t *>(
                a.q + b * a.q_stride + static_cast<int64_t>(kv * a.group + (real ? g8 : 0)) * D);
#pragma unroll
            for (int kd = 0; kd < KD; ++kd) {
                qa[kd][0] = real ? (__ldg(qrow + kd * 8 + c) & keep) ^ flip : 0u;
                qa[kd][1] = real ? (__ldg(qrow + kd * 8 + c + 4) & keep) ^ flip : 0u;
            }
        }
        float o[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
        float m_run = -INFINITY, l_run = 0.f;

        for (; f0 + warp + static_cast<int64_t>(kOwnWarps) * i < end; ++i) {
            cp_async_wait<NS - 1>();
            __syncwarp();
            const uint32_t sk = ring + (i % NS) * STAGE, sv = sk + kPosTile * ROW;
            const int valid = s_valid[warp * NS + i % NS];
            if (valid > 0) {
                float s0[2][4] = {}, s1[2][4] = {};
#pragma unroll
                for (int kd = 0; kd < KD; ++kd) {
                    uint32_t bm[4];
                    ldsm4(bm, sk + kpos * ROW + (((2 * kd + kch) ^ (kpos & 7)) << 4));
                    const uint32_t af[4] = {qa[kd][0], 0u, qa[kd][1], 0u};
                    mma_16816(s0[kd & 1], af, bm[0], bm[1]);
                    mma_16816(s1[kd & 1], af, bm[2], bm[3]);
                }
                float sc[4] = {s0[0][0] + s0[1][0], s0[0][1] + s0[1][1], s1[0][0] + s1[1][0], s1[0][1] + s1[1][1]};
                const int pos[4] = {2 * c, 2 * c + 1, 8 + 2 * c, 9 + 2 * c};
#pragma unroll
                for (int j = 0; j < 4; ++j) sc[j] = pos[j] < valid ? sc[j] * a.scale_log2 : -INFINITY;
                float tmax = fmaxf(fmaxf(sc[0], sc[1]), fmaxf(sc[2], sc[3]));
                tmax = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, 1));
                tmax = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, 2));
                const float m_new = fmaxf(m_run, tmax);  // finite: the tile has a position
                const float corr = exp2f(m_run - m_new);
                const uint32_t p01 = bf16_pair(exp2f(sc[0] - m_new), exp2f(sc[1] - m_new));
                const uint32_t p23 = bf16_pair(exp2f(sc[2] - m_new), exp2f(sc[3] - m_new));
                l_run = l_run * corr + ((__uint_as_float(p01 << 16) + __uint_as_float(p01 & 0xFFFF0000u)) +
                                        (__uint_as_float(p23 << 16) + __uint_as_float(p23 & 0xFFFF0000u)));
                m_run = m_new;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    o[n][0] *= corr;
                    o[n][1] *= corr;
                }
                const uint32_t pa[4] = {p01, 0u, p23, 0u};
#pragma unroll
                for (int jt = 0; jt < NT / 2; ++jt) {
                    uint32_t bm[4];
                    ldsm4_trans(bm, sv + vpos * ROW + (((2 * jt + vch) ^ (vpos & 7)) << 4));
                    mma_16816(o[2 * jt], pa, bm[0], bm[1]);
                    mma_16816(o[2 * jt + 1], pa, bm[2], bm[3]);
                }
            }
            __syncwarp();  // every lane has read the stage before it is refilled
            if (i + NS < my_n) issue(i + NS);
            cp_async_commit();
        }

        // merge the eight warps: every warp scales its output to the common
        // maximum, the upper four hand theirs to the lower four, these add and
        // leave four sums, which the block adds in order
        float l_sum = l_run + __shfl_xor_sync(0xffffffffu, l_run, 1);
        l_sum += __shfl_xor_sync(0xffffffffu, l_sum, 2);
        if (c == 0) {
            mm[warp * 8 + g8] = m_run;  // -inf: no tile of this item
            ml[warp * 8 + g8] = l_sum;
        }
        __syncthreads();
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kOwnWarps; ++w) M = fmaxf(M, mm[w * 8 + g8]);
        const float e = m_run == -INFINITY ? 0.f : exp2f(m_run - M);
        float *mine = mo + ((warp & 3) * 8 + g8) * MP + 2 * c;
        if (warp >= 4) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
                *reinterpret_cast<float2 *>(mine + 8 * n) = make_float2(o[n][0] * e, o[n][1] * e);
        }
        __syncthreads();
        if (warp < 4) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float2 v = *reinterpret_cast<float2 *>(mine + 8 * n);
                v.x += o[n][0] * e;
                v.y += o[n][1] * e;
                *reinterpret_cast<float2 *>(mine + 8 * n) = v;
            }
        }
        __syncthreads();
        const int64_t slot = static_cast<int64_t>(blockIdx.x) + static_cast<int64_t>(b) * Hkv + kv;
        {
            const int h = tid & 7;
            for (int d4 = tid >> 3; d4 < D / 4; d4 += kOwnThreads / 8) {
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float4 v = *reinterpret_cast<const float4 *>(mo + (w * 8 + h) * MP + d4 * 4);
                    sum.x += v.x;
                    sum.y += v.y;
                    sum.z += v.z;
                    sum.w += v.w;
                }
                *reinterpret_cast<float4 *>(a.own_o + (slot * (D / 4) + d4) * 32 + h * 4) = sum;
            }
            if (tid < 8) {
                float mx = -INFINITY, den = 0.f;
#pragma unroll
                for (int w = 0; w < kOwnWarps; ++w) mx = fmaxf(mx, mm[w * 8 + tid]);
#pragma unroll
                for (int w = 0; w < kOwnWarps; ++w)
                    if (mm[w * 8 + tid] != -INFINITY) den += exp2f(mm[w * 8 + tid] - mx) * ml[w * 8 + tid];
                a.own_ml[slot * 8 + tid] = make_float2(mx, den);
            }
        }
        __syncthreads();  // the merge buffers are free for the next item
        f = end;
    }
    cp_async_wait<0>();
    pdl_wait();  // a kernel before this one that still runs is complete before this one is
}

// Merge the partials of one (row, key-value head): grid (B Hkv, D / 32), thread
// (part of the partials, 4 dimensions, head).  First the weights 2^(m_i - M) of
// all partials per head, then the sums with every load independent.
constexpr int kMergeMax = 768;  // partials of one row: at most 256 of its own, 512 of the prefix

__global__ void __launch_bounds__(256) paged_combine_kernel(const __grid_constant__ PagedArgs a) {
    __shared__ float s_w[8][kMergeMax + 1];
    __shared__ float s_inv[8];
    __shared__ float4 s_red[4][64];
    pdl_wait();
    const int Hkv = a.c.Hkv, D = a.c.D;
    const int b = blockIdx.x / Hkv, kv = blockIdx.x % Hkv;
    if (a.seq_len[b] < 0) return;  // padding: out stays as it is
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t W = a.starts[a.B] * Hkv, s0 = a.starts[b], nt = a.starts[b + 1] - s0;
    int c0 = 0, n_own = 0;
    if (nt > 0) {
        const int np = own_pieces(W, a.ncta);
        c0 = piece_of(W, np, s0 * Hkv + kv * nt);
        n_own = piece_of(W, np, s0 * Hkv + (kv + 1) * nt - 1) - c0 + 1;
    }
    const int64_t slot0 = static_cast<int64_t>(c0) + static_cast<int64_t>(b) * Hkv + kv;
    // the prefix's partials of head h's row: first index, count, step
    const int step = a.prefix_two ? 2 : 1;
    auto prefix_parts = [&](int h, int64_t &first, int &row) {
        if (a.prefix_ncta == 0 || h >= a.group) return 0;
        const int g = b * a.group + h, blk = g / (step * 128);
        const int64_t item = static_cast<int64_t>(kv) * a.prefix_blocks + blk;
        const int64_t ntile = (a.prefix_len + 127) / 128, Wp = ntile * Hkv * a.prefix_blocks;
        const int p0 = piece_of(Wp, a.prefix_ncta, item * ntile), p1 = piece_of(Wp, a.prefix_ncta, (item + 1) * ntile - 1);
        row = g & 127;
        first = (p0 + item) * 2 + (a.prefix_two ? (g >> 7) & 1 : 0);
        return (p1 - p0 + 1) * (3 - step);
    };
    {
        const int h = warp;  // warp h: head h's weights
        int64_t first = 0;
        int row = 0;
        const int n_pre = prefix_parts(h, first, row);
        const float2 *own = a.own_ml + slot0 * 8 + h, *pre = a.prefix_ml + first * 128 + row;
        float M = -INFINITY;
        for (int i = lane; i < n_own + n_pre; i += 32) {
            const float v = i < n_own ? __ldcg(own + i * 8).x : __ldcg(pre + static_cast<int64_t>(i - n_own) * step * 128).x;
            s_w[h][i] = v;
            M = fmaxf(M, v);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
        float den = 0.f;
        for (int i = lane; i < n_own + n_pre; i += 32) {
            const float v = s_w[h][i], w = v == -INFINITY ? 0.f : exp2f(v - M);
            s_w[h][i] = w;
            den += w * (i < n_own ? __ldcg(own + i * 8).y : __ldcg(pre + static_cast<int64_t>(i - n_own) * step * 128).y);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) den += __shfl_xor_sync(0xffffffffu, den, off);
        if (lane == 0) s_inv[h] = M == -INFINITY ? 0.f : 1.0f / den;
    }
    __syncthreads();
    const int h = tid & 7, dq = (tid >> 3) & 7, part = tid >> 6;
    const int d4 = blockIdx.y * 8 + dq;
    int64_t first = 0;
    int row = 0;
    const int n_pre = prefix_parts(h, first, row);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    // a partial without weight may never have been written: it is not added
    auto add = [&](float w, const float4 &v) {
        acc.x = w > 0.f ? fmaf(w, v.x, acc.x) : acc.x;
        acc.y = w > 0.f ? fmaf(w, v.y, acc.y) : acc.y;
        acc.z = w > 0.f ? fmaf(w, v.z, acc.z) : acc.z;
        acc.w = w > 0.f ? fmaf(w, v.w, acc.w) : acc.w;
    };
    const float *src = a.own_o + (slot0 * (D / 4) + d4) * 32 + h * 4;
#pragma unroll 8
    for (int i = part; i < n_own; i += 4)
        add(s_w[h][i], __ldcg(reinterpret_cast<const float4 *>(src + static_cast<int64_t>(i) * D * 8)));
    const float *psrc = a.prefix_o + (first * (D / 4) + d4) * 512 + row * 4;
#pragma unroll 8
    for (int i = part; i < n_pre; i += 4)
        add(s_w[h][n_own + i], __ldcg(reinterpret_cast<const float4 *>(psrc + static_cast<int64_t>(i) * step * D * 128)));
    s_red[part][tid & 63] = acc;
    __syncthreads();
    if (part == 0 && h < a.group) {
#pragma unroll
        for (int i = 1; i < 4; ++i) {
            const float4 v = s_red[i][tid];
            acc.x += v.x;
            acc.y += v.y;
            acc.z += v.z;
            acc.w += v.w;
        }
        const float inv = s_inv[h];
        uint2 r;
        r.x = bf16_pair(acc.x * inv, acc.y * inv);
        r.y = bf16_pair(acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2 *>(a.out + b * a.out_stride + static_cast<int64_t>(kv * a.group + h) * D + d4 * 4) = r;
    }
}

// ------------------------------------------------------------------- host

// One row's prefix is read once either way, and without the prefix kernel
// there is a launch less.
bool paged_joins(int B, int prefix_len) { return B == 1 || prefix_len == 0; }

static int prefix_row_blocks(int rows) { return rows <= 128 ? 1 : (rows + 255) / 256; }

struct PagedLayout {
    size_t starts, own_ml, own_o, prefix_ml, prefix_o, total;
};

static PagedLayout paged_layout(int B, int Hq, int Hkv, int D, int prefix_len, int num_sms) {
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    PagedLayout L{};
    const size_t slots = static_cast<size_t>(num_sms) + static_cast<size_t>(B) * Hkv;
    L.starts = kCtrlBytes;
    L.own_ml = L.starts + up((B + 1) * sizeof(int64_t));
    L.own_o = L.own_ml + up(slots * 8 * sizeof(float2));
    L.prefix_ml = L.own_o + up(slots * 8 * D * sizeof(float));
    const size_t parts = paged_joins(B, prefix_len) ? 0 : 2 * (num_sms + static_cast<size_t>(Hkv) * prefix_row_blocks(B * (Hq / Hkv)));
    L.prefix_o = L.prefix_ml + up(parts * 128 * sizeof(float2));
    L.total = L.prefix_o + parts * 128 * D * sizeof(float);
    return L;
}

size_t paged_workspace_bytes(int B, int Hq, int Hkv, int D, int prefix_len, int num_sms) {
    return paged_layout(B, Hq, Hkv, D, prefix_len, num_sms).total;
}

template <int D>
static cudaError_t launch_own(const PagedArgs &a, cudaStream_t s) {
    constexpr int smem = own_smem_bytes(D);
    cudaError_t e = cudaFuncSetAttribute(paged_own_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // beside a prefix kernel its blocks take over the SMs as that one's end
    if (a.prefix_ncta) return launch_dependent(paged_own_kernel<D>, dim3(a.ncta), dim3(kOwnThreads), smem, s, a);
    paged_own_kernel<D><<<a.ncta, kOwnThreads, smem, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_paged(PagedArgs &a, const CUtensorMap *maps, float scale, void *ws, int num_sms, cudaStream_t s) {
    char *w = static_cast<char *>(ws);
    const PagedLayout L = paged_layout(a.B, a.Hq, a.c.Hkv, a.c.D, a.prefix_len, num_sms);
    a.starts = reinterpret_cast<int64_t *>(w + L.starts);
    a.own_ml = reinterpret_cast<float2 *>(w + L.own_ml);
    a.own_o = reinterpret_cast<float *>(w + L.own_o);
    a.prefix_ml = reinterpret_cast<float2 *>(w + L.prefix_ml);
    a.prefix_o = reinterpret_cast<float *>(w + L.prefix_o);
    a.ncta = num_sms;
    a.negate = scale < 0.f;
    a.zero_q = scale == 0.f;
    a.scale_log2 = scale == 0.f ? 1.f : fabsf(scale) * 1.4426950408889634f;
    a.join = paged_joins(a.B, a.prefix_len);
    cudaError_t e;
    if (!a.join) {
        const int rows = a.B * a.group;
        a.prefix_two = rows > 128;
        a.prefix_blocks = prefix_row_blocks(rows);
        const int64_t tiles = static_cast<int64_t>(a.c.Hkv) * a.prefix_blocks * ((a.prefix_len + 127) / 128);
        a.prefix_ncta = tiles < num_sms ? static_cast<int>(tiles) : num_sms;
        if ((e = launch_prefix(maps[0], maps[1], a, s)) != cudaSuccess) return e;
    }
    if ((e = a.c.D == 64 ? launch_own<64>(a, s) : launch_own<128>(a, s)) != cudaSuccess) return e;
    return launch_dependent(paged_combine_kernel, dim3(a.B * a.c.Hkv, a.c.D / 32), dim3(256), 0, s, a);
}

}  // namespace moe
