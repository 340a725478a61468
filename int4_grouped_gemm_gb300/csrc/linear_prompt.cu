// y[t][n] = sum_k x[t][k] (s[n][k/G] q[n][k] + z[n][k/G]) for a prompt's many tokens, on
// the fifth-generation tensor cores.
//
// With so many tokens the unpacking is done once, by a kernel of its own, and the
// product is a plain one of fp16 operands, no product of which is rounded:
//
//   weights  s (q - 8): eight bits by four with a sign are eleven, exact in fp16, at a
//            power of two of the row's own
//   tokens   bf16's eight bits are exact in fp16 at a power of two of the row's own
//            (largest element in [2^14, 2^15); what is below 2^-31 of it is off by 2^-40)
//   biases   with c = z + 8 s what is left is sum_g X[t][g] c[n][g], X = sum of the
//            group's x: three more columns of the product for each group, X as two fp16
//            parts (h1, h2, h1) times c as two (c1, c1, c2), 22 bits each; X at 2^-8 and c
//            at 2^8, which keeps sums of 128 in fp16's range
//
// linear_operands_kernel writes both operands, rows of P = K + 3 K / G columns (each
// part rounded up to 64, zeros between), and the rows' powers; matrices larger than
// the L2 are worked through in pieces of rows, so that the fp16 weights are read
// back from the L2.  (Unpacked in the product's kernel, a code is unpacked again for
// every 256 tokens: that kernel of the experts' products runs at 41 % of the tensor
// rate.)
//
// linear_prompt_kernel: tiles of 128 weight rows (M) by up to 256 tokens (N, a multiple
// of 16 picked for even rounds over the SMs), one block per SM, tiles in turn:
//
//   warp 0           loads: 64 columns of both operands a stage, 128-byte swizzle
//   warp 1           MMA issue; two accumulators in tensor memory in turn
//   warps 4-11       epilogue: a lane is a weight row, so that a warp writes 32
//                    neighbouring results of a token at a time, whatever y's stride;
//                    powers of two put back
//
// Every wait is bounded.
#include <cuda_fp16.h>

#include <algorithm>

#include "linear.cuh"

namespace moe {
namespace prompt {

constexpr int kRows = 128;                 // weight rows of a tile
constexpr int kMaxTok = 256;               // tokens of a tile
constexpr int kStep = 64;                  // columns of a stage
constexpr int kMaxStages = 8;
constexpr int kEpiWarp = 4, kEpiWarps = 8;
constexpr int kThreads = (kEpiWarp + kEpiWarps) * 32;
constexpr int kWBytes = kRows * kStep * 2;
constexpr int kMaxT = 16384;               // tokens whose operands are held at a time
constexpr size_t kWeightBytes = 40 << 20;  // of fp16 weights held at a time, about

// Columns of an operand's row.
struct Columns {
    int K, Kp, groups, P;
    __host__ __device__ Columns(int K_, int G) : K(K_), Kp((K_ + 63) / 64 * 64), groups(K_ / G), P(Kp + (3 * groups + 63) / 64 * 64) {}
};

struct Args {
    LinearArgs l;
    __half *xh, *wh;      // [tokens here][P], [rows here][P]
    int *xe, *we;         // their powers
    int t0, nt, n0, nn;   // tokens and rows of this launch
    int x_blocks;         // operands: blocks that make tokens
    int tok, t_tiles, n_tiles, stages;
};

// ------------------------------------------------------------- operands

// 2^e for e in -140 .. 140 times x, without a rounding that the result does not need.
__device__ __forceinline__ float times_power(float x, int e) {
    const int h = e / 2;
    return x * __int_as_float((h + 127) << 23) * __int_as_float((e - h + 127) << 23);
}
// e of |x| in [2^e, 2^(e+1)), -126 at least; for infinities and NaN 128.
__device__ __forceinline__ int power_of(float x) {
    const int e = static_cast<int>(__float_as_uint(x) >> 23 & 255);
    return (e ? e : 1) - 127;
}

// y in two fp16 parts.
__device__ __forceinline__ void split(float y, __half &hi, __half &lo) {
    hi = __float2half_rn(y);
    lo = __float2half_rn(y - __half2float(hi));
}

__device__ __forceinline__ void zero_columns(__half *row, int from, int to, int i, int n) {
    for (int c = from + i; c < to; c += n) row[c] = __float2half_rn(0.f);
}

constexpr int kOpThreads = 256;

// Blocks 0 .. x_blocks - 1: a token each.  The others: a weight row a warp.
__global__ void __launch_bounds__(kOpThreads) linear_operands_kernel(const __grid_constant__ Args a) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Columns c(a.l.K, a.l.G);
    const int G = a.l.G, ng = c.groups;
    __shared__ uint32_t tops[kOpThreads / 32];
    pdl_wait();
    pdl_trigger();
    if (static_cast<int>(blockIdx.x) < a.x_blocks) {
        const int t = blockIdx.x;
        const uint4 *x = reinterpret_cast<const uint4 *>(a.l.x + (a.t0 + t) * a.l.x_stride);
        __half *row = a.xh + static_cast<int64_t>(t) * c.P;
        uint32_t top = 0;
        for (int i = tid; i < c.K / 8; i += kOpThreads) {
            const uint4 v = __ldg(x + i);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) top = max(top, max(w[j] & 0x7FFFu, w[j] >> 16 & 0x7FFFu));
        }
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) tops[warp] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kOpThreads / 32; ++i) top = max(top, tops[i]);
        // (a row with an infinity or NaN keeps it)
        const int e = power_of(__uint_as_float(top << 16)), up = 14 - e;
        const int lanes = G / 8;  // of a group
        for (int i0 = 0; i0 < c.K / 8; i0 += kOpThreads) {
            const int i = i0 + tid;
            float sum = 0.f;
            if (i < c.K / 8) {
                const uint4 v = __ldg(x + i);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                uint4 o;
                uint32_t *ow = reinterpret_cast<uint32_t *>(&o);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const __half2 h = __floats2half2_rn(times_power(__uint_as_float(w[j] << 16), up),
                                                        times_power(__uint_as_float(w[j] & 0xFFFF0000u), up));
                    ow[j] = *reinterpret_cast<const uint32_t *>(&h);
                    const float2 f = __half22float2(h);
                    sum += f.x + f.y;
                }
                reinterpret_cast<uint4 *>(row)[i] = o;
            }
            for (int j = 1; j < lanes; j <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, j);
            if (i < c.K / 8 && i % lanes == 0) {
                const int g = i / lanes;
                __half h1, h2;
                split(sum * 0x1p-8f, h1, h2);
                row[c.Kp + g] = h1;
                row[c.Kp + ng + g] = h2;
                row[c.Kp + 2 * ng + g] = h1;
            }
        }
        zero_columns(row, c.K, c.Kp, tid, kOpThreads);
        zero_columns(row, c.Kp + 3 * ng, c.P, tid, kOpThreads);
        if (tid == 0) a.xe[t] = -up;
        return;
    }
    const int r = (blockIdx.x - a.x_blocks) * (kOpThreads / 32) + warp;
    if (r >= a.nn) return;
    const int64_t n = a.n0 + r;
    const uint16_t *s = a.l.s + n * a.l.ldg, *z = a.l.b + n * a.l.ldg;
    const uint32_t *q = a.l.q + n * (c.K / 8);
    __half *row = a.wh + static_cast<int64_t>(r) * c.P;
    float top = 0.f;
    for (int g = lane; g < ng; g += 32) {
        const float sg = bf16_bits_to_float(__ldg(s + g)), cg = bf16_bits_to_float(__ldg(z + g)) + 8.f * sg;
        top = fmaxf(top, fmaxf(8.f * fabsf(sg), 256.f * fabsf(cg)));
    }
    const int up = 14 - power_of(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top))));
    for (int i = lane; i < c.K / 8; i += 32) {
        const uint32_t w = __ldcs(q + i);
        const __half2 sg = __half2half2(__float2half_rn(times_power(bf16_bits_to_float(__ldg(s + i * 8 / G)), up)));
        const __half2 c1032 = __half2half2(__ushort_as_half(0x6408));
        uint4 o;
        uint32_t *ow = reinterpret_cast<uint32_t *>(&o);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // 1024 + q by a mask-and-set a pair
            const uint32_t b = mask_set(w >> (4 * j), 0x000F000Fu, 0x64006400u);
            const __half2 p = __hmul2(__hsub2(*reinterpret_cast<const __half2 *>(&b), c1032), sg);
            ow[j] = *reinterpret_cast<const uint32_t *>(&p);
        }
        reinterpret_cast<uint4 *>(row)[i] = o;
    }
    for (int g = lane; g < ng; g += 32) {
        const float sg = bf16_bits_to_float(__ldg(s + g)), cg = bf16_bits_to_float(__ldg(z + g)) + 8.f * sg;
        __half c1, c2;
        split(times_power(cg, up) * 256.f, c1, c2);
        row[c.Kp + g] = c1;
        row[c.Kp + ng + g] = c1;
        row[c.Kp + 2 * ng + g] = c2;
    }
    zero_columns(row, c.K, c.Kp, lane, 32);
    zero_columns(row, c.Kp + 3 * ng, c.P, lane, 32);
    if (lane == 0) a.we[r] = -up;
}

// -------------------------------------------------------------- product

struct Ctl {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t drain;
    uint32_t tmem;
    int abort;
};

__host__ __device__ constexpr int stage_bytes(int tok) { return kWBytes + tok * kStep * 2; }
__host__ __device__ constexpr int stages_for(int tok) {
    const int n = (kBlockSmem - 1024 - static_cast<int>(sizeof(Ctl))) / stage_bytes(tok);
    return n < kMaxStages ? n : kMaxStages;
}
__host__ __device__ constexpr int smem_bytes(int tok) {
    return stages_for(tok) * stage_bytes(tok) + 1024 + static_cast<int>(sizeof(Ctl));
}
static_assert(stages_for(kMaxTok) >= 4 && smem_bytes(kMaxTok) <= kBlockSmem, "stages");

__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, const Args &a, Ctl *s, int site) {
    return role_wait(bar, parity, a.l.wait_limit, a.l.status, &s->abort, site);
}

// Instruction descriptor: fp16 x fp16 -> fp32, A and B K-major, shape 128 x tok.
__device__ __forceinline__ uint32_t idesc_f16(int tok) {
    return (1u << 4) | (static_cast<uint32_t>(tok >> 3) << 17) | (static_cast<uint32_t>(kRows >> 4) << 24);
}

__global__ void __launch_bounds__(kThreads, 1)
    linear_prompt_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                         const __grid_constant__ Args a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int stage = stage_bytes(a.tok), stages = a.stages;
    Ctl *s = reinterpret_cast<Ctl *>(base + stages * stage);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tiles = a.t_tiles * a.n_tiles, steps = Columns(a.l.K, a.l.G).P / kStep;

    if (tid == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(&s->full[i], 1);
            mbar_init(&s->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s->acc_full[i], 1);
            mbar_init(&s->acc_empty[i], kEpiWarps);
        }
        mbar_init(&s->drain, 1);
        s->abort = 0;
        fence_mbar_init();
        prefetch_tmap(&tm_w);
        prefetch_tmap(&tm_x);
    }
    if (warp == 1) {
        tmem_alloc(&s->tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s->tmem;
    pdl_wait();
    pdl_trigger();

    if (warp == 0) {
        if (elect_one()) {
            uint32_t it = 0;
            bool ok = true;
            for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
                const int n0 = tile % a.n_tiles * kRows, t0 = tile / a.n_tiles * a.tok;
                for (int k = 0; k < steps && ok; ++k, ++it) {
                    const int st = it % stages;
                    ok = wait(&s->empty[st], ((it / stages) & 1) ^ 1, a, s, 61);
                    if (!ok) break;
                    uint8_t *at = base + st * stage;
                    mbar_arrive_expect_tx(&s->full[st], stage);
                    tma_load_2d(at, &tm_w, &s->full[st], k * kStep, n0);
                    tma_load_2d(at + kWBytes, &tm_x, &s->full[st], k * kStep, t0);
                }
            }
            // no copy of this block is in flight when it ends
            for (uint32_t i = it > static_cast<uint32_t>(stages) ? it - stages : 0; i < it; ++i)
                mbar_drain(&s->full[i % stages], (i / stages) & 1, a.l.wait_limit);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (elect_one()) {
            const uint32_t idesc = idesc_f16(a.tok);
            uint32_t it = 0, nt = 0;
            bool ok = true;
            for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x, ++nt) {
                const uint32_t acc = tmem + (nt & 1) * 256;
                ok = wait(&s->acc_empty[nt & 1], ((nt >> 1) & 1) ^ 1, a, s, 62);
                if (!ok) break;
                tc_fence_after();
                for (int k = 0; k < steps; ++k, ++it) {
                    const int st = it % stages;
                    ok = wait(&s->full[st], (it / stages) & 1, a, s, 63);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t w_at = smem_u32(base) + st * stage, x_at = w_at + kWBytes;
#pragma unroll
                    for (int j = 0; j < kStep / 16; ++j)
                        umma_bf16(acc, sdesc_k128(w_at + j * 32), sdesc_k128(x_at + j * 32), idesc, k | j);
                    umma_commit(&s->empty[st]);
                }
                if (ok) umma_commit(&s->acc_full[nt & 1]);
            }
            // every MMA issued here is complete before tensor memory is freed
            umma_commit(&s->drain);
            mbar_drain(&s->drain, 0, a.l.wait_limit);
        }
        __syncwarp();
    } else if (warp >= kEpiWarp) {
        const int quarter = warp & 3, half = (warp - kEpiWarp) >> 2;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        uint32_t nt = 0;
        for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, ++nt) {
            const int n = tile % a.n_tiles * kRows + quarter * 32 + lane, t0 = tile / a.n_tiles * a.tok;
            const int we = n < a.nn ? __ldcg(a.we + n) : 0;
            const bool ok = __all_sync(0xffffffffu, wait(&s->acc_full[nt & 1], (nt >> 1) & 1, a, s, 64));
            if (!ok) break;
            tc_fence_after();
            // sixteen tokens at a time, the halves in turn
            for (int c = half * 16; c < a.tok; c += 32) {
                float v[16];
                tmem_ld16((tmem + (nt & 1) * 256 + c) | lanes, v);
                const int left = a.nt - t0 - c;
                if (left <= 0) break;
                const int xe = lane < 16 && lane < left ? __ldcg(a.xe + t0 + c + lane) : 0;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float y = times_power(v[j], max(-250, min(250, we + __shfl_sync(0xffffffffu, xe, j))));
                    if (j < left && n < a.nn) a.l.store(a.t0 + t0 + c + j, a.n0 + n, y);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s->acc_empty[nt & 1]);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ----------------------------------------------------------------- host

struct Layout {
    size_t xe, we, xh, wh, total;
    int rows;  // weight rows held at a time
};

static Layout layout(int N, int K, int G, int T) {
    auto up = [](size_t n) { return (n + 1023) / 1024 * 1024; };
    const size_t P = Columns(K, G).P;
    Layout L{};
    const size_t most = std::max<size_t>(kWeightBytes / (P * 2) / kRows * kRows, kRows);
    L.rows = static_cast<int>(std::min<size_t>(N, most));
    L.xe = kCtrlBytes;
    L.we = L.xe + up(std::min(T, kMaxT) * sizeof(int));
    L.xh = up(L.we + L.rows * sizeof(int));
    L.wh = L.xh + up(std::min(T, kMaxT) * P * 2);
    L.total = L.wh + L.rows * P * 2;
    return L;
}

// Tokens of a tile: as many as make the rounds over the SMs cheapest, a round's cost
// being its tokens and 32 more (weights are fetched for few tokens as for many).
static int tile_tokens(int N, int T, int sms) {
    const int n_tiles = (N + kRows - 1) / kRows;
    int best = kMaxTok;
    int64_t least = INT64_MAX;
    for (int tok = kMaxTok; tok >= 32; tok -= 16) {
        const int64_t tiles = static_cast<int64_t>(n_tiles) * ((T + tok - 1) / tok);
        const int64_t cost = (tiles + sms - 1) / sms * (tok + 32);
        if (cost < least) {
            least = cost;
            best = tok;
        }
    }
    return best;
}

}  // namespace prompt

size_t linear_prompt_workspace_bytes(int N, int K, int G, int T) { return prompt::layout(N, K, G, T).total; }

cudaError_t launch_linear_prompt(const LinearArgs &l, LinearMap encode, void *ws, int num_sms, cudaStream_t s) {
    using namespace prompt;
    const Layout L = layout(l.N, l.K, l.G, l.B);
    const Columns c(l.K, l.G);
    char *w = static_cast<char *>(ws);
    Args a{};
    a.l = l;
    a.xe = reinterpret_cast<int *>(w + L.xe);
    a.we = reinterpret_cast<int *>(w + L.we);
    a.xh = reinterpret_cast<__half *>(w + L.xh);
    a.wh = reinterpret_cast<__half *>(w + L.wh);
    cudaError_t e = allow_smem<linear_prompt_kernel>();
    if (e != cudaSuccess) return e;
    for (a.t0 = 0; a.t0 < l.B; a.t0 += kMaxT) {
        a.nt = std::min(l.B - a.t0, kMaxT);
        for (a.n0 = 0; a.n0 < l.N; a.n0 += L.rows) {
            a.nn = std::min(l.N - a.n0, L.rows);
            a.x_blocks = a.n0 ? 0 : a.nt;
            const int w_blocks = (a.nn + kOpThreads / 32 - 1) / (kOpThreads / 32);
            if ((e = launch_dependent(linear_operands_kernel, dim3(a.x_blocks + w_blocks), dim3(kOpThreads), 0, s, a)) != cudaSuccess)
                return e;
            a.tok = tile_tokens(a.nn, a.nt, num_sms);
            a.stages = stages_for(a.tok);
            a.n_tiles = (a.nn + kRows - 1) / kRows;
            a.t_tiles = (a.nt + a.tok - 1) / a.tok;
            CUtensorMap mw, mx;
            if (!encode(&mw, a.wh, c.P, a.nn, kStep, kRows) || !encode(&mx, a.xh, c.P, a.nt, kStep, a.tok))
                return cudaErrorInvalidValue;
            const int tiles = a.n_tiles * a.t_tiles;
            if ((e = launch_dependent(linear_prompt_kernel, dim3(std::min(tiles, num_sms)), dim3(kThreads), smem_bytes(a.tok),
                                      s, mw, mx, a)) != cudaSuccess)
                return e;
        }
    }
    return cudaSuccess;
}

}  // namespace moe
