// y[b][n] = sum_k x[b][k] (s[n][k/G] q[n][k] + z[n][k/G]) for 1 to 64 tokens,
// the weights in the int4 format of pack_int4, read once.
//
// The sum runs group by group on the codes themselves: 128 + q is exact in
// bf16, so with D = sum over the group of (128 + q) x on mma.sync (fp32 sums)
// and X = sum of x,
//   y += s D + (z - 128 s) X
// and no weight is ever rounded.  The MMA's M = 16 is 16 weight rows, its N = 8
// eight tokens (NT such tiles), and per weight the ALU work is one shift or
// one mask-and-set for each pair.
//
// A block of eight warps takes RW tiles of 16 rows and splits K over KW = 8 / RW
// warps (few tokens: all eight, one tile of rows, so that even 2048 rows
// occupy 128 SMs; many tokens: none, 128 rows, since the tokens pass through
// shared memory once per block).  If there are too few rows for the GPU, a
// cluster of up to eight blocks splits K further and adds up through
// distributed shared memory.  The weights of a warp stream through its own ring
// of cp.async stages (16 rows x 128 k and their scales, eight deep); the tokens
// stay in shared memory if they fit, else chunks of them alternate in two
// buffers.
#include "linear.cuh"

#include <algorithm>

namespace moe {

constexpr int kLinWarps = 8;
constexpr int kLinThreads = kLinWarps * 32;
constexpr int kUnit = 128;                       // k of a stage
constexpr int kNibBytes = 16 * kUnit / 2;        // codes of a stage
constexpr int kScaleBytes = 16 * 8;              // up to four groups of 16 rows
constexpr int kStageBytes = kNibBytes + 2 * kScaleBytes;
__host__ __device__ constexpr int ring_bytes(int stages) { return kLinWarps * stages * kStageBytes; }

__device__ __forceinline__ void cp_async_n(uint32_t dst, const void *src, int bytes, bool valid) {
    if (bytes == 16)
        asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
                     : "memory");
    else if (bytes == 8)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(valid ? 8 : 0) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(valid ? 4 : 0) : "memory");
}

// Pair j of a word (elements 2j, 2j + 1 in nibbles j, j + 4) as bf16 128 + q.
__device__ __forceinline__ uint32_t code_pair(uint32_t word, int j) {
    return ((word >> (4 * j)) & 0x000F000Fu) | 0x43004300u;
}

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

template <int G, int NT, int RW, int kLinStages>
__global__ void __launch_bounds__(kLinThreads, NT <= 2 ? 2 : 1) int4_linear_kernel(const LinearArgs a) {
    constexpr int KW = kLinWarps / RW;
    constexpr int B8 = NT * 8;                    // token rows of the buffers
    constexpr int GPU_ = kUnit / G;               // groups of a unit
    constexpr int SB = GPU_ == 4 ? 8 : 4;         // bytes of scales copied per row and unit
    constexpr int XPAD = G == 32 ? 64 : 16;       // token rows start on different banks
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g8 = lane >> 2, c = lane & 3;
    const int rw = warp % RW, kw = warp / RW;
    const uint32_t ring = smem_u32(smem) + warp * kLinStages * kStageBytes;
    const int cu = a.chunk_units;                 // units of a chunk of tokens
    const int xpitch = cu * kUnit * 2 + XPAD;     // bytes
    const int xbytes = a.B * xpitch, gbytes = cu * GPU_ * B8 * 4;
    uint8_t *xbuf = smem + ring_bytes(kLinStages);            // [buffers][tokens][chunk], then group sums [buffers][group][tokens]
    uint8_t *gbuf = xbuf + a.x_buffers * xbytes;
    float *red = reinterpret_cast<float *>(gbuf + a.x_buffers * gbytes);  // sums across warps or blocks
    pdl_wait();
    pdl_trigger();

    // this block's share of K, in units, and its chunks
    const int units = (a.K + kUnit - 1) / kUnit;
    const int u0 = units * a.rank_of(blockIdx.x) / a.split, u1 = units * (a.rank_of(blockIdx.x) + 1) / a.split;
    const int nchunk = (u1 - u0 + cu - 1) / cu;
    const int first_block = blockIdx.x / a.split, row_step = gridDim.x / a.split;
    const int row_blocks = (a.N + 16 * RW - 1) / (16 * RW);

    // this warp's share of a chunk: units [from, to)
    auto share = [&](int ch, int &from, int &to) {
        const int n = min(cu, u1 - u0 - ch * cu);
        from = u0 + ch * cu + n * kw / KW;
        to = u0 + ch * cu + n * (kw + 1) / KW;
    };
    // the requests run ahead through the same units: block of rows, chunk, unit
    // and end of the share, and this lane's sources.  Lane l copies the 16-byte
    // pieces l and l + 32 of the codes' [16 rows][4 pieces], and row l % 16's
    // scales (lanes 0-15) or biases
    const int ldw = a.K / 8;
    int n_rb = first_block, n_ch = 0, n_u, n_to;
    share(0, n_u, n_to);
    const uint32_t *n_q = nullptr;
    const uint16_t *n_s = nullptr;
    bool n_row0 = false, n_row1 = false, n_srow = false;
    auto aim = [&]() {
        const int row = (n_rb * RW + rw) * 16;
        const int r = row + (lane >> 2), rs = row + (lane & 15);
        n_row0 = r < a.N;
        n_row1 = r + 8 < a.N;
        n_srow = rs < a.N;
        n_q = a.q + static_cast<int64_t>(n_row0 ? r : 0) * ldw + n_u * (kUnit / 8) + 4 * (lane & 3);
        n_s = (lane < 16 ? a.s : a.b) + static_cast<int64_t>(n_srow ? rs : 0) * a.ldg;
    };
    aim();
    uint32_t d_q, d_s;  // destinations in a stage
    {
        const int r = lane >> 2, sw = ((r >> 1) & 1) * 2 + ((r >> 2) & 1);
        d_q = ring + r * 64 + (((lane & 3) ^ sw) << 4);
        d_s = ring + kNibBytes + (lane >> 4) * kScaleBytes + (lane & 15) * 8;
    }
    auto issue = [&](int st) {
        while (n_u == n_to) {  // the share is through: the next chunk, the next block of rows
            if (n_rb >= row_blocks) return;
            if (++n_ch == nchunk) {
                n_ch = 0;
                n_rb += row_step;
                if (n_rb >= row_blocks) return;
            }
            share(n_ch, n_u, n_to);
            aim();
        }
        const bool k_ok = n_u * kUnit + 32 * (lane & 3) < a.K;
        cp_async_n(d_q + st * kStageBytes, n_q, 16, n_row0 && k_ok);
        cp_async_n(d_q + st * kStageBytes + 8 * 64, n_row1 ? n_q + 8 * static_cast<int64_t>(ldw) : n_q, 16, n_row1 && k_ok);
        cp_async_n(d_s + st * kStageBytes, n_s + (GPU_ == 1 ? n_u & ~1 : n_u * GPU_), SB, n_srow);
        n_q += kUnit / 8;
        ++n_u;
    };
#pragma unroll
    for (int i = 0; i < kLinStages - 1; ++i) {
        issue(i);
        cp_async_commit();
    }

    // chunk ch of the tokens into a buffer (all copies in flight together), then
    // its group sums: a thread takes 16 bytes of a token row, the lanes of a
    // group add up their elements
    auto load_x = [&](int ch, int buf) {
        const int k0 = (u0 + ch * cu) * kUnit;
        const int n = min(cu, u1 - u0 - ch * cu) * (kUnit / 8);  // 16-byte pieces of a row, a multiple of 16
        uint8_t *xd = xbuf + buf * xbytes;
        float *gd = reinterpret_cast<float *>(gbuf + buf * gbytes);
        for (int t = warp; t < a.B; t += kLinWarps)
            for (int p = lane; p < n; p += 32)
                cp_async_n(smem_u32(xd + t * xpitch + p * 16), a.x + t * a.x_stride + min(k0 + 8 * p, a.K - 8), 16,
                           k0 + 8 * p < a.K);
        cp_async_wait_all();
        __syncwarp();
        for (int t = warp; t < a.B; t += kLinWarps)
            for (int p = lane; p < n; p += 32) {
                const uint4 v = *reinterpret_cast<const uint4 *>(xd + t * xpitch + p * 16);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) sum += __uint_as_float(w[j] << 16) + __uint_as_float(w[j] & 0xFFFF0000u);
                const unsigned mask = 0xFFFFu << (lane & 16);  // 16 lanes are in or out together
#pragma unroll
                for (int off = 1; off < G / 8; off <<= 1) sum += __shfl_xor_sync(mask, sum, off);
                if (p % (G / 8) == 0) gd[(p / (G / 8)) * B8 + t] = sum;
            }
    };
    load_x(0, 0);
    __syncthreads();

    float y[NT][4];
    int st = 0, buf = 0;
    for (int rb = first_block; rb < row_blocks; rb += row_step) {
#pragma unroll
        for (int n = 0; n < NT; ++n) y[n][0] = y[n][1] = y[n][2] = y[n][3] = 0.f;
        for (int ch = 0; ch < nchunk; ++ch) {
            int from, to;
            share(ch, from, to);
            // (columns past the batch repeat its last token: they are not stored)
            const uint32_t xs = smem_u32(xbuf + buf * xbytes);
            uint32_t xrow[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) xrow[n] = xs + min(n * 8 + g8, a.B - 1) * xpitch;
            const float *gs = reinterpret_cast<const float *>(gbuf + buf * gbytes) + 2 * c;
            const int base = u0 + ch * cu;
            for (int u = from; u < to; ++u) {
                cp_async_wait<kLinStages - 2>();
                __syncwarp();
                const uint8_t *sp = smem + warp * kLinStages * kStageBytes + st * kStageBytes;
                const int ul = u - base;
#pragma unroll
                for (int gr = 0; gr < GPU_; ++gr) {
                    float d[NT][4];
#pragma unroll
                    for (int n = 0; n < NT; ++n) d[n][0] = d[n][1] = d[n][2] = d[n][3] = 0.f;
                    // the group's words of this thread: with groups of 32 word c of
                    // four, else words 2c, 2c + 1 of each eight (any order of k
                    // serves, as long as tokens and weights agree)
#pragma unroll
                    for (int part = 0; part < (G == 128 ? 2 : 1); ++part) {
                        constexpr int WPT = G == 32 ? 1 : 2;
                        const int w0 = G == 32 ? 4 * gr + c : 8 * (G == 128 ? part : gr) + 2 * c;  // word of the unit
                        uint32_t lo[WPT], hi[WPT];
                        {
                            const int sw = ((g8 >> 1) & 1) * 2 + ((g8 >> 2) & 1);
                            const uint8_t *at = sp + g8 * 64 + (((w0 >> 2) ^ sw) << 4) + (w0 & 3) * 4;
                            if constexpr (WPT == 1) {
                                lo[0] = *reinterpret_cast<const uint32_t *>(at);
                                hi[0] = *reinterpret_cast<const uint32_t *>(at + 8 * 64);
                            } else {
                                const uint2 l2 = *reinterpret_cast<const uint2 *>(at);
                                const uint2 h2 = *reinterpret_cast<const uint2 *>(at + 8 * 64);
                                lo[0] = l2.x;
                                lo[1] = l2.y;
                                hi[0] = h2.x;
                                hi[1] = h2.y;
                            }
                        }
#pragma unroll
                        for (int w = 0; w < WPT; ++w) {
                            uint32_t af[2][4];
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                af[j][0] = code_pair(lo[w], 2 * j);
                                af[j][1] = code_pair(hi[w], 2 * j);
                                af[j][2] = code_pair(lo[w], 2 * j + 1);
                                af[j][3] = code_pair(hi[w], 2 * j + 1);
                            }
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                uint32_t x0, x1, x2, x3;
                                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                             : "=r"(x0), "=r"(x1), "=r"(x2), "=r"(x3)
                                             : "r"(xrow[n] + ul * (kUnit * 2) + (w0 + w) * 16));
                                mma_16816(d[n], af[0], x0, x1);
                                mma_16816(d[n], af[1], x2, x3);
                            }
                        }
                    }
                    // the group's scale and bias of rows g8 and g8 + 8
                    const int gi = GPU_ == 1 ? (u & 1) : gr;
                    const uint32_t *ss = reinterpret_cast<const uint32_t *>(sp + kNibBytes + g8 * 8) + (gi >> 1);
                    auto pick = [&](uint32_t pair) {
                        return __uint_as_float((gi & 1) ? pair & 0xFFFF0000u : pair << 16);
                    };
                    const float s0 = pick(ss[0]), s1 = pick(ss[16]);
                    const float z0 = fmaf(-128.f, s0, pick(ss[kScaleBytes / 4]));
                    const float z1 = fmaf(-128.f, s1, pick(ss[kScaleBytes / 4 + 16]));
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float2 X = *reinterpret_cast<const float2 *>(gs + (ul * GPU_ + gr) * B8 + n * 8);
                        y[n][0] = fmaf(s0, d[n][0], fmaf(z0, X.x, y[n][0]));
                        y[n][1] = fmaf(s0, d[n][1], fmaf(z0, X.y, y[n][1]));
                        y[n][2] = fmaf(s1, d[n][2], fmaf(z1, X.x, y[n][2]));
                        y[n][3] = fmaf(s1, d[n][3], fmaf(z1, X.y, y[n][3]));
                    }
                }
                __syncwarp();  // the stage before this one has been read by every lane
                issue(st == 0 ? kLinStages - 1 : st - 1);
                cp_async_commit();
                st = st + 1 == kLinStages ? 0 : st + 1;
            }
            // the next chunk of tokens (of this block of rows, or the first of the
            // next one); a single one stays where it is
            if (nchunk > 1 && (ch + 1 < nchunk || rb + row_step < row_blocks)) {
                const int nb = a.x_buffers == 2 ? buf ^ 1 : buf;
                load_x(ch + 1 < nchunk ? ch + 1 : 0, nb);
                __syncthreads();
                buf = nb;
            }
        }

        // add up across the warps of a row tile and the blocks of the cluster:
        // [RW][KW][token][16 rows] (token-major, so that a token's rows are
        // stored side by side)
        const bool across = KW > 1 || a.split > 1;
        if (across) {
            float *dst = red + (rw * KW + kw) * (B8 * 16);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                dst[(n * 8 + 2 * c) * 16 + g8] = y[n][0];
                dst[(n * 8 + 2 * c + 1) * 16 + g8] = y[n][1];
                dst[(n * 8 + 2 * c) * 16 + g8 + 8] = y[n][2];
                dst[(n * 8 + 2 * c + 1) * 16 + g8 + 8] = y[n][3];
            }
            if (a.split > 1)
                cluster_sync();
            else
                __syncthreads();
            const int rank = a.rank_of(blockIdx.x);
            for (int i = tid + rank * kLinThreads; i < RW * B8 * 16; i += kLinThreads * a.split) {
                const int r = i % 16, t = i / 16 % B8, tile = i / (16 * B8);
                const int row = (rb * RW + tile) * 16 + r;
                float sum = 0.f;
                for (int sp = 0; sp < a.split; ++sp) {
                    const float *src = red + tile * KW * (B8 * 16) + t * 16 + r;
#pragma unroll
                    for (int w = 0; w < KW; ++w)
                        sum += a.split > 1 ? dsmem_ld(smem_u32(src + w * (B8 * 16)), sp) : src[w * (B8 * 16)];
                }
                if (t < a.B && row < a.N) a.store(t, row, sum);
            }
            if (a.split > 1)
                cluster_sync();
            else
                __syncthreads();
        } else {
            const int row = (rb * RW + rw) * 16 + g8;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = n * 8 + 2 * c + (e & 1), r = row + 8 * (e >> 1);
                    if (t < a.B && r < a.N) a.store(t, r, y[n][e]);
                }
        }
    }
    cp_async_wait<0>();
}

template <int G, int NT, int RW, int kLinStages>
static cudaError_t launch_s(LinearArgs a, int blocks, int smem, cudaStream_t s) {
    auto kernel = int4_linear_kernel<G, NT, RW, kLinStages>;
    const cudaError_t e = allow_smem<int4_linear_kernel<G, NT, RW, kLinStages>>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kLinThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int G, int NT, int RW>
static cudaError_t launch_t(LinearArgs a, int num_sms, cudaStream_t s) {
    constexpr int KW = kLinWarps / RW, B8 = NT * 8;
    const int units = (a.K + kUnit - 1) / kUnit;
    const int row_blocks = (a.N + 16 * RW - 1) / (16 * RW);
    // split K over a cluster while that leaves every warp two units and the
    // GPU is not yet full
    a.split = 1;
    while (a.split < 8 && row_blocks * a.split * 2 <= num_sms + num_sms / 4 && units / (a.split * 2) >= 2 * KW) a.split *= 2;
    const int share = (units + a.split - 1) / a.split;
    // all of the block's tokens if they fit, else two chunks that do
    const int per_unit = a.B * kUnit * 2 + B8 * (kUnit / G) * 4;
    constexpr int room = 96 * 1024;
    if (share * per_unit <= room) {
        a.chunk_units = share;
        a.x_buffers = 1;
    } else {
        a.chunk_units = room / 2 / per_unit / KW * KW;
        a.x_buffers = 2;
    }
    constexpr int XPAD = G == 32 ? 64 : 16;
    const int xbytes = a.B * (a.chunk_units * kUnit * 2 + XPAD), gbytes = a.chunk_units * (kUnit / G) * B8 * 4;
    const int red = KW > 1 || a.split > 1 ? RW * KW * B8 * 16 * 4 : 0;
    const int rest = a.x_buffers * (xbytes + gbytes) + red;
    // two blocks a SM if their rings fit with eight or four stages
    constexpr int half = 113 * 1024;
    const bool two8 = NT <= 2 && rest + ring_bytes(8) <= half, two4 = NT <= 2 && rest + ring_bytes(4) <= half;
    const int per_sm = two8 || two4 ? 2 : 1;
    const int groups = std::min(row_blocks, num_sms * per_sm / a.split);
    if (two4 && !two8) return launch_s<G, NT, RW, 4>(a, groups * a.split, rest + ring_bytes(4), s);
    return launch_s<G, NT, RW, 8>(a, groups * a.split, rest + ring_bytes(8), s);
}

template <int G>
static cudaError_t launch_g(const LinearArgs &a, int num_sms, cudaStream_t s) {
    if (a.B <= 16) return launch_t<G, 2, 8>(a, num_sms, s);
    if (a.B <= 32) return launch_t<G, 4, 8>(a, num_sms, s);
    return launch_t<G, 8, 8>(a, num_sms, s);
}

cudaError_t launch_linear(const LinearArgs &a, int num_sms, cudaStream_t s) {
    if (a.B <= kFewTokens) return launch_linear_few(a, num_sms, s);
    if (a.G == 32) return launch_g<32>(a, num_sms, s);
    if (a.G == 64) return launch_g<64>(a, num_sms, s);
    return launch_g<128>(a, num_sms, s);
}

}  // namespace moe
