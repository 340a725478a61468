// y[b][n] = sum_k x[b][k] (s[n][k/G] q[n][k] + z[n][k/G]) for up to 8 tokens: a
// read of the weights at memory speed, so the arithmetic has to stay within
// about three instructions a weight and lane (47 weights a clock and SM).
//
// The codes are unpacked to fp16 rather than bf16: set below the exponent of
// 1024, a nibble at bits 0-3 of a half is 1024 + q and one at bits 4-7 is
// 1024 + 16 q (bf16's mantissa is too short for that), so that eight codes take
// one shift and four mask-and-sets on the ALU, which is what bounds this kernel;
// one fused multiply-add a pair, on the other pipe, leaves q exactly.  (Unpacked
// to bf16 pairs: 74 us for 131072 x 4096, whose bytes take 42; as fp8 bytes with
// mma.sync e4m3 x e5m2, which this GPU expands to fp16 by itself: 59.)
// The token is made fp16 exactly as well: scaled by a power of two, so that the
// largest element of the block's share lies in [2^14, 2^15), the 8 significant bits of an element fit
// unless it is below 2^-31 of the largest, and then it is off by 2^-40 of that.
// mma.sync m16n8k16 multiplies and adds in fp32.  Per group of weights, with
// D = sum q x 2^e and X = 2^e sum x,
//   y 2^e += s D + z X
// and no weight is rounded.  The M = 16 of an MMA is 16 weight rows, its N = 8
// the tokens.
//
// A block of eight warps takes RW tiles of 16 rows, KW = 8 / RW warps share the
// k of a tile: one or two tiles for few rows (2048 rows occupy 128 SMs), eight for
// many (no sums across warps then) or for long tokens.  If there are too few rows for the GPU, a
// cluster of up to eight blocks shares K and adds up through distributed
// shared memory.  Each warp streams its weights through its own ring of
// cp.async stages (16 rows x 256 k and their scales).  The tokens as fp16 and
// their group sums are made once per block if they fit in shared memory, else
// chunk by chunk for each block of rows.
//
// Measured, calls: 131072 x 4096 with one token 56 us, 5.1 TB/s of the 285 MB (ALU
// 51 %, issue 66 % of their peaks; eight warps a SM and more in flight gain
// nothing); 2560 x 2048 with one token 4.0 us and 2048 x 2048 with eight 5.1, which
// is the tokens' way through shared memory, the ring's first stages and the cluster's
// sum.
#include <cuda_fp16.h>

#include <algorithm>

#include "linear.cuh"

namespace moe {
namespace few {

constexpr int kUnit = 256;                        // k of a stage
constexpr int kRowBytes = kUnit / 2;              // codes of a row in a stage
constexpr int kScaleRow = 16;                     // up to eight groups a row
constexpr int kStageBytes = 16 * (kRowBytes + 2 * kScaleRow);
__host__ __device__ constexpr int stages(int warps) { return warps == 16 ? 3 : 4; }
__host__ __device__ constexpr int ring_bytes(int warps) { return warps * stages(warps) * kStageBytes; }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void cp_async_scales(uint32_t dst, const void *src) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}

__device__ __forceinline__ uint32_t lds32(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
    return v;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The eight codes of a word as fp16 pairs (0 1), (2 3), (4 5), (6 7).
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t (&q)[4]) {
    const __half2 low = __half2half2(__ushort_as_half(0x6400));          // 1024
    const __half2 sixteenth = __half2half2(__ushort_as_half(0x2C00));    // 1/16
    const __half2 minus64 = __half2half2(__ushort_as_half(0xD400));      // -64
    const uint32_t v = w >> 8;
    const uint32_t t[4] = {mask_set(w, 0x000F000Fu, 0x64006400u), mask_set(w, 0x00F000F0u, 0x64006400u),
                           mask_set(v, 0x000F000Fu, 0x64006400u), mask_set(v, 0x00F000F0u, 0x64006400u)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = *reinterpret_cast<const __half2 *>(&t[i]);
        const __half2 r = i & 1 ? __hfma2(h, sixteenth, minus64) : __hsub2(h, low);
        q[i] = *reinterpret_cast<const uint32_t *>(&r);
    }
}

constexpr int kMaxSmem = 226 * 1024, kHalfSmem = 113 * 1024;  // a SM's, and what lets two blocks share it

// Shared memory after the rings.
struct Map {
    int pitch, xbytes, gbytes, red, total;  // bytes of a token's row, of the tokens, of the group sums
};

template <int G, int WARPS, int RW>
__host__ __device__ inline Map smem_map(int B, int units, int split) {
    Map m{};
    // token rows start 16 (groups of 32: 64) bytes apart modulo 128: the lanes'
    // reads fall on different banks
    m.pitch = units * kUnit * 2 + (G == 32 ? 64 : 16);
    m.xbytes = B * m.pitch;
    m.gbytes = units * (kUnit / G) * 8 * 4;
    m.red = RW == WARPS && split == 1 ? 0 : WARPS * 8 * 16 * 4;
    m.total = ring_bytes(WARPS) + m.xbytes + m.gbytes + m.red + 64;
    return m;
}

template <int G, int WARPS, int RW>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS) linear_few_kernel(const LinearArgs a) {
    constexpr int KW = WARPS / RW, kThreads = WARPS * 32, kStages = stages(WARPS);
    constexpr int GU = kUnit / G;                 // groups of a unit
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g8 = lane >> 2, c = lane & 3;
    const int rw = warp % RW, kw = warp / RW;
    const uint32_t ring = smem_u32(smem) + warp * kStages * kStageBytes;
    const int cu = a.chunk_units;
    const Map map = smem_map<G, WARPS, RW>(a.B, cu, a.split);
    uint8_t *xbuf = smem + ring_bytes(WARPS);     // [token] rows of fp16
    float *gbuf = reinterpret_cast<float *>(xbuf + map.xbytes);                // [group][8 tokens]
    float *red = reinterpret_cast<float *>(xbuf + map.xbytes + map.gbytes);    // [RW][KW][token][16 rows]
    int *s_top = reinterpret_cast<int *>(xbuf + map.xbytes + map.gbytes + map.red);  // [token] largest |x| as bf16 bits
    int *s_exp = s_top + 8;                        // [token] exponent of its scale
    pdl_wait();
    pdl_trigger();

    const int units = (a.K + kUnit - 1) / kUnit;
    const int rank = a.rank_of(blockIdx.x);
    const int u0 = units * rank / a.split, u1 = units * (rank + 1) / a.split;
    const int nchunk = (u1 - u0 + cu - 1) / cu;
    const int first_block = blockIdx.x / a.split, row_step = gridDim.x / a.split;
    const int row_blocks = (a.N + 16 * RW - 1) / (16 * RW);

    // this warp's share of a chunk: units [from, to)
    auto share = [&](int ch, int &from, int &to) {
        const int n = min(cu, u1 - u0 - ch * cu);
        from = u0 + ch * cu + n * kw / KW;
        to = u0 + ch * cu + n * (kw + 1) / KW;
    };
    // the requests run ahead through the same units.  Lane l copies piece l % 8
    // (16 bytes) of the codes' rows l / 8, + 4, + 8, + 12, and row l % 16's
    // scales (lanes 0-15) or biases.  Piece p of row r lies at
    // p ^ (2 (r & 3) + (r >> 2 & 1)): the pairs of pieces that a fragment load of
    // four rows meets, and the single ones of eight rows, fall on different banks
    const int ldw = a.K / 8;
    int n_rb = first_block, n_ch = 0, n_u, n_to;
    share(0, n_u, n_to);
    const uint32_t *n_q[4];
    const uint16_t *n_s = nullptr;
    auto aim = [&]() {
        const int row = (n_rb * RW + rw) * 16;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            n_q[i] = a.q + static_cast<int64_t>(min(row + (lane >> 3) + 4 * i, a.N - 1)) * ldw + n_u * (kUnit / 8) +
                     4 * (lane & 7);
        n_s = (lane < 16 ? a.s : a.b) + static_cast<int64_t>(min(row + (lane & 15), a.N - 1)) * a.ldg + n_u * GU;
    };
    aim();
    // rows l / 8 and l / 8 + 4 (and + 8, + 12 alike)
    const uint32_t d_q0 = ring + (lane >> 3) * kRowBytes + (((lane & 7) ^ 2 * (lane >> 3)) << 4);
    const uint32_t d_q1 = ring + ((lane >> 3) + 4) * kRowBytes + (((lane & 7) ^ (2 * (lane >> 3) + 1)) << 4);
    const uint32_t d_s = ring + 16 * kRowBytes + (lane >> 4) * 16 * kScaleRow + (lane & 15) * kScaleRow;
    auto issue = [&](uint32_t off) {
        if (n_u == n_to) {  // the share is through: the next chunk, the next block of rows
            do {
                if (n_rb >= row_blocks) return;
                if (++n_ch == nchunk) {
                    n_ch = 0;
                    n_rb += row_step;
                    if (n_rb >= row_blocks) return;
                }
                share(n_ch, n_u, n_to);
            } while (n_u == n_to);
            aim();
        }
        // rows past the last one repeat it (they are not stored); k past the end
        // are zero codes (the last unit only)
        if ((n_u + 1) * kUnit <= a.K) {
#pragma unroll
            for (int i = 0; i < 4; ++i) cp_async16((i & 1 ? d_q1 : d_q0) + (i >> 1) * 8 * kRowBytes + off, n_q[i]);
        } else {
            const bool ok = n_u * kUnit + 32 * (lane & 7) < a.K;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                cp_async16_zfill((i & 1 ? d_q1 : d_q0) + (i >> 1) * 8 * kRowBytes + off, ok ? n_q[i] : a.q, ok);
        }
        cp_async_scales<GU * 2>(d_s + off, n_s);
#pragma unroll
        for (int i = 0; i < 4; ++i) n_q[i] += kUnit / 8;
        n_s += GU;
        ++n_u;
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
        issue(i * kStageBytes);
        cp_async_commit();
    }

    // The tokens as fp16, scaled by a power of two each that this block's share of k
    // alone decides (the sums leave the block at their own scale): a thread
    // takes eight k of a token at a time.
    const int shift = 14 + 127;  // x 2^e: the largest element to [2^14, 2^15); 2^e and 2^-e stay normal
    auto exponent = [&](int top) { return top == 0 ? 0 : max(-112, min(126, shift - (top >> 7))); };
    auto largest = [&](const uint4 &v) {  // largest |x| as bf16 bits (NaN and infinity above all)
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) top = max(top, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
        return top;
    };
    // piece p (of n, a multiple of 32) of token t of a chunk, and the group sums: the
    // lanes of a group add up their elements
    auto convert = [&](int t, int p, const uint4 &v, int exp) {
        const float up = __uint_as_float(static_cast<uint32_t>(exp + 127) << 23);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t h[4];
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float f0 = __uint_as_float(w[j] << 16) * up, f1 = __uint_as_float(w[j] & 0xFFFF0000u) * up;
            const __half2 hh = __floats2half2_rn(f0, f1);
            h[j] = *reinterpret_cast<const uint32_t *>(&hh);
            sum += f0 + f1;
        }
        *reinterpret_cast<uint4 *>(xbuf + t * map.pitch + p * 16) = make_uint4(h[0], h[1], h[2], h[3]);
        // (all 32 lanes: n is a multiple of 32)
#pragma unroll
        for (int off = 1; off < G / 8; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (p % (G / 8) == 0) gbuf[(p / (G / 8)) * 8 + t] = sum;
    };
    auto piece = [&](int t, int k) {
        return k < a.K ? *reinterpret_cast<const uint4 *>(a.x + t * a.x_stride + k) : make_uint4(0u, 0u, 0u, 0u);
    };
    auto load_x = [&](int ch) {
        const int k0 = (u0 + ch * cu) * kUnit;
        const int n = min(cu, u1 - u0 - ch * cu) * (kUnit / 8);
#pragma unroll 4
        for (int i = tid; i < a.B * n; i += kThreads) {
            const int t = i / n, p = i - t * n;
            convert(t, p, piece(t, k0 + 8 * p), s_exp[t]);
        }
        __syncthreads();
    };
    {
        // the largest elements, by as many warps a token as there are
        constexpr int kHeld = 8;  // pieces that a lane keeps between the two passes
        const int k0 = u0 * kUnit, n = (u1 - u0) * (kUnit / 8);
        const int wpt = WARPS / a.B, t = warp / wpt, step = wpt * 32, p0 = warp % wpt * 32 + lane;  // 1 or more: at most 8 tokens
        // (one piece has a way of its own: the other's code, not yet in the
        // instruction cache, costs one token 0.4 of 4.3 us)
        const bool one = nchunk == 1 && n <= step, held = nchunk == 1 && n <= kHeld * step;
        if (tid < 8) s_top[tid] = s_exp[tid] = 0;
        __syncthreads();
        uint4 v[kHeld];
        uint32_t top = 0;
        if (t < a.B) {
            if (one) {
                v[0] = p0 < n ? piece(t, k0 + 8 * p0) : make_uint4(0u, 0u, 0u, 0u);
                top = largest(v[0]);
            } else if (held) {
#pragma unroll
                for (int j = 0; j < kHeld; ++j) v[j] = p0 + j * step < n ? piece(t, k0 + 8 * (p0 + j * step)) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int j = 0; j < kHeld; ++j) top = max(top, largest(v[j]));
            } else {
#pragma unroll 4
                for (int p = p0; p < n; p += step) top = max(top, largest(piece(t, k0 + 8 * p)));
            }
            top = __reduce_max_sync(0xffffffffu, top);
            if (lane == 0) atomicMax(&s_top[t], static_cast<int>(top));
        }
        __syncthreads();
        const int exp = t < a.B ? exponent(s_top[t]) : 0;
        if (t < a.B && p0 == 0) s_exp[t] = exp;
        if (one) {
            if (t < a.B && p0 < n) convert(t, p0, v[0], exp);
            __syncthreads();
        } else if (held) {
            if (t < a.B) {
#pragma unroll
                for (int j = 0; j < kHeld; ++j)
                    if (p0 + j * step < n) convert(t, p0 + j * step, v[j], exp);
            }
            __syncthreads();
        } else {
            __syncthreads();
            load_x(0);
        }
    }

    // the B operand's row of this lane (columns past the batch repeat its last
    // token: they are not stored)
    const uint32_t xrow = smem_u32(xbuf) + min(g8, a.B - 1) * map.pitch;
    // this lane's places in a stage: rows g8 and g8 + 8 of each 64 k (groups of
    // 32: of each group), and the rows' scales
    uint32_t at_q[kUnit / (G == 32 ? 32 : 64)];
#pragma unroll
    for (int i = 0; i < kUnit / (G == 32 ? 32 : 64); ++i) {
        const int sw = 2 * (g8 & 3) + (g8 >> 2);
        at_q[i] = ring + g8 * kRowBytes +
                  (G == 32 ? ((i ^ sw) << 4) + c * 4 : (((2 * i + (c >> 1)) ^ sw) << 4) + (c & 1) * 8);
    }
    const uint32_t at_s = ring + 16 * kRowBytes + g8 * kScaleRow;
    uint32_t st = 0, refill = (kStages - 1) * kStageBytes;  // stages read and requested next, as offsets
    for (int rb = first_block; rb < row_blocks; rb += row_step) {
        float y[4] = {0.f, 0.f, 0.f, 0.f};
        for (int ch = 0; ch < nchunk; ++ch) {
            if (nchunk > 1 && (rb != first_block || ch > 0)) {
                __syncthreads();  // every warp is done with the previous chunk
                load_x(ch);
            }
            int from, to;
            share(ch, from, to);
            const int base = u0 + ch * cu;
            for (int u = from; u < to; ++u) {
                cp_async_wait<kStages - 2>();
                __syncwarp();
                const uint32_t xo = xrow + (u - base) * (kUnit * 2);
                const float *gs = gbuf + (u - base) * (GU * 8) + 2 * c;
                constexpr int kRow8 = 8 * kScaleRow, kBias = 16 * kScaleRow;
#pragma unroll
                for (int gr = 0; gr < GU; ++gr) {
                    float d[4] = {0.f, 0.f, 0.f, 0.f};
                    auto words = [&](uint32_t lo, uint32_t hi, int w0) {
                        uint32_t ql[4], qh[4], x0, x1, x2, x3;
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(x0), "=r"(x1), "=r"(x2), "=r"(x3)
                                     : "r"(xo + w0 * 16));
                        unpack8(lo, ql);
                        unpack8(hi, qh);
                        const uint32_t a0[4] = {ql[0], qh[0], ql[1], qh[1]}, a1[4] = {ql[2], qh[2], ql[3], qh[3]};
                        mma_f16(d, a0, x0, x1);
                        mma_f16(d, a1, x2, x3);
                    };
                    if constexpr (G == 32) {
                        // word c of the group's four
                        words(lds32(at_q[gr] + st), lds32(at_q[gr] + st + 8 * kRowBytes), 4 * gr + c);
                    } else {
                        // words 2c, 2c + 1 of each eight (any order of k serves, as
                        // long as tokens and weights agree)
#pragma unroll
                        for (int blk = 0; blk < G / 64; ++blk) {
                            const int k64 = gr * (G / 64) + blk;  // which 64 k of the unit
                            const uint2 lo = lds64(at_q[k64] + st), hi = lds64(at_q[k64] + st + 8 * kRowBytes);
                            words(lo.x, hi.x, 8 * k64 + 2 * c);
                            words(lo.y, hi.y, 8 * k64 + 2 * c + 1);
                        }
                    }
                    // the group's scale and bias of rows g8 and g8 + 8
                    auto pick = [&](uint32_t pair) {
                        return __uint_as_float((gr & 1) ? pair & 0xFFFF0000u : pair << 16);
                    };
                    const uint32_t as = at_s + st + (gr / 2) * 4;
                    const float s0 = pick(lds32(as)), s1 = pick(lds32(as + kRow8));
                    const float z0 = pick(lds32(as + kBias)), z1 = pick(lds32(as + kBias + kRow8));
                    const float2 X = *reinterpret_cast<const float2 *>(gs + gr * 8);
                    y[0] = fmaf(s0, d[0], fmaf(z0, X.x, y[0]));
                    y[1] = fmaf(s0, d[1], fmaf(z0, X.y, y[1]));
                    y[2] = fmaf(s1, d[2], fmaf(z1, X.x, y[2]));
                    y[3] = fmaf(s1, d[3], fmaf(z1, X.y, y[3]));
                }
                __syncwarp();  // the stage before this one has been read by every lane
                issue(refill);
                cp_async_commit();
                refill = st;
                st = st == (kStages - 1) * kStageBytes ? 0 : st + kStageBytes;
            }
        }

        // 2^-e
        auto down = [&](int t) { return __uint_as_float(static_cast<uint32_t>(127 - s_exp[t]) << 23); };
        if (RW < WARPS || a.split > 1) {
            // add up the warps of a row tile and the blocks of the cluster
            float *dst = red + (rw * KW + kw) * (8 * 16);
            const float d0 = down(2 * c), d1 = down(2 * c + 1);
            dst[(2 * c) * 16 + g8] = y[0] * d0;
            dst[(2 * c + 1) * 16 + g8] = y[1] * d1;
            dst[(2 * c) * 16 + g8 + 8] = y[2] * d0;
            dst[(2 * c + 1) * 16 + g8 + 8] = y[3] * d1;
            if (a.split > 1)
                cluster_sync();
            else
                __syncthreads();
            for (int i = tid + rank * kThreads; i < RW * a.B * 16; i += kThreads * a.split) {
                const int r = i % 16, t = i / 16 % a.B, tile = i / (16 * a.B);
                const int row = (rb * RW + tile) * 16 + r;
                float sum = 0.f;
                for (int sp = 0; sp < a.split; ++sp) {
#pragma unroll
                    for (int w = 0; w < KW; ++w) {
                        const float *src = red + (tile * KW + w) * (8 * 16) + t * 16 + r;
                        sum += a.split > 1 ? dsmem_ld(smem_u32(src), sp) : *src;
                    }
                }
                if (row < a.N) a.store(t, row, sum);
            }
            if (a.split > 1)
                cluster_sync();
            else
                __syncthreads();
        } else {
            const int row = (rb * RW + rw) * 16 + g8;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = 2 * c + (e & 1), r = row + 8 * (e >> 1);
                if (t < a.B && r < a.N) a.store(t, r, y[e] * down(t));
            }
        }
    }
    cp_async_wait<0>();
}

template <int G, int WARPS, int RW>
static cudaError_t launch_t(LinearArgs a, int num_sms, cudaStream_t s) {
    constexpr int KW = WARPS / RW;
    const int units = (a.K + kUnit - 1) / kUnit;
    const int row_blocks = (a.N + 16 * RW - 1) / (16 * RW);
    // share K in a cluster while that leaves every warp a unit and the GPU is
    // not yet full (clusters of other numbers than powers of two measured slower:
    // they find fewer places)
    const int most = RW == WARPS ? num_sms : num_sms + num_sms / 4;
    a.split = 1;
    while (a.split < 8 && row_blocks * a.split * 2 <= most && units / (a.split * 2) >= KW) a.split *= 2;
    // all of the block's tokens at once if that leaves room for them
    a.chunk_units = (units + a.split - 1) / a.split;
    while (smem_map<G, WARPS, RW>(a.B, a.chunk_units, a.split).total > kMaxSmem) a.chunk_units = (a.chunk_units + 1) / 2;
    const int smem = smem_map<G, WARPS, RW>(a.B, a.chunk_units, a.split).total;
    const int per_sm = smem <= kHalfSmem && WARPS == 8 ? 2 : 1;
    const int groups = std::min(row_blocks, std::max(1, num_sms * per_sm / a.split));
    auto kernel = linear_few_kernel<G, WARPS, RW>;
    const cudaError_t e = allow_smem<linear_few_kernel<G, WARPS, RW>>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(groups * a.split);
    cfg.blockDim = dim3(WARPS * 32);
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

template <int G>
static cudaError_t launch_g(const LinearArgs &a, int num_sms, cudaStream_t s) {
    // row tiles a block.  A block converts all tokens of its k, so that many or
    // long tokens take eight tiles a block and share K among more blocks instead
    // (8 tokens 4096 -> 4096: one tile 10.6 us, two 10.2, eight 7.1; 8192 -> 4096:
    // 19, 19, 10).  Else one if all blocks run at once, two if they do then, and
    // eight for many rows (one token 2048 -> 3500, 6000, 16384: one tile 4.0, 5.7,
    // 10.2; two 3.9, 5.4, 8.7; eight 4.5, 5.8, 7.4).  (The border for long tokens: 131
    // rows of 8 x 32768 eight 17, one 10.7; 700 of 8 x 16384 and 8 x 32768 eight 10.0 and
    // 17.2, one 18.4 and 31; 700 of 8 x 4096 6.1 and 6.2; 700 of 1 x 8192 6.3 and 5.2.)
    //
    // A block of sixteen warps converts a chunk of the tokens for twice the rows: for
    // very many rows whose tokens do not fit at once (80000 rows, 8 x 16384 in groups
    // of 32 and 64: 294 and 330 us with eight warps, 247 and 235 with sixteen; 8 x
    // 32768: 598, 490).  Where they do, sixteen are slower (4 x 16384: 192 and 222,
    // 8 x 4096: 51 and 54, 1 x 32768: 329 and 585), and so they are in groups of 128
    // (6 x 32768: 515 and 628)
    const int tiles = (a.N + 15) / 16, units = (a.K + kUnit - 1) / kUnit;
    const int whole = smem_map<G, 8, 8>(a.B, units, 1).total;
    if constexpr (G < 128)
        if (tiles >= 8 * 4 * num_sms && whole > kMaxSmem) return launch_t<G, 16, 16>(a, num_sms, s);
    const int slots = num_sms * (whole <= kHalfSmem ? 2 : 1);
    const bool tokens = a.B * a.K >= 8192 && tiles >= num_sms / 4;
    if (tokens || tiles > 2 * slots) return launch_t<G, 8, 8>(a, num_sms, s);
    if (tiles > slots) return launch_t<G, 8, 2>(a, num_sms, s);
    return launch_t<G, 8, 1>(a, num_sms, s);
}

}  // namespace few

cudaError_t launch_linear_few(const LinearArgs &a, int num_sms, cudaStream_t s) {
    if (a.G == 32) return few::launch_g<32>(a, num_sms, s);
    if (a.G == 64) return few::launch_g<64>(a, num_sms, s);
    return few::launch_g<128>(a, num_sms, s);
}

}  // namespace moe
