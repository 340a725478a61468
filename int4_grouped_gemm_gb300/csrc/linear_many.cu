// y[b][n] = sum_k x[b][k] (s[n][k/G] q[n][k] + z[n][k/G]) for 9 to 64 tokens on the
// fifth-generation tensor cores.
//
// As with few tokens no weight is rounded: the codes themselves, exact in bf16
// as q 2^-12 (128 + q by a shift and a mask-and-set a pair, then one fused
// multiply-add), are the M = 128 side of tcgen05.mma, the tokens as they are the N
// side, and each group of weights has a sum of its own, D = sum q x 2^-12 (the
// power keeps it finite for any finite token); then, in fp32 registers,
//   y += (2^12 s) D
// (With 128 + q as the operand and z - 128 s for z, D is 17 times as large and y
// off by 2e-6 instead of 2e-7.)  The codes go straight into tensor memory, where
// the MMA reads its first operand from: a thread unpacks one row's 128 codes in
// registers and stores them to its lane.  What is in shared memory is only what
// TMA brings (packed codes, scales, tokens) and the token sums.
//
// The biases are a small product of their own, sum_g z[n][g] X[b][g] with
// X = sum of the group's x: for each 16 groups (a chunk) the row's 16 biases,
// copied to tensor memory as they are, times X as three bf16 parts (24 bits), three MMAs
// of K = 16 (and a fourth for sums that bf16 cannot hold).  X is the same
// for every tile of rows, so that it is made once per block, while the first
// tile's tokens pass by, where shared memory has room for all its chunks.  (With
// X from a row of ones in every tile and one multiply-add more a value, the
// epilogue's shuffles set the pace: 64 x 2048 x 131072 took 94 us.)
//
//   epilogue     warps 0-7, warp w: rows 32 (w % 4) .., token half w / 4: D from
//                tensor memory, y in registers
//   unpacking    warps 8-15, a thread per row, two sets of four in turn
//   16, 17, 18   loads of weights, MMA, loads of tokens
//   token sums   warps 20-23
//
// A barrier wait costs its role about 130 cycles however early the other side
// was, so the work goes in steps of 64 to 256 k and all that a
// step's MMAs need comes in on one barrier (`ready`: tokens by TMA, codes from
// the unpacking warps, the buffer of sums given back by the epilogue), all that
// waits for them on one other (`done`).
//
// Measured, calls: 64 x 2048 x 131072 59.5 us, 577 TFLOP/s and 2.8 TB/s, 16 x 4096 x
// 32768 29.3 us, 37 x 2080 x 5003 12.1.  Neither the tensor pipe (27 % busy) nor the bytes
// bound it, but a step's round through the roles, whose warps share the issue
// slots (65 % of them used).
//
// Blocks take tiles of 128 rows in turn.  If there are too few tiles for the
// GPU, a cluster of up to eight blocks shares K and adds up through distributed
// shared memory.  Every wait is bounded.
#include <algorithm>

#include "linear.cuh"

namespace moe {
namespace many {

constexpr int kRows = 128;                 // weight rows of a tile
constexpr int kEpiWarps = 8, kDeqWarp = 8, kWWarp = 16, kMmaWarp = 17, kXWarp = 18, kSumWarp = 20, kSumWarps = 4;
constexpr int kThreads = 24 * 32;
// Registers a thread: an epilogue thread of 64 tokens holds 32 sums and 64 of D.
// The launch gives 80 to each of the 768 threads (61,440 in all); epilogue,
// unpacking and the rest then hold 120, 64 and 56 (30,720 + 16,384 + 14,336).
constexpr int kLaunchRegs = 80, kEpiRegs = 120, kDeqRegs = 64, kRestRegs = 56;
static_assert(256 * kEpiRegs + 256 * kDeqRegs + 256 * kRestRegs <= kThreads * kLaunchRegs, "shares of the launch's registers");
constexpr int kMaxW = 6, kS = 2;           // stages: codes (at most), scales (a chunk of 16 groups)
constexpr int kX = 6, kA = 2;              // stages: tokens in shared memory, codes in tensor memory
constexpr int kD = 2;                      // buffers of a step's group sums
constexpr int kChunk = 16, kC = 8;         // groups of a chunk, chunks of token sums in shared memory
constexpr int kSBytes = 128 * kChunk * 2;
// k of a step: the longer, the fewer waits; tensor memory has to hold two steps'
// codes (a column for each two k) and group sums.
__host__ __device__ constexpr int step_k(int G, int tok) {
    return tok == 16 ? (G == 32 ? 128 : 256) : tok == 32 ? (G == 128 ? 256 : 128) : (G == 32 ? 64 : 128);
}
// Columns: group sums, codes, the bias products, a chunk's biases (2 x 8).
__host__ __device__ constexpr int d_cols(int G, int tok) { return step_k(G, tok) / G * tok; }
__host__ __device__ constexpr int tmem_cols(int G, int tok) { return kD * d_cols(G, tok) + kA * step_k(G, tok) / 2 + tok + 16; }
constexpr uint32_t kTmemCols = 512;
static_assert(tmem_cols(32, 16) <= 512 && tmem_cols(64, 16) <= 512 && tmem_cols(128, 16) <= 512 && tmem_cols(32, 32) <= 512 &&
                  tmem_cols(64, 32) <= 512 && tmem_cols(128, 32) <= 512 && tmem_cols(32, 64) <= 512 &&
                  tmem_cols(64, 64) <= 512 && tmem_cols(128, 64) <= 512,
              "tensor memory");
__host__ __device__ constexpr int w_bytes(int G, int tok) { return 128 * step_k(G, tok) / 2; }
__host__ __device__ constexpr int x_bytes(int G, int tok) { return step_k(G, tok) / 64 * tok * 128; }  // boxes of 64 k
// stages of codes: about 48 KB
__host__ __device__ constexpr int w_stages(int G, int tok) { return step_k(G, tok) == 256 ? 4 : 6; }

struct Ctl {
    uint64_t w_full[kMaxW], w_empty[kMaxW], s_full[kS], s_empty[kS];
    uint64_t ready[kX], done[kX];          // a step's operands and sums are there; its MMAs are complete
    uint64_t z_full;                       // a chunk's biases are in tensor memory, its products' place is free
    uint64_t sums_full[kC], x_read[kX];    // a chunk's token sums are there; a stage of tokens has been added up
    uint64_t drain;
    uint32_t tmem;
    int abort;
};

// More than half of a SM's: one block at a time, since each takes all of the
// tensor memory.
__host__ __device__ constexpr int smem_bytes(int G, int tok) {
    constexpr int least = kBlockSmem / 2 + 1024;
    const int n = kX * x_bytes(G, tok) + w_stages(G, tok) * w_bytes(G, tok) + kS * 2 * kSBytes + kC * tok * 128 +
                  static_cast<int>(sizeof(Ctl)) + 1024;
    return n > least ? n : least;
}
static_assert(smem_bytes(64, 64) <= kBlockSmem, "one block per SM");
static_assert(kX * x_bytes(32, 64) >= 64 * 128 * 4 && kX * x_bytes(32, 32) >= 32 * 128 * 4 &&
                  kX * x_bytes(32, 16) >= 16 * 128 * 4,
              "the cluster's sums lie over the tokens");

struct Maps {
    CUtensorMap q, s, b, x;
};

__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, const LinearArgs &a, Ctl *s, int site) {
    return role_wait(bar, parity, a.wait_limit, a.status, &s->abort, site);
}

__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const LinearArgs &a, Ctl *s, int site) {
    return __all_sync(0xffffffffu, wait(bar, parity, a, s, site));
}

// By predicate, without a branch.
__device__ __forceinline__ void first_lane_arrives(int lane, uint64_t *bar) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %1, 0;\n\t@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(
                     smem_u32(bar)),
                 "r"(lane)
                 : "memory");
}

// Shared memory by its own address: through a plain pointer these become generic
// accesses, with several times the latency.
__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void sts16(uint32_t at, uint16_t v) {
    asm volatile("st.shared.b16 [%0], %1;" ::"r"(at), "h"(v) : "memory");
}
__device__ __forceinline__ void sts128_zero(uint32_t at) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t at, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}

// N columns of this warp's lanes; the registers are valid after tmem_wait.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t *r) {
    if constexpr (N == 32)
        tmem_ld32(at, r);
    else if constexpr (N == 16)
        tmem_ld16_now(at, r);
    else
        tmem_ld8_now(at, r);
}
template <int N>
__device__ __forceinline__ void tmem_wait(uint32_t *r) {
    if constexpr (N == 32) tmem_wait32(r);
}

// A ring position: stage and phase parity.
template <int N>
struct Ring {
    uint32_t i = 0, ph = 0;
    __device__ __forceinline__ void next() {
        if (++i == N) {
            i = 0;
            ph ^= 1;
        }
    }
};

template <int G, int TOK>
__global__ void __launch_bounds__(kThreads, 1)
    linear_many_kernel(const __grid_constant__ Maps maps, const __grid_constant__ LinearArgs a) {
    constexpr int TW = TOK / 2;                        // tokens of an epilogue warp
    constexpr int KS = step_k(G, TOK), GU = KS / G;    // k and groups of a step
    constexpr int XB = x_bytes(G, TOK), WB = w_bytes(G, TOK), WROW = KS / 2, kW = w_stages(G, TOK);
    constexpr int DC = d_cols(G, TOK);                 // columns of a step's sums; of its codes: KS / 2
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sX = base, *sW = sX + kX * XB, *sS = sW + kW * WB;
    uint8_t *sT = sS + kS * 2 * kSBytes;               // token sums: chunks of [token][4 parts][16 groups]
    Ctl *s = reinterpret_cast<Ctl *>(sT + kC * TOK * 128);
    float *red = reinterpret_cast<float *>(sX);        // [token][128 lanes], when the last tokens have been read
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < kW; ++i) {
            mbar_init(&s->w_full[i], 1);
            mbar_init(&s->w_empty[i], 4);
        }
        for (int i = 0; i < kS; ++i) {
            mbar_init(&s->s_full[i], 1);
            mbar_init(&s->s_empty[i], kEpiWarps);
        }
        for (int i = 0; i < kX; ++i) {
            mbar_init(&s->ready[i], 1 + 4 + kEpiWarps);  // the loads' own arrival, unpacking warps, epilogue warps
            mbar_init(&s->done[i], 1);
        }
        mbar_init(&s->z_full, kEpiWarps);
        for (int i = 0; i < kC; ++i) mbar_init(&s->sums_full[i], kSumWarps);
        for (int i = 0; i < kX; ++i) mbar_init(&s->x_read[i], kSumWarps);
        mbar_init(&s->drain, 1);
        s->abort = 0;
        fence_mbar_init();
    }
    if (warp == kWWarp && lane == 0) {
        prefetch_tmap(&maps.q);
        prefetch_tmap(&maps.s);
        prefetch_tmap(&maps.b);
        prefetch_tmap(&maps.x);
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&s->tmem, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s->tmem;                     // group sums, then codes
    const uint32_t tA = tmem + kD * DC, tZ = tA + kA * KS / 2, tB = tZ + TOK;
    pdl_wait();
    pdl_trigger();

    const int units = (a.K + KS - 1) / KS, rank = a.rank_of(blockIdx.x);
    const int u0 = units * rank / a.split, u1 = units * (rank + 1) / a.split;
    const int tiles = (a.N + kRows - 1) / kRows, step = gridDim.x / a.split;
    const int first = blockIdx.x / a.split;
    // The token sums are the same for every tile: made in the first one, if all
    // chunks of this block's k have a place, else in each.
    const int c0 = u0 * GU / kChunk;
    const bool once = (u1 * GU - 1) / kChunk - c0 < kC;
    // the last step of a chunk
    auto ends = [&](int u) { return u == u1 - 1 || (u + 1) * GU % kChunk == 0; };

    if (warp >= kWWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRestRegs));
    if (warp == kWWarp) {
        if (elect_one()) {
            Ring<kW> w;
            Ring<kS> sc;
            uint32_t n_w = 0, n_s = 0;
            bool ok = true;
            for (int tile = first; tile < tiles && ok; tile += step) {
                for (int u = u0; u < u1; ++u) {
                    if (u == u0 || u * GU % kChunk == 0) {
                        ok = wait(&s->s_empty[sc.i], sc.ph ^ 1, a, s, 40);
                        if (!ok) break;
                        mbar_arrive_expect_tx(&s->s_full[sc.i], 2 * kSBytes);
                        uint8_t *dst = sS + sc.i * 2 * kSBytes;
                        const int g = u * GU / kChunk * kChunk;
                        tma_load_2d(dst, &maps.s, &s->s_full[sc.i], g, tile * kRows);
                        tma_load_2d(dst + kSBytes, &maps.b, &s->s_full[sc.i], g, tile * kRows);
                        sc.next();
                        ++n_s;
                    }
                    ok = wait(&s->w_empty[w.i], w.ph ^ 1, a, s, 41);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&s->w_full[w.i], WB);
                    tma_load_2d(sW + w.i * WB, &maps.q, &s->w_full[w.i], u * (KS / 8), tile * kRows);
                    w.next();
                    ++n_w;
                }
            }
            // no copy of this block is in flight when it ends
            for (uint32_t i = n_w > kW ? n_w - kW : 0; i < n_w; ++i) mbar_drain(&s->w_full[i % kW], (i / kW) & 1, a.wait_limit);
            for (uint32_t i = n_s > kS ? n_s - kS : 0; i < n_s; ++i) mbar_drain(&s->s_full[i % kS], (i / kS) & 1, a.wait_limit);
        }
        __syncwarp();
    } else if (warp == kXWarp) {
        if (elect_one()) {
            Ring<kX> x;
            uint32_t n_x = 0;
            bool ok = true;
            for (int tile = first; tile < tiles && ok; tile += step) {
                for (int u = u0; u < u1; ++u) {
                    // the slot's previous step (kX before this one) is complete, and
                    // its tokens have been added up
                    ok = wait(&s->done[x.i], x.ph ^ 1, a, s, 42);
                    if (ok && (!once || n_x < static_cast<uint32_t>(u1 - u0 + kX))) ok = wait(&s->x_read[x.i], x.ph ^ 1, a, s, 44);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&s->ready[x.i], XB);
#pragma unroll
                    for (int i = 0; i < KS / 64; ++i)
                        tma_load_2d(sX + x.i * XB + i * TOK * 128, &maps.x, &s->ready[x.i], u * KS + i * 64, 0);
                    x.next();
                    ++n_x;
                }
            }
            // nor one of these.  (The phases also wait for other arrivals, which after
            // a timeout elsewhere may not come: the wait then runs out, long after
            // the copies landed.)
            for (uint32_t i = n_x > kX ? n_x - kX : 0; i < n_x; ++i)
                if (!mbar_drain(&s->ready[i % kX], (i / kX) & 1, a.wait_limit)) break;
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        if (elect_one()) {
            constexpr uint32_t idesc = idesc_bf16(128, TOK);
            Ring<kX> x;
            uint32_t ab = 0, db = 0, chunk = 0;        // chunks of the block so far
            bool ok = true;
            // (a descriptor's address field counts 16 bytes)
            const uint64_t x_desc = sdesc_k128(smem_u32(sX)), t_desc = sdesc_k128(smem_u32(sT));
            for (int tile = first; tile < tiles && ok; tile += step) {
                for (int u = u0; u < u1; ++u) {
                    ok = wait(&s->ready[x.i], x.ph, a, s, 43);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t xd = x_desc + x.i * (XB / 16);
                    const uint32_t at = tA + ab * (KS / 2), dt = tmem + db * DC;
#pragma unroll
                    for (int kk = 0; kk < KS / 16; ++kk)
                        umma_bf16_ts(dt + kk / (G / 16) * TOK, at + kk * 8, xd + (kk / 4) * (TOK * 8) + (kk % 4) * 2,
                                     idesc, kk % (G / 16) != 0);
                    if (ends(u)) {
                        // the chunk's biases times the three parts of its token sums, and 2^12
                        // times the biases times what was too large for those
                        const uint32_t slot = once ? u * GU / kChunk - c0 : chunk % kC;
                        ok = wait(&s->z_full, chunk & 1, a, s, 45);
                        if (ok && (!once || tile == first)) ok = wait(&s->sums_full[slot], once ? 0 : (chunk / kC) & 1, a, s, 50);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int part = 0; part < 4; ++part)
                            umma_bf16_ts(tZ, tB + part / 3 * 8, t_desc + slot * (TOK * 8) + part * 2, idesc, part != 0);
                        ++chunk;
                    }
                    umma_commit(&s->done[x.i]);
                    x.next();
                    ab = ab + 1 == kA ? 0 : ab + 1;
                    db ^= 1;
                }
            }
            // every MMA issued here is complete before tensor memory is freed
            umma_commit(&s->drain);
            mbar_drain(&s->drain, 0, a.wait_limit);
        }
        __syncwarp();
    } else if (warp >= kSumWarp) {
        // ----------------------------------------------------- token sums
        // Two lanes a token (TOK of the 64 pairs).  Of each 128 k of a step a lane
        // adds up 64 (of a step of 64, a group of 32).
        const int pair = (tid - kSumWarp * 32) >> 1, h = tid & 1, t = min(pair, TOK - 1);
        const bool mine = pair < TOK;
        const uint32_t x_row = smem_u32(sX) + t * 128, t_row = smem_u32(sT) + t * 128;
        const uint32_t sw = (t & 7) << 4;              // 128-byte swizzle
        Ring<kX> x;
        uint32_t chunk = 0;
        bool ok = true;
        for (int tile = first; tile < tiles && ok; tile += step) {
            if (once && tile != first) break;
            for (int u = u0; u < u1; ++u) {
                ok = warp_wait(&s->ready[x.i], x.ph, a, s, 52);
                if (!ok) break;
                const uint32_t dst = t_row + chunk % kC * (TOK * 128);
                if (mine && (u == u0 || u * GU % kChunk == 0)) {
                    // groups that this block has no share of count as zero.  (The
                    // chunk that had the place before was multiplied long since:
                    // the sums of step n - 2, of another chunk, have been read.)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sts128_zero(dst + (((4 * h + i) << 4) ^ sw));
                }
                __syncwarp();
                // the sum of 16 k after 16 k, the pair's pieces on different banks
                auto add_up = [&](uint32_t src, int piece, int n) {
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < n; ++i) {
                        const uint4 v = lds128(src + (((piece ^ i) << 4) ^ sw));
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            sum[j] = fmaf(__uint_as_float(w[j] << 16), 0x1p-7f, sum[j]);
                            sum[j] = fmaf(__uint_as_float(w[j] & 0xFFFF0000u), 0x1p-7f, sum[j]);
                        }
                    }
                    return (sum[0] + sum[1]) + (sum[2] + sum[3]);
                };
                // X 2^-7, exact down to the smallest token and finite up to the largest.
                // X in three parts of 8 bits is exact to 2^-25; one that is too large
                // for that has 2^-12 of its first 8 bits in the fourth place.
                auto put = [&](float X, int group) {
                    const int at = group % kChunk * 2;
                    float top = 0.f;
                    if (fabsf(X) >= 0x1p118f) top = __bfloat162float(__float2bfloat16_rn(X * 0x1p-5f));
                    X = fmaf(top, -32.f, X) * 128.f;
#pragma unroll
                    for (int part = 0; part < 3; ++part) {
                        const __nv_bfloat16 b = __float2bfloat16_rn(X);
                        sts16(dst + ((part * 32 + at) ^ sw), __bfloat16_as_ushort(b));
                        X -= __bfloat162float(b);
                    }
                    if (top != 0.f) sts16(dst + ((96 + at) ^ sw), __bfloat16_as_ushort(__float2bfloat16_rn(top)));
                };
                const uint32_t src = x_row + x.i * XB;
                if constexpr (KS == 64) {
                    const float X = add_up(src, 4 * h, 4);
                    if (mine) put(X, 2 * u + h);
                } else {
#pragma unroll 1
                    for (int b = 0; b < KS / 128; ++b) {
                        const uint32_t box = src + (2 * b + h) * (TOK * 128);
                        if constexpr (G == 32) {
                            const float lo = add_up(box, 4 * h, 4), hi = add_up(box, 4 * (h ^ 1), 4);
                            if (mine) put(lo, u * GU + 4 * b + 2 * h + h);
                            if (mine) put(hi, u * GU + 4 * b + 2 * h + (h ^ 1));
                        } else {
                            float X = add_up(box, 4 * h, 8);
                            if constexpr (G == 128) X += __shfl_xor_sync(0xffffffffu, X, 1);
                            if (mine && (G == 64 || h == 0)) put(X, G == 64 ? u * GU + 2 * b + h : u * GU + b);
                        }
                    }
                }
                __syncwarp();
                first_lane_arrives(lane, &s->x_read[x.i]);
                if (ends(u)) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    first_lane_arrives(lane, &s->sums_full[chunk % kC]);
                    ++chunk;
                }
                x.next();
            }
        }
    }
    } else if (warp >= kDeqWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kDeqRegs));
        // ------------------------------------------------------- unpacking
        // the two sets of four warps take the steps in turn
        const int quarter = warp & 3, set_of = (warp - kDeqWarp) >> 2;
        const int r = quarter * 32 + lane;             // row of the tile
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        const int rot = KS == 256 ? r & 7 : KS == 128 ? (r >> 1) & 3 : (r >> 2) & 1;  // swizzle of the row's 16-byte pieces
        const uint32_t w_addr = smem_u32(sW);
        // 128 + q as a bf16 pair, then (128 + q) 2^-12 - 2^-5, exactly
        const __nv_bfloat162 down = u32_as_bf162(0x39803980u), off = u32_as_bf162(0xBD00BD00u);
        uint32_t n = 0;                                // steps of the block so far
        bool ok = true;
        for (int tile = first; tile < tiles && ok; tile += step) {
            for (int u = u0; u < u1; ++u, ++n) {
                if (static_cast<int>(n & 1) != set_of) continue;
                const uint32_t ws = n % kW, as = n % kA;
                ok = warp_wait(&s->w_full[ws], (n / kW) & 1, a, s, 46);
                if (!ok) break;
                const uint32_t row = w_addr + ws * WB + r * WROW;
                constexpr int kHeld = KS < 128 ? KS / 32 : 4;  // pieces in registers
                uint4 v[kHeld];
                bool free = false;
#pragma unroll kHeld
                for (int i = 0; i < KS / 32; ++i) {
                    if (i % kHeld == 0) {
#pragma unroll
                        for (int e = 0; e < kHeld; ++e) v[e] = lds128(row + (((i + e) ^ rot) << 4));
                        if (i + kHeld == KS / 32) {
                            __syncwarp();
                            first_lane_arrives(lane, &s->w_empty[ws]);
                        }
                    }
                    const uint4 &c = v[i % kHeld];
                    const uint32_t q[4] = {c.x, c.y, c.z, c.w};
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int j = 0; j < 4; ++j) p[4 * e + j] = bf162_as_u32(__hfma2(u32_as_bf162(mask_set(q[e] >> (4 * j), 0x000F000Fu, 0x43004300u)), down, off));
                    if (!free) {
                        // the MMAs of the step that had this buffer before
                        if (n >= kA) ok = warp_wait(&s->done[(n - kA) % kX], ((n - kA) / kX) & 1, a, s, 47);
                        if (!ok) break;
                        free = true;
                        tc_fence_after();
                    }
                    tmem_st16((tA + as * (KS / 2) + i * 16) | lanes, p);
                }
                if (!ok) break;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                first_lane_arrives(lane, &s->ready[n % kX]);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
        // -------------------------------------------------------- epilogue
        const int half = warp >> 2, quarter = warp & 3;
        const int r = quarter * 32 + lane;             // row of the tile
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t s_addr = smem_u32(sS) + r * (kChunk * 2);
        Ring<kS> sc;
        Ring<kX> x;                                    // step
        uint32_t ahead = kD, db = 0;                   // slot of the step that gets this one's buffer of sums
        bool ok = true;
        // the first steps find their buffers free
        if (lane == 0)
            for (int i = 0; i < kD; ++i) mbar_arrive(&s->ready[i]);
        for (int tile = first; tile < tiles; tile += step) {
            uint64_t y[TW / 2];
#pragma unroll
            for (int i = 0; i < TW / 2; ++i) y[i] = 0;
            for (int u = u0; u < u1; ++u) {
                if (u == u0 || u * GU % kChunk == 0) {
                    // the row's biases of the chunk are the first operand of its bias
                    // products.  (The last chunk's are complete, and have been read.)
                    ok = warp_wait(&s->s_full[sc.i], sc.ph, a, s, 48);
                    if (!ok) break;
                    if (half == 0) {
                        const uint32_t at = s_addr + sc.i * 2 * kSBytes + kSBytes;
                        const uint4 lo = lds128(at), hi = lds128(at + 16);
                        uint32_t b[16] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                        // (2^12 z stays finite, as its factor is mostly zero)
                        const __nv_bfloat162 most = u32_as_bf162(0x7F7F7F7Fu), least = u32_as_bf162(0xFF7FFF7Fu);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            b[8 + i] = bf162_as_u32(__hmax2(least, __hmin2(most, __hmul2(u32_as_bf162(b[i]), u32_as_bf162(0x45804580u)))));
                        tmem_st16(tB | lanes, b);
                        tmem_st_wait();
                    }
                    tc_fence_before();
                    __syncwarp();
                    first_lane_arrives(lane, &s->z_full);
                }
                uint32_t pair[(GU + 1) / 2];               // scales of two groups each
#pragma unroll
                for (int i = 0; i < (GU + 1) / 2; ++i)
                    pair[i] = lds32(s_addr + sc.i * 2 * kSBytes + ((u * GU % kChunk >> 1) + i) * 4);
                ok = warp_wait(&s->done[x.i], x.ph, a, s, 49);
                if (!ok) break;
                tc_fence_after();
                uint32_t d[GU][TW];
#pragma unroll
                for (int gu = 0; gu < GU; ++gu) tmem_ld<TW>((tmem + db * DC + gu * TOK + half * TW) | lanes, d[gu]);
#pragma unroll
                for (int gu = 0; gu < GU; ++gu) tmem_wait<TW>(d[gu]);
                tc_fence_before();
                __syncwarp();
                first_lane_arrives(lane, &s->ready[ahead]);
                x.next();
                ahead = ahead + 1 == kX ? 0 : ahead + 1;
                db ^= 1;
#pragma unroll
                for (int gu = 0; gu < GU; ++gu) {
                    const bool high = GU > 1 ? gu & 1 : u & 1;
                    const float scale = 4096.f * __uint_as_float(high ? pair[gu / 2] & 0xFFFF0000u : pair[gu / 2] << 16);
                    const uint64_t s2 = pack2(__float_as_uint(scale), __float_as_uint(scale));
#pragma unroll
                    for (int i = 0; i < TW / 2; ++i) y[i] = fma2(s2, pack2(d[gu][2 * i], d[gu][2 * i + 1]), y[i]);
                }
                if (ends(u)) {
                    uint32_t z[TW];
                    tmem_ld<TW>((tZ + half * TW) | lanes, z);
                    tmem_wait<TW>(z);
#pragma unroll
                    for (int i = 0; i < TW / 2; ++i) y[i] = add2(y[i], pack2(z[2 * i], z[2 * i + 1]));
                    __syncwarp();
                    first_lane_arrives(lane, &s->s_empty[sc.i]);
                    sc.next();
                }
            }
            if (!ok) break;
            const int row = tile * kRows + r, t0 = half * TW;
            if (a.split > 1) {
                const uint32_t at = smem_u32(red) + (t0 * 128 + r) * 4;
#pragma unroll
                for (int i = 0; i < TW / 2; ++i) {
                    const float2 v = unpack2(y[i]);
                    sts32(at + i * 1024, v.x);
                    sts32(at + i * 1024 + 512, v.y);
                }
                continue;
            }
            // the MMAs of the next tile wait for these warps: a loop without branches
            // for each type (through LinearArgs::store, a tile's end took 6500 cycles)
            const int nt = row < a.N ? a.B - t0 : 0;
            auto put = [&](auto *out, auto narrow) {
                out += t0 * a.y_stride + row;
#pragma unroll
                for (int i = 0; i < TW / 2; ++i) {
                    const float2 v = unpack2(y[i]);
                    if (2 * i < nt) *out = narrow(v.x);
                    out += a.y_stride;
                    if (2 * i + 1 < nt) *out = narrow(v.y);
                    out += a.y_stride;
                }
            };
            if (a.y_fp32)
                put(static_cast<float *>(a.y), [](float v) { return v; });
            else
                put(static_cast<__nv_bfloat16 *>(a.y), [](float v) { return __float2bfloat16_rn(v); });
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
    if (a.split > 1) {
        // one tile per cluster: every block adds up some of its tokens
        cluster_sync();
        const int per = (a.B + a.split - 1) / a.split, t0 = rank * per, t1 = min(a.B, t0 + per);
        for (int i = tid; i < (t1 - t0) * 128; i += kThreads) {
            const int t = t0 + i / 128, l = i % 128, row = first * kRows + l;
            if (row >= a.N) continue;
            float sum = 0.f;
            for (int p = 0; p < a.split; ++p) sum += dsmem_ld(smem_u32(red + t * 128 + l), p);
            a.store(t, row, sum);
        }
        cluster_sync();
    }
}

template <int G, int TOK>
static cudaError_t launch_t(const Maps &maps, LinearArgs a, int num_sms, cudaStream_t s) {
    const int units = (a.K + step_k(G, TOK) - 1) / step_k(G, TOK), tiles = (a.N + kRows - 1) / kRows;
    // share K in a cluster while there are two steps for each block (one of 256 k)
    // and all clusters run at once (one tile each)
    constexpr int least = step_k(G, TOK) == 256 ? 1 : 2;
    a.split = 1;
    while (a.split < 8 && tiles * (a.split + 1) <= num_sms * 7 / 8 && units >= (a.split + 1) * least) ++a.split;
    const auto kernel = linear_many_kernel<G, TOK>;
    const cudaError_t e = allow_smem<linear_many_kernel<G, TOK>>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(a.split > 1 ? tiles * a.split : std::min(tiles, num_sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes(G, TOK);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, maps, a);
}

template <int G>
static cudaError_t launch_g(const Maps &m, const LinearArgs &a, int num_sms, cudaStream_t s) {
    if (a.B <= 16) return launch_t<G, 16>(m, a, num_sms, s);
    if (a.B <= 32) return launch_t<G, 32>(m, a, num_sms, s);
    return launch_t<G, 64>(m, a, num_sms, s);
}

}  // namespace many

int linear_token_rows(int B) { return B <= 16 ? 16 : B <= 32 ? 32 : 64; }
int linear_code_words(int G, int B) { return many::step_k(G, linear_token_rows(B)) / 8; }

cudaError_t launch_linear_many(const CUtensorMap *maps, const LinearArgs &a, int num_sms, cudaStream_t s) {
    const many::Maps m{maps[0], maps[1], maps[2], maps[3]};
    if (a.G == 32) return many::launch_g<32>(m, a, num_sms, s);
    if (a.G == 64) return many::launch_g<64>(m, a, num_sms, s);
    return many::launch_g<128>(m, a, num_sms, s);
}

}  // namespace moe
