// y[b][n] = sum_k x[b][k] (s[n][k/G] q[n][k] + z[n][k/G]) for 9 to 64 tokens on the
// fifth-generation tensor cores.
//
// As with few tokens no weight is rounded: the codes themselves, exact in bf16
// as q 2^-12 (128 + q by a shift and a mask-and-set a pair, then one fused
// multiply-add), are the M = 128 side of tcgen05.mma, the tokens as they are the N
// side, and each group of weights has a sum of its own, D = sum q x 2^-12 (the
// power keeps it finite for any finite token); then, in fp32 registers,
//   y += (2^12 s) D + (2^12 z) X,   X = sum of the group's x 2^-12
// (With 128 + q as the operand and z - 128 s the multiply-add is saved, but D is
// 17 times as large and y off by 2e-6 instead of 2e-7.)
// X comes out of the same MMA: the last of each 32 rows of a tile is not a
// weight row but ones, so that a tile has 4 x 31 weight rows and the last lane of
// every epilogue warp finds X in its row of D.  The codes go straight into tensor
// memory, where the MMA reads its first operand from: a thread unpacks one row's
// 128 codes in registers and stores them to its lane.  What is in shared memory
// is only what TMA brings: packed codes, scales, and tokens.
//
//   epilogue     warps 0-7, warp w: rows 32 (w % 4) .., token half w / 4: D from
//                tensor memory, y in registers
//   unpacking    warps 8-15, a thread per row, two sets of four in turn
//   loads, MMA   warps 16 and 17 (18 and 19 complete the warpgroup)
//
// A barrier wait costs its role about 130 cycles however early the other side
// was, so the work goes in steps of 128 k (groups of 32: 64 k) and all that a
// step's MMAs need comes in on one barrier (`ready`: tokens by TMA, codes from
// the unpacking warps, the buffer of sums given back by the epilogue), all that
// waits for them on one other (`done`).  With a barrier for each and steps of 64
// k, 64 x 2048 x 131072 took 136 us, with steps of 128 k 104.
//
// Blocks take tiles of 124 rows in turn.  If there are too few tiles for the
// GPU, a cluster of up to eight blocks shares K and adds up through distributed
// shared memory.  Every wait is bounded.
#include <algorithm>

#include "linear.cuh"

namespace moe {
namespace many {

constexpr int kRows = 124;                 // weight rows of a tile: 31 in each 32 lanes
constexpr int kEpiWarps = 8, kDeqWarp = 8, kTmaWarp = 16, kMmaWarp = 17, kThreads = 20 * 32;
// Registers a thread: an epilogue thread of 64 tokens holds 32 sums and 32 of
// D.  The launch gives 96 to each of the 640 threads (61,440 in all); epilogue,
// unpacking and the rest then hold 128, 72 and 80 (32,768 + 18,432 + 10,240).
constexpr int kLaunchRegs = 96, kEpiRegs = 128, kDeqRegs = 72, kRestRegs = 80;
static_assert(256 * kEpiRegs + 256 * kDeqRegs + 128 * kRestRegs <= kThreads * kLaunchRegs, "shares of the launch's registers");
constexpr int kW = 6, kS = 3;              // stages: codes, scales (8 groups)
constexpr int kX = 6, kA = 3;              // stages: tokens in shared memory, codes in tensor memory (64 columns)
constexpr int kD = 2;                      // buffers of group sums, two groups each (128 columns)
constexpr int kSBytes = 128 * 8 * 2;
constexpr uint32_t kTmemCols = 512;        // kD * 128 + kA * 64 = 448, rounded up
__host__ __device__ constexpr int step_k(int G) { return G == 32 ? 64 : 128; }
__host__ __device__ constexpr int w_bytes(int G) { return 128 * step_k(G) / 2; }

__host__ __device__ constexpr int x_bytes(int G, int tok) { return step_k(G) / 64 * tok * 128; }  // boxes of 64 k

struct Ctl {
    uint64_t w_full[kW], w_empty[kW], s_full[kS], s_empty[kS];
    uint64_t ready[kX], done[kX];          // a step's operands and sums are there; its MMAs are complete
    uint64_t drain;
    uint32_t tmem;
    int abort;
};

// More than half of a SM's: one block at a time, since each takes all of the
// tensor memory.
__host__ __device__ constexpr int smem_bytes(int G, int tok) {
    constexpr int least = kBlockSmem / 2 + 1024;
    const int n = kX * x_bytes(G, tok) + kW * w_bytes(G) + kS * 2 * kSBytes + tok * 128 * 4 +
                  static_cast<int>(sizeof(Ctl)) + 1024;
    return n > least ? n : least;
}
static_assert(smem_bytes(64, 64) <= kBlockSmem, "one block per SM");

struct Maps {
    CUtensorMap q, s, b, x;
};

__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, const LinearArgs &a, Ctl *s, int site) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
        if (*reinterpret_cast<volatile int *>(&s->abort)) return false;
        if (clock64() - t0 > a.wait_limit) {
            record_status(a.status, MOE_ERR_TIMEOUT - site);
            *reinterpret_cast<volatile int *>(&s->abort) = 1;
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const LinearArgs &a, Ctl *s, int site) {
    return __all_sync(0xffffffffu, wait(bar, parity, a, s, site));
}

// Shared memory by its own address: through a plain pointer these become generic
// accesses, with several times the latency.
__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void sts32(uint32_t at, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}

// (w & mask) | set in one instruction
__device__ __forceinline__ uint32_t mask_set(uint32_t w, uint32_t mask, uint32_t set) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(set));
    return r;
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
    constexpr int KS = step_k(G), GU = KS / G;         // k and groups (one or two) of a step
    constexpr int XB = x_bytes(G, TOK), WB = w_bytes(G), WROW = KS / 2;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sX = base, *sW = sX + kX * XB, *sS = sW + kW * WB;
    float *red = reinterpret_cast<float *>(sS + kS * 2 * kSBytes);  // [token][128 lanes]
    Ctl *s = reinterpret_cast<Ctl *>(red + TOK * 128);
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
        mbar_init(&s->drain, 1);
        s->abort = 0;
        fence_mbar_init();
    }
    if (warp == kTmaWarp && lane == 0) {
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
    const uint32_t tA = tmem + kD * 128;
    pdl_wait();
    pdl_trigger();

    const int units = (a.K + KS - 1) / KS, rank = a.rank_of(blockIdx.x);
    const int u0 = units * rank / a.split, u1 = units * (rank + 1) / a.split;
    const int tiles = (a.N + kRows - 1) / kRows, step = gridDim.x / a.split;
    const int first = blockIdx.x / a.split;

    if (warp >= kTmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRestRegs));
    if (warp == kTmaWarp) {
        if (lane == 0) {
            Ring<kW> w;
            Ring<kX> x;
            Ring<kS> sc;
            uint32_t n_w = 0, n_s = 0, n_x = 0;
            bool ok = true;
            for (int tile = first; tile < tiles && ok; tile += step) {
                int block = -1;
                for (int u = u0; u < u1 && ok; ++u) {
                    const int need = u * GU / 8;       // block of 8 groups that the step's lie in
                    if (need != block) {
                        block = need;
                        ok = wait(&s->s_empty[sc.i], sc.ph ^ 1, a, s, 40);
                        if (!ok) break;
                        mbar_arrive_expect_tx(&s->s_full[sc.i], 2 * kSBytes);
                        uint8_t *dst = sS + sc.i * 2 * kSBytes;
                        tma_load_2d(dst, &maps.s, &s->s_full[sc.i], block * 8, tile * kRows);
                        tma_load_2d(dst + kSBytes, &maps.b, &s->s_full[sc.i], block * 8, tile * kRows);
                        sc.next();
                        ++n_s;
                    }
                    ok = wait(&s->w_empty[w.i], w.ph ^ 1, a, s, 41);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&s->w_full[w.i], WB);
                    tma_load_2d(sW + w.i * WB, &maps.q, &s->w_full[w.i], u * (KS / 8), tile * kRows);
                    w.next();
                    ++n_w;
                    // the slot's previous step (kX before this one) is complete
                    ok = wait(&s->done[x.i], x.ph ^ 1, a, s, 42);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&s->ready[x.i], XB);
#pragma unroll
                    for (int i = 0; i < KS / 64; ++i)
                        tma_load_2d(sX + x.i * XB + i * TOK * 128, &maps.x, &s->ready[x.i], u * KS + i * 64, 0);
                    x.next();
                    ++n_x;
                }
            }
            // no copy of this block is in flight when it ends.  (The tokens' phases
            // also wait for other arrivals, which after a timeout elsewhere may
            // not come: the wait then runs out, long after the copies landed.)
            for (uint32_t i = n_w > kW ? n_w - kW : 0; i < n_w; ++i) mbar_wait(&s->w_full[i % kW], (i / kW) & 1, a.wait_limit);
            for (uint32_t i = n_x > kX ? n_x - kX : 0; i < n_x; ++i)
                if (!mbar_wait(&s->ready[i % kX], (i / kX) & 1, a.wait_limit)) break;
            for (uint32_t i = n_s > kS ? n_s - kS : 0; i < n_s; ++i) mbar_wait(&s->s_full[i % kS], (i / kS) & 1, a.wait_limit);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        if (elect_one()) {
            constexpr uint32_t idesc = idesc_bf16(128, TOK);
            Ring<kX> x;
            uint32_t ab = 0, db = 0;
            bool ok = true;
            const uint32_t x_addr = smem_u32(sX);
            for (int tile = first; tile < tiles && ok; tile += step) {
                for (int u = u0; u < u1; ++u) {
                    ok = wait(&s->ready[x.i], x.ph, a, s, 43);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t xa = x_addr + x.i * XB, at = tA + ab * 64, dt = tmem + db * 128;
#pragma unroll
                    for (int kk = 0; kk < KS / 16; ++kk)
                        umma_bf16_ts(dt + kk / (G / 16) * 64, at + kk * 8, sdesc_k128(xa + (kk / 4) * (TOK * 128) + (kk % 4) * 32),
                                     idesc, kk % (G / 16) != 0);
                    umma_commit(&s->done[x.i]);
                    x.next();
                    ab = ab + 1 == kA ? 0 : ab + 1;
                    db ^= 1;
                }
            }
            // every MMA issued here is complete before tensor memory is freed
            umma_commit(&s->drain);
            mbar_wait(&s->drain, 0, a.wait_limit);
        }
        __syncwarp();
    }
    } else if (warp >= kDeqWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kDeqRegs));
        // ------------------------------------------------------- unpacking
        // the two sets of four warps take the steps in turn
        const int quarter = warp & 3, set_of = (warp - kDeqWarp) >> 2;
        const int r = quarter * 31 + min(lane, 30);    // row of the tile
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        const int rot = KS == 128 ? (r >> 1) & 3 : (r >> 2) & 1;  // swizzle of the row's 16-byte pieces
        const uint32_t w_addr = smem_u32(sW);
        // (w & mask) | set: 128 + q as a bf16 pair, or 129 in the last lane; then
        // (128 + q) 2^-12 - 2^-5, exactly
        const uint32_t mask = lane == 31 ? 0u : 0x000F000Fu, set = lane == 31 ? 0x43014301u : 0x43004300u;
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
                uint4 v[KS / 32];
#pragma unroll
                for (int i = 0; i < KS / 32; ++i) v[i] = lds128(row + ((i ^ rot) << 4));
                __syncwarp();
                if (lane == 0) mbar_arrive(&s->w_empty[ws]);
                bool free = false;
#pragma unroll
                for (int i = 0; i < KS / 32; ++i) {
                    const uint32_t q[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int j = 0; j < 4; ++j) p[4 * e + j] = bf162_as_u32(__hfma2(u32_as_bf162(mask_set(q[e] >> (4 * j), mask, set)), down, off));
                    if (!free) {
                        // the MMAs of the step that had this buffer before
                        if (n >= kA) ok = warp_wait(&s->done[(n - kA) % kX], ((n - kA) / kX) & 1, a, s, 47);
                        if (!ok) break;
                        free = true;
                        tc_fence_after();
                    }
                    tmem_st16((tA + as * 64 + i * 16) | lanes, p);
                }
                if (!ok) break;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s->ready[n % kX]);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
        // -------------------------------------------------------- epilogue
        const int half = warp >> 2, quarter = warp & 3;
        const int r = quarter * 31 + min(lane, 30);    // row of the tile (the last lane: X)
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t s_addr = smem_u32(sS) + r * 16;
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
            int block = -1;
            uint4 sv = make_uint4(0u, 0u, 0u, 0u), bv = sv;
            for (int g = u0 * GU; g < u1 * GU && ok; g += GU) {
                if (g / 8 != block) {
                    // the row's scales and biases of eight groups
                    block = g / 8;
                    ok = warp_wait(&s->s_full[sc.i], sc.ph, a, s, 48);
                    if (!ok) break;
                    sv = lds128(s_addr + sc.i * 2 * kSBytes);
                    bv = lds128(s_addr + sc.i * 2 * kSBytes + kSBytes);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s->s_empty[sc.i]);
                    sc.next();
                }
                ok = warp_wait(&s->done[x.i], x.ph, a, s, 49);
                if (!ok) break;
                tc_fence_after();
                uint32_t d[GU][TW];
#pragma unroll
                for (int gu = 0; gu < GU; ++gu) tmem_ld<TW>((tmem + db * 128 + gu * 64 + half * TW) | lanes, d[gu]);
#pragma unroll
                for (int gu = 0; gu < GU; ++gu) tmem_wait<TW>(d[gu]);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s->ready[ahead]);
                x.next();
                ahead = ahead + 1 == kX ? 0 : ahead + 1;
                db ^= 1;
                const int pair = (g & 7) >> 1;
                const uint32_t sw = pair == 0 ? sv.x : pair == 1 ? sv.y : pair == 2 ? sv.z : sv.w;
                const uint32_t bw = pair == 0 ? bv.x : pair == 1 ? bv.y : pair == 2 ? bv.z : bv.w;
#pragma unroll
                for (int gu = 0; gu < GU; ++gu) {
                    const bool high = GU == 2 ? gu == 1 : (g & 1);
                    const float scale = 4096.f * __uint_as_float(high ? sw & 0xFFFF0000u : sw << 16);
                    const float bias = 4096.f * __uint_as_float(high ? bw & 0xFFFF0000u : bw << 16);
                    const uint64_t s2 = pack2(__float_as_uint(scale), __float_as_uint(scale));
                    const uint64_t b2 = pack2(__float_as_uint(bias), __float_as_uint(bias));
                    const uint32_t *e = d[gu];
#pragma unroll
                    for (int i = 0; i < TW / 4; ++i) {
                        // X is the last lane's D
                        uint4 X;
                        X.x = __shfl_sync(0xffffffffu, e[4 * i], 31);
                        X.y = __shfl_sync(0xffffffffu, e[4 * i + 1], 31);
                        X.z = __shfl_sync(0xffffffffu, e[4 * i + 2], 31);
                        X.w = __shfl_sync(0xffffffffu, e[4 * i + 3], 31);
                        y[2 * i] = fma2(s2, pack2(e[4 * i], e[4 * i + 1]), fma2(b2, pack2(X.x, X.y), y[2 * i]));
                        y[2 * i + 1] =
                            fma2(s2, pack2(e[4 * i + 2], e[4 * i + 3]), fma2(b2, pack2(X.z, X.w), y[2 * i + 1]));
                    }
                }
            }
            if (a.split == 1) {
                if (!ok) break;
                const int row = tile * kRows + r;
                if (lane < 31 && row < a.N) {
#pragma unroll
                    for (int i = 0; i < TW / 2; ++i) {
                        const float2 v = unpack2(y[i]);
                        const int t = half * TW + 2 * i;
                        if (t < a.B) a.store(t, row, v.x);
                        if (t + 1 < a.B) a.store(t + 1, row, v.y);
                    }
                }
                continue;
            }
#pragma unroll
            for (int i = 0; i < TW / 2; ++i) {
                const float2 v = unpack2(y[i]);
                const uint32_t at = smem_u32(red) + ((half * TW + 2 * i) * 128 + quarter * 32 + lane) * 4;
                sts32(at, v.x);
                sts32(at + 512, v.y);
            }
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
            const int t = t0 + i / 128, l = i % 128, row = first * kRows + l / 32 * 31 + l % 32;
            if (l % 32 == 31 || row >= a.N) continue;
            float sum = 0.f;
            for (int p = 0; p < a.split; ++p) sum += dsmem_ld(smem_u32(red + t * 128 + l), p);
            a.store(t, row, sum);
        }
        cluster_sync();
    }
}

template <int G, int TOK>
static cudaError_t launch_t(const Maps &maps, LinearArgs a, int num_sms, cudaStream_t s) {
    const int units = (a.K + step_k(G) - 1) / step_k(G), tiles = (a.N + kRows - 1) / kRows;
    // share K in a cluster while there are two steps for each block and all
    // clusters run at once (one tile each)
    a.split = 1;
    while (a.split < 8 && tiles * (a.split + 1) <= num_sms * 7 / 8 && units >= (a.split + 1) * 2) ++a.split;
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

int linear_code_words(int G) { return many::step_k(G) / 8; }
int linear_token_rows(int B) { return B <= 16 ? 16 : B <= 32 ? 32 : 64; }

cudaError_t launch_linear_many(const CUtensorMap *maps, const LinearArgs &a, int num_sms, cudaStream_t s) {
    const many::Maps m{maps[0], maps[1], maps[2], maps[3]};
    if (a.G == 32) return many::launch_g<32>(m, a, num_sms, s);
    if (a.G == 64) return many::launch_g<64>(m, a, num_sms, s);
    return many::launch_g<128>(m, a, num_sms, s);
}

}  // namespace moe
