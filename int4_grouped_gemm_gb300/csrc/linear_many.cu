// y[b][n] = sum_k x[b][k] (s[n][k/G] q[n][k] + z[n][k/G]) for 9 to 64 tokens on the
// fifth-generation tensor cores.
//
// As with few tokens no weight is rounded: the codes themselves, 128 + q in
// bf16 (one shift or one mask-and-set a pair), are the M = 128 side of
// tcgen05.mma, the tokens as they are the N side, and each group of weights
// has a sum of its own, D = sum (128 + q) x; then, in fp32 registers,
//   y += s D + (z - 128 s) X,   X = sum of the group's x
// X comes out of the same MMA: the last of the 128 rows of a tile is not a
// weight row but ones, so that a tile has 127 weight rows and D's row 127 is X.
// The codes go straight into tensor memory, where the MMA reads its first
// operand from: a thread unpacks one row's 64 codes in registers and stores
// them to its lane.  What is in shared memory is only what TMA brings: packed
// codes, scales, and tokens.
//
//   warps 0-7    epilogue, warp w: rows 32 (w % 4) .., token half w / 4: D from
//                tensor memory, y in registers
//   warps 8-11   unpacking, a thread per row
//   warp 12      TMA loads
//   warp 13      MMA issue
//
// Blocks take tiles of 127 rows in turn.  If there are too few tiles for the
// GPU, a cluster of up to four blocks shares K and adds up through distributed
// shared memory.  Every wait is bounded.
#include <algorithm>

#include "linear.cuh"

namespace moe {
namespace many {

constexpr int kRows = 127;                 // weight rows of a tile
constexpr int kEpiWarps = 8, kDeqWarp = 8, kTmaWarp = 12, kMmaWarp = 13, kThreads = 14 * 32;
constexpr int kUnit = 128;                 // k of a stage of codes
constexpr int kW = 6, kX = 8, kS = 3;      // stages: codes (128 k), tokens (64 k), scales (8 groups)
constexpr int kA = 4, kD = 4;              // buffers in tensor memory: codes (64 k, 32 columns), group sums
constexpr int kWBytes = 128 * kUnit / 2, kSBytes = 128 * 8 * 2;
constexpr uint32_t kTmemCols = 512;        // kD * 64 + kA * 32 = 384, rounded up

__host__ __device__ constexpr int x_bytes(int tok) { return tok * 128; }

struct Ctl {
    uint64_t w_full[kW], w_empty[kW], x_full[kX], x_empty[kX], s_full[kS], s_empty[kS];
    uint64_t a_full[kA], a_empty[kA], d_full[kD], d_empty[kD];
    uint64_t sum_full[2][kD];              // X of the token half is in shared memory
    uint64_t drain;
    alignas(16) float sums[kD][64];        // X
    uint32_t tmem;
    int abort;
};

// More than half of a SM's: one block at a time, since each takes all of the
// tensor memory.
__host__ __device__ constexpr int smem_bytes(int tok) {
    constexpr int least = kBlockSmem / 2 + 1024;
    const int n = kX * x_bytes(tok) + kW * kWBytes + kS * 2 * kSBytes + tok * 128 * 4 + static_cast<int>(sizeof(Ctl)) + 1024;
    return n > least ? n : least;
}
static_assert(smem_bytes(64) <= kBlockSmem, "one block per SM");
static_assert(offsetof(Ctl, sums) % 16 == 0, "X is read in 16-byte pieces");

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
    constexpr int HG = G == 32 ? 2 : 1;                // groups that end in a 64-k half (128: one in two halves)
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sX = base, *sW = sX + kX * x_bytes(TOK), *sS = sW + kW * kWBytes;
    float *red = reinterpret_cast<float *>(sS + kS * 2 * kSBytes);  // [token][128 rows]
    Ctl *s = reinterpret_cast<Ctl *>(red + TOK * 128);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < kW; ++i) {
            mbar_init(&s->w_full[i], 1);
            mbar_init(&s->w_empty[i], 4);
        }
        for (int i = 0; i < kX; ++i) {
            mbar_init(&s->x_full[i], 1);
            mbar_init(&s->x_empty[i], 1);
        }
        for (int i = 0; i < kS; ++i) {
            mbar_init(&s->s_full[i], 1);
            mbar_init(&s->s_empty[i], kEpiWarps);
        }
        for (int i = 0; i < kA; ++i) {
            mbar_init(&s->a_full[i], 4);
            mbar_init(&s->a_empty[i], 1);
        }
        for (int i = 0; i < kD; ++i) {
            mbar_init(&s->d_full[i], 1);
            mbar_init(&s->d_empty[i], kEpiWarps);
            mbar_init(&s->sum_full[0][i], 1);
            mbar_init(&s->sum_full[1][i], 1);
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
    const uint32_t tA = tmem + kD * 64;
    pdl_wait();
    pdl_trigger();

    const int units = (a.K + kUnit - 1) / kUnit, rank = a.rank_of(blockIdx.x);
    const int u0 = units * rank / a.split, u1 = units * (rank + 1) / a.split;
    const int tiles = (a.N + kRows - 1) / kRows, step = gridDim.x / a.split;
    const int first = blockIdx.x / a.split;

    if (warp == kTmaWarp) {
        if (lane == 0) {
            Ring<kW> w;
            Ring<kX> x;
            Ring<kS> sc;
            uint32_t n_w = 0, n_x = 0, n_s = 0;
            bool ok = true;
            for (int tile = first; tile < tiles && ok; tile += step) {
                int block = -1;
                for (int u = u0; u < u1 && ok; ++u) {
                    const int need = u * (kUnit / 32) * 32 / G / 8;  // block of 8 groups that the unit's lie in
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
                    mbar_arrive_expect_tx(&s->w_full[w.i], kWBytes);
                    tma_load_2d(sW + w.i * kWBytes, &maps.q, &s->w_full[w.i], u * (kUnit / 8), tile * kRows);
                    w.next();
                    ++n_w;
                    for (int h = 0; h < 2 && ok; ++h) {
                        ok = wait(&s->x_empty[x.i], x.ph ^ 1, a, s, 42);
                        if (!ok) break;
                        mbar_arrive_expect_tx(&s->x_full[x.i], x_bytes(TOK));
                        tma_load_2d(sX + x.i * x_bytes(TOK), &maps.x, &s->x_full[x.i], u * kUnit + h * 64, 0);
                        x.next();
                        ++n_x;
                    }
                }
            }
            // no copy of this block is in flight when it ends
            for (uint32_t i = n_w > kW ? n_w - kW : 0; i < n_w; ++i) mbar_wait(&s->w_full[i % kW], (i / kW) & 1, a.wait_limit);
            for (uint32_t i = n_x > kX ? n_x - kX : 0; i < n_x; ++i) mbar_wait(&s->x_full[i % kX], (i / kX) & 1, a.wait_limit);
            for (uint32_t i = n_s > kS ? n_s - kS : 0; i < n_s; ++i) mbar_wait(&s->s_full[i % kS], (i / kS) & 1, a.wait_limit);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        if (elect_one()) {
            constexpr uint32_t idesc = idesc_bf16(128, TOK);
            Ring<kX> x;
            Ring<kA> ab;
            Ring<kD> db;
            bool ok = true;
            for (int tile = first; tile < tiles && ok; tile += step) {
                for (int h = 2 * u0; h < 2 * u1 && ok; ++h) {  // 64 k each
                    ok = wait(&s->x_full[x.i], x.ph, a, s, 43) && wait(&s->a_full[ab.i], ab.ph, a, s, 44);
                    if (!ok) break;
                    const uint32_t xa = smem_u32(sX + x.i * x_bytes(TOK)), at = tA + ab.i * 32;
#pragma unroll
                    for (int g = 0; g < HG; ++g) {
                        if (G < 128 || (h & 1) == 0) {
                            ok = wait(&s->d_empty[db.i], db.ph ^ 1, a, s, 45);
                            if (!ok) break;
                        }
                        tc_fence_after();
                        const uint32_t dt = tmem + db.i * 64;
#pragma unroll
                        for (int kk = g * (4 / HG); kk < (g + 1) * (4 / HG); ++kk)
                            umma_bf16_ts(dt, at + kk * 8, sdesc_k128(xa + kk * 32), idesc,
                                         kk != g * (4 / HG) || (G == 128 && (h & 1)));
                        if (G < 128 || (h & 1)) {
                            umma_commit(&s->d_full[db.i]);
                            db.next();
                        }
                    }
                    if (!ok) break;
                    umma_commit(&s->a_empty[ab.i]);
                    umma_commit(&s->x_empty[x.i]);
                    ab.next();
                    x.next();
                }
            }
            // every MMA issued here is complete before tensor memory is freed
            umma_commit(&s->drain);
            mbar_wait(&s->drain, 0, a.wait_limit);
        }
        __syncwarp();
    } else if (warp >= kDeqWarp) {
        // ------------------------------------------------------- unpacking
        const int r = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int rot = (r >> 1) & 3;                  // 64-byte swizzle of the row's 16-byte pieces
        // (w & mask) | set: 128 + q as a bf16 pair, or ones in the last row
        const uint32_t mask = r == kRows ? 0u : 0x000F000Fu, set = r == kRows ? 0x3F803F80u : 0x43004300u;
        Ring<kW> w;
        Ring<kA> ab;
        bool ok = true;
        for (int tile = first; tile < tiles && ok; tile += step) {
            for (int u = u0; u < u1 && ok; ++u) {
                ok = warp_wait(&s->w_full[w.i], w.ph, a, s, 46);
                if (!ok) break;
                const uint8_t *row = sW + w.i * kWBytes + r * 64;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint4 v0 = *reinterpret_cast<const uint4 *>(row + (((2 * h) ^ rot) << 4));
                    const uint4 v1 = *reinterpret_cast<const uint4 *>(row + (((2 * h + 1) ^ rot) << 4));
                    const uint32_t q[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
                    uint32_t p[32];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) p[4 * i + j] = mask_set(q[i] >> (4 * j), mask, set);
                    ok = warp_wait(&s->a_empty[ab.i], ab.ph ^ 1, a, s, 47);
                    if (!ok) break;
                    tc_fence_after();
                    tmem_st16((tA + ab.i * 32) | lanes, p);
                    tmem_st16((tA + ab.i * 32 + 16) | lanes, p + 16);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s->a_full[ab.i]);
                    ab.next();
                }
                if (!ok) break;
                if (lane == 0) mbar_arrive(&s->w_empty[w.i]);
                w.next();
            }
        }
    } else {
        // -------------------------------------------------------- epilogue
        const int half = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        Ring<kS> sc;
        Ring<kD> db;
        bool ok = true;
        for (int tile = first; tile < tiles; tile += step) {
            uint64_t y[TW / 2];
#pragma unroll
            for (int i = 0; i < TW / 2; ++i) y[i] = 0;
            int block = -1;
            uint4 sv = make_uint4(0u, 0u, 0u, 0u), bv = sv;
            const int g0 = u0 * kUnit / G, g1 = u1 * kUnit / G;
            for (int g = g0; g < g1 && ok; ++g) {
                if (g / 8 != block) {
                    // the row's scales and biases of eight groups
                    block = g / 8;
                    ok = warp_wait(&s->s_full[sc.i], sc.ph, a, s, 48);
                    if (!ok) break;
                    const uint8_t *src = sS + sc.i * 2 * kSBytes + r * 16;
                    sv = *reinterpret_cast<const uint4 *>(src);
                    bv = *reinterpret_cast<const uint4 *>(src + kSBytes);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s->s_empty[sc.i]);
                    sc.next();
                }
                ok = warp_wait(&s->d_full[db.i], db.ph, a, s, 49);
                if (!ok) break;
                tc_fence_after();
                uint32_t d[TW];
                const uint32_t at = (tmem + db.i * 64 + half * TW) | lanes;
                if constexpr (TW == 32) {
                    tmem_ld32(at, d);
                    tmem_wait32(d);
                } else if constexpr (TW == 16) {
                    tmem_ld16_now(at, d);
                } else {
                    tmem_ld8_now(at, d);
                }
                float *sums = s->sums[db.i] + half * TW;
                if (r == kRows) {
#pragma unroll
                    for (int i = 0; i < TW; i += 4)
                        *reinterpret_cast<uint4 *>(sums + i) = make_uint4(d[i], d[i + 1], d[i + 2], d[i + 3]);
                    mbar_arrive(&s->sum_full[half][db.i]);
                }
                __syncwarp();
                ok = warp_wait(&s->sum_full[half][db.i], db.ph, a, s, 50);
                if (!ok) break;
                const int gi = g & 7;
                const uint32_t sw = (gi >> 1) == 0 ? sv.x : (gi >> 1) == 1 ? sv.y : (gi >> 1) == 2 ? sv.z : sv.w;
                const uint32_t bw = (gi >> 1) == 0 ? bv.x : (gi >> 1) == 1 ? bv.y : (gi >> 1) == 2 ? bv.z : bv.w;
                const float scale = __uint_as_float(gi & 1 ? sw & 0xFFFF0000u : sw << 16);
                const float bias = fmaf(-128.f, scale, __uint_as_float(gi & 1 ? bw & 0xFFFF0000u : bw << 16));
                const uint64_t s2 = pack2(__float_as_uint(scale), __float_as_uint(scale));
                const uint64_t b2 = pack2(__float_as_uint(bias), __float_as_uint(bias));
#pragma unroll
                for (int i = 0; i < TW / 4; ++i) {
                    const uint4 X = *reinterpret_cast<const uint4 *>(sums + 4 * i);
                    y[2 * i] = fma2(s2, pack2(d[4 * i], d[4 * i + 1]), fma2(b2, pack2(X.x, X.y), y[2 * i]));
                    y[2 * i + 1] = fma2(s2, pack2(d[4 * i + 2], d[4 * i + 3]), fma2(b2, pack2(X.z, X.w), y[2 * i + 1]));
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s->d_empty[db.i]);
                db.next();
            }
            if (a.split == 1) {
                if (!ok) break;
                const int row = tile * kRows + r;
                if (r < kRows && row < a.N) {
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
                red[(half * TW + 2 * i) * 128 + r] = v.x;
                red[(half * TW + 2 * i + 1) * 128 + r] = v.y;
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
            const int t = t0 + i / 128, r = i % 128, row = first * kRows + r;
            if (r >= kRows || row >= a.N) continue;
            float sum = 0.f;
            for (int p = 0; p < a.split; ++p) sum += dsmem_ld(smem_u32(red + t * 128 + r), p);
            a.store(t, row, sum);
        }
        cluster_sync();
    }
}

template <int G, int TOK>
static cudaError_t launch_t(const Maps &maps, LinearArgs a, int num_sms, cudaStream_t s) {
    const int units = (a.K + kUnit - 1) / kUnit, tiles = (a.N + kRows - 1) / kRows;
    // share K in a cluster while there are two units for each block and all
    // clusters run at once (one tile each)
    a.split = 1;
    while (a.split < 4 && tiles * a.split * 2 <= num_sms * 7 / 8 && units >= a.split * 4) a.split *= 2;
    const auto kernel = linear_many_kernel<G, TOK>;
    const cudaError_t e = allow_smem<linear_many_kernel<G, TOK>>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(a.split > 1 ? tiles * a.split : std::min(tiles, num_sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes(TOK);
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

cudaError_t launch_linear_many(const CUtensorMap *maps, const LinearArgs &a, int num_sms, cudaStream_t s) {
    const many::Maps m{maps[0], maps[1], maps[2], maps[3]};
    if (a.G == 32) return many::launch_g<32>(m, a, num_sms, s);
    if (a.G == 64) return many::launch_g<64>(m, a, num_sms, s);
    return many::launch_g<128>(m, a, num_sms, s);
}

}  // namespace moe
