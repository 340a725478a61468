// Log probabilities of given tokens, the entropy and the most probable tokens of
// rows of scores, in one pass over the scores.
//
//   sums     with a reference r, S = sum e^(x - r) and U = sum e^(x - r) (x - r):
//            log sum e^x = r + log S, entropy = log S - U / S.  Each thread has a
//            reference of its own, the maximum of its first eight scores, which it
//            moves only when a score exceeds it by 8 (S and U are then scaled): e^8
//            costs nothing of fp32's accuracy, and a running maximum would be moved
//            in most batches by one of a warp's lanes
//   top      each warp keeps the 32 best scores so far, sorted, a lane each, as one
//            64-bit number of value and id.  Of a batch of 256 scores it looks at the
//            lanes' maxima only, which the sums need anyway; where one exceeds the
//            n-th best, the scores that do go to a buffer, and 32 of them are
//            sorted and merged with the list by exchanges between lanes (15 + 6
//            steps).  For scores in random order that is n log(V / 8n) of V / 8 scores a
//            warp; in rising order every score is sorted
//   work     a row is cut into parts where there are too few rows for the GPU, a
//            block of eight warps each, whose sums and lists are merged through shared
//            memory; scores_merge_kernel merges the parts.  Short rows of many are a
//            warp's each
//
// Bound by the bytes of the scores: 64 bytes a thread are in flight.
#include "scores.cuh"

#include <algorithm>

namespace moe {

typedef unsigned long long u64;

constexpr int kWarps = 8;             // of a block
constexpr int kBatch = 256;           // scores that a warp takes at a time, eight a lane
constexpr int kPartBatches = 16;      // of a part at least
constexpr float kLogRaise = 8.f;
constexpr float kLeast = -3.402823466e38f;

// A score's place in the order of alternatives: larger scores first, NaN before
// all, equal ones (zeros of both signs too) by lower id; 0: none.
__device__ __forceinline__ u64 rank_key(float x, int id) {
    const uint32_t u = x != x ? 0x7FFFFFFFu : __float_as_uint(x + 0.f);
    const uint32_t up = u & 0x80000000u ? ~u : u | 0x80000000u;
    return static_cast<u64>(up) << 32 | ~static_cast<uint32_t>(id);
}
__device__ __forceinline__ float key_score(u64 k) {
    const uint32_t up = static_cast<uint32_t>(k >> 32);
    return __uint_as_float(up & 0x80000000u ? up & 0x7FFFFFFFu : ~up);
}
__device__ __forceinline__ int key_id(u64 k) { return static_cast<int>(~static_cast<uint32_t>(k)); }

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// 2^x by the hardware's approximation (relative error about 2^-22).
__device__ __forceinline__ float exp2_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float exp_of(float t) { return exp2_of(t * 1.4426950408889634f); }

// ------------------------------------------------------------------ lists

template <typename K>
__device__ __forceinline__ K larger(K a, K b) { return a > b ? a : b; }
template <typename K>
__device__ __forceinline__ K smaller(K a, K b) { return a < b ? a : b; }

// A bitonic sequence of 32 (a lane each) into descending order.
template <typename K>
__device__ __forceinline__ K bitonic_merge(K k, int lane) {
#pragma unroll
    for (int j = 16; j; j >>= 1) {
        const K o = __shfl_xor_sync(0xffffffffu, k, j);
        k = lane & j ? smaller(k, o) : larger(k, o);
    }
    return k;
}

template <typename K>
__device__ __forceinline__ K sort32(K k, int lane) {
#pragma unroll
    for (int size = 2; size < 32; size <<= 1) {
#pragma unroll
        for (int j = size >> 1; j; j >>= 1) {
            const K o = __shfl_xor_sync(0xffffffffu, k, j);
            k = ((lane & size) == 0) == ((lane & j) == 0) ? larger(k, o) : smaller(k, o);
        }
    }
    return bitonic_merge(k, lane);
}

// The 32 best of two descending lists.
__device__ __forceinline__ u64 merge32(u64 a, u64 b, int lane) {
    return bitonic_merge(larger(a, __shfl_sync(0xffffffffu, b, 31 - lane)), lane);
}

// The float before x (plus infinity or finite): y > before(x) where y >= x; NaN for
// minus infinity.
__device__ __forceinline__ float before(float x) {
    const uint32_t u = __float_as_uint(x);
    return __uint_as_float(u == 0 || u == 0x80000000u ? 0x80000001u : u & 0x80000000u ? u + 1 : u - 1);
}

// The 32 best of a warp's scores so far.
struct Best {
    u64 list = 0;           // this lane's
    float above = NAN;      // a score that is not `<=` this may be among the n best
    int waiting = 0;        // scores in the buffer

    // equal: a score equal to the n-th best may still have a lower id, which is so
    // within a batch, but not from one to the next
    __device__ __forceinline__ void set_above(int n, bool equal) {
        const u64 k = __shfl_sync(0xffffffffu, list, n - 1);
        const float x = key_score(k), y = x != x ? INFINITY : x;
        // fewer than n: NaN, which takes all; the n-th a NaN: only NaN comes before it
        above = k == 0 ? NAN : equal ? before(y) : y;
    }
    __device__ __forceinline__ void sort_in(const u64 *buffer, int n, int lane) {
        __syncwarp();
        const u64 k = lane < waiting ? buffer[lane] : 0;
        const u64 rest = 32 + lane < waiting ? buffer[32 + lane] : 0;
        __syncwarp();
        list = merge32(list, sort32(k, lane), lane);
        if (waiting > 32) const_cast<u64 *>(buffer)[lane] = rest;
        waiting = waiting > 32 ? waiting - 32 : 0;
        set_above(n, true);
    }
    __device__ __forceinline__ void offer(float x, int id, bool real, u64 *buffer, int n, int lane) {
        const bool take = real && !(x <= above);
        const unsigned m = __ballot_sync(0xffffffffu, take);
        if (!m) return;
        if (take) buffer[waiting + __popc(m & ((1u << lane) - 1))] = rank_key(x, id);
        waiting += __popc(m);
        if (waiting >= 32) sort_in(buffer, n, lane);
    }
    // Scores of one lane alone.
    template <typename F>
    __device__ __forceinline__ void offer_lane(const float (&x)[8], int of, F id, u64 *buffer, int n, int lane) {
        int k = 0;
        if (lane == of) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (!(x[i] <= above) && id(i) >= 0) buffer[waiting + k++] = rank_key(x[i], id(i));
        }
        waiting += __shfl_sync(0xffffffffu, k, of);
        if (waiting >= 32) sort_in(buffer, n, lane);
    }
};

// ------------------------------------------------------------------- sums

struct Sums {
    float r, S, U;

    __device__ __forceinline__ void move(float to) {
        const float d = r - to, c = exp_of(d);
        U = S > 0.f && c > 0.f ? c * (U + d * S) : 0.f;  // (d may be minus infinity)
        S *= c;
        r = to;
    }
    __device__ __forceinline__ void add(const Sums &o) {
        Sums b = o;
        const float to = max_nan(r, b.r);
        move(to);
        b.move(to);
        S += b.S;
        U += b.U;
    }
};

// What a row's sums and list say, by a warp.
__device__ __forceinline__ void finish_row(const ScoresArgs &a, int t, int target, float given, const Sums &s, u64 list, int lane) {
    // a NaN, a plus infinity, or no score above minus infinity: no distribution
    const bool none = !(s.r < INFINITY) || !(s.S > 0.f);
    const float logS = none ? NAN : logf(s.S);
    if (lane == 0) {
        if (a.logprob) {
            if (target >= a.V) record_status(a.status, MOE_ERR_TOKEN_ID);
            a.logprob[t] = target < a.V ? (given - s.r) - logS : NAN;
        }
        if (a.entropy) a.entropy[t] = logS - s.U / s.S;
    }
    if (lane < a.n_top) {
        const int64_t at = static_cast<int64_t>(t) * a.n_top + lane;
        a.top_ids[at] = key_id(list);
        a.top_logprobs[at] = (key_score(list) - s.r) - logS;
    }
}

// Merges the sums and lists of each WPR warps, halves at a time; the first of them
// returns with all.
template <int WPR>
__device__ __forceinline__ void merge_warps(Sums &s, u64 &list, bool top, int warp, int lane) {
    __shared__ Sums sums[kWarps];
    __shared__ u64 lists[kWarps][32];
    const int mine = warp % WPR;
#pragma unroll
    for (int half = WPR / 2; half; half >>= 1) {
        if (mine >= half && mine < 2 * half) {
            if (lane == 0) sums[warp] = s;
            if (top) lists[warp][lane] = list;
        }
        __syncthreads();
        if (mine < half) {
            s.add(sums[warp + half]);
            if (top) list = merge32(list, lists[warp + half][lane], lane);
        }
    }
}

__device__ __forceinline__ void merge_lanes(Sums &s) {
#pragma unroll
    for (int i = 16; i; i >>= 1) {
        const Sums o{__shfl_xor_sync(0xffffffffu, s.r, i), __shfl_xor_sync(0xffffffffu, s.S, i),
                     __shfl_xor_sync(0xffffffffu, s.U, i)};
        s.add(o);
    }
}

// ------------------------------------------------------------------- main

template <typename E>
__device__ __forceinline__ float score(const E *p) {
    if constexpr (sizeof(E) == 4)
        return __ldcs(p);
    else
        return bf16_bits_to_float(__ldcs(reinterpret_cast<const unsigned short *>(p)));
}

// A lane's eight scores of a batch: of the row's vectors of 16 bytes (which start
// at its first 16-byte boundary or the one before it) vector lane of each 32.
// Batches wait in shared memory, each lane's own 128 bytes of it, so that
// sorting does not stop the loads.
template <typename E>
struct Ring {
    static constexpr int VEC = 16 / sizeof(E), N = 8 / VEC, STAGES = 8 / N;
    uint4 *mine;  // [stage][N][32 lanes], this lane's

    // first: index in the row of the batch's first score; hi: the row's end (0: no batch)
    __device__ __forceinline__ void load(int stage, const E *row, int64_t first, int64_t hi, int lane) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int64_t e = first + (i * 32 + lane) * VEC;
            uint4 *to = mine + (stage * N + i) * 32;
            if (e >= 0 && e + VEC <= hi) {
                cp_async<16>(to, row + e);
            } else if (hi > 0) {
                // minus infinity where there is no score
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    auto at = [&](int64_t k) { return k >= 0 && k < hi ? __float_as_uint(score(row + k)) : 0xFF800000u; };
                    w[j] = sizeof(E) == 4 ? at(e + j) : at(e + 2 * j) >> 16 | at(e + 2 * j + 1);
                }
                *to = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        cp_async_commit();
    }
    __device__ __forceinline__ void read(int stage, float (&x)[8]) const {
        cp_async_wait<STAGES - 1>();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint4 v = mine[(stage * N + i) * 32];
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (sizeof(E) == 4) {
                    x[i * 4 + j] = __uint_as_float(w[j]);
                } else {
                    x[2 * j] = __uint_as_float(w[j] << 16);
                    x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
                }
            }
        }
    }
    __device__ __forceinline__ static int index(int i, int lane) { return (i / VEC * 32 + lane) * VEC + i % VEC; }
};

// ROWS: rows of a block, each for 8 / ROWS warps.
template <typename E, bool TOP, int ROWS>
__global__ void __launch_bounds__(kWarps * 32, 4) scores_kernel(const __grid_constant__ ScoresArgs a) {
    constexpr int WPR = kWarps / ROWS;
    __shared__ u64 buffers[TOP ? kWarps : 1][TOP ? 64 : 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    __shared__ uint4 ring_at[kWarps][8][32];
    const int t = ROWS > 1 ? blockIdx.x * ROWS + warp / WPR : blockIdx.x / a.parts;
    const int part = ROWS > 1 ? 0 : blockIdx.x % a.parts;
    const int mine = warp % WPR;  // of the row's warps
    // (a block's warps stay together until their lists are merged, also without a row)
    const int target = t < a.T ? (a.targets ? a.targets[t] : 0) : -1;
    if (WPR == 1 && target < 0) return;
    const E *row = static_cast<const E *>(a.x) + t * a.stride;
    const float given = a.logprob && target >= 0 && target < a.V ? score(row + target) : 0.f;
    u64 *buffer = buffers[TOP ? warp : 0];

    // batch b of the row: scores off + 256 b .. (off <= 0, to a 16-byte boundary)
    const int off = -static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(E));
    const int batches = (a.V - off + kBatch - 1) / kBatch;
    const int b1 = target < 0 ? 0 : ROWS > 1 ? batches : min(batches, (part + 1) * a.part_batches);
    int b = (ROWS > 1 ? 0 : part * a.part_batches) + mine;

    Sums s{kLeast, 0.f, 0.f};
    Best best;
    u64 S2 = 0, U2 = 0;  // pairs of partial sums
    const u64 log2e = pack2(0x3FB8AA3Bu, 0x3FB8AA3Bu);
    // the warps' ceil(n / warps)-th best: n scores at least are not below the least of them
    __shared__ u64 quantiles[kWarps];
    const int nth_share = TOP ? (a.n_top + WPR - 1) / WPR - 1 : 0;
    if (TOP && WPR > 1) {
        if (threadIdx.x < kWarps) quantiles[threadIdx.x] = 0;
        __syncthreads();
    }
    // what the block's warps together leave of `above`
    auto share = [&]() {
        if (WPR == 1) return;
        const u64 nth = __shfl_sync(0xffffffffu, best.list, nth_share);
        if (lane == 0) *const_cast<volatile u64 *>(quantiles + warp) = nth;
        u64 q = *const_cast<volatile u64 *>(quantiles + warp - mine + lane % WPR);
#pragma unroll
        for (int i = WPR / 2; i; i >>= 1) q = smaller(q, __shfl_xor_sync(0xffffffffu, q, i));
        // (zero: a warp has too few yet; before(minus infinity) and a NaN among the best
        // take all, as NaN)
        const float y = before(key_score(q));
        if (q && y == y && !(y <= best.above)) best.above = y;
    };
    const Ring<E> ring{&ring_at[warp][0][lane]};
    constexpr int STAGES = Ring<E>::STAGES;
    auto load = [&](int stage, int b) { ring.load(stage, row, off + static_cast<int64_t>(b) * kBatch, b < b1 ? a.V : 0, lane); };
#pragma unroll
    for (int i = 0; i < STAGES; ++i) load(i, b + i * WPR);
    bool first = true;
    for (int stage = 0; b < b1; b += WPR, stage = (stage + 1) % STAGES) {
        const int at = off + b * kBatch;
        float x[8];
        ring.read(stage, x);
        const float top = max3_nan(max3_nan(x[0], x[1], x[2]), max3_nan(x[3], x[4], x[5]), max_nan(x[6], x[7]));
        if (first || !(top <= s.r + kLogRaise)) {
            const float to = max_nan(top, kLeast), d = s.r - to, c = exp_of(d);
            const u64 c2 = pack2(__float_as_uint(c), __float_as_uint(c)), d2 = pack2(__float_as_uint(d), __float_as_uint(d));
            const float2 v = unpack2(S2);
            U2 = v.x + v.y > 0.f && c > 0.f ? fma2(c2, fma2(d2, S2, U2), 0) : 0;
            S2 = fma2(c2, S2, 0);
            s.r = to;
        }
        const u64 minus_r = pack2(__float_as_uint(-s.r), __float_as_uint(-s.r));
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            float2 d = unpack2(add2(pack2(__float_as_uint(x[i]), __float_as_uint(x[i + 1])), minus_r));
            // (a score of minus infinity weighs nothing: e^-10000 = 0)
            d.x = fmaxf(d.x, -10000.f);
            d.y = fmaxf(d.y, -10000.f);
            const u64 d2 = pack2(__float_as_uint(d.x), __float_as_uint(d.y));
            const float2 y = unpack2(fma2(d2, log2e, 0));
            const u64 e2 = pack2(__float_as_uint(exp2_of(y.x)), __float_as_uint(exp2_of(y.y)));
            S2 = add2(S2, e2);
            U2 = fma2(e2, d2, U2);
        }
        load(stage, b + STAGES * WPR);  // (its scores are in registers)
        if (TOP) {
            if (first && at >= 0 && at + kBatch <= a.V) {
                // the n-th of the lanes' maxima is not above the n-th best
                const uint32_t k = sort32(static_cast<uint32_t>(rank_key(top, 0) >> 32), lane);
                const float nth = key_score(static_cast<u64>(__shfl_sync(0xffffffffu, k, a.n_top - 1)) << 32);
                if (nth > -INFINITY) best.above = before(nth);
            }
            const unsigned lanes = __ballot_sync(0xffffffffu, !(top <= best.above));
            if (lanes) {
                auto id_of = [&](int i) {
                    const int id = at + Ring<E>::index(i, lane);
                    return id < a.V ? id : -1;
                };
                if ((lanes & (lanes - 1)) == 0) {
                    best.offer_lane(x, __ffs(lanes) - 1, id_of, buffer, a.n_top, lane);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) best.offer(x[i], id_of(i), id_of(i) >= 0, buffer, a.n_top, lane);
                }
                if (first && best.waiting) best.sort_in(buffer, a.n_top, lane);
                best.set_above(a.n_top, false);
                share();
            }
        }
        first = false;
    }
    if (TOP) {
        while (best.waiting) best.sort_in(buffer, a.n_top, lane);
    }
    const float2 S1 = unpack2(S2), U1 = unpack2(U2);
    s.S = S1.x + S1.y;
    s.U = U1.x + U1.y;
    merge_lanes(s);
    merge_warps<WPR>(s, best.list, TOP, warp, lane);
    if (mine || target < 0) return;
    if (a.parts == 1) {
        finish_row(a, t, target, given, s, best.list, lane);
    } else {
        if (lane == 0) a.part_sums[blockIdx.x] = make_float4(s.r, s.S, s.U, 0.f);
        if (TOP) a.part_top[static_cast<int64_t>(blockIdx.x) * 32 + lane] = best.list;
    }
}

// Merges a row's parts: a block a row.
template <typename E>
__global__ void __launch_bounds__(kWarps * 32) scores_merge_kernel(const __grid_constant__ ScoresArgs a) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = blockIdx.x;
    pdl_wait();
    pdl_trigger();
    const int target = a.targets ? a.targets[t] : 0;
    if (target < 0) return;
    const float given = a.logprob && target < a.V ? score(static_cast<const E *>(a.x) + t * a.stride + target) : 0.f;
    Sums s{kLeast, 0.f, 0.f};
    u64 list = 0;
    const int64_t base = static_cast<int64_t>(t) * a.parts;
    // a lane a part of the sums, a warp a part of the lists
    for (int p = threadIdx.x; p < a.parts; p += kWarps * 32) {
        const float4 v = __ldcg(a.part_sums + base + p);
        s.add(Sums{v.x, v.y, v.z});
    }
    if (a.n_top)
        for (int p = warp; p < a.parts; p += kWarps) list = merge32(list, __ldcg(a.part_top + (base + p) * 32 + lane), lane);
    merge_lanes(s);
    merge_warps<kWarps>(s, list, a.n_top > 0, warp, lane);
    if (warp == 0) finish_row(a, t, target, given, s, list, lane);
}

// ------------------------------------------------------------------- host

// Parts of a row: as many as leave each SM its four blocks, of 4096 scores at least.
static int row_parts(int T, int V, int sms) {
    const int most = std::max(1, V / (kBatch * kPartBatches));
    return std::max(1, std::min(4 * sms / T, most));
}

size_t scores_workspace_bytes(int T, int V, int n_top, int max_sms) {
    const int parts = row_parts(T, V, max_sms);
    const size_t blocks = parts > 1 ? static_cast<size_t>(T) * parts : 0;
    return kCtrlBytes + blocks * (sizeof(float4) + (n_top ? 32 * sizeof(u64) : 0));
}

template <typename E, bool TOP, int ROWS>
static cudaError_t launch_rows(const ScoresArgs &a, cudaStream_t s) {
    return launch_dependent(scores_kernel<E, TOP, ROWS>, dim3((a.T + ROWS - 1) / ROWS * a.parts), dim3(kWarps * 32), 0, s, a);
}

template <typename E, bool TOP>
static cudaError_t launch_e(ScoresArgs &a, void *ws, int num_sms, cudaStream_t s) {
    a.parts = row_parts(a.T, a.V, num_sms);
    if (a.parts == 1) {
        // the fewer warps a row has, the fewer lists are made and merged: as few as
        // leave each SM its 32 warps, or as the row has batches for
        const int most = 4 * num_sms * kWarps / a.T, need = a.V / kBatch;
        a.part_batches = 1 << 30;
        if (most < 2 || need < 2) return launch_rows<E, TOP, 8>(a, s);
        if (most < 4 || need < 4) return launch_rows<E, TOP, 4>(a, s);
        if (most < 8 || need < 8) return launch_rows<E, TOP, 2>(a, s);
        return launch_rows<E, TOP, 1>(a, s);
    }
    // (up to a vector before the row counts with it)
    const int batches = (a.V + 16 / static_cast<int>(sizeof(E)) - 1 + kBatch - 1) / kBatch;
    a.part_batches = (batches + a.parts - 1) / a.parts;
    a.part_sums = reinterpret_cast<float4 *>(static_cast<char *>(ws) + kCtrlBytes);
    a.part_top = reinterpret_cast<u64 *>(a.part_sums + static_cast<size_t>(a.T) * a.parts);
    const cudaError_t e = launch_rows<E, TOP, 1>(a, s);
    if (e != cudaSuccess) return e;
    return launch_dependent(scores_merge_kernel<E>, dim3(a.T), dim3(kWarps * 32), 0, s, a);
}

cudaError_t launch_scores(ScoresArgs &a, void *ws, int num_sms, cudaStream_t s) {
    if (a.fp32) return a.n_top ? launch_e<float, true>(a, ws, num_sms, s) : launch_e<float, false>(a, ws, num_sms, s);
    return a.n_top ? launch_e<__nv_bfloat16, true>(a, ws, num_sms, s) : launch_e<__nv_bfloat16, false>(a, ws, num_sms, s);
}

}  // namespace moe
