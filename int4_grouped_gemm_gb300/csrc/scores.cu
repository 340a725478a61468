// Log probabilities of given tokens, the entropy and the most probable tokens of
// rows of scores, in one pass over the scores.
//
//   sums     with a reference r, S = sum e^(x - r) and U = sum e^(x - r) (x - r):
//            log sum e^x = r + log S, entropy = log S - U / S.  r is a warp's largest
//            score so far, the same in all lanes, so that the row's largest one counts as
//            exactly 1 at the end and log S and U / S are small where a token is nearly
//            certain.  (With a reference of each thread's own that scores may exceed by 8,
//            log S and x - r cancelled: a log probability of -3.4e-4 was off by 7e-7, now by
//            6e-8.)  It is found by a vote for each batch, and moved (S and U are then
//            scaled) about log n times in n batches, where the maximum of each lane would
//            be moved in most of them by one of 32: 4096 x 50021 bf16 96.6 us, with the
//            threads' own references 95.8, fp32 133.0 and 132.6
//   top      the pass keeps, of each lane's scores, the maximum of every eighth part
//            (the sums need the maxima anyway).  At its end the warps' ceil(n / warps)-th
//            largest of these maxima, the least of them, is a value that n scores at least
//            reach; the few eighths that reach it are read again, 1 to 2 n of the row's
//            256 to 2048.  At most 64 of their scores reach it nearly always: the row's
//            first warp puts them in order by counting the larger ones.  More are sorted
//            32 at a time and merged with the list of the 32 best, a lane each, by
//            exchanges between lanes (15 + 6 steps).  (A list kept during the pass, by
//            each warp, took as many instructions as the sums in long rows, and several
//            times as many in short ones: 257 x 50021 with 5 alternatives 39 us, so 16 to 19)
//   work     a row is cut into parts where there are too few rows for the GPU, a
//            block of eight warps each, whose sums are merged through shared memory and
//            whose scores that reach the n are sorted by the first one;
//            scores_merge_kernel merges the parts.  Short rows of many are a warp's each
//
// Bound by the bytes of fp32 scores: 96 to 128 bytes a thread are in flight, 4096 x 131072
// with 8 alternatives take 319 to 325 us, 6.6 TB/s.  bf16 ones are bound by the instructions
// (issue slots 65 %, ALU 57 %): 4096 x 50021 97 us, 4.2 TB/s.
#include "scores.cuh"

#include <algorithm>

namespace moe {

typedef unsigned long long u64;

constexpr int kWarps = 8;             // of a block
constexpr int kBatch = 256;           // scores that a warp takes at a time, eight a lane
constexpr int kPartBatches = 16;      // of a part at least
constexpr int kEighths = 8;           // parts of a lane's scores whose maxima are kept
constexpr float kLeast = -3.402823466e38f;

// A score's place in the order of alternatives: larger scores first, NaN before
// all, zeros of both signs equal; never 0.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = x != x ? 0x7FFFFFFFu : __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
// ... and equal ones by lower id; 0: none.
__device__ __forceinline__ u64 rank_key(uint32_t order, int id) { return static_cast<u64>(order) << 32 | ~static_cast<uint32_t>(id); }
__device__ __forceinline__ float score_of(uint32_t order) {
    return __uint_as_float(order & 0x80000000u ? order & 0x7FFFFFFFu : ~order);
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

// The 32 best of the scores that a warp looks at, which are those of `least` (an
// order) at least.
struct Best {
    u64 list = 0, nth = 0;  // this lane's; the n-th
    uint32_t least;
    int waiting = 0;        // scores in the buffer (of 64)

    __device__ __forceinline__ void sort_in(u64 *buffer, int n, int lane) {
        __syncwarp();
        const u64 k = lane < waiting ? buffer[lane] : 0;
        const u64 rest = 32 + lane < waiting ? buffer[32 + lane] : 0;
        __syncwarp();
        list = merge32(list, sort32(k, lane), lane);
        if (waiting > 32) buffer[lane] = rest;
        waiting = waiting > 32 ? waiting - 32 : 0;
        nth = __shfl_sync(0xffffffffu, list, n - 1);
        least = larger(least, static_cast<uint32_t>(nth >> 32));
    }
    // Each lane's x[0 .. N - 1], of ids at .. at + N - 1 (those in 0 .. hi - 1 count).
    template <int N>
    __device__ __forceinline__ void offer(const float (&x)[N], int at, int hi, u64 *buffer, int n, int lane) {
        const float from = score_of(least);
        unsigned hits = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) hits |= (hi > 0 && !(x[j] < from)) << j;
        while (__any_sync(0xffffffffu, hits != 0)) {
            const int j = __ffs(hits) - 1;
            float y = x[0];
#pragma unroll
            for (int i = 1; i < N; ++i) y = i == j ? x[i] : y;
            const uint32_t o = order_of(y);
            const u64 key = rank_key(o, at + j);
            const bool take = hits && at + j >= 0 && at + j < hi && o >= least && key > nth;
            hits &= hits - 1;
            const unsigned m = __ballot_sync(0xffffffffu, take);
            if (take) buffer[waiting + __popc(m & ((1u << lane) - 1))] = key;
            waiting += __popc(m);
            if (waiting >= 32) sort_in(buffer, n, lane);
        }
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
    // Those of each `of` neighbouring lanes (taken to the largest reference of the warp).
    template <int of>
    __device__ __forceinline__ void add_lanes() {
        move(score_of(__reduce_max_sync(0xffffffffu, order_of(r))));
#pragma unroll
        for (int i = of / 2; i; i >>= 1) {
            S += __shfl_xor_sync(0xffffffffu, S, i);
            U += __shfl_xor_sync(0xffffffffu, U, i);
        }
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
        a.top_logprobs[at] = (score_of(static_cast<uint32_t>(list >> 32)) - s.r) - logS;
    }
}

// A padding row's results, by a warp.
__device__ __forceinline__ void fill_row(const ScoresArgs &a, int t, int lane) {
    if (lane == 0) {
        if (a.logprob) a.logprob[t] = NAN;
        if (a.entropy) a.entropy[t] = NAN;
    }
    if (lane < a.n_top) {
        const int64_t at = static_cast<int64_t>(t) * a.n_top + lane;
        a.top_ids[at] = -1;
        a.top_logprobs[at] = NAN;
    }
}

// Merges the sums, and with `top` the lists (halves at a time), of each WPR warps; the
// first of them returns with all.
template <int WPR>
__device__ __forceinline__ void merge_warps(Sums &s, u64 &list, bool top, int warp, int lane) {
    __shared__ Sums sums[kWarps];
    __shared__ u64 lists[kWarps][32];
    const int mine = warp % WPR;
    if (WPR > 1) {
        if (lane == 0) sums[warp] = s;
        __syncthreads();
        if (mine == 0) {
            s = sums[warp + lane % WPR];
            s.add_lanes<WPR>();
        }
    }
    if (!top) return;
#pragma unroll
    for (int half = WPR / 2; half; half >>= 1) {
        if (mine >= half && mine < 2 * half) lists[warp][lane] = list;
        __syncthreads();
        if (mine < half) list = merge32(list, lists[warp + half][lane], lane);
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

    // The vector from score e of the row on, minus infinity where there is no score.
    __device__ __forceinline__ static uint4 edge(const E *row, int64_t e, int64_t hi) {
        auto at = [&](int64_t k) { return k >= 0 && k < hi ? __float_as_uint(score(row + k)) : 0xFF800000u; };
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = sizeof(E) == 4 ? at(e + j) : at(e + 2 * j) >> 16 | at(e + 2 * j + 1);
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ static void unpack(float *x, const uint4 &v) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (sizeof(E) == 4) {
                x[j] = __uint_as_float(w[j]);
            } else {
                x[2 * j] = __uint_as_float(w[j] << 16);
                x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
            }
        }
    }
    __device__ __forceinline__ static void fetch(float *x, const E *row, int64_t e, int64_t hi) {
        unpack(x, e >= 0 && e + VEC <= hi ? __ldcg(reinterpret_cast<const uint4 *>(row + e)) : edge(row, e, hi));
    }
    // first: index in the row of the batch's first score; hi: the row's end (0: no batch)
    __device__ __forceinline__ void load(int stage, const E *row, int first, int hi, int lane) const {
        const bool inner = first >= 0 && first + kBatch <= hi;  // (all lanes alike)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = first + (i * 32 + lane) * VEC;
            uint4 *to = mine + (stage * N + i) * 32;
            if (inner || (e >= 0 && e + VEC <= hi))
                cp_async<16>(to, row + e);
            else if (hi > 0)
                *to = edge(row, e, hi);
        }
        cp_async_commit();
    }
    __device__ __forceinline__ void read(int stage, float (&x)[8]) const {
        cp_async_wait<STAGES - 1>();
#pragma unroll
        for (int i = 0; i < N; ++i) unpack(x + i * VEC, mine[(stage * N + i) * 32]);
    }
};

// ROWS: rows of a block, each for 8 / ROWS warps.
template <typename E, bool TOP, int ROWS>
__global__ void __launch_bounds__(kWarps * 32, 4) scores_kernel(const __grid_constant__ ScoresArgs a) {
    constexpr int WPR = kWarps / ROWS;
    __shared__ u64 buffers[TOP ? kWarps : 1][TOP ? 64 : 1];
    __shared__ uint32_t maxima[TOP ? kWarps : 1][kEighths][32], shares[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    __shared__ uint4 ring_at[kWarps][8][32];
    const int t = ROWS > 1 ? blockIdx.x * ROWS + warp / WPR : blockIdx.x / a.parts;
    const int part = ROWS > 1 ? 0 : blockIdx.x % a.parts;
    const int mine = warp % WPR;  // of the row's warps
    // (a block's warps stay together until their lists are merged, also without a row)
    const int target = t < a.T ? (a.targets ? a.targets[t] : 0) : -1;
    if (a.fill && t < a.T && target < 0 && mine == 0 && part == 0) fill_row(a, t, lane);
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
    u64 S2 = 0, U2 = 0;  // pairs of partial sums
    const u64 log2e = pack2(0x3FB8AA3Bu, 0x3FB8AA3Bu);
    const int b0 = b, own = b < b1 ? (b1 - b + WPR - 1) / WPR : 0;  // this warp's first batch and their number
    const int eighth = max(1, (own + kEighths - 1) / kEighths);
    float most = -INFINITY;  // of the eighth
    int left = eighth, done = 0;
    const Ring<E> ring{&ring_at[warp][0][lane]};
    constexpr int STAGES = Ring<E>::STAGES;
    auto load = [&](int stage, int b) { ring.load(stage, row, off + b * kBatch, b < b1 ? a.V : 0, lane); };
#pragma unroll
    for (int i = 0; i < STAGES; ++i) load(i, b + i * WPR);
    for (int stage = 0; b < b1; b += WPR, stage = (stage + 1) % STAGES) {
        float x[8];
        ring.read(stage, x);
        const float top = max3_nan(max3_nan(x[0], x[1], x[2]), max3_nan(x[3], x[4], x[5]), max_nan(x[6], x[7]));
        // (NaN goes through: to is NaN then, and stays)
        if (__any_sync(0xffffffffu, !(top <= s.r))) {
            const float to = score_of(__reduce_max_sync(0xffffffffu, order_of(max_nan(top, s.r))));
            const float d = s.r - to, c = exp_of(d);
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
            most = max_nan(most, top);
            if (--left == 0) {
                maxima[warp][done++][lane] = order_of(most);
                left = eighth;
                most = -INFINITY;
            }
        }
    }
    const float2 S1 = unpack2(S2), U1 = unpack2(U2);
    s.S = S1.x + S1.y;
    s.U = U1.x + U1.y;
    s.add_lanes<32>();
    Best best;
    if (TOP) {
        if (left < eighth) maxima[warp][done++][lane] = order_of(most);
        // the share-th largest of the warp's maxima
        const int batches_here = ROWS > 1 ? batches : max(0, b1 - part * a.part_batches);
        const int with = min(WPR, max(1, batches_here)), share = (a.n_top + with - 1) / with;
        uint32_t m[kEighths], mx = 0, nth = 0;
#pragma unroll
        for (int i = 0; i < kEighths; ++i) m[i] = i < done ? maxima[warp][i][lane] : 0;
#pragma unroll
        for (int i = 0; i < kEighths; ++i) mx = larger(mx, m[i]);
        if (share > 4) {
            // (of the lanes' own maxima: lower, but in few steps)
            nth = __shfl_sync(0xffffffffu, sort32(mx, lane), share - 1);
        } else {
            for (int k = 0;;) {
                nth = __reduce_max_sync(0xffffffffu, mx);
                if (++k == share) break;
                // one of them, of the first lane that has it, goes
                bool goes = lane == __ffs(__ballot_sync(0xffffffffu, mx == nth)) - 1;
                mx = 0;
#pragma unroll
                for (int i = 0; i < kEighths; ++i) {
                    if (goes && m[i] == nth) {
                        m[i] = 0;
                        goes = false;
                    }
                    mx = larger(mx, m[i]);
                }
            }
        }
        if (WPR > 1) {
            // (a warp without batches has no say)
            if (lane == 0) shares[warp] = own ? nth : 0xFFFFFFFFu;
            __syncthreads();
            nth = shares[warp - mine + lane % WPR];
#pragma unroll
            for (int i = WPR / 2; i; i >>= 1) nth = smaller(nth, __shfl_xor_sync(0xffffffffu, nth, i));
        }
        best.least = nth;
        // the eighths that reach it
        auto look = [&](int at, int hi) {
            float x[Ring<E>::VEC];
            Ring<E>::fetch(x, row, at, hi);
            best.offer(x, at, hi, buffer, a.n_top, lane);
        };
        const int each = eighth * Ring<E>::N;  // vectors of an eighth
        auto vector = [&](int i, int v, int of) {
            return off + (b0 + (i * eighth + v / Ring<E>::N) * WPR) * kBatch + (v % Ring<E>::N * 32 + of) * Ring<E>::VEC;
        };
        // (the ring is empty)
        unsigned char *few = reinterpret_cast<unsigned char *>(&ring_at[warp][0][0]);
        int n_few = 0;
        __syncwarp();
        for (int i = 0; i < done; ++i) {
            const bool reaches = maxima[warp][i][lane] >= nth;
            const unsigned lanes = __ballot_sync(0xffffffffu, reaches);
            const int vectors = min(eighth, own - i * eighth) * Ring<E>::N;
            if (__popc(lanes) * ((vectors + 31) / 32) >= vectors) {
                // many lanes of a short eighth: all of it
                for (int v = 0; v < vectors; ++v) look(vector(i, v, lane), a.V);
            } else {
                if (reaches) few[n_few + __popc(lanes & ((1u << lane) - 1))] = static_cast<unsigned char>(i * 32 + lane);
                n_few += __popc(lanes);
            }
        }
        __syncwarp();
        // ... the others together, a lane a vector
        for (int p = lane; p - lane < n_few * each; p += 32) {
            const int k = p / each, v = p - k * each, of = k < n_few ? few[k] : 0;
            look(vector(of >> 5, v, of & 31), k < n_few && (of >> 5) * eighth + v / Ring<E>::N < own ? a.V : 0);
        }
    }
    bool merged = false;  // the lists are
    if (TOP && WPR > 1) {
        // nearly always a row's warps have at most 64 scores that none has sorted yet: the
        // first of them sorts them all
        __shared__ int counts[kWarps];
        if (lane == 0) counts[warp] = best.nth ? 65 : best.waiting;
        __syncthreads();
        const int count = counts[lane % kWarps];
        int of_row = count;
#pragma unroll
        for (int i = WPR / 2; i; i >>= 1) of_row += __shfl_xor_sync(0xffffffffu, of_row, i);
        merged = __all_sync(0xffffffffu, of_row <= 64);
        if (merged && mine == 0) {
            // each lane's two by the number of larger ones among them all
            u64 k[2] = {0, 0};
            int at = lane, all = 0;
#pragma unroll
            for (int w = 0; w < WPR; ++w) {
                const int n = __shfl_sync(0xffffffffu, count, warp + w);
                if (at >= 0 && at < n) k[0] = buffers[warp + w][at];
                if (at + 32 >= 0 && at + 32 < n) k[1] = buffers[warp + w][at + 32];
                at -= n;
                all += n;
            }
            u64 *list = buffer;
            __syncwarp();
            list[lane] = k[0];
            list[32 + lane] = k[1];
            __syncwarp();
            int rank[2] = {0, 0};
#pragma unroll 8
            for (int i = 0; i < all; ++i) {
                const u64 o = list[i];
                rank[0] += o > k[0];
                rank[1] += o > k[1];
            }
            __syncwarp();
            list[lane] = 0;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (k[i] && rank[i] < 32) list[rank[i]] = k[i];
            __syncwarp();
            best.list = list[lane];
        }
    }
    if (TOP && !merged && best.waiting) best.sort_in(buffer, a.n_top, lane);
    merge_warps<WPR>(s, best.list, TOP && !merged, warp, lane);
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
#pragma unroll 4
        for (int p = warp; p < a.parts; p += kWarps) list = merge32(list, __ldcg(a.part_top + (base + p) * 32 + lane), lane);
    s.add_lanes<32>();
    merge_warps<kWarps>(s, list, a.n_top > 0, warp, lane);
    if (warp == 0) finish_row(a, t, target, given, s, list, lane);
}

// ------------------------------------------------------------------- host

// Parts of a row: as many as give each SM two blocks, of 4096 scores at least.  (With
// four a block's beginning and end and the merge cost more than they bring: 64 rows of
// 131072 20.3 us where two take 16.3, 257 of 50021 21.5 and 16.7.)
static int most_parts(int V) { return std::max(1, V / (kBatch * kPartBatches)); }
static int row_parts(int T, int V, int sms) { return std::max(1, std::min(2 * sms / T, most_parts(V))); }

// (also for fewer rows, which have more parts)
size_t scores_workspace_bytes(int T, int V, int n_top, int max_sms) {
    const int most = most_parts(V);
    const size_t blocks = most > 1 ? std::min<size_t>(static_cast<size_t>(T) * most, 2 * max_sms) : 0;
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
        // a warp has 16 KB of a row (4096 x 50021 fp32 131 us, with 32 KB 139; bf16 97, with
        // 8 KB 116), or less where there are not 32 warps for each SM
        const int batches = a.V / kBatch, fill = 4 * num_sms * kWarps / a.T;
        const int warps = std::max(batches * static_cast<int>(sizeof(E)) / 64, std::min(fill, batches / 2));
        a.part_batches = 1 << 30;
        if (warps < 2) return launch_rows<E, TOP, 8>(a, s);
        if (warps < 4) return launch_rows<E, TOP, 4>(a, s);
        if (warps < 8) return launch_rows<E, TOP, 2>(a, s);
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
