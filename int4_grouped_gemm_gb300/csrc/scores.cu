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
constexpr int kPartBatches = 8;       // of a part at least
constexpr int kWarpRow = 4096;        // scores of the longest row that is a warp's
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

__device__ __forceinline__ float exp_of(float t) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(t * 1.4426950408889634f));
    return y;
}

// ------------------------------------------------------------------ lists

__device__ __forceinline__ u64 larger(u64 a, u64 b) { return a > b ? a : b; }
__device__ __forceinline__ u64 smaller(u64 a, u64 b) { return a < b ? a : b; }

// A bitonic sequence of 32 (a lane each) into descending order.
__device__ __forceinline__ u64 bitonic_merge(u64 k, int lane) {
#pragma unroll
    for (int j = 16; j; j >>= 1) {
        const u64 o = __shfl_xor_sync(0xffffffffu, k, j);
        k = lane & j ? smaller(k, o) : larger(k, o);
    }
    return k;
}

__device__ __forceinline__ u64 sort32(u64 k, int lane) {
#pragma unroll
    for (int size = 2; size < 32; size <<= 1) {
#pragma unroll
        for (int j = size >> 1; j; j >>= 1) {
            const u64 o = __shfl_xor_sync(0xffffffffu, k, j);
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

// Merges the warps' sums and lists; the first warp returns with the block's.
__device__ __forceinline__ void merge_warps(Sums &s, u64 &list, bool top, int warp, int lane) {
    __shared__ Sums sums[kWarps];
    __shared__ u64 lists[kWarps][32];
    if (lane == 0) sums[warp] = s;
    if (top) lists[warp][lane] = list;
    __syncthreads();
    if (warp) return;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
        s.add(sums[w]);
        if (top) list = merge32(list, lists[w][lane], lane);
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
template <typename E>
struct Batch {
    static constexpr int VEC = 16 / sizeof(E), N = 8 / VEC;
    uint4 v[N];

    // first: index in the row of the batch's first score; lo, hi: the row's (or part's) first and end
    __device__ __forceinline__ void load(const E *row, int64_t first, int64_t hi, int lane) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int64_t e = first + (i * 32 + lane) * VEC;
            if (e >= 0 && e + VEC <= hi) {
                v[i] = __ldcs(reinterpret_cast<const uint4 *>(row + e));
            } else {
                // minus infinity where there is no score
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (sizeof(E) == 4) {
                        w[j] = e + j >= 0 && e + j < hi ? __float_as_uint(score(row + e + j)) : 0xFF800000u;
                    } else {
                        const uint32_t lo16 = e + 2 * j >= 0 && e + 2 * j < hi ? __float_as_uint(score(row + e + 2 * j)) : 0xFF800000u;
                        const uint32_t hi16 =
                            e + 2 * j + 1 >= 0 && e + 2 * j + 1 < hi ? __float_as_uint(score(row + e + 2 * j + 1)) : 0xFF800000u;
                        w[j] = lo16 >> 16 | hi16;
                    }
                }
                v[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
    __device__ __forceinline__ void scores(float (&x)[8]) const {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (sizeof(E) == 4)
                x[i] = __uint_as_float(w[i]);
            else
                x[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
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
    const int t = ROWS > 1 ? blockIdx.x * ROWS + warp : blockIdx.x / a.parts;
    const int part = ROWS > 1 ? 0 : blockIdx.x % a.parts;
    if (t >= a.T) return;
    const int target = a.targets ? a.targets[t] : 0;
    if (target < 0) return;
    const E *row = static_cast<const E *>(a.x) + t * a.stride;
    const float given = a.logprob && target < a.V ? score(row + target) : 0.f;
    u64 *buffer = buffers[TOP ? warp : 0];

    // batch b of the row: scores off + 256 b .. (off <= 0, to a 16-byte boundary)
    const int off = -static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(E));
    const int batches = (a.V - off + kBatch - 1) / kBatch;
    const int b1 = ROWS > 1 ? batches : min(batches, (part + 1) * a.part_batches);
    int b = ROWS > 1 ? 0 : part * a.part_batches + warp;

    Sums s{kLeast, 0.f, 0.f};
    Best best;
    float2 S2 = make_float2(0.f, 0.f), U2 = make_float2(0.f, 0.f);
    Batch<E> cur, nxt;
    cur.load(row, off + static_cast<int64_t>(b) * kBatch, b < b1 ? a.V : 0, lane);
    bool first = true;
    for (; b < b1; b += WPR) {
        const int at = off + b * kBatch;
        nxt.load(row, at + static_cast<int64_t>(WPR) * kBatch, b + WPR < b1 ? a.V : 0, lane);
        float x[8];
        cur.scores(x);
        float top = max_nan(max_nan(max_nan(x[0], x[1]), max_nan(x[2], x[3])),
                            max_nan(max_nan(x[4], x[5]), max_nan(x[6], x[7])));
        if (first || !(top <= s.r + kLogRaise)) {
            const float to = max_nan(top, kLeast);
            const float d = s.r - to, c = exp_of(d);
            U2 = S2.x + S2.y > 0.f && c > 0.f ? make_float2(c * (U2.x + d * S2.x), c * (U2.y + d * S2.y)) : make_float2(0.f, 0.f);
            S2 = make_float2(S2.x * c, S2.y * c);
            s.r = to;
        }
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            // (a score of minus infinity weighs nothing: e^-10000 = 0)
            const float t0 = fmaxf(x[i] - s.r, -10000.f), t1 = fmaxf(x[i + 1] - s.r, -10000.f);
            const float e0 = exp_of(t0), e1 = exp_of(t1);
            S2.x += e0;
            S2.y += e1;
            U2.x = fmaf(e0, t0, U2.x);
            U2.y = fmaf(e1, t1, U2.y);
        }
        if (TOP) {
            if (first && at >= 0 && at + kBatch <= a.V) {
                // the n-th of the lanes' maxima is not above the n-th best
                const float nth = key_score(__shfl_sync(0xffffffffu, sort32(rank_key(top, lane), lane), a.n_top - 1));
                if (nth > -INFINITY) best.above = before(nth);
            }
            if (__any_sync(0xffffffffu, !(top <= best.above))) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int id = at + Batch<E>::index(i, lane);
                    best.offer(x[i], id, id >= 0 && id < a.V, buffer, a.n_top, lane);
                }
                if (first && best.waiting) best.sort_in(buffer, a.n_top, lane);
                best.set_above(a.n_top, false);
            }
        }
        first = false;
        cur = nxt;
    }
    if (TOP) {
        while (best.waiting) best.sort_in(buffer, a.n_top, lane);
    }
    s.S = S2.x + S2.y;
    s.U = U2.x + U2.y;
    merge_lanes(s);
    if (ROWS > 1) {
        finish_row(a, t, target, given, s, best.list, lane);
        return;
    }
    merge_warps(s, best.list, TOP, warp, lane);
    if (warp) return;
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
    merge_warps(s, list, a.n_top > 0, warp, lane);
    if (warp == 0) finish_row(a, t, target, given, s, list, lane);
}

// ------------------------------------------------------------------- host

// Parts of a row: as many as give four blocks to each SM, of 2048 scores at least.
static int row_parts(int T, int V, int sms) {
    if (T >= 4 * sms) return 1;
    const int most = std::max(1, V / (kBatch * kPartBatches));
    return std::min((4 * sms + T - 1) / T, most);
}

size_t scores_workspace_bytes(int T, int V, int n_top, int max_sms) {
    // (rows and parts: at most four blocks and one more a row for each SM, where there are parts at all)
    const size_t blocks = T >= 4 * max_sms ? 0 : static_cast<size_t>(T) * row_parts(T, V, max_sms);
    return kCtrlBytes + blocks * (sizeof(float4) + (n_top ? 32 * sizeof(u64) : 0));
}

template <typename E, bool TOP>
static cudaError_t launch_e(ScoresArgs &a, void *ws, int num_sms, cudaStream_t s) {
    if (a.V <= kWarpRow && (a.T >= 2 * num_sms || a.V <= kBatch * kPartBatches)) {
        a.parts = 1;
        return launch_dependent(scores_kernel<E, TOP, kWarps>, dim3((a.T + kWarps - 1) / kWarps), dim3(kWarps * 32), 0, s, a);
    }
    a.parts = row_parts(a.T, a.V, num_sms);
    // (up to a vector before the row counts with it)
    const int batches = (a.V + 16 / static_cast<int>(sizeof(E)) - 1 + kBatch - 1) / kBatch;
    a.part_batches = (batches + a.parts - 1) / a.parts;
    a.part_sums = reinterpret_cast<float4 *>(static_cast<char *>(ws) + kCtrlBytes);
    a.part_top = reinterpret_cast<u64 *>(a.part_sums + static_cast<size_t>(a.T) * a.parts);
    const cudaError_t e = launch_dependent(scores_kernel<E, TOP, 1>, dim3(a.T * a.parts), dim3(kWarps * 32), 0, s, a);
    if (e != cudaSuccess || a.parts == 1) return e;
    return launch_dependent(scores_merge_kernel<E>, dim3(a.T), dim3(kWarps * 32), 0, s, a);
}

cudaError_t launch_scores(ScoresArgs &a, void *ws, int num_sms, cudaStream_t s) {
    if (a.fp32) return a.n_top ? launch_e<float, true>(a, ws, num_sms, s) : launch_e<float, false>(a, ws, num_sms, s);
    return a.n_top ? launch_e<__nv_bfloat16, true>(a, ws, num_sms, s) : launch_e<__nv_bfloat16, false>(a, ws, num_sms, s);
}

}  // namespace moe
