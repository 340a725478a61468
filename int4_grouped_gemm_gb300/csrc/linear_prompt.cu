// y[t][n] = sum_k x[t][k] (s[n][k/G] q[n][k] + z[n][k/G]) for a prompt's many tokens, on
// the fifth-generation tensor cores.
//
// The product is a plain one of fp16 operands, no product of which is rounded:
//
//   weights  s (q - 8): eight bits by four with a sign are eleven, exact in fp16, at a
//            power of two of the row's own
//   tokens   bf16's eight bits are exact in fp16 at a power of two of the row's own
//            (largest element in [2^14, 2^15); what is below 2^-31 of it is off by 2^-39)
//   biases   with c = z + 8 s what is left is sum_g X[t][g] c[n][g], X = sum of the
//            group's x: three more columns of the product for each group, X as two fp16
//            parts (h1, 2^11 h2, h1) times c as two (c1, 2^-11 c1, c2), 22 bits each; X at
//            2^-8 and c at 2^8, which keeps sums of 128 in fp16's range.  h2 at 2^11,
//            since a group's sum may be far below the token's largest element: its parts
//            end at 2^-42 of that one so, at 2^-31 without
//
// linear_operands_kernel makes the tokens' operand, rows of P = K + 3 K / G columns
// (each part rounded up to 64, zeros between), the rows' powers, and of the weights
// the bias columns and the scales in fp16.  The codes themselves are unpacked
//   of large matrices for few tiles of tokens (codes_up_to) by the product's kernel,
//   again for each tile: the matrix is then read as it is;
//   else by the operands kernel, once, into rows of P columns too, large matrices a
//   piece of rows at a time, so that they are read back from the L2.
// (256 x 2048 x 16384 28 us the first way, 52 the second; 512 x 2048 x 131072 fp32 256
// and 496; 1024 x 2048 x 8192 38 and 42, 2048 67 and 62; 512 x 2048 x 4096 23 and 20.)
//
// linear_prompt_kernel: pairs of blocks, on two SMs, work on tiles of 256 weight rows
// by up to 256 tokens (a multiple of 32 picked for even rounds over the pairs) with
// tcgen05.mma across both: a block holds its 128 rows and half of the tokens, so
// that each SM fetches 32 KB for 512 cycles of MMA.  (One block alone, 128 rows by
// 192 to 256 tokens, fetches 40 to 48 KB in the time, more than the 64 bytes a
// cycle that reach a SM: the product of
// 4096 x 4096 x 4096 took 99 us so, 90 in pairs.)
//
//   warp 0           loads: 64 columns of both operands a stage, 128-byte swizzle;
//                    both blocks' loads complete on the first one's barrier
//   warp 1           MMA issue, in the pair's first block; two accumulators in
//                    tensor memory, a tile each in turn.  The MMA cuts sums off towards
//                    zero, which adds up: 2e-6 of y over 2176 columns, proportional to
//                    their number.  fp32 results are therefore summed over at most
//                    kChunk stages at a time: the first chunk stays in one accumulator,
//                    to which the epilogue's warps add the others, rounded, as they
//                    come from the other one (7e-7 of y)
//   warp 3           loads of packed codes, a ring of their own
//   warps 12-27      unpacking: a thread a row's 64 codes of a stage, four sets of four
//                    warps in turn
//   warp 2           tells the pair's first block what was unpacked here (pair_arrive)
//   warps 4-11, 4-15 where nothing is unpacked here (8192 x 256 x 8192 fp32 63 us, with
//                    eight 67.5): epilogue: a lane is a weight row, so that a warp writes
//                    32 neighbouring results of a token at a time, whatever y's
//                    stride; powers of two put back
//
// What bounds it.  4096 x 2048 x 2560 in 38 to 42 us (by GPU): the operands, 6 to 8 us (their
// bytes: 16384 x 2048 tokens pass at 5.5 TB/s, read and written), and a product of three
// rounds over the pairs in 32 us, tensor pipe 63 %.  Its tiles of 192 tokens fetch 28 KB in
// 384 cycles, 75 bytes a cycle where 64 reach a SM, so that 86 % is the most it could be.
// 1021 x 2080 x 5003 fp32 in 34 to 42: tiles of 160 tokens, 83 bytes a cycle, and chunks: 42 %
// of 28 us.  512 x 2048 x 131072 fp32 in 256 to 271: 29 to 31 us for scales, biases and
// tokens, then a product in which the tensor pipe is busy for 55 %, the issue slots for
// 48 %, and every stage waits for its unpacking.  65 tokens 14 to 15 us: two launches and
// 34 stages one after another on 30 pairs; K is not split here.
//
// Every wait is bounded.
#include <cuda_fp16.h>

#include <algorithm>

#include "linear.cuh"

namespace moe {
namespace prompt {

constexpr int kRows = 128;                 // weight rows of a block, of a tile
constexpr int kPairRows = 2 * kRows;
constexpr int kMaxTok = 256;               // tokens of a tile
constexpr int kStep = 64;                  // columns of a stage
constexpr int kMaxStages = 8;
constexpr int kChunk = 13;                 // stages that are summed by MMAs alone, for fp32 results
constexpr int kEpiWarp = 4;
__host__ __device__ constexpr int epi_warps(bool codes) { return codes ? 8 : 12; }
constexpr int kDeqWarp = kEpiWarp + epi_warps(true), kSets = 4, kSetWarps = 4, kDeqWarps = kSets * kSetWarps;
constexpr int kQ = 8, kQBytes = kRows * kStep / 2;  // stages of packed codes
constexpr int threads(bool codes) { return (codes ? kDeqWarp + kDeqWarps : kEpiWarp + epi_warps(false)) * 32; }
constexpr size_t kCodesBytes = 8 << 20;    // of fp16 weights for each tile of tokens, above which the product's
constexpr int kCodesTiles[2] = {4, 8};     // kernel unpacks them: of the fewest and of the most tiles that count
constexpr int kWBytes = kRows * kStep * 2;
constexpr int kMaxT = 16384;               // tokens whose operands are held at a time
constexpr size_t kPieceBytes = 80 << 20;   // of what is made of the weights for a piece of rows, about

// Columns of an operand's row: codes up to Kp, then biases.
struct Columns {
    int K, Kp, groups, P;
    int Gp;  // scales of a row in fp16, up to a multiple of 8
    __host__ __device__ Columns(int K_, int G)
        : K(K_), Kp((K_ + 63) / 64 * 64), groups(K_ / G), P(Kp + (3 * groups + 63) / 64 * 64), Gp((groups + 7) / 8 * 8) {}
};

struct Args {
    LinearArgs l;
    __half *xh;           // [tokens here][P]
    __half *wh;           // [rows of this piece][P - code_steps 64]
    __half *sh;           // [rows of this piece][Gp]: scales, where the product unpacks
    int *xe, *we;         // their powers
    int t0, nt, n0, nn;   // tokens and rows of this launch
    int x_blocks;         // operands: blocks that make tokens
    int code_steps;       // of a tile's steps, the first ones whose weights the product unpacks
    int gshift;           // log2 of the group
    int tok, t_tiles, n_tiles, stages;
    int chunk;            // stages of a chunk; all of a tile's: no chunks
};

// ------------------------------------------------------------- operands

// 2^e for e in -250 .. 250 times x, without a rounding that the result does not need.
__device__ __forceinline__ float times_power(float x, int e) {
    const int h = e / 2;
    return x * __int_as_float((h + 127) << 23) * __int_as_float((e - h + 127) << 23);
}
// e of |x| in [2^e, 2^(e+1)), -126 at least; for infinities and NaN 128.
__device__ __forceinline__ int power_of(float x) {
    const int e = static_cast<int>(__float_as_uint(x) >> 23 & 255);
    return (e ? e : 1) - 127;
}
// ... of x >= 0, subnormal numbers too (0: -150).
__device__ __forceinline__ int power_of_any(float x) {
    const uint32_t u = __float_as_uint(x);
    return u >> 23 ? power_of(x) : -118 - __clz(u);
}

// y in two fp16 parts, the lower one `up` times too large.
constexpr float kLowUp = 0x1p11f;
__device__ __forceinline__ void split(float y, __half &hi, __half &lo, float up = 1.f) {
    hi = __float2half_rn(y);
    lo = __float2half_rn((y - __half2float(hi)) * up);
}

__device__ __forceinline__ void zero_columns(__half *row, int from, int to, int i, int n) {
    for (int c = from + i; c < to; c += n) row[c] = __float2half_rn(0.f);
}

// Eight codes times their scale, (q - 8) s, exact.
__device__ __forceinline__ uint4 unpack8(uint32_t w, __half2 s) {
    const __half2 c1032 = __half2half2(__ushort_as_half(0x6408));
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        // 1024 + q by a mask-and-set a pair
        const uint32_t b = mask_set(w >> (4 * j), 0x000F000Fu, 0x64006400u);
        const __half2 p = __hmul2(__hsub2(*reinterpret_cast<const __half2 *>(&b), c1032), s);
        o[j] = *reinterpret_cast<const uint32_t *>(&p);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

constexpr int kOpThreads = 256, kOpRows = kOpThreads / 32;
constexpr int kBareRows = 4;
constexpr int kHeld = 8;  // of a token's vectors of eight, those that a lane keeps between the passes

// A row a warp: blocks 0 .. x_blocks - 1 tokens, the others weights, whose rows without
// codes are little work each: kBareRows of them a warp (512 x 2048 x 131072 fp32 267 us,
// one a warp 295).
template <bool CODES>
__global__ void __launch_bounds__(kOpThreads, 3) linear_operands_kernel(const __grid_constant__ Args a) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Columns c(a.l.K, a.l.G);
    const int ng = c.groups;
    pdl_wait();
    pdl_trigger();
    if (static_cast<int>(blockIdx.x) < a.x_blocks) {
        const int t = blockIdx.x * kOpRows + warp, n = c.K / 8;
        if (t >= a.nt) return;
        const uint4 *x = reinterpret_cast<const uint4 *>(a.l.x + (a.t0 + t) * a.l.x_stride);
        __half *row = a.xh + static_cast<int64_t>(t) * c.P;
        __shared__ float group_sums[kOpRows][kHeld * 8];
        uint4 held[kHeld];
        auto fetch = [&](int from) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i)
                held[i] = from + i * 32 + lane < n ? __ldcg(x + from + i * 32 + lane) : make_uint4(0u, 0u, 0u, 0u);
        };
        // (NaN does not count: it stays NaN at any power)
        __nv_bfloat162 most = u32_as_bf162(0u);
        auto look = [&](const uint4 &v) {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) most = __hmax2(most, u32_as_bf162(w[j] & 0x7FFF7FFFu));
        };
        fetch(0);
#pragma unroll
        for (int i = 0; i < kHeld; ++i) look(held[i]);
#pragma unroll 4
        for (int i = kHeld * 32 + lane; i < n; i += 32) look(__ldcg(x + i));
        const uint32_t tops = bf162_as_u32(most), top = __reduce_max_sync(0xffffffffu, max(tops & 0xFFFFu, tops >> 16));
        // (a row with an infinity keeps it)
        const int up = 14 - power_of(__uint_as_float(top << 16)), up1 = min(up, 127);
        const int lane_shift = a.gshift - 3;  // log2 of a group's lanes
        const uint32_t f1 = (up1 + 127) << 23, f2 = (up - up1 + 127) << 23;
        auto put = [&](const uint4 &v, int i, float *to) {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint32_t o[4];
            uint64_t sums = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint64_t y = fma2(pack2(w[j] << 16, w[j] & 0xFFFF0000u), pack2(f1, f1), 0);
                if (up > 127) y = fma2(y, pack2(f2, f2), 0);
                const float2 f = unpack2(y);
                const __half2 h = __floats2half2_rn(f.x, f.y);
                o[j] = *reinterpret_cast<const uint32_t *>(&h);
                sums = add2(sums, y);
            }
            const float2 two = unpack2(sums);
            float sum = two.x + two.y;
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            if (lane_shift > 2) sum += __shfl_xor_sync(0xffffffffu, sum, 4);
            if (lane_shift > 3) sum += __shfl_xor_sync(0xffffffffu, sum, 8);
            if (i >= n) return;
            reinterpret_cast<uint4 *>(row)[i] = make_uint4(o[0], o[1], o[2], o[3]);
            if ((lane & ((1 << lane_shift) - 1)) == 0) to[lane >> lane_shift] = sum;
        };
        for (int from = 0; from < n; from += kHeld * 32) {
            if (from) fetch(from);
#pragma unroll
            for (int i = 0; i < kHeld; ++i)
                if (from + i * 32 < n) put(held[i], from + i * 32 + lane, group_sums[warp] + (i * 32 >> lane_shift));
            __syncwarp();
            const int g0 = from >> lane_shift, here = min(kHeld * 32, n - from) >> lane_shift;
            for (int g = lane; g < here; g += 32) {
                __half h1, h2;
                split(group_sums[warp][g] * 0x1p-8f, h1, h2, kLowUp);
                row[c.Kp + g0 + g] = h1;
                row[c.Kp + ng + g0 + g] = h2;
                row[c.Kp + 2 * ng + g0 + g] = h1;
            }
            __syncwarp();
        }
        zero_columns(row, c.K, c.Kp, lane, 32);
        zero_columns(row, c.Kp + 3 * ng, c.P, lane, 32);
        if (lane == 0) a.xe[t] = -up;
        return;
    }
    constexpr int each = CODES ? 1 : kBareRows;  // rows of a warp
    const int r0 = ((blockIdx.x - a.x_blocks) * kOpRows + warp) * each, codes = CODES ? c.Kp : 0;
    // (c at 2^-16: z, s and 256 c stay within fp32 so, and any bf16 number times that is exact)
    constexpr int kDown = 16;
    auto scales = [&](int r, int g, float &sg, float &cg) {
        const int64_t at = static_cast<int64_t>(a.n0 + r) * a.l.ldg + g;
        sg = bf16_bits_to_float(__ldg(a.l.s + at));
        cg = fmaf(sg, 0x1p-13f, bf16_bits_to_float(__ldg(a.l.b + at)) * 0x1p-16f);
    };
    float held_s[each], held_c[each];  // those of group `lane`
#pragma unroll
    for (int i = 0; i < each; ++i) {
        held_s[i] = held_c[i] = 0.f;
        if (r0 + i < a.nn && lane < ng) scales(r0 + i, lane, held_s[i], held_c[i]);
    }
#pragma unroll
    for (int i = 0; i < each; ++i) {
        const int r = r0 + i;
        if (r >= a.nn) return;
        __half *row = a.wh + static_cast<int64_t>(r) * (codes + c.P - c.Kp), *bias = row + codes;
        float top = fmaxf(0x1p-13f * fabsf(held_s[i]), 256.f * fabsf(held_c[i]));
        for (int g = lane + 32; g < ng; g += 32) {
            float sg, cg;
            scales(r, g, sg, cg);
            top = fmaxf(top, fmaxf(0x1p-13f * fabsf(sg), 256.f * fabsf(cg)));
        }
        const int up = 14 - power_of_any(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)))) - kDown;
        for (int g = lane; g < ng; g += 32) {
            float sg = held_s[i], cg = held_c[i];
            if (g >= 32) scales(r, g, sg, cg);
            __half c1, c2;
            split(times_power(cg, up + kDown) * 256.f, c1, c2);
            bias[g] = c1;
            bias[ng + g] = __float2half_rn(__half2float(c1) / kLowUp);
            bias[2 * ng + g] = c2;
            if (!CODES) a.sh[static_cast<int64_t>(r) * c.Gp + g] = __float2half_rn(times_power(sg, up));
        }
        zero_columns(bias, 3 * ng, c.P - c.Kp, lane, 32);
        if (lane == 0) a.we[r] = -up;
        if constexpr (CODES) {
            const uint16_t *s = a.l.s + static_cast<int64_t>(a.n0 + r) * a.l.ldg;
            const uint32_t *q = a.l.q + static_cast<int64_t>(a.n0 + r) * (c.K / 8);
#pragma unroll 4
            for (int k = lane; k < c.K / 8; k += 32) {
                const __half sg = __float2half_rn(times_power(bf16_bits_to_float(__ldg(s + (k * 8 >> a.gshift))), up));
                reinterpret_cast<uint4 *>(row)[k] = unpack8(__ldcs(q + k), __half2half2(sg));
            }
            zero_columns(row, c.K, c.Kp, lane, 32);
        }
    }
}

// -------------------------------------------------------------- product

struct Ctl {
    uint64_t full[kMaxStages], empty[kMaxStages];  // (full: of both blocks' loads, in the first one)
    uint64_t q_full[kQ], q_empty[kQ];              // packed codes
    uint64_t unpacked[kMaxStages];                 // codes of the stage are in their place
    uint64_t acc_full[2], acc_empty[2];            // (acc_empty: of both, in the first one)
    uint64_t drain;
    uint32_t tmem;
    int abort;
};

__host__ __device__ constexpr int stage_bytes(int tok) { return kWBytes + tok / 2 * kStep * 2; }
__host__ __device__ constexpr int fixed_bytes(bool codes) {
    return 1024 + static_cast<int>(sizeof(Ctl)) + (codes ? kQ * kQBytes : 0);
}
__host__ __device__ constexpr int stages_for(int tok, bool codes) {
    const int n = (kBlockSmem - fixed_bytes(codes)) / stage_bytes(tok);
    return n < kMaxStages ? n : kMaxStages;
}
__host__ __device__ constexpr int smem_bytes(int tok, bool codes) {
    // (more than half of a SM's: one block at a time, since each takes all of the tensor memory)
    const int n = stages_for(tok, codes) * stage_bytes(tok) + fixed_bytes(codes);
    return n > kBlockSmem / 2 + 1024 ? n : kBlockSmem / 2 + 1024;
}
static_assert(stages_for(kMaxTok, true) >= 4 && smem_bytes(kMaxTok, true) <= kBlockSmem &&
                  smem_bytes(kMaxTok, false) <= kBlockSmem && smem_bytes(32, true) <= kBlockSmem,
              "stages");

__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, const Args &a, Ctl *s, int site) {
    return role_wait(bar, parity, a.l.wait_limit, a.l.status, &s->abort, site);
}

// Instruction descriptor: fp16 x fp16 -> fp32, A and B K-major, shape 256 x tok over a pair.
__device__ __forceinline__ uint32_t idesc_f16(int tok) {
    return (1u << 4) | (static_cast<uint32_t>(tok >> 3) << 17) | (static_cast<uint32_t>(kPairRows >> 4) << 24);
}

// Of a pair of blocks: the address of the first block's copy of a shared variable.
__device__ __forceinline__ uint32_t in_first(const void *p) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
    return r;
}
// Arrives on a barrier of the pair's first block, whose MMA thread acts on it.  The arrival
// is of cluster scope, what comes before it is ordered in this block alone: a release
// of cluster scope waits for all that the thread's block has under way, 0.3 to 0.6 us
// for each stage (512 x 2048 x 131072 435 us, so 268).  That is enough, because nothing
// that the MMA thread's own accesses would have to see is handed over:
//   unpacked codes   lie in this block's shared memory, of which there is one copy, in
//                    this SM.  Each writer has fenced them for the asynchronous proxy and
//                    arrived on `unpacked` (release, block scope), the thread here has
//                    seen that phase end (acquire, block scope): the bytes are in their
//                    place before the arrival leaves, and the only one to read them is
//                    this SM's tensor core, for an MMA that is issued behind the arrival
//   tensor memory    an accumulator's loads and stores of this warp are complete
//                    (tcgen05.wait) and its values in registers before it arrives
__device__ __forceinline__ void pair_arrive(uint32_t bar) {
    asm volatile("fence.acq_rel.cta;\n\tmbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// A box into this block's shared memory, complete on a barrier of the pair.
__device__ __forceinline__ void pair_load_2d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrive on `bar` of both blocks when every MMA issued so far by this thread is done.
__device__ __forceinline__ void pair_commit(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// A role's place in the ring of stages.  (By division of a count by the number of
// stages, which is not a constant, the roles' instructions were twice as many.)
struct Ring {
    int at = 0;
    uint32_t phase = 0;

    __device__ __forceinline__ void advance(int by, int stages) {
        if ((at += by) >= stages) {
            at -= stages;
            phase ^= 1;
        }
    }
};

// The unpacking warps' part: the sets take a block's stages in turn, a thread its
// row of 128.
__device__ __forceinline__ void unpack_role(const Args &a, Ctl *s, uint8_t *base, int stage, int steps, int tiles, int rank,
                                            int pair, int pairs) {
    const Columns c(a.l.K, a.l.G);
    const int set = (threadIdx.x / 32 - kDeqWarp) / kSetWarps, r = (threadIdx.x - kDeqWarp * 32) % kRows, lane = threadIdx.x & 31;
    const int stages = a.stages;
    // (16-byte piece j of the row at j ^ (r % 8) of its 128 bytes)
    const uint32_t row = smem_u32(base) + r * 128 + ((r & 7) << 4);
    const uint32_t packed = smem_u32(base) + stages * stage + r * 32 + ((r >> 2 & 1) << 4);
    // the set's next stage with codes, whose scales are fetched one ahead: tile and step
    int next_tile = pair, next_k = set, before = 0;  // (stages of the tiles before, modulo kSets)
    __half2 ahead = __half2half2(__ushort_as_half(0));
    auto fetch = [&]() {
        // (a tile may have fewer stages with codes than there are sets)
        while (next_k >= a.code_steps && next_tile < tiles) {
            next_tile += pairs;
            before = (before + steps) % kSets;
            next_k = (set - before + kSets) % kSets;
        }
        if (next_tile >= tiles) return;
        const int n = min(next_tile % a.n_tiles * kPairRows + rank * kRows + r, a.nn - 1);
        const __half *at = a.sh + static_cast<int64_t>(n) * c.Gp + (next_k * kStep >> a.gshift);
        // (a stage's one or two scales)
        ahead = a.gshift == 5 ? __ldcg(reinterpret_cast<const __half2 *>(at)) : __half2half2(__ldcg(at));
        next_k += kSets;
    };
    fetch();
    Ring ring;
    ring.advance(set, stages);
    uint32_t codes_before = 0;  // stages with codes of the tiles before
    bool ok = true;
    int k = set;
    for (int tile = pair; tile < tiles && ok; tile += pairs, codes_before += a.code_steps, k -= steps) {
        for (; k < a.code_steps; k += kSets, ring.advance(kSets, stages)) {
            const __half2 sg = ahead;
            fetch();
            const uint32_t qi = codes_before + k;
            ok = __all_sync(0xffffffffu, wait(&s->q_full[qi % kQ], (qi / kQ) & 1, a, s, 65));
            if (!ok) break;
            uint32_t w[8];
#pragma unroll
            for (int h = 0; h < 2; ++h)
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w[4 * h]), "=r"(w[4 * h + 1]), "=r"(w[4 * h + 2]), "=r"(w[4 * h + 3])
                             : "r"((packed + qi % kQ * kQBytes) ^ (h << 4))
                             : "memory");
            ok = __all_sync(0xffffffffu, wait(&s->empty[ring.at], ring.phase ^ 1, a, s, 66));
            if (!ok) break;
            const __half2 s0 = __low2half2(sg), s1 = __high2half2(sg);
            const uint32_t to = row + ring.at * stage;
            auto put = [&](int j, const uint4 &v) {
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to ^ (j << 4)), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                             : "memory");
            };
#pragma unroll
            for (int j = 0; j < 4; ++j) put(j, unpack8(w[j], s0));
            if (k * kStep + kStep <= c.K) {
#pragma unroll
                for (int j = 4; j < 8; ++j) put(j, unpack8(w[j], s1));
            } else {
                // only 32 of the codes are there
#pragma unroll
                for (int j = 4; j < 8; ++j) put(j, make_uint4(0u, 0u, 0u, 0u));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&s->q_empty[qi % kQ]);
                mbar_arrive(&s->unpacked[ring.at]);
            }
        }
        for (; k < steps && ok; k += kSets, ring.advance(kSets, stages)) {
            ok = __all_sync(0xffffffffu, wait(&s->empty[ring.at], ring.phase ^ 1, a, s, 67));
            if (ok && lane == 0) mbar_arrive(&s->unpacked[ring.at]);
        }
    }
}

// CODES: the first code_steps steps' weights are unpacked here.
template <bool CODES>
__global__ void __launch_bounds__(threads(CODES), 1)
    linear_prompt_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                         const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ Args a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int stage = stage_bytes(a.tok), stages = a.stages;
    Ctl *s = reinterpret_cast<Ctl *>(base + stages * stage + (CODES ? kQ * kQBytes : 0));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tiles = a.t_tiles * a.n_tiles, steps = Columns(a.l.K, a.l.G).P / kStep;
    const int rank = blockIdx.x & 1, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (tid == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(&s->full[i], CODES ? 3 : 1);  // (the loads' and both blocks' unpacking's)
            mbar_init(&s->empty[i], 1);
            mbar_init(&s->unpacked[i], kSetWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s->acc_full[i], 1);
            mbar_init(&s->acc_empty[i], 2 * epi_warps(CODES));
        }
        for (int i = 0; i < kQ; ++i) {
            mbar_init(&s->q_full[i], 1);
            mbar_init(&s->q_empty[i], kSetWarps);
        }
        mbar_init(&s->drain, 1);
        s->abort = 0;
        fence_mbar_init();
        prefetch_tmap(&tm_w);
        prefetch_tmap(&tm_x);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s->tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both blocks' barriers are there
    tc_fence_after();
    const uint32_t tmem = s->tmem;
    pdl_wait();
    pdl_trigger();

    if (warp == 0) {
        if (elect_one()) {
            Ring ring;
            int loaded = 0;
            bool ok = true;
            for (int tile = pair; tile < tiles && ok; tile += pairs) {
                const int n0 = tile % a.n_tiles * kPairRows + rank * kRows, t0 = tile / a.n_tiles * a.tok + rank * (a.tok / 2);
                for (int k = 0; k < steps; ++k, ring.advance(1, stages)) {
                    ok = wait(&s->empty[ring.at], ring.phase ^ 1, a, s, 61);
                    if (!ok) break;
                    const uint32_t at = smem_u32(base + ring.at * stage), bar = in_first(&s->full[ring.at]);
                    // (the other block's bytes may come before they are expected: the phase
                    // cannot end before this arrival)
                    const bool codes = CODES && k < a.code_steps;
                    if (rank == 0) mbar_arrive_expect_tx(&s->full[ring.at], 2 * (codes ? stage - kWBytes : stage));
                    if (!codes) pair_load_2d(at, &tm_w, bar, (CODES ? k - a.code_steps : k) * kStep, n0);
                    pair_load_2d(at + kWBytes, &tm_x, bar, k * kStep, t0);
                    loaded = min(loaded + 1, stages);
                }
            }
            // no copy of this block is in flight when it ends: the MMAs that read the last
            // ones are complete, or two milliseconds have passed for each
            ring.at -= loaded;
            if (ring.at < 0) {
                ring.at += stages;
                ring.phase ^= 1;
            }
            for (; loaded; --loaded, ring.advance(1, stages)) mbar_wait(&s->empty[ring.at], ring.phase, 1 << 22);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            const uint32_t idesc = idesc_f16(a.tok);
            Ring ring;
            uint32_t nt = 0;
            bool ok = true;
            const bool chunks = a.chunk < steps;
            uint32_t nc = 0;  // chunks that went to the second accumulator
            for (int tile = pair; tile < tiles && ok; tile += pairs, ++nt) {
                const uint32_t which = chunks ? 0 : nt & 1, uses = chunks ? nt : nt >> 1;
                uint32_t acc = tmem + which * 256;
                ok = wait(&s->acc_empty[which], (uses & 1) ^ 1, a, s, 62);
                if (!ok) break;
                tc_fence_after();
                for (int k = 0, in_chunk = 0; k < steps; ++k, ++in_chunk, ring.advance(1, stages)) {
                    if (in_chunk == a.chunk) {
                        if (k > a.chunk) pair_commit(&s->acc_full[1]);
                        in_chunk = 0;
                        acc = tmem + 256;
                        ok = wait(&s->acc_empty[1], (nc & 1) ^ 1, a, s, 70);
                        ++nc;
                        if (!ok) break;
                        tc_fence_after();
                    }
                    ok = wait(&s->full[ring.at], ring.phase, a, s, 63);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t w_at = smem_u32(base) + ring.at * stage, x_at = w_at + kWBytes;
#pragma unroll
                    for (int j = 0; j < kStep / 16; ++j)
                        pair_mma(acc, sdesc_k128(w_at + j * 32), sdesc_k128(x_at + j * 32), idesc, in_chunk | j);
                    pair_commit(&s->empty[ring.at]);
                }
                if (ok) pair_commit(&s->acc_full[chunks ? 1 : which]);
            }
            // every MMA issued here is complete before tensor memory is freed
            asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(&s->drain))
                         : "memory");
            mbar_drain(&s->drain, 0, a.l.wait_limit);
        }
        __syncwarp();
    } else if (warp == 2) {
        if (CODES && elect_one()) {
            Ring ring;
            for (int left = pair < tiles ? (tiles - pair + pairs - 1) / pairs * steps : 0; left; --left, ring.advance(1, stages)) {
                if (!wait(&s->unpacked[ring.at], ring.phase, a, s, 68)) break;
                pair_arrive(in_first(&s->full[ring.at]));
            }
        }
        __syncwarp();
    } else if (warp == 3) {
        if (CODES && elect_one()) {
            uint32_t it = 0;
            bool ok = true;
            for (int tile = pair; tile < tiles && ok; tile += pairs) {
                const int n0 = a.n0 + tile % a.n_tiles * kPairRows + rank * kRows;
                for (int k = 0; k < a.code_steps && ok; ++k, ++it) {
                    ok = wait(&s->q_empty[it % kQ], ((it / kQ) & 1) ^ 1, a, s, 69);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&s->q_full[it % kQ], kQBytes);
                    tma_load_2d(base + stages * stage + it % kQ * kQBytes, &tm_q, &s->q_full[it % kQ], k * (kStep / 8), n0);
                }
            }
            for (uint32_t i = it > kQ ? it - kQ : 0; i < it; ++i) mbar_drain(&s->q_full[i % kQ], (i / kQ) & 1, a.l.wait_limit);
        }
        __syncwarp();
    } else if (CODES && warp >= kDeqWarp) {
        unpack_role(a, s, base, stage, steps, tiles, rank, pair, pairs);
    } else if (warp >= kEpiWarp) {
        constexpr int SETS = epi_warps(CODES) / 4;  // of four warps, in turn
        const int quarter = warp & 3, set = (warp - kEpiWarp) >> 2;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        const bool chunks = a.chunk < steps;
        constexpr int E = CODES ? 16 : 32;
        auto load = [&](uint32_t from, uint32_t (&v)[E]) {
            if constexpr (CODES)
                tmem_ld16_issue(from | lanes, v);
            else
                tmem_ld32(from | lanes, v);
        };
        auto loaded = [&](uint32_t (&v)[E]) {
            if constexpr (CODES)
                tmem_wait16(v);
            else
                tmem_wait32(v);
        };
        uint32_t nt = 0, nc = 0;
        bool ok = true;
        for (int tile = pair; tile < tiles; tile += pairs, ++nt) {
            const int n = tile % a.n_tiles * kPairRows + rank * kRows + quarter * 32 + lane, t0 = tile / a.n_tiles * a.tok;
            const int we = n < a.nn ? __ldcg(a.we + n) : 0;
            // tokens' powers, a lane a token, some tokens ahead
            auto powers = [&](int c) {
                return lane < E && c + lane < min(a.tok, a.nt - t0) ? __ldcg(a.xe + t0 + c + lane) : 0;
            };
            int ahead = powers(set * E);
            // all chunks but the last one: added to the first
            for (int k = 2 * a.chunk; chunks && k < steps && ok; k += a.chunk, ++nc) {
                ok = __all_sync(0xffffffffu, wait(&s->acc_full[1], nc & 1, a, s, 71));
                if (!ok) break;
                tc_fence_after();
                for (int c = set * E; c < a.tok; c += SETS * E) {
                    uint32_t v[E], u[E];
                    load(tmem + c, v);
                    load(tmem + 256 + c, u);
                    loaded(v);
                    loaded(u);
#pragma unroll
                    for (int j = 0; j < E; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(u[j]));
#pragma unroll
                    for (int j = 0; j < E; j += 16) tmem_st16((tmem + c + j) | lanes, v + j);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) pair_arrive(in_first(&s->acc_empty[1]));
            }
            if (!ok) break;
            const uint32_t which = chunks ? 1 : nt & 1;
            ok = __all_sync(0xffffffffu, wait(&s->acc_full[which], (chunks ? nc++ : nt >> 1) & 1, a, s, 64));
            if (!ok) break;
            tc_fence_after();
            // some tokens at a time, the sets of warps in turn; the powers as two factors where they
            // are near enough to one that neither leaves fp32's range
            for (int c = set * E; c < a.tok; c += SETS * E) {
                const int left = a.nt - t0 - c;
                if (left <= 0) break;
                uint32_t v[E], u[E];
                load(tmem + (nt & 1 && !chunks ? 256 : 0) + c, v);
                if (chunks) load(tmem + 256 + c, u);
                const int xe = ahead;
                ahead = powers(c + SETS * E);
                const bool near = __all_sync(0xffffffffu, abs(xe) <= 60 && abs(we) <= 60);
                const float xf = near ? __int_as_float((xe + 127) << 23) : 0.f, wf = __int_as_float(((near ? we : 0) + 127) << 23);
                loaded(v);
                if (chunks) {
                    loaded(u);
#pragma unroll
                    for (int j = 0; j < E; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(u[j]));
                }
                char *at = static_cast<char *>(a.l.y) + ((a.t0 + t0 + c) * a.l.y_stride + a.n0 + n) * (a.l.y_fp32 ? 4 : 2);
                auto write = [&](auto put) {
                    if (left >= E) {
#pragma unroll
                        for (int j = 0; j < E; ++j) put(j);
                    } else {
#pragma unroll
                        for (int j = 0; j < E; ++j)
                            if (j < left) put(j);
                    }
                };
                auto scaled = [&](int j) { return __uint_as_float(v[j]) * __shfl_sync(0xffffffffu, xf, j) * wf; };
                if (!near) {
#pragma unroll
                    for (int j = 0; j < E; ++j) {
                        const int e = max(-250, min(250, we + __shfl_sync(0xffffffffu, xe, j)));
                        if (j < left && n < a.nn) a.l.store(a.t0 + t0 + c + j, a.n0 + n, times_power(__uint_as_float(v[j]), e));
                    }
                } else if (a.l.y_fp32) {
                    const int64_t step = a.l.y_stride * 4;
                    write([&](int j) {
                        const float y = scaled(j);
                        if (n < a.nn) *reinterpret_cast<float *>(at) = y;
                        at += step;
                    });
                } else {
                    const int64_t step = a.l.y_stride * 2;
                    write([&](int j) {
                        const float y = scaled(j);
                        if (n < a.nn) *reinterpret_cast<__nv_bfloat16 *>(at) = __float2bfloat16_rn(y);
                        at += step;
                    });
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                pair_arrive(in_first(&s->acc_empty[which]));
                if (chunks) pair_arrive(in_first(&s->acc_empty[0]));
            }
        }
    }

    // neither block goes while the other may still reach its shared or tensor memory
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// ----------------------------------------------------------------- host

struct Layout {
    size_t xe, we, xh, sh, wh, total;
    int rows;        // weight rows of a piece
    int code_steps;  // (0: codes are unpacked before the product)
};

// Tokens up to which the product's kernel unpacks the codes: unpacking before it costs
// as many bytes as the weights have in fp16, unpacking in it some time for every tile.
static int codes_up_to(int N, const Columns &c) {
    const size_t tiles = (static_cast<size_t>(N) * c.P * sizeof(__half) - 1) / kCodesBytes;
    return tiles < kCodesTiles[0] ? 0 : static_cast<int>(std::min<size_t>(tiles, kCodesTiles[1])) * kMaxTok;
}

static Layout layout(int N, int K, int G, int T) {
    auto up = [](size_t n) { return (n + 1023) / 1024 * 1024; };
    const Columns c(K, G);
    Layout L{};
    L.code_steps = T <= codes_up_to(N, c) ? c.Kp / kStep : 0;
    const size_t width = (c.P - L.code_steps * kStep) * sizeof(__half);  // of a row of wh
    const size_t most = std::max<size_t>(kPieceBytes / width / kPairRows * kPairRows, kPairRows);
    L.rows = static_cast<int>(std::min<size_t>(N, most));
    L.xe = kCtrlBytes;
    L.we = L.xe + up(std::min(T, kMaxT) * sizeof(int));
    L.xh = L.we + up(L.rows * sizeof(int));
    L.sh = L.xh + up(std::min(T, kMaxT) * static_cast<size_t>(c.P) * sizeof(__half));
    L.wh = L.sh + (L.code_steps ? up(L.rows * static_cast<size_t>(c.Gp) * sizeof(__half)) : 0);
    L.total = L.wh + L.rows * width;
    return L;
}

// Tokens of a tile: as many as make the rounds over the pairs of SMs cheapest, a
// round's cost being its tokens and 32 more (weights are fetched for few tokens as
// for many).
static int tile_tokens(int N, int T, int pairs) {
    const int n_tiles = (N + kPairRows - 1) / kPairRows;
    int best = kMaxTok;
    int64_t least = INT64_MAX;
    for (int tok = kMaxTok; tok >= 32; tok -= 32) {
        const int64_t tiles = static_cast<int64_t>(n_tiles) * ((T + tok - 1) / tok);
        const int64_t cost = (tiles + pairs - 1) / pairs * (tok + 32);
        if (cost < least) {
            least = cost;
            best = tok;
        }
    }
    return best;
}

}  // namespace prompt

// (a call of fewer tokens may take the way that needs more; kLinearMaxB and fewer need
// none, and 0 stands for what is not supported)
size_t linear_prompt_workspace_bytes(int N, int K, int G, int T) {
    if (T <= kLinearMaxB) return kCtrlBytes;
    const size_t all = prompt::layout(N, K, G, T).total;
    const int few = prompt::codes_up_to(N, prompt::Columns(K, G));  // (these take other room)
    return few && few < T ? std::max(all, prompt::layout(N, K, G, few).total) : all;
}

cudaError_t launch_linear_prompt(const LinearArgs &l, LinearMap encode, void *ws, int num_sms, cudaStream_t s) {
    using namespace prompt;
    const Layout L = layout(l.N, l.K, l.G, l.B);
    const Columns c(l.K, l.G);
    char *w = static_cast<char *>(ws);
    Args a{};
    a.l = l;
    a.gshift = l.G == 32 ? 5 : l.G == 64 ? 6 : 7;
    a.xe = reinterpret_cast<int *>(w + L.xe);
    a.xh = reinterpret_cast<__half *>(w + L.xh);
    const auto operands = L.code_steps ? linear_operands_kernel<false> : linear_operands_kernel<true>;
    const auto kernel = L.code_steps ? linear_prompt_kernel<true> : linear_prompt_kernel<false>;
    cudaError_t e = L.code_steps ? allow_smem<linear_prompt_kernel<true>>() : allow_smem<linear_prompt_kernel<false>>();
    if (e != cudaSuccess) return e;
    a.we = reinterpret_cast<int *>(w + L.we);
    a.sh = reinterpret_cast<__half *>(w + L.sh);
    a.wh = reinterpret_cast<__half *>(w + L.wh);
    a.code_steps = L.code_steps;
    for (a.t0 = 0; a.t0 < l.B; a.t0 += kMaxT) {
        a.nt = std::min(l.B - a.t0, kMaxT);
        for (a.n0 = 0; a.n0 < l.N; a.n0 += L.rows) {
            a.nn = std::min(l.N - a.n0, L.rows);
            a.x_blocks = a.n0 ? 0 : (a.nt + kOpRows - 1) / kOpRows;
            const int w_rows = kOpRows * (L.code_steps ? kBareRows : 1), w_blocks = (a.nn + w_rows - 1) / w_rows;
            if ((e = launch_dependent(operands, dim3(a.x_blocks + w_blocks), dim3(kOpThreads), 0, s, a)) != cudaSuccess)
                return e;
            a.tok = tile_tokens(a.nn, a.nt, num_sms / 2);
            a.stages = stages_for(a.tok, a.code_steps > 0);
            a.n_tiles = (a.nn + kPairRows - 1) / kPairRows;
            const int steps = c.P / kStep, parts = l.y_fp32 ? (steps + kChunk - 1) / kChunk : 1;
            a.chunk = (steps + parts - 1) / parts;
            a.t_tiles = (a.nt + a.tok - 1) / a.tok;
            CUtensorMap mw, mx, mq;
            if (!encode(&mw, a.wh, true, c.P - a.code_steps * kStep, a.nn, kStep, kRows) ||
                !encode(&mx, a.xh, true, c.P, a.nt, kStep, a.tok / 2) ||
                !encode(&mq, l.q, false, c.K / 8, l.N, kStep / 8, kRows))
                return cudaErrorInvalidValue;
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(2 * std::min(a.n_tiles * a.t_tiles, num_sms / 2));
            cfg.blockDim = dim3(threads(a.code_steps > 0));
            cfg.dynamicSmemBytes = smem_bytes(a.tok, a.code_steps > 0);
            cfg.stream = s;
            cudaLaunchAttribute attr[2];
            attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[0].val.programmaticStreamSerializationAllowed = 1;
            attr[1].id = cudaLaunchAttributeClusterDimension;
            attr[1].val.clusterDim.x = 2;
            attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 2;
            if ((e = cudaLaunchKernelEx(&cfg, kernel, mw, mx, mq, a)) != cudaSuccess) return e;
        }
    }
    return cudaSuccess;
}

}  // namespace moe
