// A tile of attention on the fifth-generation tensor cores: 128 rows of queries
// (MMA M) against 128 positions, S = Q K^T, P = 2^(S - m), O += P V, as the kernels
// of the shared prefix and of prompts run it.
//
//   S, P, O  in tensor memory: S (fp32, 128 columns), P over it, and O (fp32, D
//            columns).  P is an operand straight from tensor memory, so that the
//            second product's shared-memory reads are V alone.  A weight is two
//            bf16 parts (|p - hi - lo| <= 2^-17 p; of each 64 positions the upper
//            ones over the first half of their scores' columns, the lower ones over
//            the other), each with MMAs of its own: rounded to one part (by up to
//            2^-8) weights would put as large an error on the output as its own
//            rounding does
//   softmax  one thread per row: no exchange between threads.  m need not be the
//            maximum, only a reference that keeps 2^(s - m) in range, the same in
//            l and O: fp32 and bf16 hold a weight of 2^-24 as exactly as one of
//            1.  So m starts 24 above the first scores and stays as it is until
//            one exceeds it by more than 8 (it goes to the integer 24 above that
//            one then, which scales O, l and the tile's weights by a power of
//            two), and the weights need not wait for the tile's maximum
#pragma once

#include "paged.cuh"

namespace moe {

constexpr int kRows = 128;               // rows of a sub-tile (MMA M)
constexpr int kPos = 128;                // positions of a tile
// How far the reference is set above a score, and which excess of a score over it
// moves it (log2).  Together the 32 by which scores may rise before O has to be
// scaled: with 8 alone a call whose scores spread by 4 took 147 us instead of 130,
// by 8 154.  Weights of up to 2^9 leave values of up to 2^105 and down to 2^-90 and
// their sums in fp32's range (with 0 and 32 values of 2^95 gave infinities).
constexpr float kAbove = 24.f, kRaise = 8.f;

__host__ __device__ constexpr int tile_bytes(int D) { return kPos * D * 2; }

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1, int c2,
                                            int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

// Descriptor of values as the MN-major B operand (dimensions contiguous, 128-byte
// swizzle): 64 dimensions x 8 positions are 1024 bytes; the next 64 dimensions
// are a half tile (kPos x 128 bytes) away, the next 8 positions 1024 bytes.
__device__ __forceinline__ uint64_t sdesc_mn128(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>((kPos * 128) >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

constexpr uint32_t kBTransposed = 1u << 16;  // instruction descriptor: B is MN-major
constexpr uint32_t kANegated = 1u << 13;     // A's signs are flipped

// 2^x by the hardware's approximation (relative error about 2^-22; results
// below 2^-126 are zero).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Where a box of a tile's positions is: lane `box * halves + half` of the loading
// warp fetches one.  A page outside the pool lies past the tensor map (zeros) and
// is recorded.
struct TileBox {
    int page, row;
};
__device__ __forceinline__ TileBox tile_box(const Pages &c, const int *pages, int p, int *status) {
    TileBox b{pages[p >> c.page_shift], p & ((1 << c.page_shift) - 1)};
    if (b.page < 0 || b.page >= c.n_pages) {
        record_status(status, MOE_ERR_PAGE);
        b.page = c.n_pages;
    }
    return b;
}

// S = Q K^T of a tile: q and k K-major in halves of 64 dimensions; flags: kANegated or 0.
template <int D>
__device__ __forceinline__ void tile_scores(uint32_t sS, uint32_t q_addr, uint32_t k_addr, uint32_t flags = 0) {
    const uint32_t id_s = idesc_bf16(kRows, kPos) | flags;
    constexpr int HALF = kPos * 128;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk / 4) * HALF + (kk % 4) * 32;
        umma_bf16(sS, sdesc_k128(q_addr + off), sdesc_k128(k_addr + off), id_s, kk != 0);
    }
}

// O += P V for the tile's positions 64 half .. 64 half + 63 (O = for the first,
// with add = 0).
template <int D>
__device__ __forceinline__ void tile_values(uint32_t sO, uint32_t sS, uint32_t v_addr, int half, uint32_t add) {
    constexpr uint32_t id_o = idesc_bf16(kRows, D) | kBTransposed;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int kk = 4 * half + i;
        umma_bf16_ts(sO, sS + half * 32 + kk * 8, sdesc_mn128(v_addr + kk * 2048), id_o, add | kk);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int kk = 4 * half + i;
        umma_bf16_ts(sO, sS + half * 32 + 32 + kk * 8, sdesc_mn128(v_addr + kk * 2048), id_o, 1);
    }
}

// The softmax of one tile for this thread's row, from the scores in tensor memory
// to the weights in their place: sS, sO with the warp's lanes; m, l and `any`
// (whether a tile of this row came before) are the row's state; p_full[h] hears
// that the weights of half h are there.  mask(y, n0) takes the scores n0 .. n0 + 31
// that have no weight to minus infinity; meanwhile() runs while the scores are on
// their way, and ends the tile by false.
template <int D, typename Mask, typename Meanwhile>
__device__ __forceinline__ bool tile_softmax(uint32_t sS, uint32_t sO, float scale_log2, float &m, float &l, bool any,
                                             uint64_t *p_full, Mask mask, Meanwhile meanwhile) {
    uint32_t xa[32], xb[32], xc[32];
    tmem_ld32(sS, xa);
    tmem_ld32(sS + 32, xb);
    if (!meanwhile()) {
        // (no load is under way when tensor memory is freed)
        tmem_wait32(xa);
        tmem_wait32(xb);
        return false;
    }
    uint64_t l2[2] = {0, 0};
    auto top = [&](const uint32_t *y, const uint32_t *z) {
        float t[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
            t[0] = max3(t[0], __uint_as_float(y[e]), __uint_as_float(y[e + 1]));
            t[1] = max3(t[1], __uint_as_float(z[e]), __uint_as_float(z[e + 1]));
        }
        return fmaxf(t[0], t[1]) * scale_log2;
    };
    // Move the reference of the rows whose score exceeds it by too
    // much (the warp's 32 rows together; p: weights of this tile so
    // far, in words): rare but for a block's first tile
    auto raise = [&](float tm, int p) {
        // (from the score itself: a step from m would lose it if m is far away)
        const float m_new = tm > m + kRaise ? ceilf(tm) + kAbove : m;
        const float corr = ex2(m - m_new);
        m = m_new;
        l *= corr;
        const uint64_t c2 = pack2(__float_as_uint(corr), __float_as_uint(corr));
        l2[0] = fma2(l2[0], c2, 0);
        l2[1] = fma2(l2[1], c2, 0);
        if (p) {
            tmem_st_wait();
            const __nv_bfloat162 cb = __float2bfloat162_rn(corr);
#pragma unroll 1
            for (int d = 0; d < p; d += 16) {
                uint32_t v[16];
                tmem_ld16_now(sS + d, v);
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = bf162_as_u32(__hmul2(u32_as_bf162(v[e]), cb));
                tmem_st16(sS + d, v);
            }
        }
        if (any) {
#pragma unroll 1
            for (int d = 0; d < D; d += 16) {
                uint32_t v[16];
                tmem_ld16_now(sO + d, v);
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * corr);
                tmem_st16(sO + d, v);
            }
        }
    };
    // weights, in two bf16 parts for the product; l sums them in fp32
    const uint64_t minus1 = pack2(0xBF800000u, 0xBF800000u);
    const uint64_t scale2 = pack2(__float_as_uint(scale_log2), __float_as_uint(scale_log2));
    auto weigh = [&](const uint32_t *y, int n0) {
        const uint64_t neg_m = pack2(__float_as_uint(-m), __float_as_uint(-m));
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            float2 w = unpack2(fma2(pack2(y[2 * e], y[2 * e + 1]), scale2, neg_m));
            w.x = ex2(w.x);
            w.y = ex2(w.y);
            const uint64_t w2 = pack2(__float_as_uint(w.x), __float_as_uint(w.y));
            hi[e] = bf162_as_u32(__floats2bfloat162_rn(w.x, w.y));
            const float2 r = unpack2(fma2(pack2(hi[e] << 16, hi[e] & 0xFFFF0000u), minus1, w2));
            lo[e] = bf162_as_u32(__floats2bfloat162_rn(r.x, r.y));
            l2[e & 1] = add2(l2[e & 1], w2);
        }
        // (positions 64 on have their columns from 64 on)
        tmem_st16(sS + n0 / 2 + n0 / 64 * 32, hi);
        tmem_st16(sS + n0 / 2 + n0 / 64 * 32 + 32, lo);
    };
    tmem_wait32(xa);
    tmem_wait32(xb);
    mask(xa, 0);
    mask(xb, 32);
    float tm = top(xa, xb);
    if (!any)
        m = fmaxf(ceilf(tm) + kAbove, kLeastRef);
    else if (__any_sync(0xffffffffu, tm > m + kRaise))
        raise(tm, 0);
    tmem_ld32(sS + 64, xc);
    weigh(xa, 0);
    tmem_ld32(sS + 96, xa);
    weigh(xb, 32);
    tmem_wait32(xc);
    tmem_wait32(xa);
    mask(xc, 64);
    mask(xa, 96);
    tm = top(xc, xa);
    if (__any_sync(0xffffffffu, tm > m + kRaise)) raise(tm, 64);
    tmem_st_wait();
    tc_fence_before();
    mbar_arrive(&p_full[0]);
    weigh(xc, 64);
    weigh(xa, 96);
    tmem_st_wait();
    tc_fence_before();
    mbar_arrive(&p_full[1]);
    const float2 lsum = unpack2(add2(l2[0], l2[1]));
    l += lsum.x + lsum.y;
    return true;
}

}  // namespace moe
