// Attention of a whole batch over a shared prefix on the fifth-generation
// tensor cores.
//
// Every query row of the batch that shares a key-value head (B rows times the
// group) attends to the same keys and values, so the prefix is one dense
// problem per key-value head: S = Q K^T, P = 2^(S - m), O = P V with up to
// thousands of rows.  Both products run as tcgen05.mma with M = 128 rows.
//
//   work     128 positions x one block of rows is a tile; all tiles of all
//            blocks and key-value heads are one list, cut into even pieces,
//            one per SM; a piece leaves one partial (m, l, O) per block it
//            meets, for the combine kernel
//   rows     blocks of 256 rows as two sub-tiles of 128 (slot 0 and 1) that
//            share the keys and values in shared memory: while one slot is in
//            its softmax, the tensor core works for the other.  Up to 128 rows
//            in all: one sub-tile; slot 0 takes the even and slot 1 the odd
//            tiles, each with a partial of its own
//   tile     per slot as in attn_tile.cuh; S and O of both take 512 columns of
//            tensor memory at D = 128.  With weights of one bf16 part instead of
//            two a call with 128 rows behind 131072 positions took 106 us instead of
//            129, and rows lost accuracy by sharing their prefix
//
//   warps 0-3, 4-7   softmax of slot 0, 1 (warp w: rows 32 (w % 4) ..)
//   warp 8           loads: 64-dimension boxes of page rows by TMA, 128-byte
//                    swizzle, keys and values in turn through one ring
//   warps 9, 10      MMA issue of slot 0, 1: a tile's second product and then
//                    the slot's next first one.  A token goes to and fro between
//                    the two, so that the slots stay half a period apart (left
//                    alone they fell into step, both in their softmax or both
//                    at the tensor core: with weights of one part 5,300 cycles
//                    for a tile of both instead of 3,400) and
//                    one's barrier waits and commits pass while the other issues
//
// Measured, this kernel alone: 128 rows of 16 heads behind 131072 positions 119 us,
// 1.15 PFLOP/s and the tensor pipe 81 % busy, the lower parts of the weights a
// third of it (the rest is each slot's wait from its scores to its first weights,
// which the other slot's products do not quite cover); 32 rows behind 32749
// positions 22 us: 103 pieces of five tiles of about 3 us, then two partials of
// 64 KB each.
//
// A position outside the pool is loaded as zeros (the page coordinate lies
// past the tensor map) and recorded.  Every wait is bounded.
#include "attn_tile.cuh"

namespace moe {

constexpr int kKvStages = 4;             // key or value tiles in flight
constexpr int kPrefixThreads = 11 * 32;
struct PrefixCtl {
    uint64_t kv_full[kKvStages], kv_empty[kKvStages];
    uint64_t q_free;         // every role is past the previous block of rows
    uint64_t q_full;         // queries of the block are in shared memory
    uint64_t s_full[2];      // scores of the slot's tile are in tensor memory
    uint64_t p_full[2][2];   // weights of its positions 0-63, 64-127 are (and O is ready to be added to)
    uint64_t o_full[2];      // O of the block of rows is complete
    uint64_t token[2];       // the slot's issuer may go on
    uint64_t drain;
    uint32_t tmem;
    int abort;
};

__host__ __device__ constexpr int prefix_smem_bytes(int D) {
    return 2 * kRows * D * 2 + kKvStages * tile_bytes(D) + 1024 + static_cast<int>(sizeof(PrefixCtl));
}
static_assert(prefix_smem_bytes(128) <= 227 * 1024, "one block per SM");

__device__ __forceinline__ bool prefix_wait(uint64_t *bar, uint32_t parity, const PagedArgs &a, PrefixCtl *s, int site) {
    return role_wait(bar, parity, a.wait_limit, a.status, &s->abort, site);
}

template <int D>
__global__ void __launch_bounds__(kPrefixThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ PagedArgs a) {
    constexpr int HALVES = D / 64;                 // 64-dimension halves of a row
    constexpr int HALF = kPos * 128;               // bytes of one half of a tile
    constexpr int TILE = tile_bytes(D);
    constexpr int QSUB = kRows * D * 2;
    constexpr uint32_t kTmemCols = 512;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = base, *sKV = base + 2 * QSUB;
    PrefixCtl *s = reinterpret_cast<PrefixCtl *>(sKV + kKvStages * TILE);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool two = a.prefix_two;                 // 256-row blocks; else the slots share the tiles

    if (tid == 0) {
        for (int i = 0; i < kKvStages; ++i) {
            mbar_init(&s->kv_full[i], 1);
            mbar_init(&s->kv_empty[i], two ? 2 : 1);
        }
        mbar_init(&s->q_free, 256 + 2);
        mbar_init(&s->q_full, 256);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s->s_full[i], 1);
            mbar_init(&s->p_full[i][0], kRows);
            mbar_init(&s->p_full[i][1], kRows);
            mbar_init(&s->o_full[i], 1);
            mbar_init(&s->token[i], 1);
        }
        mbar_init(&s->drain, 2);
        s->abort = 0;
        fence_mbar_init();
    }
    if (warp == 8 && lane == 0) {
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }
    if (warp == 9) {
        tmem_alloc(&s->tmem, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s->tmem;
    pdl_wait();
    pdl_trigger();

    // this block's piece of the list; item = (key-value head, block of rows)
    const int ntile = a.prefix_tiles, nblk = a.prefix_blocks;
    const int rows = a.B * a.group;
    const int64_t W = static_cast<int64_t>(a.c.Hkv) * nblk * ntile;
    const int64_t f0 = static_cast<int64_t>(blockIdx.x) * a.prefix_per, f1 = f0 + a.prefix_per < W ? f0 + a.prefix_per : W;
    const int item0 = static_cast<int>(f0 / ntile), tile0 = static_cast<int>(f0 % ntile);
    const int count = static_cast<int>(f1 - f0);  // tiles of this piece
    const int per_block = two ? 2 * kRows : kRows;

    if (warp == 8) {
        // ------------------------------------------------------------ loads
        const int ps = a.c.page_shift;
        const int box_rows = ps >= 7 ? kPos : 1 << ps;
        uint32_t it = 0;
        bool ok = true;
        int item = item0, t = tile0;
        for (int j = 0; j < count && ok; ++j, ++t) {
            if (t == ntile) {
                t = 0;
                ++item;
            }
            const int kv = item / nblk, p0 = t * kPos;
            const int left = a.prefix_len - p0;
            const int boxes = ((left < kPos ? left : kPos) + box_rows - 1) / box_rows;
            // lane j: half j % HALVES of box j / HALVES (at most 16 boxes of 2 halves)
            const int bx = lane / HALVES, half = lane % HALVES;
            TileBox at{0, 0};
            if (bx < boxes) at = tile_box(a.c, a.prefix_pages, p0 + bx * box_rows, a.status);
            for (int m = 0; m < 2 && ok; ++m, ++it) {  // keys, then values
                const int st = it % kKvStages;
                ok = prefix_wait(&s->kv_empty[st], ((it / kKvStages) & 1) ^ 1, a, s, 21);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(&s->kv_full[st], boxes * box_rows * D * 2);
                __syncwarp();
                if (bx < boxes)
                    tma_load_4d(smem_u32(sKV + st * TILE + half * HALF + bx * box_rows * 128), m ? &tm_v : &tm_k,
                                &s->kv_full[st], half * 64, at.row, kv, at.page);
            }
        }
        // no copy of this block is in flight when it ends
        for (uint32_t i = it > kKvStages ? it - kKvStages : 0; i < it; ++i)
            mbar_drain(&s->kv_full[i % kKvStages], (i / kKvStages) & 1, a.wait_limit);
    } else if (warp >= 9) {
        // -------------------------------------------------------- MMA issue
        // (one thread, elected rather than picked by lane number: the compiler
        // then keeps the descriptors in uniform registers, and eight MMAs issue
        // in 450 instead of 680 cycles)
        if (elect_one()) {
            const int slot = __shfl_sync(__activemask(), warp, 0) - 9;
            const uint32_t sS = tmem + slot * 128, sO = tmem + 256 + slot * D;
            const uint32_t q_addr = smem_u32(sQ + (two ? slot * QSUB : 0)), kv_addr = smem_u32(sKV);
            uint32_t it0 = 0, nq = 0;              // ring entry of the block's first tile, blocks of rows
            uint32_t done = 0, tok = 0;            // this slot's tiles so far, tokens taken
            bool ok = true;
            int t = tile0;
            for (int j = 0, item = item0; j < count && ok; ++item, t = 0) {
                const int nt = ntile - t < count - j ? ntile - t : count - j;  // tiles of this block here
                // steps of the block: a tile for one slot.  With 256 rows every
                // tile for both slots in turn (n / 2, n % 2), else tile n for
                // slot n % 2, or all for slot 0 where slot 1 has no rows
                const bool both = two && item % nblk * per_block + kRows < rows;
                const bool alone = two && !both;
                const int steps = both ? 2 * nt : nt, next = alone ? 1 : 2;
                auto scores = [&](int n) {
                    const uint32_t e = it0 + 2 * (both ? n >> 1 : n), st = e % kKvStages;
                    // S overwrites the slot's previous weights: their product was
                    // issued before, by this thread, and the tensor core takes
                    // MMAs in the order of issue
                    ok = prefix_wait(&s->kv_full[st], (e / kKvStages) & 1, a, s, 25);
                    if (!ok) return;
                    tc_fence_after();
                    tile_scores<D>(sS, q_addr, kv_addr + st * TILE);
                };
                // (s_full also says that the previous tile's second product is complete)
                auto scores_end = [&](int n) {
                    umma_commit(&s->s_full[slot]);
                    umma_commit(&s->kv_empty[(it0 + 2 * (both ? n >> 1 : n)) % kKvStages]);
                };
                mbar_arrive(&s->q_free);
                ok = prefix_wait(&s->q_full, nq & 1, a, s, 22);
                ++nq;
                if (alone && slot == 1) {
                    // no rows here: give the tiles back
                    for (uint32_t e = it0; e < it0 + 2 * nt && ok; ++e) {
                        ok = prefix_wait(&s->kv_full[e % kKvStages], (e / kKvStages) & 1, a, s, 23);
                        if (ok) mbar_arrive(&s->kv_empty[e % kKvStages]);
                    }
                } else {
                    if (slot < steps && ok) {
                        scores(slot);
                        if (ok) scores_end(slot);
                    }
                    for (int n = slot; n < steps && ok; n += next, ++done) {
                        const uint32_t e = it0 + 2 * (both ? n >> 1 : n) + 1, st = e % kKvStages;
                        const uint32_t v_addr = kv_addr + st * TILE;
                        ok = prefix_wait(&s->kv_full[st], (e / kKvStages) & 1, a, s, 26);
                        if (n > 0 && !alone) ok = ok && prefix_wait(&s->token[slot], tok++ & 1, a, s, 33);
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            ok = ok && prefix_wait(&s->p_full[slot][half], done & 1, a, s, 27);
                            if (!ok) break;
                            tc_fence_after();
                            tile_values<D>(sO, sS, v_addr, half, n < next ? 0 : 1);
                        }
                        if (!ok) break;
                        if (n + next < steps) scores(n + next);
                        if (!ok) break;
                        if (n + 1 < steps && !alone) mbar_arrive(&s->token[slot ^ 1]);
                        if (n + next < steps)
                            scores_end(n + next);
                        else
                            umma_commit(&s->o_full[slot]);
                        umma_commit(&s->kv_empty[st]);
                    }
                }
                it0 += 2 * nt;
                j += nt;
            }
            // every MMA issued here is complete before tensor memory is freed
            umma_commit(&s->drain);
            mbar_drain(&s->drain, 0, a.wait_limit);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------- softmax
        const int slot = warp >> 2, r = tid & 127;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t sS = (tmem + slot * 128) | lanes, sO = (tmem + 256 + slot * D) | lanes;
        uint32_t it = 0;
        uint32_t turn = 0;                             // parities: blocks of rows (1), of those with tiles (2), this slot's tiles (4)
        bool ok = true;
        int t = tile0;
        for (int j = 0, item = item0; j < count && ok; ++item, t = 0) {
            const int kv = item / nblk, blk = item % nblk;
            const int end = j + (ntile - t) < count ? j + (ntile - t) : count;

            // the block's queries into shared memory (K-major, 128-byte swizzle):
            // eight threads a row's 16-byte chunks; rows past the batch are zeros.
            // The slots have seen the scores of the previous block's last tile and
            // the issuers are past it, so that nothing reads the old ones
            mbar_arrive(&s->q_free);
            ok = prefix_wait(&s->q_free, turn & 1, a, s, 32);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            turn ^= 1;
            {
                // all copies in flight together (as plain loads and stores they cost
                // 10 of the 18 us of a short prefix)
                constexpr int CH = D / 8;
                const int ch = tid % CH, h0 = kv * a.group;
                uint8_t *dst = sQ + (ch / 8) * HALF;
                // (g / group by a 16-bit reciprocal: exact for g < 8192, group <= 8)
                const uint32_t recip = (65536 + a.group - 1) / a.group;
#pragma unroll 2
                for (int row = tid / CH; row < per_block; row += 256 / CH) {
                    const int g = blk * per_block + row;
                    const int b = g < rows ? static_cast<int>((g * recip) >> 16) : 0, h = g < rows ? g - b * a.group : 0;
                    cp_async16_zfill(smem_u32(dst + (row / kRows) * QSUB + (row % kRows) * 128 + (((ch % 8) ^ (row & 7)) << 4)),
                                 a.q + b * a.q_stride + static_cast<int64_t>(h0 + h) * D + ch * 8, g < rows);
                }
                cp_async_wait_all();
                if (a.negate || a.zero_q) {
                    // each thread turns the chunks that it copied
                    for (int row = tid / CH; row < per_block; row += 256 / CH) {
                        uint4 *q4 = reinterpret_cast<uint4 *>(dst + (row / kRows) * QSUB + (row % kRows) * 128 +
                                                              (((ch % 8) ^ (row & 7)) << 4));
                        uint4 v = *q4;
                        v = a.zero_q ? make_uint4(0u, 0u, 0u, 0u)
                                     : make_uint4(v.x ^ 0x80008000u, v.y ^ 0x80008000u, v.z ^ 0x80008000u, v.w ^ 0x80008000u);
                        *q4 = v;
                    }
                }
                fence_proxy_async_smem();
                mbar_arrive(&s->q_full);
            }
            const int row0 = blk * per_block + (two ? slot * kRows : 0);  // this slot's first row
            const bool active = row0 < rows;
            const bool warp_real = row0 + (warp & 3) * 32 < rows;  // a warp without rows only keeps step
            float m = -INFINITY, l = 0.f;
            bool any = false;
            for (int n = 0; j < end; ++j, ++t, ++n, it += 2) {
                if (!active || (!two && (n & 1) != slot)) continue;
                const int valid = a.prefix_len - t * kPos;
                ok = prefix_wait(&s->s_full[slot], turn >> 2, a, s, 28);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                if (!warp_real && valid >= kPos) {
                    mbar_arrive(&s->p_full[slot][0]);
                    mbar_arrive(&s->p_full[slot][1]);
                    any = true;
                    turn ^= 4;
                    continue;
                }
                // scores past the prefix's end have no weight
                auto mask = [&](uint32_t *y, int n0) {
                    if (n0 + 32 > valid) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (n0 + e >= valid) y[e] = 0xFF800000u;
                    }
                };
                auto meanwhile = [&]() {
                    if (valid >= kPos) return true;
                    // value rows past the prefix's end may hold anything: zeros
                    const uint32_t vi = (it + 1) % kKvStages;
                    if (!__all_sync(0xffffffffu, prefix_wait(&s->kv_full[vi], ((it + 1) / kKvStages) & 1, a, s, 30)))
                        return false;
                    for (int i = valid * 8 + r; i < kPos * 8; i += kRows)
#pragma unroll
                        for (int h = 0; h < HALVES; ++h)
                            *reinterpret_cast<uint4 *>(sKV + vi * TILE + h * HALF + i * 16) = make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();
                    return true;
                };
                ok = tile_softmax<D>(sS, sO, a.scale_log2, m, l, any, s->p_full[slot], mask, meanwhile);
                if (!ok) break;
                any = true;
                turn ^= 4;
            }
            if (!ok) break;
            // this piece's partial of the block
            if (active) {
                const int64_t part = (static_cast<int64_t>(blockIdx.x) + item) * 2 + slot;
                if (any) {  // also without rows: the next block's first tile comes after this
                    ok = prefix_wait(&s->o_full[slot], turn >> 1 & 1, a, s, 31);
                    turn ^= 2;
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    float *dst = a.prefix_o + part * (D * kRows) + r * 4;
                    if (warp_real)
#pragma unroll
                    for (int d = 0; d < D; d += 32) {
                        uint32_t v[32];
                        tmem_ld32(sO + d, v);
                        tmem_wait32(v);
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            if (row0 + r < rows)
                                *reinterpret_cast<float4 *>(dst + (d + e) / 4 * (kRows * 4)) = make_float4(
                                    __uint_as_float(v[e]), __uint_as_float(v[e + 1]), __uint_as_float(v[e + 2]),
                                    __uint_as_float(v[e + 3]));
                    }
                    tc_fence_before();
                }
                a.prefix_ml[part * kRows + r] = make_float2(any ? m : -INFINITY, l);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D>
static cudaError_t launch_t(const CUtensorMap &k, const CUtensorMap &v, const PagedArgs &a, cudaStream_t s) {
    constexpr int smem = prefix_smem_bytes(D);
    const cudaError_t e = allow_smem<prefix_kernel<D>>();
    if (e != cudaSuccess) return e;
    return launch_dependent(prefix_kernel<D>, dim3(a.prefix_ncta), dim3(kPrefixThreads), smem, s, k, v, a);
}

cudaError_t launch_prefix(const CUtensorMap &k, const CUtensorMap &v, const PagedArgs &a, cudaStream_t s) {
    return a.c.D == 64 ? launch_t<64>(k, v, a, s) : launch_t<128>(k, v, a, s);
}

}  // namespace moe
