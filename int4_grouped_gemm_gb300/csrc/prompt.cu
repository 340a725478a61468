// Causal attention of packed sequences of query tokens over the paged cache, on the
// fifth-generation tensor cores.
//
//   rows     all heads that share a key-value head are rows of one product: a
//            sub-tile of 128 rows is tq = 128 / group tokens (16 of 8 heads), a
//            block two sub-tiles (slot 0 and 1), which share the keys and values in
//            shared memory; while one slot is in its softmax, the tensor core works
//            for the other.  With the heads together a block spans few tokens, so
//            that little of its last tile lies above the diagonal
//   work     a block against 128 positions is a tile: first the shared prefix's, then
//            the sequence's own up to the block's last token.  The tiles of all
//            blocks and key-value heads are one list, cut into even pieces, one per
//            SM.  Blocks that lie within a piece write their rows of out; of those
//            that a cut runs through every piece leaves a partial (m, l, O), and
//            prompt_combine_kernel joins them
//   plan     lengths and starts are on the device (a captured call is replayed with
//            others): prompt_plan_kernel makes the list
//   tile     as in attn_tile.cuh
//
//   warps 0-3, 4-7   softmax of slot 0, 1 (warp w: rows 32 (w % 4) ..)
//   warp 8           loads: 64-dimension boxes of page rows by TMA, 128-byte
//                    swizzle, keys and values in turn through one ring
//   warps 9, 10      MMA issue of slot 0, 1, in turn by a token to and fro
//
// Masks.  A row's scores past its own position become minus infinity.  What the
// value rows hold there would still meet a weight of zero in the product, and zero
// times NaN or infinity is NaN: rows past the block's last token become zeros, and
// in tiles that only some of the block's tokens see whole, values that are not
// finite become zeros and are added, as they are, to the rows that see them when
// the block is written.
//
// A position outside the pool is loaded as zeros (the page coordinate lies past
// the tensor map) and recorded.  Every wait is bounded.
#include "attn_tile.cuh"
#include "prompt.cuh"

namespace moe {

constexpr int kStages = 4;               // key or value tiles in flight
constexpr int kThreads = 11 * 32;
constexpr int kDiag = 3;                 // tiles that a block's own tokens (at most 256) lie in

struct PromptCtl {
    uint64_t kv_full[kStages], kv_empty[kStages];
    uint64_t q_free;         // every role is past the previous block of rows
    uint64_t q_full;         // queries of the block are in shared memory
    uint64_t s_full[2];      // scores of the slot's tile are in tensor memory
    uint64_t p_full[2][2];   // weights of its positions 0-63, 64-127 are (and O is ready to be added to)
    uint64_t o_full[2];      // O of the block of rows is complete
    uint64_t token[2];       // the slot's issuer may go on
    uint64_t drain;
    uint32_t tmem;
    int abort;
    uint32_t broken[kDiag][4];  // positions of the block's own tiles with values that are not finite
    int any_broken;
};

__host__ __device__ constexpr int prompt_smem_bytes(int D) {
    return 2 * kRows * D * 2 + kStages * tile_bytes(D) + 1024 + static_cast<int>(sizeof(PromptCtl));
}
static_assert(prompt_smem_bytes(128) <= kBlockSmem, "one block per SM");

// ------------------------------------------------------------------ plan

__device__ __forceinline__ int tiles_of(int positions) { return (positions + kPos - 1) / kPos; }

// Inclusive sum over the block's threads; `total` gets the sum of all.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *warp_sums, int64_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, v, i);
        if (lane >= i) v += o;
    }
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    int64_t before = 0;
    total = 0;
    for (int i = 0; i < warps; ++i) {
        const int64_t w = warp_sums[i];
        before += i < warp ? w : 0;
        total += w;
    }
    __syncthreads();
    return v + before;
}

// The largest i < n with at[i] <= v (at[0] <= v).
template <typename T>
__device__ __forceinline__ int last_not_above(const T *at, int n, T v) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at[mid] <= v)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

constexpr int kPlanThreads = 1024;

// One block: the sequences' blocks of rows, their tiles, and where the pieces begin.
// A sequence that is padding, or whose rows or length are out of range, has none.
__global__ void __launch_bounds__(kPlanThreads) prompt_plan_kernel(const __grid_constant__ PromptArgs a) {
    __shared__ int64_t warp_sums[kPlanThreads / 32];
    const int tid = threadIdx.x, span = 2 * a.tq;
    pdl_wait();
    pdl_trigger();
    int nblocks = 0;
    for (int b0 = 0; b0 < a.n_seq; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int n = 0;
        if (b < a.n_seq) {
            const int r0 = a.q_start[b], r1 = a.q_start[b + 1], len = a.seq_len[b];
            if (r0 < 0 || r1 < r0 || r1 > a.T || len > static_cast<int64_t>(a.table_ld) << a.c.page_shift)
                record_status(a.status, MOE_ERR_PAGE);
            else if (len >= 0)
                n = (r1 - r0 + span - 1) / span;
        }
        int64_t total;
        const int64_t upto = block_scan(n, warp_sums, total);
        // (rows of several sequences at once, by starts that go back, may be more than
        // there is room for)
        if (b < a.n_seq) a.seq_blocks[b] = static_cast<int>(min(nblocks + upto - n, static_cast<int64_t>(a.max_blocks)));
        nblocks = static_cast<int>(min(nblocks + total, static_cast<int64_t>(a.max_blocks)));
    }
    if (tid == 0) a.seq_blocks[a.n_seq] = nblocks;
    __syncthreads();
    const int prefix_tiles = tiles_of(a.prefix_len);
    int64_t tiles = 0;
    for (int i0 = 0; i0 < nblocks; i0 += kPlanThreads) {
        const int i = i0 + tid;
        int n = 0;
        if (i < nblocks) {
            // (of sequences without blocks, which start where the next one does, the last
            // at i or before is the one that has it)
            const int b = last_not_above(a.seq_blocks, a.n_seq, i);
            const int r0 = a.q_start[b], r1 = a.q_start[b + 1], first = (i - a.seq_blocks[b]) * span;
            PromptBlock k;
            k.seq = b;
            k.row0 = r0 + first;
            k.pos0 = a.seq_len[b] - (r1 - r0) + first;
            k.ntok = r1 - k.row0 < span ? r1 - k.row0 : span;
            a.blocks[i] = k;
            const int end = k.pos0 + k.ntok;
            n = prefix_tiles + (end > 0 ? tiles_of(end) : 0);
            n = n > 0 ? n : 1;  // rows that see nothing are written too
        }
        int64_t total;
        const int64_t upto = block_scan(n, warp_sums, total);
        if (i < nblocks) a.start[i] = tiles + upto - n;
        tiles += total;
    }
    const int64_t all = tiles * a.c.Hkv, per = (all + a.ncta - 1) / a.ncta;
    if (tid == 0) {
        a.start[nblocks] = tiles;
        *a.plan = PromptPlan{tiles, per, nblocks};
    }
    __syncthreads();
    for (int c = tid; c < a.ncta; c += kPlanThreads)
        if (c * per < all) a.piece_block[c] = last_not_above(a.start, nblocks, c * per % tiles);
}

// ------------------------------------------------------------------ main

__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, const PromptArgs &a, PromptCtl *s, int site) {
    return role_wait(bar, parity, a.wait_limit, a.status, &s->abort, site);
}

// A piece's way through the list: its part of one (key-value head, block) after
// another.
struct Walk {
    int left;       // tiles of the piece from here on
    int kv, blk;
    int t, n;       // first tile of the block here, tiles of it here
    bool whole;     // all of them
    PromptBlock k;

    __device__ __forceinline__ void load(const PromptArgs &a) {
        const int4 v = __ldcg(reinterpret_cast<const int4 *>(a.blocks + blk));
        k = PromptBlock{v.x, v.y, v.z, v.w};
        const int of = static_cast<int>(__ldcg(a.start + blk + 1) - __ldcg(a.start + blk));
        n = of - t < left ? of - t : left;
        whole = n == of;
    }
    // False: there are fewer tiles than pieces.
    __device__ __forceinline__ bool first(const PromptArgs &a) {
        const int64_t tiles = __ldcg(&a.plan->tiles), per = __ldcg(&a.plan->per), f0 = blockIdx.x * per;
        const int64_t rest = tiles * a.c.Hkv - f0;
        if (rest <= 0) return false;
        left = static_cast<int>(rest < per ? rest : per);
        kv = static_cast<int>(f0 / tiles);
        blk = __ldcg(a.piece_block + blockIdx.x);
        t = static_cast<int>(f0 % tiles - __ldcg(a.start + blk));
        load(a);
        return true;
    }
    __device__ __forceinline__ bool next(const PromptArgs &a) {
        left -= n;
        if (left <= 0) return false;
        t = 0;
        if (++blk == __ldcg(&a.plan->nblocks)) {
            blk = 0;
            ++kv;
        }
        load(a);
        return true;
    }
};

// For scales below zero the queries with their signs flipped, for zero zeros: each
// of 256 threads turns the 16-byte chunks (from column `dst` on) that it copied.
template <int D>
__device__ __noinline__ void turn_queries(uint8_t *dst, bool zero) {
    constexpr int CH = D / 8;
    const int ch = threadIdx.x % CH;
    for (int row = threadIdx.x / CH; row < 2 * kRows; row += 256 / CH) {
        uint4 *q4 = reinterpret_cast<uint4 *>(dst + (row / kRows) * (kRows * D * 2) + (row % kRows) * 128 +
                                              (((ch % 8) ^ (row & 7)) << 4));
        const uint4 v = *q4;
        *q4 = zero ? make_uint4(0u, 0u, 0u, 0u)
                   : make_uint4(v.x ^ 0x80008000u, v.y ^ 0x80008000u, v.z ^ 0x80008000u, v.w ^ 0x80008000u);
    }
}

// Makes the value rows of a tile safe to be met by weights of zero, by a slot's 128
// threads: those from `valid` on may hold anything and become zeros, and in the
// block's own tile number `own` (-1: another) what is not finite does and is noted.
// (Not inlined: a tile's softmax takes all registers.)
template <int D>
__device__ __noinline__ void clean_values(PromptCtl *s, uint4 *v, int valid, int own) {
    const int r = threadIdx.x & 127;
    constexpr int HALF = kPos * 128 / 16;
    for (int i = valid * 8 + r; i < kPos * 8; i += kRows)
#pragma unroll
        for (int h = 0; h < D / 64; ++h) v[h * HALF + i] = make_uint4(0u, 0u, 0u, 0u);
    if (own < 0) return;
    for (int i = r; i < valid * 8; i += kRows)
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
            // (an exponent of all ones carries into the sign's place)
            uint32_t x[4], bad = 0;
            *reinterpret_cast<uint4 *>(x) = v[h * HALF + i];
#pragma unroll
            for (int e = 0; e < 4; ++e) bad |= (x[e] & 0x7F807F80u) + 0x00800080u;
            if (bad & 0x80008000u) {
                // (noted before they go, so that who finds zeros finds the note)
                atomicOr(&s->broken[own][i >> 8], 1u << (i >> 3 & 31));
                *reinterpret_cast<volatile int *>(&s->any_broken) = 1;
                __threadfence_block();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t b = (x[e] & 0x7F807F80u) + 0x00800080u;
                    if (b & 0x8000u) x[e] &= 0xFFFF0000u;
                    if (b & 0x80000000u) x[e] &= 0xFFFFu;
                }
                v[h * HALF + i] = *reinterpret_cast<uint4 *>(x);
            }
        }
}

// Adds the values noted as not finite to the rows (of a warp, at own position
// `pos`) that see them; first: the position of the first note.
template <int D>
__device__ __noinline__ void mend_rows(const PromptArgs &a, PromptCtl *s, uint32_t sO, int blk, int kv, int first, int pos) {
    const int *table = a.table + static_cast<int64_t>(a.blocks[blk].seq) * a.table_ld;
    for (int d = 0; d < D; d += 16) {
        uint32_t o[16];
        tmem_ld16_now(sO + d, o);
        for (int j = 0; j < kDiag * kPos; ++j) {
            const int p = first + j;
            if (p > pos || !(s->broken[j >> 7][(j >> 5) & 3] >> (j & 31) & 1)) continue;
            const int page = table[p >> a.c.page_shift];
            if (page < 0 || page >= a.c.n_pages) continue;
            const __nv_bfloat16 *x = a.c.v + page * a.c.page_stride + kv * a.c.head_stride +
                                     (p & ((1 << a.c.page_shift) - 1)) * a.c.pos_stride + d;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float f = __bfloat162float(x[e]);
                if (!(fabsf(f) < INFINITY)) o[e] = __float_as_uint(__uint_as_float(o[e]) + f);
            }
        }
        __syncwarp();
        tmem_st16(sO + d, o);
    }
    tmem_st_wait();
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ PromptArgs a) {
    constexpr int HALVES = D / 64;                 // 64-dimension halves of a row
    constexpr int HALF = kPos * 128;               // bytes of one half of a tile
    constexpr int TILE = tile_bytes(D);
    constexpr int QSUB = kRows * D * 2;
    constexpr uint32_t kTmemCols = 512;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = base, *sKV = base + 2 * QSUB;
    PromptCtl *s = reinterpret_cast<PromptCtl *>(sKV + kStages * TILE);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&s->kv_full[i], 1);
            mbar_init(&s->kv_empty[i], 2);
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

    const int ptiles = tiles_of(a.prefix_len);

    if (warp == 8) {
        // ------------------------------------------------------------ loads
        const int ps = a.c.page_shift;
        const int box_rows = ps >= 7 ? kPos : 1 << ps;
        // lane j: half j % HALVES of box j / HALVES (at most 8 boxes of 2 halves)
        const int bx = lane / HALVES, half = lane % HALVES;
        uint32_t it = 0;
        Walk w;
        bool ok = w.first(a);
        if (ok) do {
            for (int t = w.t; t < w.t + w.n && ok; ++t) {
                const bool pre = t < ptiles;
                const int p0 = (pre ? t : t - ptiles) * kPos;
                const int left = (pre ? a.prefix_len : w.k.pos0 + w.k.ntok) - p0;
                const int boxes = left <= 0 ? 0 : ((left < kPos ? left : kPos) + box_rows - 1) / box_rows;
                TileBox at{0, 0};
                if (bx < boxes)
                    at = tile_box(a.c, pre ? a.prefix_pages : a.table + static_cast<int64_t>(w.k.seq) * a.table_ld,
                                  p0 + bx * box_rows, a.status);
                for (int m = 0; m < 2 && ok; ++m, ++it) {  // keys, then values
                    const int st = it % kStages;
                    ok = wait(&s->kv_empty[st], ((it / kStages) & 1) ^ 1, a, s, 41);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&s->kv_full[st], boxes * box_rows * D * 2);
                    __syncwarp();
                    if (bx < boxes)
                        tma_load_4d(smem_u32(sKV + st * TILE + half * HALF + bx * box_rows * 128), m ? &tm_v : &tm_k,
                                    &s->kv_full[st], half * 64, at.row, w.kv, at.page);
                }
            }
        } while (ok && w.next(a));
        // no copy of this block is in flight when it ends
        for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i)
            mbar_drain(&s->kv_full[i % kStages], (i / kStages) & 1, a.wait_limit);
    } else if (warp >= 9) {
        // -------------------------------------------------------- MMA issue
        if (elect_one()) {
            const int slot = __shfl_sync(__activemask(), warp, 0) - 9;
            const uint32_t sS = tmem + slot * 128, sO = tmem + 256 + slot * D;
            const uint32_t q_addr = smem_u32(sQ + slot * QSUB), kv_addr = smem_u32(sKV);
            uint32_t it0 = 0, nq = 0;              // ring entry of the block's first tile, blocks of rows
            uint32_t done = 0, tok = 0;            // this slot's tiles so far, tokens taken
            Walk w;
            bool ok = w.first(a);
            if (ok) do {
                const int nt = w.n;
                // a tile for both slots in turn (step n: tile n / 2, slot n % 2), or all for
                // slot 0 where slot 1 has no tokens
                const bool both = w.k.ntok > a.tq;
                const int steps = both ? 2 * nt : nt, next = both ? 2 : 1;
                auto scores = [&](int n) {
                    const uint32_t e = it0 + 2 * (both ? n >> 1 : n), st = e % kStages;
                    // S overwrites the slot's previous weights: their product was
                    // issued before, by this thread, and the tensor core takes
                    // MMAs in the order of issue
                    ok = wait(&s->kv_full[st], (e / kStages) & 1, a, s, 42);
                    if (!ok) return;
                    tc_fence_after();
                    tile_scores<D>(sS, q_addr, kv_addr + st * TILE);
                };
                // (s_full also says that the previous tile's second product is complete)
                auto scores_end = [&](int n) {
                    umma_commit(&s->s_full[slot]);
                    umma_commit(&s->kv_empty[(it0 + 2 * (both ? n >> 1 : n)) % kStages]);
                };
                mbar_arrive(&s->q_free);
                ok = wait(&s->q_full, nq & 1, a, s, 43);
                ++nq;
                if (!both && slot == 1) {
                    // no rows here: give the tiles back
                    for (uint32_t e = it0; e < it0 + 2 * nt && ok; ++e) {
                        ok = wait(&s->kv_full[e % kStages], (e / kStages) & 1, a, s, 44);
                        if (ok) mbar_arrive(&s->kv_empty[e % kStages]);
                    }
                } else {
                    if (slot < steps && ok) {
                        scores(slot);
                        if (ok) scores_end(slot);
                    }
                    for (int n = slot; n < steps && ok; n += next, ++done) {
                        const uint32_t e = it0 + 2 * (both ? n >> 1 : n) + 1, st = e % kStages;
                        const uint32_t v_addr = kv_addr + st * TILE;
                        ok = wait(&s->kv_full[st], (e / kStages) & 1, a, s, 45);
                        if (n > 0 && both) ok = ok && wait(&s->token[slot], tok++ & 1, a, s, 46);
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            ok = ok && wait(&s->p_full[slot][half], done & 1, a, s, 47);
                            if (!ok) break;
                            tc_fence_after();
                            tile_values<D>(sO, sS, v_addr, half, n < next ? 0 : 1);
                        }
                        if (!ok) break;
                        if (n + next < steps) scores(n + next);
                        if (!ok) break;
                        if (n + 1 < steps && both) mbar_arrive(&s->token[slot ^ 1]);
                        if (n + next < steps)
                            scores_end(n + next);
                        else
                            umma_commit(&s->o_full[slot]);
                        umma_commit(&s->kv_empty[st]);
                    }
                }
                it0 += 2 * nt;
            } while (ok && w.next(a));
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
        const int group = a.group, tq = a.tq;
        // (rows / group by a 16-bit reciprocal: exact for rows below 8192, group <= 8)
        const uint32_t recip = (65536 + group - 1) / group;
        auto token_of = [&](int row) { return static_cast<int>((row * recip) >> 16); };
        const int tl = slot * tq + token_of(r);          // this row's token in the block
        const int tl_warp = slot * tq + token_of((warp & 3) * 32);  // its warp's first
        uint32_t it = 0, turn = 0;                       // ring entry; parities: blocks of rows (1), those with rows of this slot (2), its tiles (4)
        Walk w;
        bool ok = w.first(a);
        if (ok) do {
            const PromptBlock &k = w.k;
            // the block's queries into shared memory (K-major, 128-byte swizzle):
            // eight threads a row's 16-byte chunks; rows without a token are zeros.
            // The slots have seen the scores of the previous block's last tile and
            // the issuers are past it, so that nothing reads the old ones
            mbar_arrive(&s->q_free);
            ok = wait(&s->q_free, turn & 1, a, s, 48);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            turn ^= 1;
            {
                // all copies in flight together
                // (UNROLL: as the other unrolling makes the compiler spill two registers)
                constexpr int CH = D / 8, UNROLL = D == 128 ? 1 : 2;
                const int ch = tid % CH, h0 = w.kv * group;
                uint8_t *dst = sQ + (ch / 8) * HALF;
#pragma unroll UNROLL
                for (int row = tid / CH; row < 2 * kRows; row += 256 / CH) {
                    const int sub = row / kRows, g = row % kRows, i = token_of(g), tok = sub * tq + i;
                    const bool real = i < tq && tok < k.ntok;
                    cp_async16_zfill(smem_u32(dst + sub * QSUB + g * 128 + (((ch % 8) ^ (row & 7)) << 4)),
                                     a.q + static_cast<int64_t>(real ? k.row0 + tok : k.row0) * a.q_stride +
                                         static_cast<int64_t>(h0 + (real ? g - i * group : 0)) * D + ch * 8,
                                     real);
                }
                if (tid < kDiag * 4) (&s->broken[0][0])[tid] = 0;
                if (tid == kDiag * 4) s->any_broken = 0;
                cp_async_wait_all();
                if (a.negate || a.zero_q) turn_queries<D>(dst, a.zero_q);
                fence_proxy_async_smem();
                mbar_arrive(&s->q_full);
            }
            const bool active = slot * tq < k.ntok;      // this slot has rows
            const bool warp_real = tl_warp < k.ntok && token_of((warp & 3) * 32) < tq;
            const bool real = token_of(r) < tq && tl < k.ntok;
            const int diag0 = (k.pos0 > 0 ? k.pos0 : 0) / kPos;  // first own tile that not all of the block's tokens see whole
            float m = -INFINITY, l = 0.f;
            if (!active) {
                it += 2 * w.n;
                continue;
            }
            for (int t = w.t; t < w.t + w.n; ++t, it += 2) {
                const bool pre = t < ptiles;
                const int p0 = (pre ? t : t - ptiles) * kPos;
                const int left = (pre ? a.prefix_len : k.pos0 + k.ntok) - p0;  // positions of the tile
                const int valid = left < 0 ? 0 : left < kPos ? left : kPos;
                // what this row sees of it; whether its warp's rows all see it whole
                const int sees = pre ? valid : min(valid, k.pos0 + tl + 1 - p0);
                const bool full = (pre ? valid : min(valid, k.pos0 + tl_warp + 1 - p0)) == kPos;
                const bool diag = !pre && k.pos0 + 1 - p0 < valid;
                ok = wait(&s->s_full[slot], turn >> 2, a, s, 49);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                auto mask = [&](uint32_t *y, int n0) {
                    if (!full) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (n0 + e >= sees) y[e] = 0xFF800000u;
                    }
                };
                if (valid < kPos || diag) {
                    const uint32_t vi = (it + 1) % kStages;
                    ok = wait(&s->kv_full[vi], ((it + 1) / kStages) & 1, a, s, 50);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    clean_values<D>(s, reinterpret_cast<uint4 *>(sKV + vi * TILE), valid, diag ? t - ptiles - diag0 : -1);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (warp_real) {
                    tile_softmax<D>(sS, sO, a.scale_log2, m, l, t != w.t, s->p_full[slot], mask, []() { return true; });
                } else {
                    // a warp without rows only keeps step
                    mbar_arrive(&s->p_full[slot][0]);
                    mbar_arrive(&s->p_full[slot][1]);
                }
                turn ^= 4;
            }
            if (!ok) break;
            // the block's rows, or this piece's partial of them
            ok = wait(&s->o_full[slot], turn >> 1 & 1, a, s, 51);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            turn ^= 2;
            tc_fence_after();
            const int64_t part = (blockIdx.x * 2 + (w.t == 0)) * 2 + slot;
            const int pos = k.pos0 + tl;
            const bool sees = a.prefix_len || pos >= 0;  // a row that sees nothing is zeros
            const float inv = 1.0f / l;
            if (warp_real) {
                if (*reinterpret_cast<volatile int *>(&s->any_broken))
                    mend_rows<D>(a, s, sO, w.blk, w.kv, diag0 * kPos, real ? pos : -1);
#pragma unroll 1
                for (int d = 0; d < D; d += 32) {
                    uint32_t v[32];
                    tmem_ld32(sO + d, v);
                    tmem_wait32(v);
                    if (real && w.whole) {
                        __nv_bfloat16 *dst = a.out + static_cast<int64_t>(k.row0 + tl) * a.out_stride +
                                             static_cast<int64_t>(w.kv * group + r - token_of(r) * group) * D + d;
                        uint32_t o[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            o[e] = sees ? pack2_bf16(__uint_as_float(v[2 * e]) * inv, __uint_as_float(v[2 * e + 1]) * inv) : 0u;
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            *reinterpret_cast<uint4 *>(dst + 2 * e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    } else if (real) {
                        float *dst = a.part_o + part * (D * kRows) + r * 4;
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4 *>(dst + (d + e) / 4 * (kRows * 4)) = make_float4(
                                __uint_as_float(v[e]), __uint_as_float(v[e + 1]), __uint_as_float(v[e + 2]),
                                __uint_as_float(v[e + 3]));
                    }
                    __syncwarp();
                }
                if (!w.whole) a.part_ml[part * kRows + r] = make_float2(m, l);
            }
            tc_fence_before();
        } while (ok && w.next(a));
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// --------------------------------------------------------------- combine

// Joins the partials of the blocks that cuts run through: grid (cuts, sub-tiles,
// D / 32), the cut that is a block's first works for it.  Thread: row, half of the 32 dimensions.
template <int D>
__global__ void __launch_bounds__(256) prompt_combine_kernel(const __grid_constant__ PromptArgs a) {
    pdl_wait();
    pdl_trigger();
    const int64_t tiles = __ldcg(&a.plan->tiles), per = __ldcg(&a.plan->per);
    const int c = blockIdx.x + 1, sub = blockIdx.y;
    const int64_t f = c * per;
    if (f >= tiles * a.c.Hkv) return;
    const int kv = static_cast<int>(f / tiles), blk = __ldcg(a.piece_block + c);
    const int64_t first = __ldcg(a.start + blk) + kv * tiles, end = __ldcg(a.start + blk + 1) + kv * tiles;
    if (first == f || first < f - per) return;  // no block is cut here, or not for the first time
    const int n = static_cast<int>((end - 1) / per) - c + 2;  // pieces that it lies in
    const int4 b4 = __ldcg(reinterpret_cast<const int4 *>(a.blocks + blk));
    const PromptBlock k{b4.x, b4.y, b4.z, b4.w};
    const int r = threadIdx.x & 127, d0 = blockIdx.z * 8 + (threadIdx.x >> 7) * 4;  // dimensions in fours
    const int i = r / a.group, tl = sub * a.tq + i;
    if (i >= a.tq || tl >= k.ntok) return;
    float m = -INFINITY, l = 0.f;
    float4 acc[4] = {};
    for (int p = 0; p < n; ++p) {
        // the first piece's partial is of the block that ends later, the others' of the one that began before
        const int64_t part = ((c - 1 + p) * 2 + (p == 0)) * 2 + sub;
        const float2 t = __ldcg(a.part_ml + part * kRows + r);
        float4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = __ldcg(reinterpret_cast<const float4 *>(a.part_o + part * (D * kRows) + (d0 + j) * (kRows * 4) + r * 4));
        const float mn = fmaxf(m, t.x), c0 = exp2f(m - mn), c1 = exp2f(t.x - mn);
        m = mn;
        l = l * c0 + t.y * c1;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[j] = make_float4(acc[j].x * c0 + v[j].x * c1, acc[j].y * c0 + v[j].y * c1, acc[j].z * c0 + v[j].z * c1,
                                 acc[j].w * c0 + v[j].w * c1);
    }
    const float inv = 1.0f / l;  // (a block that sees nothing has one tile: no cut)
    const bool sees = a.prefix_len || k.pos0 + tl >= 0;
    uint4 o[2];
    uint32_t *w = reinterpret_cast<uint32_t *>(o);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        w[2 * j] = sees ? pack2_bf16(acc[j].x * inv, acc[j].y * inv) : 0u;
        w[2 * j + 1] = sees ? pack2_bf16(acc[j].z * inv, acc[j].w * inv) : 0u;
    }
    uint4 *dst = reinterpret_cast<uint4 *>(a.out + static_cast<int64_t>(k.row0 + tl) * a.out_stride +
                                           static_cast<int64_t>(kv * a.group + r - i * a.group) * D + d0 * 4);
    dst[0] = o[0];
    dst[1] = o[1];
}

// ------------------------------------------------------------------- host

struct PromptLayout {
    size_t plan, seq_blocks, start, blocks, piece_block, part_ml, part_o, total;
    int max_blocks;
};

static PromptLayout prompt_layout(int T, int n_seq, int group, int D, int sms) {
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    PromptLayout L{};
    L.max_blocks = T / (2 * (kRows / group)) + n_seq;
    const size_t blocks = L.max_blocks;
    L.plan = kCtrlBytes;
    L.seq_blocks = L.plan + up(sizeof(PromptPlan));
    L.start = L.seq_blocks + up((n_seq + 1) * sizeof(int));
    L.blocks = L.start + up((blocks + 1) * sizeof(int64_t));
    L.piece_block = L.blocks + up(blocks * sizeof(PromptBlock));
    L.part_ml = L.piece_block + up(sms * sizeof(int));
    L.part_o = L.part_ml + static_cast<size_t>(sms) * 4 * kRows * sizeof(float2);
    L.total = L.part_o + static_cast<size_t>(sms) * 4 * kRows * D * sizeof(float);
    return L;
}

size_t prompt_workspace_bytes(int T, int n_seq, int Hq, int Hkv, int D, int max_sms) {
    return prompt_layout(T, n_seq, Hq / Hkv, D, max_sms).total;
}

template <int D>
static cudaError_t launch_t(const PromptArgs &a, const CUtensorMap *maps, cudaStream_t s) {
    cudaError_t e = allow_smem<prompt_kernel<D>>();
    if (e != cudaSuccess) return e;
    if ((e = launch_dependent(prompt_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, a)) != cudaSuccess) return e;
    if ((e = launch_dependent(prompt_kernel<D>, dim3(a.ncta), dim3(kThreads), prompt_smem_bytes(D), s, maps[0], maps[1],
                              a)) != cudaSuccess)
        return e;
    return launch_dependent(prompt_combine_kernel<D>, dim3(a.ncta - 1, 2, D / 32), dim3(256), 0, s, a);
}

cudaError_t launch_prompt(PromptArgs &a, const CUtensorMap *maps, void *ws, int num_sms, cudaStream_t s) {
    char *w = static_cast<char *>(ws);
    const PromptLayout L = prompt_layout(a.T, a.n_seq, a.group, a.c.D, num_sms);
    a.tq = kRows / a.group;
    a.ncta = num_sms;
    a.max_blocks = L.max_blocks;
    a.negate = a.scale < 0.f;
    a.zero_q = a.scale == 0.f;
    a.scale_log2 = a.scale == 0.f ? 1.f : fabsf(a.scale) * 1.4426950408889634f;
    a.plan = reinterpret_cast<PromptPlan *>(w + L.plan);
    a.seq_blocks = reinterpret_cast<int *>(w + L.seq_blocks);
    a.start = reinterpret_cast<int64_t *>(w + L.start);
    a.blocks = reinterpret_cast<PromptBlock *>(w + L.blocks);
    a.piece_block = reinterpret_cast<int *>(w + L.piece_block);
    a.part_ml = reinterpret_cast<float2 *>(w + L.part_ml);
    a.part_o = reinterpret_cast<float *>(w + L.part_o);
    return a.c.D == 64 ? launch_t<64>(a, maps, s) : launch_t<128>(a, maps, s);
}

}  // namespace moe
