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
//            the sequence's own up to the block's last token.  All blocks and
//            key-value heads are one list, a block as long as its tiles and
//            kSwitch (what changing blocks costs), cut into even pieces, one per SM.
//            A block that lies within a piece has its rows of out written; of one
//            that a cut runs through every piece leaves a partial (m, l, O), and
//            prompt_combine_kernel joins them.  Lengths and starts are on the device
//            (a captured call is replayed with others): each piece adds up the
//            list's length from them and finds its beginning, in one warp (a kernel
//            before this one that laid the list out took 4 us of a short call, sums over
//            the whole block 1)
//   tile     as in attn_tile.cuh
//
//   warps 0-3, 4-7   softmax of slot 0, 1 (warp w: rows 32 (w % 4) ..)
//   warp 8           goes along the list and tells the others each block; loads:
//                    64-dimension boxes of page rows by TMA, 128-byte swizzle, keys and
//                    values in turn through one ring
//   warps 9, 10      MMA issue of slot 0, 1, in turn by a token to and fro
//
// Between two blocks the tensor core does not stop: a slot's queries of the next
// one are fetched by TMA when the last scores of this one are there, and its first
// scores follow this one's last second product, while the softmax threads write the
// rows.
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
//
// What bounds it.  D = 128: the tensor core.  16384 tokens of 16 heads on 2 in 885 to 971 us
// (by GPU) are 1130 to 1240 TFLOP/s, half as much again with the second parts of the
// weights.  D = 64: the softmax
// warps, busy 2700 of a tile's 3660 cycles (8192 tokens 215 us).  Two threads a row (16
// softmax warps of 96 registers) took 1127 us where this then took 980, the scores of
// each half of the next tile behind this one's values 988 (and 10 % more at D = 64);
// rows written by way of shared memory 1 % less, at D = 64 7 % more.  A call of a few
// tiles is a chain of first steps: 77 tokens 10.4 us, of which the plan 2.2, pages and
// keys 2, one tile's softmax 1.9, the rows 1.8.  Many short sequences cost a block each,
// and the plan one look at each length a piece: 32768 rows of 512 sequences 97 us, 65536
// of 4096 283, of 16384 1000, of 65536 3790 (a row each).
#include "attn_tile.cuh"
#include "prompt.cuh"

namespace moe {

constexpr int kStages = 4;               // key or value tiles in flight
constexpr int kThreads = 11 * 32;
constexpr int kDiag = 3;                 // tiles that a block's own tokens (at most 256) lie in
constexpr int kItems = 4;                // blocks that the loads may be ahead
// What changing blocks counts, in tiles: with 0, 1, 4 of them 4096 tokens take 115, 89
// and 79 us, with 2 76.
constexpr int kSwitch = 2;
constexpr int kAhead = 4;                // sequences whose lengths a lane fetches together

// A piece's part of a block: tiles t .. t + n - 1 (n = 0: no more).
struct Item {
    int row0, ntok, pos0;    // first row of q, tokens, own position of the first (negative: none)
    int kv, seq;
    int t, n;
    int whole;               // these are all its tiles
    uint32_t broken[kDiag][4];  // positions of the block's own tiles with values that are not finite
    int any_broken;
};

// ------------------------------------------------------------------ list

__device__ __forceinline__ int tiles_of(int positions) { return (positions + kPos - 1) / kPos; }

// sum_{i < n} floor((a i + b) / 128): the terms' own sum less their remainders'.  Those
// come back after 128 / g terms, g the largest power of two in a (128 at most), and are
// then b mod g and its steps of g, each once; what is left is at most 63 terms for an
// even a.
__device__ __forceinline__ int64_t floor_sum(int n, int a, int64_t b) {
    static_assert(kPos == 128, "the divisor");
    const int log_g = min(__ffs(a) - 1, 7), g = 1 << log_g, period = 128 >> log_g;
    const int once = period * static_cast<int>(b & (g - 1)) + g * (period * (period - 1) / 2);
    int some = 0, at = static_cast<int>(b & 127);
#pragma unroll 4
    for (int left = n & (period - 1); left > 0; --left, at += a) some += at & 127;
    const int64_t rest = static_cast<int64_t>(n >> (7 - log_g)) * once + some;
    return (static_cast<int64_t>(n) * (n - 1) / 2 * a + b * n - rest) >> 7;
}

// a / b for a >= 0, b > 0 (nearly always of 32 bits, whose division is far quicker).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// A sequence's rows; none for padding and for what is out of range.
struct Seq {
    int row0, n, pos0;

    __device__ __forceinline__ Seq() : row0(0), n(0), pos0(0) {}
    __device__ __forceinline__ Seq(const PromptArgs &a, int b)
        : Seq(a, __ldcg(a.q_start + b), __ldcg(a.q_start + b + 1), __ldcg(a.seq_len + b)) {}
    __device__ __forceinline__ Seq(const PromptArgs &a, int r0, int r1, int len) : row0(0), n(0), pos0(0) {
        if (r0 < 0 || r1 < r0 || r1 > a.T || len > static_cast<int64_t>(a.table_ld) << a.c.page_shift) {
            record_status(a.status, MOE_ERR_PAGE);
        } else if (len >= 0) {
            row0 = r0;
            n = r1 - r0;
            pos0 = len - n;
        }
    }
    __device__ __forceinline__ int blocks(int span) const { return (n + span - 1) / span; }
    // Tiles of block j: a block that sees nothing has one too, since its rows are written.
    __device__ __forceinline__ int tiles(const PromptArgs &a, int j) const {
        const int span = 2 * a.tq, end = pos0 + min((j + 1) * span, n);
        return max(tiles_of(a.prefix_len) + (end > 0 ? tiles_of(end) : 0), 1);
    }
    // Length of the first j blocks in the list.
    __device__ __forceinline__ int64_t length(const PromptArgs &a, int j) const {
        const int span = 2 * a.tq, nb = blocks(span), prefix = tiles_of(a.prefix_len);
        int64_t sum = 0;
        if (j == nb && nb > 0) sum = kSwitch + tiles(a, --j);
        if (j == 0) return sum;
        const int none = pos0 >= 0 ? 0 : min(j, -pos0 / span);  // blocks before the first position
        return sum + static_cast<int64_t>(j) * (kSwitch + prefix) + (prefix ? 0 : none) +
               floor_sum(j - none, span, pos0 + (none + 1) * static_cast<int64_t>(span) + kPos - 1);
    }
};

struct PromptCtl {
    uint64_t kv_full[kStages], kv_empty[kStages];
    uint64_t item_full[kItems], item_empty[kItems];
    uint64_t q_full[2], q_empty[2];  // the slot's queries of the block
    uint64_t s_full[2];      // scores of the slot's tile are in tensor memory
    uint64_t p_full[2][2];   // weights of its positions 0-63, 64-127 are (and O is ready to be added to)
    uint64_t o_full[2];      // O of the block of rows is complete
    uint64_t token[2];       // the slot's issuer may go on
    uint64_t drain;
    Item items[kItems];
    uint32_t tmem;
    int abort;
};

__host__ __device__ constexpr int prompt_smem_bytes(int D) {
    return 2 * kRows * D * 2 + kStages * tile_bytes(D) + 1024 + static_cast<int>(sizeof(PromptCtl));
}
static_assert(prompt_smem_bytes(128) <= kBlockSmem, "one block per SM");

// A warp's way along the list, all lanes alike.
struct Walk {
    int64_t per;             // length of a piece
    int64_t left;            // of the piece from here on
    int kv, seq, blk, nb;
    int t, n, of;            // first tile of the block here, tiles of it here, of it at all
    int row0, ntok, pos0;

    // The part of block blk of its sequence, of which the piece has what lies from
    // `at` (negative: before its tiles) on.
    __device__ __forceinline__ void block(const PromptArgs &a, const Seq &q, int64_t at) {
        const int span = 2 * a.tq;
        nb = q.blocks(span);
        row0 = q.row0 + blk * span;
        ntok = min(q.n - blk * span, span);
        pos0 = q.pos0 + blk * span;
        of = q.tiles(a, blk);
        t = at > kSwitch ? static_cast<int>(at - kSwitch) : 0;
        left -= at < kSwitch ? kSwitch - at : 0;
        n = static_cast<int>(min(static_cast<int64_t>(of - t), left));
    }
    // False: nothing (more) for this piece.  Every piece adds up the list for itself,
    // one lane a run of sequences.
    __device__ __forceinline__ bool first(const PromptArgs &a) {
        const int lane = threadIdx.x & 31, span = 2 * a.tq;
        const int run = (a.n_seq + 31) / 32;
        int64_t own = 0, rows = 0;
        Seq q;
        for (int i = 0; i < run; i += kAhead) {
            int r[kAhead + 1], len[kAhead];
#pragma unroll
            for (int e = 0; e <= kAhead; ++e) {
                const int b = lane * run + min(i + e, run);
                r[e] = __ldcg(a.q_start + min(b, a.n_seq));
                if (e < kAhead) len[e] = __ldcg(a.seq_len + min(b, a.n_seq - 1));
            }
#pragma unroll
            for (int e = 0; e < kAhead; ++e) {
                if (i + e >= run) break;
                q = lane * run + i + e < a.n_seq ? Seq(a, r[e], r[e + 1], len[e]) : Seq();
                own += q.length(a, q.blocks(span));
                rows += q.n;
            }
        }
        int64_t upto = own;
#pragma unroll
        for (int i = 1; i < 32; i <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, upto, i);
            if (lane >= i) upto += o;
            rows += __shfl_xor_sync(0xffffffffu, rows, i);
        }
        int64_t each = __shfl_sync(0xffffffffu, upto, 31);  // length of one key-value head's list
        // (starts that go back may give more rows than there are: none is worked on then)
        if (rows > a.T) {
            record_status(a.status, MOE_ERR_PAGE);
            each = 0;
        }
        per = quotient(each * a.c.Hkv + a.ncta - 1, a.ncta);
        left = min(each * a.c.Hkv - blockIdx.x * per, per);
        if (left <= 0) return false;
        kv = static_cast<int>(quotient(blockIdx.x * per, each));
        int64_t at = blockIdx.x * per - kv * each;
        // the sequence: the lane's run, then in it
        const int l = __ffs(__ballot_sync(0xffffffffu, at < upto)) - 1;
        at -= __shfl_sync(0xffffffffu, upto - own, l);
        seq = l * run;
        int k = l;
        if (run > 1) {
            for (;; seq += 32) {
                if (seq >= a.n_seq) return false;  // (the lengths have changed meanwhile)
                q = lane < run && seq + lane < a.n_seq ? Seq(a, seq + lane) : Seq();
                own = upto = q.length(a, q.blocks(span));
#pragma unroll
                for (int i = 1; i < 32; i <<= 1) {
                    const int64_t o = __shfl_up_sync(0xffffffffu, upto, i);
                    if (lane >= i) upto += o;
                }
                const unsigned m = __ballot_sync(0xffffffffu, at < upto);
                if (m) {
                    k = __ffs(m) - 1;
                    at -= __shfl_sync(0xffffffffu, upto - own, k);
                    seq += k;
                    break;
                }
                at -= __shfl_sync(0xffffffffu, upto, 31);
            }
        }
        q.row0 = __shfl_sync(0xffffffffu, q.row0, k);
        q.n = __shfl_sync(0xffffffffu, q.n, k);
        q.pos0 = __shfl_sync(0xffffffffu, q.pos0, k);
        // its last block that begins at `at` or before, by 32 looks at a time
        int lo = 0, hi = q.blocks(span);
        int64_t begin = 0;
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32, j = lo + lane * step;
            const int64_t b = q.length(a, min(j, hi - 1));
            const int last = 31 - __clz(__ballot_sync(0xffffffffu, j < hi && b <= at));
            begin = __shfl_sync(0xffffffffu, b, last);
            lo += last * step;
            hi = min(hi, lo + step);
        }
        blk = lo;
        block(a, q, at - begin);
        return n > 0 || next(a);
    }
    __device__ __forceinline__ bool next(const PromptArgs &a) {
        left -= n;
        if (left <= 0) return false;
        if (++blk == nb) {
            // the next sequence with rows, of this key-value head or the next
            const int lane = threadIdx.x & 31;
            blk = 0;
            for (int b = seq + 1;; b += 32) {
                if (b >= a.n_seq) {
                    b = 0;
                    if (++kv >= a.c.Hkv) return false;
                }
                const bool has = b + lane < a.n_seq && Seq(a, b + lane).n > 0;
                const unsigned m = __ballot_sync(0xffffffffu, has);
                if (m) {
                    seq = b + __ffs(m) - 1;
                    break;
                }
            }
        }
        block(a, Seq(a, seq), 0);
        return n > 0;
    }
};

// ------------------------------------------------------------------ main

__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, const PromptArgs &a, PromptCtl *s, int site) {
    return role_wait(bar, parity, a.wait_limit, a.status, &s->abort, site);
}

__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const PromptArgs &a, PromptCtl *s, int site) {
    return __all_sync(0xffffffffu, wait(bar, parity, a, s, site));
}

// Makes the value rows of a tile safe to be met by weights of zero, by a slot's 128
// threads: those from `valid` on may hold anything and become zeros, and in the
// block's own tile number `own` (-1: another) what is not finite does and is noted.
// (Not inlined: a tile's softmax takes all registers.)
template <int D>
__device__ __noinline__ void clean_values(Item *item, uint4 *v, int valid, int own) {
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
                atomicOr(&item->broken[own][i >> 8], 1u << (i >> 3 & 31));
                *reinterpret_cast<volatile int *>(&item->any_broken) = 1;
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
__device__ __noinline__ void mend_rows(const PromptArgs &a, const Item *item, uint32_t sO, int first, int pos) {
    const int *table = a.table + static_cast<int64_t>(item->seq) * a.table_ld;
    for (int d = 0; d < D; d += 16) {
        uint32_t o[16];
        tmem_ld16_now(sO + d, o);
        for (int j = 0; j < kDiag * kPos; ++j) {
            const int p = first + j;
            if (p > pos || !(item->broken[j >> 7][(j >> 5) & 3] >> (j & 31) & 1)) continue;
            const int page = table[p >> a.c.page_shift];
            if (page < 0 || page >= a.c.n_pages) continue;
            const __nv_bfloat16 *x = a.c.v + page * a.c.page_stride + item->kv * a.c.head_stride +
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

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PromptArgs a) {
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
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&s->item_full[i], 1);
            mbar_init(&s->item_empty[i], 256 + 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s->q_full[i], 1);
            mbar_init(&s->q_empty[i], 1);
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
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }
    if (warp == 9) {
        tmem_alloc(&s->tmem, kTmemCols);
        tmem_relinquish();
    }
    pdl_wait();
    pdl_trigger();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s->tmem;
    const int ptiles = tiles_of(a.prefix_len);

    if (warp == 8) {
        // ------------------------------------------------------------ loads
        const int ps = a.c.page_shift;
        const int box_rows = ps >= 7 ? kPos : 1 << ps;
        // lane j: half j % HALVES of box j / HALVES (at most 8 boxes of 2 halves)
        const int bx = lane / HALVES, half = lane % HALVES;
        uint32_t it = 0, ni = 0, nq[2] = {0, 0};  // ring entries, blocks, a slot's blocks
        Walk w;
        bool more = w.first(a), ok = true;
        // the block that the piece begins in, which may be cut there
        const bool cut = more && w.t > 0 && w.t <= w.per;
        const PromptCut here{0, w.kv, w.row0, w.ntok, w.pos0};
        const int64_t to_end = w.of - w.t;
        for (;; ++ni) {
            Item *k = s->items + ni % kItems;
            ok = warp_wait(&s->item_empty[ni % kItems], (ni / kItems & 1) ^ 1, a, s, 40);
            if (!ok) break;
            if (lane < kDiag * 4) (&k->broken[0][0])[lane] = 0;
            if (lane == 0) {
                k->row0 = w.row0;
                k->ntok = w.ntok;
                k->pos0 = w.pos0;
                k->kv = w.kv;
                k->seq = w.seq;
                k->t = w.t;
                k->n = more ? w.n : 0;
                k->whole = w.n == w.of;
                k->any_broken = 0;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&s->item_full[ni % kItems]);
            if (!more) break;
            for (int t = w.t; t < w.t + w.n && ok; ++t) {
                const bool pre = t < ptiles;
                const int p0 = (pre ? t : t - ptiles) * kPos;
                const int left = (pre ? a.prefix_len : w.pos0 + w.ntok) - p0;
                const int boxes = left <= 0 ? 0 : ((left < kPos ? left : kPos) + box_rows - 1) / box_rows;
                TileBox at{0, 0};
                if (bx < boxes)
                    at = tile_box(a.c, pre ? a.prefix_pages : a.table + static_cast<int64_t>(w.seq) * a.table_ld,
                                  p0 + bx * box_rows, a.status);
                for (int m = 0; m < 2 && ok; ++m, ++it) {  // keys, then values
                    const int st = it % kStages;
                    ok = warp_wait(&s->kv_empty[st], ((it / kStages) & 1) ^ 1, a, s, 41);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&s->kv_full[st], boxes * box_rows * D * 2);
                    __syncwarp();
                    if (bx < boxes)
                        tma_load_4d(smem_u32(sKV + st * TILE + half * HALF + bx * box_rows * 128), m ? &tm_v : &tm_k,
                                    &s->kv_full[st], half * 64, at.row, w.kv, at.page);
                    // with a block's first keys its queries: a slot's tokens with the heads
                    // of this key-value head (tokens past the block's last are rows that
                    // nobody reads)
                    if (t > w.t || m) continue;
                    for (int slot = 0; slot < 2 && ok; ++slot) {
                        if (slot * a.tq >= w.ntok) continue;
                        ok = warp_wait(&s->q_empty[slot], (nq[slot] & 1) ^ 1, a, s, 54);
                        if (!ok) break;
                        ++nq[slot];
                        if (lane == 0) {
                            mbar_arrive_expect_tx(&s->q_full[slot], a.tq * a.group * D * 2);
                            for (int h = 0; h < HALVES; ++h)
                                tma_load_3d(smem_u32(sQ + slot * QSUB + h * HALF), &tm_q, &s->q_full[slot], h * 64,
                                            w.kv * a.group, w.row0 + slot * a.tq);
                        }
                    }
                }
            }
            if (!ok) break;
            more = w.next(a);
        }
        // what there is to join at the piece's beginning: of a block that the piece
        // before begins, all its pieces
        if (lane == 0 && blockIdx.x) {
            PromptCut c{};
            if (cut) {
                c = here;
                c.pieces = static_cast<int>(quotient(blockIdx.x * w.per + to_end - 1, w.per)) -
                           static_cast<int>(blockIdx.x) + 2;
            }
            a.cuts[blockIdx.x] = c;
        }
        // no copy of this block is in flight when it ends
        for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i)
            mbar_drain(&s->kv_full[i % kStages], (i / kStages) & 1, a.wait_limit);
        for (int slot = 0; slot < 2; ++slot)
            if (nq[slot]) mbar_drain(&s->q_full[slot], (nq[slot] - 1) & 1, a.wait_limit);
    } else if (warp >= 9) {
        // -------------------------------------------------------- MMA issue
        if (elect_one()) {
            const int slot = __shfl_sync(__activemask(), warp, 0) - 9;
            const uint32_t sS = tmem + slot * 128, sO = tmem + 256 + slot * D;
            const uint32_t q_addr = smem_u32(sQ + slot * QSUB), kv_addr = smem_u32(sKV);
            uint32_t it0 = 0, nq = 0;              // ring entry of the block's first tile, this slot's blocks
            uint32_t done = 0, tok = 0;            // this slot's tiles so far, tokens taken
            bool ok = true;
            for (uint32_t ni = 0;; ++ni) {
                ok = wait(&s->item_full[ni % kItems], ni / kItems & 1, a, s, 42);
                if (!ok) break;
                const volatile Item *k = s->items + ni % kItems;
                const int nt = k->n;
                // a tile for both slots in turn (step n: tile n / 2, slot n % 2), or all for
                // slot 0 where slot 1 has no tokens
                const bool both = k->ntok > a.tq;
                mbar_arrive(&s->item_empty[ni % kItems]);
                if (!nt) break;
                const int steps = both ? 2 * nt : nt, next = both ? 2 : 1;
                auto scores = [&](int n) {
                    const uint32_t e = it0 + 2 * (both ? n >> 1 : n), st = e % kStages;
                    // S overwrites the slot's previous weights: their product was
                    // issued before, by this thread, and the tensor core takes
                    // MMAs in the order of issue
                    ok = wait(&s->kv_full[st], (e / kStages) & 1, a, s, 43);
                    if (!ok) return;
                    tc_fence_after();
                    tile_scores<D>(sS, q_addr, kv_addr + st * TILE, a.negate ? kANegated : 0);
                };
                // (s_full also says that the previous tile's second product is complete)
                auto scores_end = [&](int n) {
                    umma_commit(&s->s_full[slot]);
                    umma_commit(&s->kv_empty[(it0 + 2 * (both ? n >> 1 : n)) % kStages]);
                    if (n + next >= steps) umma_commit(&s->q_empty[slot]);
                };
                if (!both && slot == 1) {
                    // no rows here: give the tiles back
                    for (uint32_t e = it0; e < it0 + 2 * nt && ok; ++e) {
                        ok = wait(&s->kv_full[e % kStages], (e / kStages) & 1, a, s, 44);
                        if (ok) mbar_arrive(&s->kv_empty[e % kStages]);
                    }
                } else {
                    ok = wait(&s->q_full[slot], nq++ & 1, a, s, 45);
                    if (ok) scores(slot);
                    if (ok) scores_end(slot);
                    for (int n = slot; n < steps && ok; n += next, ++done) {
                        const uint32_t e = it0 + 2 * (both ? n >> 1 : n) + 1, st = e % kStages;
                        const uint32_t v_addr = kv_addr + st * TILE;
                        ok = wait(&s->kv_full[st], (e / kStages) & 1, a, s, 46);
                        if (n > 0 && both) ok = ok && wait(&s->token[slot], tok++ & 1, a, s, 47);
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            ok = ok && wait(&s->p_full[slot][half], done & 1, a, s, 48);
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
                if (!ok) break;
                it0 += 2 * nt;
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
        const int group = a.group, tq = a.tq;
        // (rows / group by a 16-bit reciprocal: exact for rows below 8192, group <= 8)
        const uint32_t recip = (65536 + group - 1) / group;
        auto token_of = [&](int row) { return static_cast<int>((row * recip) >> 16); };
        const int tl = slot * tq + token_of(r);          // this row's token in the block
        uint32_t it = 0, turn = 0;                       // ring entry; parities: this slot's blocks (1), its tiles (2)
        bool ok = true;
        for (uint32_t ni = 0;; ++ni) {
            ok = warp_wait(&s->item_full[ni % kItems], ni / kItems & 1, a, s, 49);
            if (!ok) break;
            // (read again where it is used: a tile's softmax takes all registers)
            volatile Item *item = s->items + ni % kItems;
            if (!item->n) break;
            const bool active = slot * tq < item->ntok;
            const bool warp_real = slot * tq + token_of((warp & 3) * 32) < item->ntok && token_of((warp & 3) * 32) < tq;
            float m = -INFINITY, l = 0.f;
            if (!active) it += 2 * item->n;
            for (int t = item->t; active && t < item->t + item->n; ++t, it += 2) {
                const int pos0 = item->pos0, ntok = item->ntok;
                const bool pre = t < ptiles;
                const int p0 = (pre ? t : t - ptiles) * kPos;
                const int left = (pre ? a.prefix_len : pos0 + ntok) - p0;  // positions of the tile
                const int valid = left < 0 ? 0 : left < kPos ? left : kPos;
                // what this row sees of it; whether its warp's rows all see it whole
                const int sees = pre ? valid : min(valid, pos0 + tl + 1 - p0);
                const bool full = __all_sync(0xffffffffu, sees == kPos);
                const bool diag = !pre && pos0 + 1 - p0 < valid;  // not all of the block's tokens see it whole
                auto mask = [&](uint32_t *y, int n0) {
                    if (!full) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (n0 + e >= sees) y[e] = 0xFF800000u;
                    }
                };
                if (valid < kPos || diag) {
                    const uint32_t vi = (it + 1) % kStages;
                    ok = warp_wait(&s->kv_full[vi], ((it + 1) / kStages) & 1, a, s, 52);
                    if (!ok) break;
                    clean_values<D>(s->items + ni % kItems, reinterpret_cast<uint4 *>(sKV + vi * TILE), valid,
                                    diag ? t - ptiles - max(pos0, 0) / kPos : -1);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                ok = warp_wait(&s->s_full[slot], turn >> 1 & 1, a, s, 50);
                if (!ok) break;
                tc_fence_after();
                if (warp_real) {
                    tile_softmax<D>(sS, sO, a.scale_log2, m, l, m != -INFINITY, s->p_full[slot], mask, []() { return true; });
                } else {
                    // a warp without rows only keeps step
                    mbar_arrive(&s->p_full[slot][0]);
                    mbar_arrive(&s->p_full[slot][1]);
                }
                turn ^= 2;
            }
            if (!ok) break;
            if (active) {
                // the block's rows, or this piece's partial of them
                ok = warp_wait(&s->o_full[slot], turn & 1, a, s, 53);
                if (!ok) break;
                turn ^= 1;
                tc_fence_after();
                const int pos0 = item->pos0;
                const bool real = token_of(r) < tq && tl < item->ntok, whole = item->whole;
                const int64_t part = (blockIdx.x * 2 + (item->t == 0)) * 2 + slot;
                const bool sees = a.prefix_len || pos0 + tl >= 0;  // a row that sees nothing is zeros
                const float inv = 1.0f / l;
                if (warp_real) {
                    if (item->any_broken)
                        mend_rows<D>(a, s->items + ni % kItems, sO, max(pos0, 0) / kPos * kPos, real ? pos0 + tl : -1);
                    __nv_bfloat16 *row = a.out + static_cast<int64_t>(item->row0 + tl) * a.out_stride +
                                         static_cast<int64_t>(item->kv * group + r - token_of(r) * group) * D;
#pragma unroll 1
                    for (int d = 0; d < D; d += 32) {
                        uint32_t v[32];
                        tmem_ld32(sO + d, v);
                        tmem_wait32(v);
                        if (real && whole) {
                            uint32_t o[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = sees ? pack2_bf16(__uint_as_float(v[2 * e]) * inv, __uint_as_float(v[2 * e + 1]) * inv) : 0u;
#pragma unroll
                            for (int e = 0; e < 16; e += 4)
                                *reinterpret_cast<uint4 *>(row + d + 2 * e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
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
                    if (!whole) a.part_ml[part * kRows + r] = make_float2(m, l);
                }
                tc_fence_before();
            }
            mbar_arrive(&s->item_empty[ni % kItems]);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// --------------------------------------------------------------- combine

// Joins the partials of the blocks that cuts run through: grid (cuts, sub-tiles, D / 32).
// Thread: row, half of the 32 dimensions.
template <int D>
__global__ void __launch_bounds__(256) prompt_combine_kernel(const __grid_constant__ PromptArgs a) {
    pdl_wait();
    pdl_trigger();
    const int c = blockIdx.x + 1, sub = blockIdx.y;
    const int4 k = __ldcg(reinterpret_cast<const int4 *>(a.cuts + c));  // pieces, kv, row0, ntok
    const int r = threadIdx.x & 127, d0 = blockIdx.z * 8 + (threadIdx.x >> 7) * 4;  // dimensions in fours
    const int i = r / a.group, tl = sub * a.tq + i;
    if (!k.x || i >= a.tq || tl >= k.w) return;
    float m = -INFINITY, l = 0.f;
    float4 acc[4] = {};
    for (int p = 0; p < k.x; ++p) {
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
    const bool sees = a.prefix_len || __ldcg(&a.cuts[c].pos0) + tl >= 0;
    const float inv = 1.0f / l;
    uint4 o[2];
    uint32_t *w = reinterpret_cast<uint32_t *>(o);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        w[2 * j] = sees ? pack2_bf16(acc[j].x * inv, acc[j].y * inv) : 0u;
        w[2 * j + 1] = sees ? pack2_bf16(acc[j].z * inv, acc[j].w * inv) : 0u;
    }
    uint4 *dst = reinterpret_cast<uint4 *>(a.out + static_cast<int64_t>(k.z + tl) * a.out_stride +
                                           static_cast<int64_t>(k.y * a.group + r - i * a.group) * D + d0 * 4);
    dst[0] = o[0];
    dst[1] = o[1];
}

// ------------------------------------------------------------------- host

struct PromptLayout {
    size_t cuts, part_ml, part_o, total;
};

static PromptLayout prompt_layout(int D, int sms) {
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    PromptLayout L{};
    L.cuts = kCtrlBytes;
    L.part_ml = L.cuts + up(sms * sizeof(PromptCut));
    L.part_o = L.part_ml + static_cast<size_t>(sms) * 4 * kRows * sizeof(float2);
    L.total = L.part_o + static_cast<size_t>(sms) * 4 * kRows * D * sizeof(float);
    return L;
}

size_t prompt_workspace_bytes(int D, int max_sms) { return prompt_layout(D, max_sms).total; }

template <int D>
static cudaError_t launch_t(const PromptArgs &a, const CUtensorMap *maps, cudaStream_t s) {
    cudaError_t e = allow_smem<prompt_kernel<D>>();
    if (e != cudaSuccess) return e;
    if ((e = launch_dependent(prompt_kernel<D>, dim3(a.ncta), dim3(kThreads), prompt_smem_bytes(D), s, maps[0], maps[1],
                              maps[2], a)) != cudaSuccess)
        return e;
    // (blocks of one tile are never cut)
    const int64_t longest = static_cast<int64_t>(a.table_ld) << a.c.page_shift;
    if (!a.prefix_len && longest <= kPos) return cudaSuccess;
    return launch_dependent(prompt_combine_kernel<D>, dim3(a.ncta - 1, 2, D / 32), dim3(256), 0, s, a);
}

cudaError_t launch_prompt(PromptArgs &a, const CUtensorMap *maps, void *ws, int num_sms, cudaStream_t s) {
    char *w = static_cast<char *>(ws);
    const PromptLayout L = prompt_layout(a.c.D, num_sms);
    a.tq = prompt_tokens(a.group);
    a.ncta = num_sms;
    a.negate = a.scale < 0.f;
    // (zero: the least factor instead, with which a masked score stays minus infinity)
    a.scale_log2 = a.scale == 0.f ? 0x1p-126f : fabsf(a.scale) * 1.4426950408889634f;
    a.cuts = reinterpret_cast<PromptCut *>(w + L.cuts);
    a.part_ml = reinterpret_cast<float2 *>(w + L.part_ml);
    a.part_o = reinterpret_cast<float *>(w + L.part_o);
    return a.c.D == 64 ? launch_t<64>(a, maps, s) : launch_t<128>(a, maps, s);
}

}  // namespace moe
