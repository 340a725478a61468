// Appending to a paged key-value cache and attending over it.
#include <type_traits>

#include "paged.cuh"

namespace moe {

// The rotation angle pos * f as the cosine and sine of its fraction of a turn.
// f / 2 pi, less whole turns, is kept as a 64-bit fraction, so that its product
// with a position loses whole turns by itself.  The fraction is made from f's 24
// bits times 128 bits of 1 / 2 pi in integers and is off by less than 2^-62 for any
// f below 2^63, so that the angle is off by 2^-30 of a turn at position 2^32, less than
// its own rounding to fp32.  (A product in fp64 loses what stands before the
// point: with f = 100 it was off by 2^-20 of a turn at position 2^30.)
__device__ __forceinline__ uint64_t turn_fraction(float f) {
    constexpr uint32_t kInv2Pi[4] = {0x7D4D3770u, 0x7F09D5F4u, 0x9391054Au, 0x28BE60DBu};  // 2^128 / 2 pi, from the lowest
    const uint32_t u = __float_as_uint(f), biased = u >> 23 & 255u;
    const uint32_t m = (u & 0x7FFFFFu) | (biased ? 0x800000u : 0u);  // f = m 2^(e - 150)
    const int e = biased ? biased : 1;
    uint32_t w[5];
    uint64_t carry = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        carry += static_cast<uint64_t>(m) * kInv2Pi[i];
        w[i] = static_cast<uint32_t>(carry);
        carry >>= 32;
    }
    w[4] = static_cast<uint32_t>(carry);
    // the 64 bits below the point: the product shifted down by 128 + 150 - 64 - e
    const int s = max(214 - e, 0), at = s >> 5;
    uint32_t lo = 0, mid = 0, hi = 0;
#pragma unroll
    for (int i = 0; i < 5; ++i) {
        lo = i == at ? w[i] : lo;
        mid = i == at + 1 ? w[i] : mid;
        hi = i == at + 2 ? w[i] : hi;
    }
    const uint64_t frac = static_cast<uint64_t>(__funnelshift_r(mid, hi, s)) << 32 | __funnelshift_r(lo, mid, s);
    return u >> 31 ? 0 - frac : frac;
}
__device__ __forceinline__ float2 angle_cs(uint32_t pos, uint64_t f) {
    const uint32_t frac = __umulhi(static_cast<uint32_t>(f), pos) + static_cast<uint32_t>(f >> 32) * pos;
    float2 r;
    sincospif(static_cast<float>(static_cast<int32_t>(frac)) * 0x1p-31f, &r.y, &r.x);
    return r;
}

// A block takes a few tokens (one when there are few, so that every SM has a
// share, up to eight).  First the tokens' places and their angles' cosines and
// sines into shared memory, one per thread and pair, shared by all heads (the
// frequencies' fractions of a turn once per pair and block); then 16-byte pieces: of a
// rotated head the pair of pieces whose elements turn into one another (halves:
// pieces j and j + rot / 16 of the head; interleaved: a piece by itself),
// otherwise plain copies.  Bound by the bytes, each read and written once, and at
// few tokens by the three dependent reads (index, page, piece): a call with 8192
// tokens of 16 + 2 x 2 heads of 128 takes 18.3 us (84 MB, 4.6 TB/s), one with 8
// tokens 2.9, its host side included.
constexpr int kAppendThreads = 256;
constexpr int kAppendTokens = 8;

// cs: (cos, sin) of two pairs of elements in each
__device__ __forceinline__ uint4 turn_piece(const uint4 &x, const float4 &cs0, const float4 &cs1) {
    // interleaved: (x0, x1) by the first, ...
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    const float c[4] = {cs0.x, cs0.z, cs1.x, cs1.z}, s[4] = {cs0.y, cs0.w, cs1.y, cs1.w};
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float a = __uint_as_float(w[j] << 16), b = __uint_as_float(w[j] & 0xFFFF0000u);
        r[j] = bf162_as_u32(__floats2bfloat162_rn(a * c[j] - b * s[j], b * c[j] + a * s[j]));
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

__device__ __forceinline__ void turn_halves(uint4 &x, uint4 &y, const float4 *cs, int step) {
    uint32_t *wx = reinterpret_cast<uint32_t *>(&x), *wy = reinterpret_cast<uint32_t *>(&y);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float4 c = cs[j * step];
        const float a0 = __uint_as_float(wx[j] << 16), a1 = __uint_as_float(wx[j] & 0xFFFF0000u);
        const float b0 = __uint_as_float(wy[j] << 16), b1 = __uint_as_float(wy[j] & 0xFFFF0000u);
        wx[j] = bf162_as_u32(__floats2bfloat162_rn(a0 * c.x - b0 * c.y, a1 * c.z - b1 * c.w));
        wy[j] = bf162_as_u32(__floats2bfloat162_rn(b0 * c.x + a0 * c.y, b1 * c.z + a1 * c.w));
    }
}

// ITEMS: a thread's work items in flight together
template <int D, int ITEMS>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendArgs a, int per_block) {
    constexpr int P = D / 8;  // 16-byte pieces of a head
    // (cos, sin) of the pairs, those of 16 p, 16 p + 2, .. (two each) side by side for
    // all p: threads with neighbouring pieces read neighbouring places
    __shared__ float4 s_cs[kAppendTokens][D / 4];
    __shared__ int64_t s_slot[kAppendTokens];  // the token's place in the pools, -1: none
    __shared__ uint64_t s_turn[D / 2];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x;
    const int t0 = blockIdx.x * per_block, nt = min(per_block, a.T - t0);
    const int ps = a.c.page_shift, half = a.rot / 2;
    if (tid < nt) {
        const int seq = a.seq[t0 + tid], idx = a.index[t0 + tid];
        int64_t slot = -1;
        if (seq >= 0 && idx >= 0) {  // else padding
            const bool in_table = seq < a.n_seq && (idx >> ps) < a.table_ld;
            const int page = in_table ? a.table[static_cast<int64_t>(seq) * a.table_ld + (idx >> ps)] : -1;
            if (page >= 0 && page < a.c.n_pages)
                slot = page * a.c.page_stride + (idx & ((1 << ps) - 1)) * a.c.pos_stride;
            else
                record_status(a.status, MOE_ERR_PAGE);
        }
        s_slot[tid] = slot;
    }
    if (tid >= kAppendThreads - half) s_turn[tid - (kAppendThreads - half)] = turn_fraction(a.inv_freq[tid - (kAppendThreads - half)]);
    __syncthreads();
    for (int i = tid; i < nt * half; i += kAppendThreads) {
        const int t = i / half, p = i - t * half;
        reinterpret_cast<float2 *>(s_cs[t])[(p % 8 / 2 * (D / 16) + p / 8) * 2 + p % 2] = angle_cs(static_cast<uint32_t>(a.index[t0 + t]) + static_cast<uint32_t>(a.pos_offset), s_turn[p]);
    }
    __syncthreads();

    // work items of a token: rotated heads (halves) HP = P / 2 pairs of pieces,
    // else P pieces; queries, keys, then values (P plain pieces each, in pairs)
    const int Hq = a.q ? a.Hq : 0, Hkv = a.c.Hkv;
    constexpr int HP = P / 2;
    const int per_token = (Hq + 2 * Hkv) * HP;
    const int rp = a.rot / 16;  // pieces of a rotated half
    for (int i0 = tid; i0 < nt * per_token; i0 += ITEMS * kAppendThreads) {
        uint4 x[ITEMS], y[ITEMS];
        __nv_bfloat16 *dst[ITEMS];
        int tt[ITEMS], pp[ITEMS], p0[ITEMS], p1[ITEMS];
        bool rotated[ITEMS];
#pragma unroll
        for (int e = 0; e < ITEMS; ++e) {
            const int i = i0 + e * kAppendThreads, t = i / per_token, r = i - t * per_token, h = r / HP, p = r % HP;
            dst[e] = nullptr;
            if (i >= nt * per_token) continue;
            const int64_t slot = s_slot[t];
            if (slot < 0) continue;
            const __nv_bfloat16 *src;
            if (h < Hq) {
                src = a.q + (t0 + t) * a.q_stride + h * D;
                dst[e] = a.q_out + (t0 + t) * a.qo_stride + h * D;
            } else if (h < Hq + Hkv) {
                src = a.k + (t0 + t) * a.k_stride + (h - Hq) * D;
                dst[e] = a.c.k + slot + (h - Hq) * a.c.head_stride;
            } else {
                src = a.v + (t0 + t) * a.v_stride + (h - Hq - Hkv) * D;
                dst[e] = a.c.v + slot + (h - Hq - Hkv) * a.c.head_stride;
            }
            // two pieces a thread: the pair of a rotation by halves, or neighbours
            // (not rotated are 2 rp, 2 rp + 1 and on: 2 p, 2 p + 1 from p = rp on)
            rotated[e] = h < Hq + Hkv;
            const bool paired = rotated[e] && !a.interleaved && p < rp;
            tt[e] = t;
            pp[e] = p;
            p0[e] = paired ? p : 2 * p;
            p1[e] = paired ? p + rp : 2 * p + 1;
            x[e] = *reinterpret_cast<const uint4 *>(src + p0[e] * 8);
            y[e] = *reinterpret_cast<const uint4 *>(src + p1[e] * 8);
        }
#pragma unroll
        for (int e = 0; e < ITEMS; ++e) {
            if (!dst[e]) continue;
            const float4 *cs = s_cs[tt[e]] + pp[e];
            if (rotated[e]) {
                if (!a.interleaved) {
                    if (pp[e] < rp) turn_halves(x[e], y[e], cs, HP);
                } else {
                    if (p0[e] * 8 < a.rot) x[e] = turn_piece(x[e], cs[0], cs[HP]);
                    if (p1[e] * 8 < a.rot) y[e] = turn_piece(y[e], cs[2 * HP], cs[3 * HP]);
                }
            }
            *reinterpret_cast<uint4 *>(dst[e] + p0[e] * 8) = x[e];
            *reinterpret_cast<uint4 *>(dst[e] + p1[e] * 8) = y[e];
        }
    }
}

cudaError_t launch_append(const AppendArgs &a, int num_sms, cudaStream_t s) {
    // as many tokens a block as leave every SM four blocks
    int per = a.T / (4 * num_sms);
    per = per < 1 ? 1 : per > kAppendTokens ? kAppendTokens : per;
    const dim3 grid((a.T + per - 1) / per), block(kAppendThreads);
    // two items of a thread in flight together if a block has more than one for each
    // (prompt of 8192: 19 -> 17.9 us; four: 24; where there is one only, two in the
    // code cost 0.8 of 4.3 us)
    const int heads = (a.q ? a.Hq : 0) + 2 * a.c.Hkv;
    if (per * heads * (a.c.D / 16) <= kAppendThreads)
        return a.c.D == 64 ? launch_dependent(append_kernel<64, 1>, grid, block, 0, s, a, per)
                           : launch_dependent(append_kernel<128, 1>, grid, block, 0, s, a, per);
    return a.c.D == 64 ? launch_dependent(append_kernel<64, 2>, grid, block, 0, s, a, per)
                       : launch_dependent(append_kernel<128, 2>, grid, block, 0, s, a, per);
}

// ------------------------------------------------------------- attention
//
// Row b, query head h, key-value head g = h / group: o = softmax(scale q . K) V
// over the prefix and the row's own positions, by the online softmax: over any
// part of the positions a reference m (here the maximum), sum l = sum 2^(s - m)
// and output O = sum 2^(s - m) v (scores in units of log2), and parts merge as
// m = max m_i, l = sum 2^(m_i - m) l_i, O likewise.
//
// paged_own_kernel: every key and value is read once for the (at most 8) query
// heads that share it, so the work is bound by those bytes.  The rows' positions
// are cut into tiles of 16 (never across a page), all tiles of all rows and
// key-value heads (items) form one list, and the list is cut into even pieces,
// whatever the lengths: a batch of one long and many short rows fills the GPU
// like one row does.  Two ways, by the average item (the kernel sees the
// lengths, the host does not):
//   long items   a piece per block; warp w takes tiles w, w + 8, ... of it, and
//                at an item's end the warps' (m, l, O) are merged in shared
//                memory into one partial (about a microsecond an item)
//   short items  (up to 32 tiles on average) a piece per warp, which writes a
//                partial of its own for each item: no block-wide barriers
// Each warp streams its tiles through its own ring of cp.async stages (24 KB),
// which runs on across the items of the piece.  Alone, block (or warp) n takes
// piece n.  Behind a prefix kernel the first blocks, on the SMs that it leaves
// free, start with a piece each, and the other pieces are taken from a counter:
// the first blocks work through them while the prefix is under way, and blocks
// that come late find nothing left and go.  (Which block took a piece does not
// show in the result.)
//   scores   mma.sync m16n8k16, the heads as M, 16 positions as N
//   output   O += P V, P from the score registers as two bf16 parts (|p - hi -
//            lo| <= 2^-17 p): the heads fill only half of the MMA's 16 rows, the
//            upper parts are rows 0-7 and the lower ones rows 8-15, and the two
//            results are added when the item is through.  l sums the fp32 values
// Measured, calls with the merge: 8 rows of up to 32768 positions (134 MB of keys
// and values) 31 us, 4.3 TB/s, of which the merge's launch and the start (lengths,
// pages, first tiles: three dependent reads) are 8 (this kernel alone 28.5, the
// merge 5); 128 rows of up to 512 13.1 us; one row of 1000 9.5 to 9.8, all of it
// latency.
constexpr int kOwnWarps = 8;
constexpr int kOwnThreads = kOwnWarps * 32;
constexpr int kPosTile = 16;
constexpr int kShortItem = 32;   // tiles of an average item up to which pieces go to warps
constexpr int kBlockTiles = 8;   // tiles that a block's piece has at least (one per warp) ...
constexpr int kWarpTiles = 4;    // ... and a warp's, if there are fewer items than pieces

__host__ __device__ constexpr int own_stages(int D) { return D == 128 ? 3 : 6; }
__host__ __device__ constexpr int own_stage_bytes(int D) { return 2 * kPosTile * D * 2; }
__host__ __device__ constexpr int own_ring_bytes(int D) { return kOwnWarps * own_stages(D) * own_stage_bytes(D); }
__host__ __device__ constexpr int merge_pitch(int D) { return D + 8; }
__host__ __device__ constexpr int own_merge_bytes(int D) { return kOwnWarps / 2 * 8 * merge_pitch(D) * 4; }
constexpr int kMaxRows = 1024;
__host__ __device__ constexpr int own_smem_bytes(int D) {
    return own_ring_bytes(D) + own_merge_bytes(D) + 2 * kOwnWarps * 8 * 4 + kOwnWarps * own_stages(D) * 4 +
           (kMaxRows + 1) * 8;
}
static_assert(kOwnWarps == 8, "a shift by 3 divides by the warps");
static_assert(own_smem_bytes(128) <= 227 * 1024 && own_smem_bytes(64) <= 227 * 1024, "one block per SM");

// a / b of two numbers that are not negative: nearly always both fit 32 bits,
// where a division takes a fraction of the instructions.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return (a | b) >> 32 ? a / b : static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
}

__host__ __device__ __forceinline__ int tiles16(int n) { return (n + kPosTile - 1) / kPosTile; }

// Row b's own positions: none for a padding row, the table's room at most.
__device__ __forceinline__ int own_len(const PagedArgs &a, int b, bool &over) {
    const int n = a.seq_len[b];
    const int64_t room = static_cast<int64_t>(a.table_ld) << a.c.page_shift;
    over = n > room;
    return n < 0 ? 0 : over ? static_cast<int>(room) : n;
}

template <int D>
__global__ void __launch_bounds__(kOwnThreads, 1) paged_own_kernel(const __grid_constant__ PagedArgs a) {
    constexpr int KD = D / 16;          // MMA k-steps of the scores
    constexpr int NT = D / 8;           // 8-dimension MMA tiles of the output
    constexpr int CH = D * 2 / 16;      // 16-byte chunks of a row
    constexpr int ROW = D * 2;
    constexpr int NS = own_stages(D), STAGE = own_stage_bytes(D), MP = merge_pitch(D);
    extern __shared__ __align__(128) uint8_t smem[];
    float *mo = reinterpret_cast<float *>(smem + own_ring_bytes(D));          // [4 warps][8 heads][MP]
    float *mm = reinterpret_cast<float *>(smem + own_ring_bytes(D) + own_merge_bytes(D));  // [warp][head]
    float *ml = mm + kOwnWarps * 8;
    int *s_valid = reinterpret_cast<int *>(ml + kOwnWarps * 8);               // [warp][stage]
    int64_t *s_start = reinterpret_cast<int64_t *>(s_valid + kOwnWarps * NS);  // [B + 1]
    __shared__ int64_t s_warp[kOwnWarps];
    __shared__ int s_rows[kOwnWarps];
    __shared__ int s_piece;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g8 = lane >> 2, c = lane & 3;
    // the first kernel of the call waits for what came before it; after a prefix
    // kernel (which has waited) it need not wait for that one, and its blocks
    // take over the SMs as that one's end
    if (!a.prefix_ncta) pdl_wait();
    pdl_trigger();
    if (a.prefix_ncta && static_cast<int>(blockIdx.x) >= a.own_first) {
        // everything taken already?
        if (tid == 0) s_piece = __ldcg(a.pieces) > 0 && __ldcg(a.pieces + 1) >= __ldcg(a.pieces) - 1;
        __syncthreads();
        if (s_piece) {
            pdl_wait();
            return;
        }
    }
    const int Hkv = a.c.Hkv, ps = a.c.page_shift;
    const int ntp = a.join ? tiles16(a.prefix_len) : 0;

    // tiles of the rows before each row, and the number of rows that have any
    int64_t items = 0;
    if (a.B <= 31) {
        // a row a lane, the same in every warp
        int64_t n = 0;
        if (lane < a.B) {
            bool over;
            const int len = own_len(a, lane, over);
            n = a.seq_len[lane] < 0 ? 0 : ntp + tiles16(len);
            if (over && blockIdx.x == 0 && warp == 0) record_status(a.status, MOE_ERR_PAGE);
        }
        items = __popc(__ballot_sync(0xffffffffu, n > 0));
        int64_t scan = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, scan, off);
            if (lane >= off) scan += v;
        }
        if (warp == 0 && lane <= a.B) {
            s_start[lane] = scan - n;
            if (blockIdx.x == 0) a.starts[lane] = scan - n;
        }
        __syncthreads();
    } else {
        // one or four rows a thread, then a scan
        auto scan_rows = [&](auto each) {
            constexpr int R = decltype(each)::value;
            int64_t n[R], sum = 0;
            int filled = 0;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int b = tid * R + i;
                n[i] = 0;
                if (b < a.B) {
                    bool over;
                    const int len = own_len(a, b, over);
                    n[i] = a.seq_len[b] < 0 ? 0 : ntp + tiles16(len);
                    if (over && blockIdx.x == 0) record_status(a.status, MOE_ERR_PAGE);
                }
                sum += n[i];
                filled += n[i] > 0;
            }
            int64_t scan = sum;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int64_t v = __shfl_up_sync(0xffffffffu, scan, off);
                if (lane >= off) scan += v;
            }
            filled = __reduce_add_sync(0xffffffffu, filled);
            if (lane == 31) {
                s_warp[warp] = scan;
                s_rows[warp] = filled;
            }
            __syncthreads();
            scan -= sum;
            for (int w = 0; w < warp; ++w) scan += s_warp[w];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int b = tid * R + i;
                if (b <= a.B) {
                    s_start[b] = scan;
                    if (blockIdx.x == 0) a.starts[b] = scan;
                }
                scan += n[i];
            }
            if (tid == kOwnThreads - 1 && a.B == R * kOwnThreads) {
                s_start[a.B] = scan;
                if (blockIdx.x == 0) a.starts[a.B] = scan;
            }
        };
        if (a.B <= kOwnThreads)
            scan_rows(std::integral_constant<int, 1>());
        else
            scan_rows(std::integral_constant<int, kMaxRows / kOwnThreads>());
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kOwnWarps; ++w) items += s_rows[w];
    }
    items *= Hkv;
    const int64_t W = s_start[a.B] * Hkv;
    // tiles of a piece: as many pieces as there are blocks or warps, or fewer
    // where that leaves less than an item or a few tiles for each
    const bool by_warp = W <= kShortItem * items;
    int64_t most = by_warp ? (W + kWarpTiles - 1) / kWarpTiles : (W + kBlockTiles - 1) / kBlockTiles;
    most = most > items ? most : items;
    const int64_t cap = by_warp ? a.ncta * kOwnWarps : a.ncta;
    most = most < cap ? most : cap;
    const int64_t per = most ? quotient(W + most - 1, most) : 0;
    const int n_pieces = per ? static_cast<int>(quotient(W + per - 1, per)) : 0;
    const int given = a.prefix_ncta ? (by_warp ? a.own_first * kOwnWarps : a.own_first) : n_pieces;  // not by the counter
    if (blockIdx.x == 0 && tid == 0) {
        a.starts[a.B + 1] = per;
        if (a.prefix_ncta) __stcg(a.pieces, max(n_pieces - given, 0) + 1);
    }
    const int stride = by_warp ? 1 : kOwnWarps;
    // this warp's piece, and its tiles in it: first + stride i, i < my_n.  The
    // pieces of warps go round the blocks, so that a few of them meet no other
    const int spread = a.prefix_ncta ? a.own_first : a.ncta;
    int piece = by_warp ? warp * spread + blockIdx.x : blockIdx.x;
    int64_t f0 = 0, f1 = 0, first = 0;
    int my_n = 0;

    // the row of tile f: the last one that starts at or before it
    auto row_of = [&](int64_t f) {
        int lo = 0, hi = a.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_start[mid] * Hkv <= f)
                lo = mid;
            else
                hi = mid - 1;
        }
        return lo;
    };

    // lane j describes tile 32 k + j of this warp: where its first key is, and
    // how many positions it has (none if the page is outside the pool)
    int64_t d_at = 0;
    int d_valid = 0;
    auto describe = [&](int i) {
        d_valid = 0;
        if (i >= my_n) return;
        const int64_t f = first + static_cast<int64_t>(stride) * i;
        const int b = row_of(f);
        const int64_t nt = s_start[b + 1] - s_start[b];
        const int64_t in_row = f - s_start[b] * Hkv;
        const int kv = static_cast<int>(quotient(in_row, nt));
        int t = static_cast<int>(in_row - kv * nt);
        const int *pages = a.table + static_cast<int64_t>(b) * a.table_ld;
        bool over;
        int n = own_len(a, b, over);
        if (t < ntp) {
            pages = a.prefix_pages;
            n = a.prefix_len;
        } else {
            t -= ntp;
        }
        const int p0 = t * kPosTile;
        const int page = pages[p0 >> ps];
        if (page < 0 || page >= a.c.n_pages) {
            record_status(a.status, MOE_ERR_PAGE);
            return;
        }
        d_at = page * a.c.page_stride + kv * a.c.head_stride + (p0 & ((1 << ps) - 1)) * a.c.pos_stride;
        d_valid = n - p0 < kPosTile ? n - p0 : kPosTile;
    };
    const uint32_t ring = smem_u32(smem) + warp * NS * STAGE;
    // tile i into stage i % NS: keys then values, chunk ch of row r at
    // ch ^ (r & 7); rows past the last position are zeros.  Lane l copies chunk
    // l % CH of rows l / CH, + RS, + 2 RS, ..  (A tile lies within a page, so that
    // the addresses of all its rows are inside the pool; those of a tile without
    // a page are page 0's, and nothing is read)
    constexpr int RS = 32 / CH;
    const int r0 = lane / CH;
    const int64_t from = (r0 * a.c.pos_stride + lane % CH * 8) * 2, row_bytes = a.c.pos_stride * (2 * RS);
    const int64_t to_v = reinterpret_cast<const char *>(a.c.v) - reinterpret_cast<const char *>(a.c.k);
    const uint32_t at_row = r0 * ROW, at_chunk = (lane % CH ^ r0) << 4;
    auto issue = [&](int i) {
        if ((i & 31) == 0) describe(i + lane);
        const int64_t at = __shfl_sync(0xffffffffu, d_at, i & 31);
        const int valid = __shfl_sync(0xffffffffu, d_valid, i & 31);
        const uint32_t st = ring + (i % NS) * STAGE + at_row;
        if (lane == 0) s_valid[warp * NS + i % NS] = valid;
        const char *src = reinterpret_cast<const char *>(a.c.k + at) + from;
#pragma unroll
        for (int j = 0; j < kPosTile / RS; ++j) {
            const bool ok = r0 + j * RS < valid;
            // (r0 and j RS have no bit in common)
            const uint32_t dst = st + j * RS * ROW + (at_chunk ^ (j * RS & 7) << 4);
            cp_async16_zfill(dst, src, ok);
            cp_async16_zfill(dst + kPosTile * ROW, src + to_v, ok);
            src += row_bytes;
        }
    };
    // ldmatrix lane roles: matrix mi = lane / 8, row rr = lane % 8
    const int mi = lane >> 3, rr = lane & 7;
    const int kpos = (mi >> 1) * 8 + rr, kch = mi & 1;
    const int vpos = (mi & 1) * 8 + rr, vch = mi >> 1;
    const uint32_t flip = a.negate ? 0x80008000u : 0u, keep = a.zero_q ? 0u : 0xFFFFFFFFu;

    // the item's queries as the A operand: thread (g8, c) holds
    // q[g8][16 kd + 2c, +1] and [16 kd + 2c + 8, +9]
    uint32_t qa[KD][2];
    auto load_q = [&](int b, int kv) {
        const bool real = g8 < a.group;
        const uint32_t *qrow = reinterpret_cast<const uint32_t *>(
            a.q + b * a.q_stride + static_cast<int64_t>(kv * a.group + (real ? g8 : 0)) * D);
#pragma unroll
        for (int kd = 0; kd < KD; ++kd) {
            qa[kd][0] = real ? (__ldg(qrow + kd * 8 + c) & keep) ^ flip : 0u;
            qa[kd][1] = real ? (__ldg(qrow + kd * 8 + c + 4) & keep) ^ flip : 0u;
        }
    };

    for (bool given_one = static_cast<int>(blockIdx.x) < spread;; given_one = false) {
        if (!given_one) {
            if (!a.prefix_ncta) break;
            if (by_warp) {
                if (lane == 0) piece = given + atomicAdd(a.pieces + 1, 1);
                piece = __shfl_sync(0xffffffffu, piece, 0);
            } else {
                __syncthreads();  // the piece before has been read by every warp
                if (tid == 0) s_piece = given + atomicAdd(a.pieces + 1, 1);
                __syncthreads();
                piece = s_piece;
            }
        }
        if (piece >= n_pieces) break;
        f0 = piece * per;
        f1 = f0 + per < W ? f0 + per : W;
        first = by_warp ? f0 : f0 + warp;
        my_n = f1 > first ? static_cast<int>((f1 - first + stride - 1) >> (by_warp ? 0 : 3)) : 0;
#pragma unroll 1
        for (int j = 0; j < NS; ++j) {
            if (j < my_n) issue(j);
            cp_async_commit();
        }
        int i = 0, b = row_of(f0);
        int64_t nt = s_start[b + 1] - s_start[b];  // tiles of the row's items
        int kv = static_cast<int>(quotient(f0 - s_start[b] * Hkv, nt));
        int64_t end = s_start[b] * Hkv + (kv + 1) * nt;  // end of this item
        load_q(b, kv);
        for (int64_t f = f0; f < f1;) {
            const int64_t stop = end < f1 ? end : f1;
            float o[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
            float m_run = -INFINITY, l_run = 0.f;

            for (; first + static_cast<int64_t>(stride) * i < stop; ++i) {
                cp_async_wait<NS - 1>();
                __syncwarp();
                const uint32_t sk = ring + (i % NS) * STAGE, sv = sk + kPosTile * ROW;
                const int valid = s_valid[warp * NS + i % NS];
                if (valid > 0) {
                    float s0[2][4] = {}, s1[2][4] = {};
#pragma unroll
                    for (int kd = 0; kd < KD; ++kd) {
                        uint32_t bm[4];
                        ldsm_x4(bm, sk + kpos * ROW + (((2 * kd + kch) ^ (kpos & 7)) << 4));
                        const uint32_t af[4] = {qa[kd][0], 0u, qa[kd][1], 0u};
                        mma_16816(s0[kd & 1], af, bm[0], bm[1]);
                        mma_16816(s1[kd & 1], af, bm[2], bm[3]);
                    }
                    float sc[4] = {s0[0][0] + s0[1][0], s0[0][1] + s0[1][1], s1[0][0] + s1[1][0], s1[0][1] + s1[1][1]};
                    const int pos[4] = {2 * c, 2 * c + 1, 8 + 2 * c, 9 + 2 * c};
#pragma unroll
                    for (int j = 0; j < 4; ++j) sc[j] = pos[j] < valid ? sc[j] * a.scale_log2 : -INFINITY;
                    float tmax = fmaxf(fmaxf(sc[0], sc[1]), fmaxf(sc[2], sc[3]));
                    tmax = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, 1));
                    tmax = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, 2));
                    const float m_new = fmaxf(fmaxf(m_run, tmax), kLeastRef);
                    const float corr = exp2f(m_run - m_new);
                    float p[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) p[j] = exp2f(sc[j] - m_new);
                    l_run = l_run * corr + ((p[0] + p[1]) + (p[2] + p[3]));
                    m_run = m_new;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        o[n][0] *= corr;
                        o[n][1] *= corr;
                        o[n][2] *= corr;
                        o[n][3] *= corr;
                    }
                    uint32_t pa[4];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t hi = pack2_bf16(p[2 * j], p[2 * j + 1]);
                        pa[2 * j] = hi;
                        pa[2 * j + 1] = pack2_bf16(p[2 * j] - __uint_as_float(hi << 16),
                                                  p[2 * j + 1] - __uint_as_float(hi & 0xFFFF0000u));
                    }
#pragma unroll
                    for (int jt = 0; jt < NT / 2; ++jt) {
                        uint32_t bm[4];
                        ldsm_x4_trans(bm, sv + vpos * ROW + (((2 * jt + vch) ^ (vpos & 7)) << 4));
                        mma_16816(o[2 * jt], pa, bm[0], bm[1]);
                        mma_16816(o[2 * jt + 1], pa, bm[2], bm[3]);
                    }
                }
                __syncwarp();  // every lane has read the stage before it is refilled
                if (i + NS < my_n) issue(i + NS);
                cp_async_commit();
            }

            const int64_t slot = static_cast<int64_t>(piece) + static_cast<int64_t>(b) * Hkv + kv;
            // the next item; its queries are on their way while this one is written
            f = stop;
            if (f < f1) {
                if (++kv == Hkv) {
                    kv = 0;
                    do ++b;
                    while (s_start[b + 1] == s_start[b]);
                    nt = s_start[b + 1] - s_start[b];
                }
                end += nt;
                load_q(b, kv);
            }

            // both parts of the weights
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                o[n][0] += o[n][2];
                o[n][1] += o[n][3];
            }
            float l_sum = l_run + __shfl_xor_sync(0xffffffffu, l_run, 1);
            l_sum += __shfl_xor_sync(0xffffffffu, l_sum, 2);
            if (by_warp) {
                float *dst = a.own_o + slot * (8 * D) + (c >> 1) * 32 + g8 * 4 + (c & 1) * 2;
#pragma unroll
                for (int n = 0; n < NT; ++n) *reinterpret_cast<float2 *>(dst + n * 64) = make_float2(o[n][0], o[n][1]);
                if (c == 0) a.own_ml[slot * 8 + g8] = make_float2(m_run, l_sum);
                continue;
            }
            // merge the eight warps: every warp scales its output to the common
            // maximum, the upper four hand theirs to the lower four, these add and
            // leave four sums, which the block adds in order
            if (c == 0) {
                mm[warp * 8 + g8] = m_run;  // -inf: no tile of this item
                ml[warp * 8 + g8] = l_sum;
            }
            __syncthreads();
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kOwnWarps; ++w) M = fmaxf(M, mm[w * 8 + g8]);
            const float e = m_run == -INFINITY ? 0.f : exp2f(m_run - M);
            float *mine = mo + ((warp & 3) * 8 + g8) * MP + 2 * c;
            if (warp >= 4) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    *reinterpret_cast<float2 *>(mine + 8 * n) = make_float2(o[n][0] * e, o[n][1] * e);
            }
            __syncthreads();
            if (warp < 4) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float2 v = *reinterpret_cast<float2 *>(mine + 8 * n);
                    v.x += o[n][0] * e;
                    v.y += o[n][1] * e;
                    *reinterpret_cast<float2 *>(mine + 8 * n) = v;
                }
            }
            __syncthreads();
            {
                const int h = tid & 7;
                for (int d4 = tid >> 3; d4 < D / 4; d4 += kOwnThreads / 8) {
                    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const float4 v = *reinterpret_cast<const float4 *>(mo + (w * 8 + h) * MP + d4 * 4);
                        sum.x += v.x;
                        sum.y += v.y;
                        sum.z += v.z;
                        sum.w += v.w;
                    }
                    *reinterpret_cast<float4 *>(a.own_o + (slot * (D / 4) + d4) * 32 + h * 4) = sum;
                }
                if (tid < 8) {
                    float mx = -INFINITY, den = 0.f;
#pragma unroll
                    for (int w = 0; w < kOwnWarps; ++w) mx = fmaxf(mx, mm[w * 8 + tid]);
#pragma unroll
                    for (int w = 0; w < kOwnWarps; ++w)
                        if (mm[w * 8 + tid] != -INFINITY) den += exp2f(mm[w * 8 + tid] - mx) * ml[w * 8 + tid];
                    a.own_ml[slot * 8 + tid] = make_float2(mx, den);
                }
            }
            __syncthreads();  // the merge buffers are free for the next item
        }
    }
    cp_async_wait<0>();
    pdl_wait();  // a kernel before this one that still runs is complete before this one is
}

// Merge the partials of one (row, key-value head): grid (B Hkv, D / 32), thread
// (one of kParts shares of the partials, 4 dimensions, head).  Every thread runs
// the online merge over its partials, four at a time (their loads
// independent), the shares meet in shared memory.  Bound by latency, so there
// are as many shares as keep the GPU's threads busy: 128 rows without a prefix
// took 13 us in all with 2 shares and 18 with 8, one row of 32768 positions 21
// and 14.  (A merge by the last block to finish an item, in the kernel above,
// took 1 to 4 us more: its fence, its atomic and one block's reads cost more than
// this launch.)
constexpr int kBatch = 4;

template <int kParts>
__global__ void __launch_bounds__(kParts * 64, 16 / kParts) paged_combine_kernel(const __grid_constant__ PagedArgs a) {
    __shared__ float4 s_acc[kParts][64];
    __shared__ float2 s_ml[kParts][64];
    pdl_wait();
    pdl_trigger();
    const int Hkv = a.c.Hkv, D = a.c.D;
    const int b = blockIdx.x / Hkv, kv = blockIdx.x % Hkv;
    const int tid = threadIdx.x, h = tid & 7, dq = (tid >> 3) & 7, part = tid >> 6;
    const int d4 = blockIdx.y * 8 + dq;
    const int len = a.seq_len[b];
    const int64_t s0 = a.starts[b], nt = a.starts[b + 1] - s0, per = a.starts[a.B + 1];
    if (a.prefix_ncta && blockIdx.x == 0 && blockIdx.y == 0 && tid < 2) a.pieces[tid] = 0;  // for the next call
    if (len < 0) return;  // padding: out stays as it is

    // its own partials: those of the pieces that its tiles lie in
    int n_own = 0;
    const float2 *own_ml = a.own_ml;
    const float *own_o = a.own_o;
    if (nt > 0) {
        const int64_t f = s0 * Hkv + kv * nt, p0 = quotient(f, per);
        n_own = static_cast<int>(quotient(f + nt - 1, per) - p0) + 1;
        const int64_t slot = p0 + static_cast<int64_t>(b) * Hkv + kv;
        own_ml += slot * 8 + h;
        own_o += (slot * (D / 4) + d4) * 32 + h * 4;
    }
    // the prefix's partials of head h's row
    int n_pre = 0;
    int64_t step = 1;
    const float2 *pre_ml = a.prefix_ml;
    const float *pre_o = a.prefix_o;
    if (a.prefix_ncta && h < a.group) {
        const int g = b * a.group + h, sub = a.prefix_two ? (g >> 7) & 1 : 0;
        const int64_t item = static_cast<int64_t>(kv) * a.prefix_blocks + (a.prefix_two ? g >> 8 : 0);
        const int64_t f = item * a.prefix_tiles, p0 = f / a.prefix_per;
        n_pre = static_cast<int>((f + a.prefix_tiles - 1) / a.prefix_per - p0) + 1;
        if (a.prefix_two)
            step = 2;
        else
            n_pre *= 2;  // a partial of the even and one of the odd tiles
        const int64_t slot = 2 * (p0 + item) + sub;
        pre_ml += slot * 128 + (g & 127);
        pre_o += (slot * (D / 4) + d4) * 512 + (g & 127) * 4;
    }
    const int n = n_own + n_pre;
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = part; i0 < n; i0 += kParts * kBatch) {
        float2 t[kBatch];
        float4 v[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int i = i0 + kParts * j;
            t[j] = make_float2(-INFINITY, 0.f);
            v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < n_own) {
                t[j] = __ldcg(own_ml + i * 8);
                v[j] = __ldcg(reinterpret_cast<const float4 *>(own_o + static_cast<int64_t>(i) * D * 8));
            } else if (i < n) {
                t[j] = __ldcg(pre_ml + (i - n_own) * step * 128);
                v[j] = __ldcg(reinterpret_cast<const float4 *>(pre_o + (i - n_own) * step * D * 128));
            }
        }
        float mx = m;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) mx = fmaxf(mx, t[j].x);
        if (mx == -INFINITY) continue;
        const float corr = exp2f(m - mx);
        m = mx;
        l *= corr;
        acc = make_float4(acc.x * corr, acc.y * corr, acc.z * corr, acc.w * corr);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            // a partial without a tile (-inf) may never have been written
            const bool has = t[j].x != -INFINITY;
            const float w = exp2f(t[j].x - mx);
            l += has ? w * t[j].y : 0.f;
            acc.x += has ? w * v[j].x : 0.f;
            acc.y += has ? w * v[j].y : 0.f;
            acc.z += has ? w * v[j].z : 0.f;
            acc.w += has ? w * v[j].w : 0.f;
        }
    }
    s_acc[part][tid & 63] = acc;
    s_ml[part][tid & 63] = make_float2(m, l);
    __syncthreads();
    if (part == 0 && h < a.group) {
        float2 t[kParts];
        float mx = -INFINITY, den = 0.f;
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            t[i] = s_ml[i][tid];
            mx = fmaxf(mx, t[i].x);
        }
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (mx != -INFINITY) {
#pragma unroll
            for (int i = 0; i < kParts; ++i) {
                const float w = exp2f(t[i].x - mx);
                const float4 v = s_acc[i][tid];
                den += w * t[i].y;
                acc.x += w * v.x;
                acc.y += w * v.y;
                acc.z += w * v.z;
                acc.w += w * v.w;
            }
        }
        const float inv = mx == -INFINITY ? 0.f : 1.0f / den;  // no position at all: zeros
        uint2 r;
        r.x = pack2_bf16(acc.x * inv, acc.y * inv);
        r.y = pack2_bf16(acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2 *>(a.out + b * a.out_stride + static_cast<int64_t>(kv * a.group + h) * D + d4 * 4) = r;
    }
}

// ------------------------------------------------------------------- host

// One row's prefix is read once either way, and without the prefix kernel
// there is a launch less.
bool paged_joins(int B, int prefix_len) { return B == 1 || prefix_len == 0; }

static int prefix_row_blocks(int rows) { return rows <= 128 ? 1 : (rows + 255) / 256; }

struct PagedLayout {
    size_t starts, own_ml, own_o, prefix_ml, prefix_o, total;
};

static PagedLayout paged_layout(int B, int Hq, int Hkv, int D, int prefix_len, int num_sms) {
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    PagedLayout L{};
    const size_t slots = static_cast<size_t>(num_sms) * kOwnWarps + static_cast<size_t>(B) * Hkv;
    L.starts = kCtrlBytes;
    L.own_ml = L.starts + up((B + 2) * sizeof(int64_t));
    L.own_o = L.own_ml + up(slots * 8 * sizeof(float2));
    L.prefix_ml = L.own_o + up(slots * 8 * D * sizeof(float));
    const size_t parts = paged_joins(B, prefix_len) ? 0 : 2 * (num_sms + static_cast<size_t>(Hkv) * prefix_row_blocks(B * (Hq / Hkv)));
    L.prefix_o = L.prefix_ml + up(parts * 128 * sizeof(float2));
    L.total = L.prefix_o + parts * 128 * D * sizeof(float);
    return L;
}

size_t paged_workspace_bytes(int B, int Hq, int Hkv, int D, int prefix_len, int num_sms) {
    return paged_layout(B, Hq, Hkv, D, prefix_len, num_sms).total;
}

template <int D>
static cudaError_t launch_own(const PagedArgs &a, cudaStream_t s) {
    constexpr int smem = own_smem_bytes(D);
    const cudaError_t e = allow_smem<paged_own_kernel<D>>();
    if (e != cudaSuccess) return e;
    return launch_dependent(paged_own_kernel<D>, dim3(a.ncta), dim3(kOwnThreads), smem, s, a);
}

cudaError_t launch_paged(PagedArgs &a, const CUtensorMap *maps, float scale, void *ws, int num_sms, cudaStream_t s) {
    char *w = static_cast<char *>(ws);
    const PagedLayout L = paged_layout(a.B, a.Hq, a.c.Hkv, a.c.D, a.prefix_len, num_sms);
    a.starts = reinterpret_cast<int64_t *>(w + L.starts);
    a.own_ml = reinterpret_cast<float2 *>(w + L.own_ml);
    a.own_o = reinterpret_cast<float *>(w + L.own_o);
    a.prefix_ml = reinterpret_cast<float2 *>(w + L.prefix_ml);
    a.prefix_o = reinterpret_cast<float *>(w + L.prefix_o);
    a.pieces = reinterpret_cast<int *>(w) + 8;  // in the control block, zero between calls
    a.ncta = num_sms;
    a.negate = scale < 0.f;
    a.zero_q = scale == 0.f;
    a.scale_log2 = scale == 0.f ? 1.f : fabsf(scale) * 1.4426950408889634f;
    a.join = paged_joins(a.B, a.prefix_len);
    cudaError_t e;
    if (!a.join) {
        const int rows = a.B * a.group;
        a.prefix_two = rows > 128;
        a.prefix_blocks = prefix_row_blocks(rows);
        a.prefix_tiles = (a.prefix_len + 127) / 128;
        const int64_t tiles = static_cast<int64_t>(a.c.Hkv) * a.prefix_blocks * a.prefix_tiles;
        // (short pieces one tile longer, which leaves SMs for the rows' own positions: 32
        // rows behind 65536 positions 30.3 us instead of 35.8, 64 behind 32768 31.8 and
        // 36.0; 32 of short rows behind 32749 26.6 instead of 22.9)
        a.prefix_per = static_cast<int>((tiles + num_sms - 1) / num_sms);
        if (a.prefix_per >= 2 && a.prefix_per <= 8) ++a.prefix_per;
        a.prefix_ncta = static_cast<int>((tiles + a.prefix_per - 1) / a.prefix_per);
        a.own_first = num_sms - a.prefix_ncta;
        if ((e = launch_prefix(maps[0], maps[1], a, s)) != cudaSuccess) return e;
    }
    if ((e = a.c.D == 64 ? launch_own<64>(a, s) : launch_own<128>(a, s)) != cudaSuccess) return e;
    const dim3 grid(a.B * a.c.Hkv, a.c.D / 32);
    const int blocks = a.B * a.c.Hkv * (a.c.D / 32);
    if (blocks >= 4 * num_sms) return launch_dependent(paged_combine_kernel<2>, grid, dim3(2 * 64), 0, s, a);
    if (blocks >= 2 * num_sms) return launch_dependent(paged_combine_kernel<4>, grid, dim3(4 * 64), 0, s, a);
    if (blocks >= num_sms / 2) return launch_dependent(paged_combine_kernel<8>, grid, dim3(8 * 64), 0, s, a);
    return launch_dependent(paged_combine_kernel<16>, grid, dim3(16 * 64), 0, s, a);
}

}  // namespace moe
