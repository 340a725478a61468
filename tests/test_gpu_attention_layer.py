"""The operators of the attention sub-layer against plain implementations in
64 bits: int4_linear, gqa_append and gqa_paged_attention at the sizes, layouts
and masks where they can go wrong, and a run of them together.

Tolerances.  A bf16 output is the fp32 result rounded once: at most 2^-8 of
the value (half a step), plus the fp32 computation's own error, which is
bounded below per operator in terms of the magnitudes that enter its sums."""
import math

import numpy as np
import pytest
import torch

from int4_grouped_gemm_gb300 import _lib, attention, moe, synthetic

pytestmark = pytest.mark.gpu

BF16 = torch.finfo(torch.bfloat16).eps / 2   # 2^-8: a rounding to bf16
FP32 = torch.finfo(torch.float32).eps / 2    # 2^-24


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16)


# ------------------------------------------------------------------- linear


def make_int4(g, N, K, G):
    """A random int4 matrix in the library's layout (device) and its exact
    values in fp64."""
    pitch = moe.ld_groups(K, G)
    q = torch.randint(0, 16, (N, K), generator=g, dtype=torch.int64)
    words = torch.zeros(N, K // 8, dtype=torch.int64)
    for e in range(8):
        words |= q[:, e::8] << (4 * (e // 2 + 4 * (e % 2)))
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)
    s = (torch.rand(N, K // G, generator=g) * 0.01 + 0.001).to(torch.bfloat16)
    z = (torch.randn(N, K // G, generator=g) * 0.03).to(torch.bfloat16)
    sp = torch.zeros(N, pitch, dtype=torch.bfloat16)
    zp = torch.zeros(N, pitch, dtype=torch.bfloat16)
    sp[:, :K // G], zp[:, :K // G] = s, z
    w = q.double() * s.double().repeat_interleave(G, 1) + z.double().repeat_interleave(G, 1)
    m = moe.QMatrix(words.cuda(), sp.view(torch.int16).cuda(), zp.view(torch.int16).cuda(), N, K, G)
    return m, w


def linear_bound(x, w, K):
    """The fp32 error of y: products s q x are summed as codes offset by up to
    136 (so up to 144 s |x| per term, and 144 s |x| again where the offset is
    taken off) in K rounded additions; sqrt is not used: this is a worst case
    with the terms' absolute values, for additions in any order of depth
    K / 16 + 64 (tensor products of 16, then groups, warps and blocks)."""
    scale = 0.011 * 144 * 2
    mag = x.abs().double().sum(1, keepdim=True) * scale + x.abs().double() @ w.abs().t()
    return mag * (K / 16 + 64) * FP32


LINEAR = [  # B, K, N, group
    (1, 32, 1, 32), (1, 64, 7, 64), (1, 128, 16, 128), (2, 96, 17, 32), (8, 2048, 160, 64), (9, 2080, 33, 32),
    (16, 192, 129, 64), (17, 1152, 250, 128), (31, 256, 64, 64), (33, 160, 515, 32), (64, 1024, 272, 64),
    (63, 4224, 31, 128), (5, 32768, 24, 64), (64, 8192, 40, 32), (1, 2048, 2560, 64), (3, 4096, 20000, 128),
]


@pytest.mark.parametrize("fp32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("B,K,N,G", LINEAR)
def test_linear_against_64_bits(B, K, N, G, fp32):
    g = gen(B * 7 + K + N)
    m, w = make_int4(g, N, K, G)
    x = randn(g, B, K)
    y = moe.linear(m, x.cuda(), dtype=torch.float32 if fp32 else torch.bfloat16).cpu().double()
    want = x.double() @ w.t()
    tol = linear_bound(x, w, K) + (0 if fp32 else want.abs() * BF16 * 1.01)
    assert ((y - want).abs() <= tol).all(), ((y - want).abs() - tol).max()


def test_linear_strided_rows_and_untouched_neighbours():
    """x a column range of a wider tensor, y a column range too: nothing
    outside it is written, and the rest of x is not read (NaN there)."""
    g = gen(5)
    m, w = make_int4(g, 77, 320, 64)
    xb = torch.full((11, 320 + 48), float("nan"), dtype=torch.bfloat16)
    xb[:, 16:336] = randn(g, 11, 320)
    yb = torch.full((11, 100), 3.0, dtype=torch.bfloat16, device="cuda")
    moe.linear(m, xb.cuda()[:, 16:336], yb[:, 8:85])
    want = xb[:, 16:336].double() @ w.t()
    got = yb.cpu().double()
    assert (got[:, :8] == 3).all() and (got[:, 85:] == 3).all()
    assert ((got[:, 8:85] - want).abs() <= linear_bound(xb[:, 16:336], w, 320) + want.abs() * BF16 * 1.01).all()


def test_linear_odd_row_stride_of_y():
    g = gen(6)
    m, w = make_int4(g, 33, 128, 64)
    x = randn(g, 19, 128)
    for dtype in (torch.bfloat16, torch.float32):
        yb = torch.zeros(19, 35, dtype=dtype, device="cuda")
        moe.linear(m, x.cuda(), yb[:, :33])
        want = x.double() @ w.t()
        assert ((yb[:, :33].cpu().double() - want).abs() <= linear_bound(x, w, 128) + want.abs() * BF16 * 1.01).all()
        assert (yb[:, 33:] == 0).all()


def test_linear_of_packed_weights_repeats_and_replays():
    """Weights packed by pack_int4; the same call twice, on another stream and
    from a replayed graph gives the same bits."""
    w = synthetic.make_weight_matrix(520, 512, seed=3, device="cuda")
    m = moe.pack_matrix(w, 64)
    x = synthetic.make_tokens(512, 12, seed=4, device="cuda")
    a = moe.linear(m, x)
    b = torch.empty_like(a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    moe.linear(m, x, b, stream=s)
    torch.cuda.synchronize()
    graph, c = torch.cuda.CUDAGraph(), torch.empty_like(a)
    with torch.cuda.graph(graph):
        moe.linear(m, x, c)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)
    ref = x.double() @ w.double().t()
    # 15 steps over a group's range: |w - packed| <= half a step plus the bf16 rounding of scale and bias
    assert (a.double() - ref).abs().max() < 0.1 * ref.abs().max()


@pytest.mark.parametrize("B", [1, 5, 8, 9, 16, 40])
def test_linear_a_broken_token_stays_alone(B):
    """NaN and infinity in one token (a padding row, say) leave the others'
    results as they are, bit for bit."""
    g = gen(40 + B)
    m, w = make_int4(g, 150, 256, 64)
    x = randn(g, B, 256).cuda()
    want = moe.linear(m, x, dtype=torch.float32)
    for bad in (float("nan"), float("inf")):
        broken = x.clone()
        broken[B // 2, 17] = bad
        got = moe.linear(m, broken, dtype=torch.float32)
        for b in range(B):
            if b == B // 2:
                assert not torch.isfinite(got[b]).any()
            else:
                assert torch.equal(got[b], want[b])


@pytest.mark.parametrize("B", [1, 3, 12])
@pytest.mark.parametrize("top", [1e-38, 1e-20, 1e20, 3e38])
def test_linear_tokens_of_any_magnitude(B, top):
    """Tokens whose largest element is tiny, huge or subnormal (the few-token
    kernel scales by powers of two), and tokens that span 30 binary orders."""
    g = gen(50)
    m, w = make_int4(g, 40, 128, 32)
    w = w * (1.0 if top < 1e30 else 1e-3)     # (the largest results would not be finite)
    if top >= 1e30:
        s = m.scale.view(torch.bfloat16).float() * 1e-3
        z = m.bias.view(torch.bfloat16).float() * 1e-3
        m = moe.QMatrix(m.q, s.to(torch.bfloat16).view(torch.int16), z.to(torch.bfloat16).view(torch.int16), 40, 128, 32)
        qs = torch.zeros(40, 128, dtype=torch.float64)
        words = m.q.cpu().long() & 0xFFFFFFFF
        for e in range(8):
            qs[:, e::8] = ((words >> (4 * (e // 2 + 4 * (e % 2)))) & 15).double()
        sc = m.scale.cpu().view(torch.bfloat16)[:, :4].double().repeat_interleave(32, 1)
        zc = m.bias.cpu().view(torch.bfloat16)[:, :4].double().repeat_interleave(32, 1)
        w = qs * sc + zc
    x = randn(g, B, 128).double()
    x = x / x.abs().max(1, keepdim=True).values * top
    x[:, ::3] *= 2.0 ** -15
    x[:, 1::3] *= 2.0 ** -30
    x = x.to(torch.bfloat16)
    y = moe.linear(m, x.cuda(), dtype=torch.float32).cpu().double()
    want = x.double() @ w.t()
    # and an element below 2^-31 of the token's largest is off by 2^-40 of that
    tol = linear_bound(x, w, 128) + x.abs().double().max(1, keepdim=True).values * 2.0 ** -40 * w.abs().sum(1) + 1e-43
    assert ((y - want).abs() <= tol).all()


# ------------------------------------------------------------------- append


def make_tables(g, n_seq, ld, n_pages):
    perm = torch.randperm(n_pages, generator=g)[:n_seq * ld]
    return perm.view(n_seq, ld).to(torch.int32)


def pools(n_pages, Hkv, page, D, heads_first, fill=None):
    shape = (n_pages, Hkv, page, D) if heads_first else (n_pages, page, Hkv, D)
    out = []
    for _ in range(2):
        t = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        if fill is not None:
            t.fill_(fill)
        out.append(t if heads_first else t.transpose(1, 2))
    return out


def rotate64(x, pos, inv_freq, interleaved):
    y = x.double().clone()
    rot = 2 * len(inv_freq)
    ang = pos.double()[:, None] * inv_freq.double()
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    i0, i1 = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x[..., i0].double(), x[..., i1].double()
    y[..., i0], y[..., i1] = a * c - b * s, b * c + a * s
    return y


def rotate_tol(x, want, rot, interleaved):
    """fp32: the angle's fraction of a turn is off by 2^-24 of a turn at far
    positions and 2^-25 by its rounding (2 pi of that in radians, 2^-20.8 in
    all), cosine and sine by 2^-23, the two products by 2^-23 each: below 2^-20
    of |a| + |b|; then the rounding to bf16."""
    if rot == 0:
        return torch.zeros_like(want)
    pair = torch.zeros_like(want)
    i0, i1 = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    pair[..., i0] = pair[..., i1] = x[..., i0].double().abs() + x[..., i1].double().abs()
    return pair * 2 ** -20 + want.abs() * BF16 * (pair > 0)


APPEND = [  # T, n_seq, Hq, Hkv, D, rot, interleaved, page, heads_first, first, offset
    (1, 1, 1, 1, 64, 64, False, 16, True, 0, 0),
    (1, 1, 16, 2, 128, 128, False, 64, True, 4095, 0),
    (8, 8, 16, 2, 128, 128, True, 16, False, 31, 1 << 30),
    (37, 3, 12, 4, 128, 64, False, 32, True, 15, 131072),
    (100, 4, 5, 5, 64, 16, True, 64, False, 0, 1000001),
    (65, 2, 8, 1, 64, 0, False, 128, True, 3, 7),
    (29, 2, 24, 3, 128, 48, False, 16, True, 1, 12345),
    (257, 7, 256, 32, 64, 32, True, 16, True, 9, 0),
    (300, 1, 40, 8, 128, 128, False, 256, False, 100, 77),
]


@pytest.mark.parametrize("in_place", [False, True], ids=["out", "in_place"])
@pytest.mark.parametrize("T,n_seq,Hq,Hkv,D,rot,inter,page,hf,first,offset", APPEND)
def test_append_against_64_bits(T, n_seq, Hq, Hkv, D, rot, inter, page, hf, first, offset, in_place):
    g = gen(T + D + rot)
    per = -(-T // n_seq)
    ld = (first + per) // page + 1
    n_pages = n_seq * ld + 3
    table = make_tables(g, n_seq, ld, n_pages)
    seq = torch.arange(T) % n_seq
    index = first + torch.arange(T) // n_seq
    kp, vp = pools(n_pages, Hkv, page, D, hf, fill=2.0)
    cache = attention.PagedCache(kp, vp)
    # queries, keys and values side by side in one buffer, as a projection leaves them
    qkv = randn(g, T, Hq + 2 * Hkv, D)
    dev = qkv.cuda()
    q, k, v = dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:]
    inv = None if rot == 0 else (1e6 ** (-torch.arange(0, rot, 2).double() / rot)).float()
    got = cache.append(q, k, v, seq.int().cuda(), index.int().cuda(), table.cuda(), None if rot == 0 else inv.cuda(),
                       pos_offset=offset, interleaved=inter, q_out=q if in_place else None)
    assert int(cache.status[0]) == 0
    if in_place:
        assert got.data_ptr() == q.data_ptr()
        assert torch.equal(dev[:, Hq:].cpu(), qkv[:, Hq:])
    pos = index + offset
    kw = qkv[:, Hq:Hq + Hkv].double() if rot == 0 else rotate64(qkv[:, Hq:Hq + Hkv], pos, inv, inter)
    qw = qkv[:, :Hq].double() if rot == 0 else rotate64(qkv[:, :Hq], pos, inv, inter)
    assert ((got.cpu().double() - qw).abs() <= rotate_tol(qkv[:, :Hq], qw, rot, inter)).all()
    pages, off = table[seq, index // page].long(), index % page
    kc, vc = kp.cpu(), vp.cpu()
    at = kc[pages, :, off].double()
    assert ((at - kw).abs() <= rotate_tol(qkv[:, Hq:Hq + Hkv], kw, rot, inter)).all()
    assert torch.equal(vc[pages, :, off], qkv[:, Hq + Hkv:])
    # every other place is as it was
    for c in (kc, vc):
        c = c.clone()
        c[pages, :, off] = 2.0
        assert (c == 2.0).all()


def test_append_padding_and_bad_places():
    """Padding tokens leave cache and q_out alone; places outside the table or
    the pool are skipped and recorded, the other tokens written."""
    g = gen(1)
    kp, vp = pools(6, 2, 16, 64, True, fill=1.0)
    cache = attention.PagedCache(kp, vp)
    table = torch.tensor([[4, 1], [3, 9], [-1, 2]], dtype=torch.int32).cuda()
    q, k, v = randn(g, 8, 4, 64).cuda(), randn(g, 8, 2, 64).cuda(), randn(g, 8, 2, 64).cuda()
    out = torch.full_like(q, 5.0)
    inv = (1e4 ** (-torch.arange(0, 64, 2).double() / 64)).float().cuda()
    # good, padding, padding, bad page 9, page -1, sequence 3, index past the table, good
    seq = torch.tensor([0, -1, 0, 1, 2, 3, 0, 2], dtype=torch.int32).cuda()
    index = torch.tensor([17, 0, -1, 16, 5, 0, 32, 31], dtype=torch.int32).cuda()
    cache.append(q[:3], k[:3], v[:3], seq[:3], index[:3], table, inv, q_out=out[:3])
    assert _lib.moe_read_device_status(cache.status) == 0
    cache.append(q, k, v, seq, index, table, inv, q_out=out)
    assert _lib.moe_read_device_status(cache.status) == _lib.MOE_ERR_PAGE
    assert _lib.moe_read_device_status(cache.status) == 0    # read and cleared
    assert (out[1:3] == 5).all() and not (out[0] == 5).all() and not (out[7] == 5).all()
    assert torch.equal(vp[1, :, 1], v[0]) and torch.equal(vp[2, :, 15], v[7])
    vp[1, :, 1] = kp[1, :, 1] = vp[2, :, 15] = kp[2, :, 15] = 1.0
    assert (kp == 1).all() and (vp == 1).all()


def test_append_on_a_side_stream_and_replayed():
    """A captured append follows the positions of the moment."""
    g = gen(33)
    kp, vp = pools(5, 2, 16, 64, True, fill=0.0)
    cache = attention.PagedCache(kp, vp)
    q, k, v = (randn(g, 2, h, 64).cuda() for h in (4, 2, 2))
    table = torch.tensor([[3, 1], [4, 2]], dtype=torch.int32).cuda()
    seq = torch.tensor([0, 1], dtype=torch.int32).cuda()
    index = torch.tensor([0, 0], dtype=torch.int32).cuda()
    inv = (1e4 ** (-torch.arange(0, 64, 2).double() / 64)).float().cuda()
    out = torch.zeros_like(q)
    cache.append(q, k, v, seq, index, table, inv, q_out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.append(q, k, v, seq, index, table, inv, q_out=out)
    for i, j in ((5, 31), (16, 2)):
        index.copy_(torch.tensor([i, j], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = rotate64(q.cpu(), torch.tensor([i, j]), inv.cpu(), False)
        assert ((out.cpu().double() - want).abs() <= rotate_tol(q.cpu(), want, 64, False)).all()
        for t, at in ((0, i), (1, j)):
            assert torch.equal(vp[table[t, at // 16], :, at % 16], v[t])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = cache.append(q, k, v, seq, index, table, inv, stream=side)
    side.synchronize()
    assert torch.equal(again, out)


@pytest.mark.parametrize("f", [0.0, 1.0, -0.75, 3.0, 100.0, 1e-7, 2 ** -20])
def test_append_angles_of_any_frequency_far_out(f):
    """cos and sin of p f by the exact product, p up to 2^31 - 1, f of either
    sign and beyond a turn per position."""
    g = gen(34)
    kp, vp = pools(1, 1, 65536, 64, True)
    cache = attention.PagedCache(kp, vp)
    T = 200
    index = torch.randint(0, 65536, (T,), generator=g)
    index = torch.unique(index)
    T = len(index)
    k = randn(g, T, 1, 64).cuda()
    inv = torch.full((8,), f)
    zero = torch.zeros(T, dtype=torch.int32).cuda()
    for off in (0, 1 << 20, 1 << 30):
        cache.append(None, k, k, zero, index.int().cuda(), torch.zeros(1, 1, dtype=torch.int32).cuda(), inv.cuda(),
                     pos_offset=off)
        # fp64's own cos of a large angle is exact to the product's rounding,
        # 2^-53 of it: 2^-22 of a radian at 2^31, like the kernel's
        want = rotate64(k.cpu(), index + off, inv, False)
        got = kp[0, :, index.cuda()].transpose(0, 1).cpu().double()
        tol = rotate_tol(k.cpu(), want, 16, False)
        tol[..., :16] += abs(f) * (index + off).double()[:, None, None] * 2 ** -52 * 8
        assert ((got - want).abs() <= tol).all()


def test_append_without_queries_and_beyond_32_bit_offsets():
    """Keys and values alone; pages whose offsets pass 2^32 elements."""
    n_pages, Hkv, page, D = 9, 2, 16, 64
    stride = 1 << 29       # elements between pages: page 8 starts at 2^32
    buf = torch.zeros(8 * stride + 2 * Hkv * page * D, dtype=torch.bfloat16, device="cuda")
    kp = buf.as_strided((n_pages, Hkv, page, D), (stride, page * D, D, 1))
    vp = buf[Hkv * page * D:].as_strided((n_pages, Hkv, page, D), (stride, page * D, D, 1))
    cache = attention.PagedCache(kp, vp)
    g = gen(2)
    k, v = randn(g, 3, Hkv, D).cuda(), randn(g, 3, Hkv, D).cuda()
    table = torch.tensor([[0, 8, 7]], dtype=torch.int32).cuda()
    seq = torch.zeros(3, dtype=torch.int32).cuda()
    index = torch.tensor([15, 16, 33], dtype=torch.int32).cuda()
    assert cache.append(None, k, v, seq, index, table, None) is None
    assert torch.equal(kp[8, :, 0], k[1]) and torch.equal(vp[7, :, 1], v[2]) and torch.equal(vp[0, :, 15], v[0])
    assert int(torch.count_nonzero(buf[stride // 2:stride])) == 0
    q = randn(g, 1, 4, D).cuda()
    out = cache.attend(q, table, torch.tensor([34], dtype=torch.int32).cuda())
    kk = torch.cat([kp[p] for p in (0, 8, 7)], dim=1)[:, :34].double()
    vv = torch.cat([vp[p] for p in (0, 8, 7)], dim=1)[:, :34].double()
    want = attend64(q.double(), kk[None], vv[None], 1 / 8)
    assert ((out.double() - want[0]).abs() <= attend_tol(want[0], vv)).all()


# ------------------------------------------------------------------- attend


def attend64(q, k, v, scale):
    """q [B, Hq, D], k, v [B, Hkv, n, D] in fp64 -> [B, Hq, D]; n = 0: zeros."""
    B, Hq, D = q.shape
    Hkv, n = k.shape[1], k.shape[2]
    if n == 0:
        return torch.zeros_like(q)
    s = (q.view(B, Hkv, Hq // Hkv, D) @ k.transpose(2, 3)) * scale
    return (torch.softmax(s, -1) @ v).view(B, Hq, D)


def attend_tol(want, v):
    """A score is off by its fp32 sums, at most 2^-20 of scale sum |q_i k_i|
    (D <= 128 rounded additions), which stays below 512 here: a weight is off
    by 2^-11 of itself at most.  A weight is rounded to bf16 (2^-8 of it, in
    the numerator and in the denominator), so a sum of weights times values is
    off by at most (2 2^-8 + 2^-11) max |v|; then the output's rounding."""
    return float(v.abs().max()) * (2 * BF16 + 2 ** -11) + want.abs() * BF16


class Setup:
    def __init__(self, B, Hq, Hkv, D, page, prefix, lens, heads_first=True, seed=0, k_std=1.0, spare=2):
        g = gen(seed)
        self.lens, self.prefix, self.D = lens, prefix, D
        n_p = -(-prefix // page)
        own = [-(-max(n, 0) // page) for n in lens]
        total = n_p + sum(own) + spare
        perm = torch.randperm(total, generator=g).to(torch.int32)
        # everything behind a sequence's end, and every unused page, is NaN
        kp, vp = pools(total, Hkv, page, D, heads_first, fill=float("nan"))
        table = torch.full((B, max(1, max(own))), 0, dtype=torch.int32)
        at = n_p
        self.k, self.v = [], []
        pk, pv = randn(g, Hkv, prefix, D, std=k_std).cuda(), randn(g, Hkv, prefix, D).cuda()
        self._fill(kp, vp, perm[:n_p], pk, pv, page)
        for b in range(B):
            n = max(lens[b], 0)
            table[b, :own[b]] = perm[at:at + own[b]]
            kb, vb = randn(g, Hkv, n, D, std=k_std).cuda(), randn(g, Hkv, n, D).cuda()
            self._fill(kp, vp, perm[at:at + own[b]], kb, vb, page)
            at += own[b]
            self.k.append(torch.cat((pk, kb), 1))
            self.v.append(torch.cat((pv, vb), 1))
        self.cache = attention.PagedCache(kp, vp)
        self.table = table.cuda()
        self.prefix_pages = perm[:n_p].cuda() if n_p else None
        self.seq_len = torch.tensor(lens, dtype=torch.int32).cuda()
        self.q = randn(g, B, Hq, D).cuda()

    @staticmethod
    def _fill(kp, vp, pages, k, v, page):
        n = k.shape[1]
        for i, p in enumerate(pages.tolist()):
            m = min(page, n - i * page)
            kp[p, :, :m], vp[p, :, :m] = k[:, i * page:i * page + m], v[:, i * page:i * page + m]

    def run(self, **kw):
        return self.cache.attend(self.q, self.table, self.seq_len, self.prefix_pages, self.prefix, **kw)

    def check(self, out, scale=None):
        scale = 1 / math.sqrt(self.D) if scale is None else scale
        assert torch.isfinite(out).all()
        for b, n in enumerate(self.lens):
            if n < 0:
                continue
            want = attend64(self.q[b:b + 1].double(), self.k[b][None].double(), self.v[b][None].double(), scale)[0]
            if self.k[b].shape[1] == 0:
                assert (out[b] == 0).all()
                continue
            err = (out[b].double() - want).abs()
            tol = attend_tol(want, self.v[b])
            assert (err <= tol).all(), (b, n, (err - tol).max())
            # the roundings of many weights are independent: far below the worst case on average
            if self.k[b].shape[1] > 64:
                assert err.mean() <= 2 * BF16 * want.abs().mean() + 2 ** -11 * float(self.v[b].abs().mean())


ATTEND = [  # B, Hq, Hkv, D, page, prefix, lens, heads_first
    (1, 1, 1, 64, 16, 0, [1], True),
    (1, 16, 2, 128, 16, 0, [0], True),
    (2, 8, 1, 128, 16, 0, [15, 17], False),
    (3, 12, 4, 128, 32, 0, [0, 33, 1], True),
    (1, 16, 2, 128, 64, 0, [4097], True),
    (5, 14, 2, 64, 128, 0, [129, 1000, 0, 64, 3], False),
    (4, 64, 64, 64, 16, 0, [5, 70, 16, 31], True),
    (2, 256, 32, 64, 16, 0, [100, 257], True),
    (1, 16, 2, 128, 64, 1, [0], True),
    (1, 8, 1, 64, 16, 128, [1], False),
    (3, 6, 2, 128, 16, 127, [0, 5, 200], True),
    (2, 3, 3, 64, 256, 129, [1, 1], True),
    (16, 16, 2, 128, 64, 1000, [1 + 7 * i for i in range(16)], True),
    (17, 8, 1, 128, 16, 333, [0] * 17, True),
    (33, 8, 1, 64, 32, 2050, [3] * 33, False),
    (70, 15, 3, 128, 16, 700, [i % 5 for i in range(70)], True),
    (100, 32, 4, 64, 64, 1500, [i for i in range(100)], False),
    (9, 56, 8, 128, 1024, 3000, [40, 0, 1, 2, 16, 15, 1025, 900, 7], True),
    (300, 8, 1, 128, 16, 260, [i % 40 for i in range(300)], True),
    # long among short (pieces per warp), short among long (pieces per block)
    (41, 8, 1, 128, 16, 0, [9000] + [1] * 40, True),
    (5, 16, 2, 64, 32, 0, [6000, 1, 5000, 0, 7], False),
    (41, 8, 1, 64, 16, 200, [2000] + [2] * 40, False),
    (6, 16, 2, 128, 64, 300, [4000, 3, 2500, -1, 0, 700], True),
    # the most rows: 8192 of the prefix, 32 blocks of 256
    (1024, 8, 1, 64, 16, 130, [1 + i % 3 for i in range(1024)], True),
    (1023, 1, 1, 128, 16, 0, [i % 20 for i in range(1023)], True),
    # a page of the largest size, and one that holds the whole prefix
    (2, 8, 1, 64, 65536, 1000, [900, 5], True),
    # padding at both ends and between
    (20, 16, 2, 128, 16, 64, [-1, -1, 30, -1, 5] + [-1] * 14 + [17], True),
]


@pytest.mark.parametrize("B,Hq,Hkv,D,page,prefix,lens,hf", ATTEND)
def test_attend_against_64_bits(B, Hq, Hkv, D, page, prefix, lens, hf):
    s = Setup(B, Hq, Hkv, D, page, prefix, lens, hf, seed=B + Hq + prefix)
    ws = s.cache.workspace(B, Hq, prefix)
    # (padding rows keep what out held)
    out = s.run(out=torch.full_like(s.q, 3.0), ws=ws)
    assert _lib.moe_read_device_status(ws) == 0
    s.check(out)
    assert (out[s.seq_len < 0] == 3).all()
    # the same bits again, in the workspace as it is now
    assert torch.equal(out, s.run(out=torch.full_like(s.q, 3.0), ws=ws))


@pytest.mark.parametrize("k_std,scale", [(6.0, None), (1.0, 0.0), (1.0, -0.3), (30.0, None)])
def test_attend_peaked_uniform_and_negative_scales(k_std, scale):
    s = Setup(6, 16, 2, 128, 32, 777, [0, 1, 50, 300, 16, 999], seed=3, k_std=k_std)
    s.check(s.run(scale=scale), scale)


def test_attend_rising_scores():
    """Keys along the query, each larger than the last: the running maximum
    moves at every position, in the prefix and in the own part."""
    s = Setup(4, 8, 1, 128, 16, 600, [300, 0, 150, 1], seed=4)
    kp = s.cache.k
    ramp = torch.linspace(0.0, 4.0, 900).to(torch.bfloat16)
    dirn = s.q[0, 0].sign()
    for b in range(4):
        n = s.k[b].shape[1]
        s.k[b] = (ramp[:n, None].cuda() * dirn)[None].expand(1, n, 128).contiguous()
    Setup._fill(kp, s.cache.v, s.prefix_pages, s.k[0][:, :600], s.v[0][:, :600], 16)
    for b in range(4):
        Setup._fill(kp, s.cache.v, s.table[b, :-(-s.lens[b] // 16)], s.k[b][:, 600:], s.v[b][:, 600:], 16)
    s.check(s.run())


def test_attend_leaves_padding_rows_alone_and_takes_strided_rows():
    s = Setup(6, 16, 2, 128, 16, 100, [5, -1, 0, 40, -7, -1], seed=5)
    wide = torch.full((6, 20, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :16] = s.q
    s.q = wide[:, :16]
    out = torch.full((6, 24, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    s.run(out=out[:, 8:])
    s.check(out[:, 8:])
    assert (out[:, :8] == 7).all()
    for b in (1, 4, 5):
        assert (out[b] == 7).all()
    # in place of the queries
    want = out[:, 8:].clone()
    keep = s.q.clone()
    s.run(out=s.q)
    for b in (0, 2, 3):
        assert torch.equal(s.q[b], want[b])
    for b in (1, 4, 5):
        assert torch.equal(s.q[b], keep[b])


def test_attend_bad_pages_and_lengths_are_recorded_not_followed():
    s = Setup(4, 16, 2, 128, 16, 64, [40, 20, 40, 3], seed=6)
    ws = s.cache.workspace(4, 16, 64)
    good = s.run(ws=ws).clone()
    table, lens, pages = s.table.clone(), s.seq_len.clone(), s.prefix_pages.clone()
    for bad in (-1, s.cache.n_pages, 2 ** 31 - 1):
        s.table = table.clone()
        s.table[1, 0] = bad
        out = s.run(ws=ws)
        assert _lib.moe_read_device_status(ws) == _lib.MOE_ERR_PAGE
        for b in (0, 2, 3):                       # the other rows do not suffer
            assert torch.equal(out[b], good[b])
    s.table = table
    s.seq_len = lens.clone()
    s.seq_len[2] = 16 * table.shape[1] + 1        # past the table
    out = s.run(ws=ws)
    assert _lib.moe_read_device_status(ws) == _lib.MOE_ERR_PAGE
    for b in (0, 1, 3):
        assert torch.equal(out[b], good[b])
    s.seq_len = lens
    s.prefix_pages = pages.clone()
    s.prefix_pages[3] = s.cache.n_pages
    s.run(ws=ws)
    assert _lib.moe_read_device_status(ws) == _lib.MOE_ERR_PAGE
    s.prefix_pages = pages
    assert torch.equal(s.run(ws=ws), good) and _lib.moe_read_device_status(ws) == 0


def test_attend_agrees_with_the_one_sequence_call():
    """One sequence in one page per sequence: gqa_decode_attention's own
    cache layout, to the same 64-bit values."""
    cfg = synthetic.AttnConfig("one", Hq=16, Hkv=2, D=128, L=1000, L_cap=1024, seed=9)
    q, k, v = (t.cuda() for t in synthetic.make_attention(cfg))
    cache = attention.PagedCache(k[None], v[None])      # one page of 1024 positions
    out = cache.attend(q[None], torch.zeros(1, 1, dtype=torch.int32).cuda(),
                       torch.tensor([1000], dtype=torch.int32).cuda())
    want = attend64(q[None].double(), k[None, :, :1000].double(), v[None, :, :1000].double(), 1 / math.sqrt(128))
    assert ((out.double() - want).abs() <= attend_tol(want, v)).all()


def test_attend_replays_with_new_lengths_and_on_two_streams():
    """A captured call follows the lengths, tables and queries of the moment;
    two calls at once with a workspace each do not disturb one another."""
    s = Setup(5, 16, 2, 128, 16, 300, [100, 200, 3, 0, 77], seed=7)
    ws, ws2 = s.cache.workspace(5, 16, 300), s.cache.workspace(5, 16, 300)
    full = s.run(ws=ws).clone()
    out = torch.zeros_like(full)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run(out=out, ws=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, full)
    lens = s.lens
    s.lens = [1, 199, 0, 0, 16]
    s.seq_len.copy_(torch.tensor(s.lens, dtype=torch.int32))
    keep_k, keep_v = s.k, s.v
    s.k = [k[:, :300 + n] for k, n in zip(keep_k, s.lens)]
    s.v = [v[:, :300 + n] for v, n in zip(keep_v, s.lens)]
    graph.replay()
    torch.cuda.synchronize()
    s.check(out)
    s.seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    oa, ob = torch.zeros_like(full), torch.zeros_like(full)
    for _ in range(5):
        s.run(out=oa, ws=ws, stream=a)
        s.run(out=ob, ws=ws2, stream=b)
    torch.cuda.synchronize()
    assert torch.equal(oa, full) and torch.equal(ob, full)


def test_attend_pools_that_share_a_buffer_and_offsets_past_32_bits():
    """Keys and values of a page side by side; pages 2^29 elements apart, so
    that the prefix's and the rows' pages lie past 2^32 elements."""
    Hkv, page, D, n_pages = 2, 16, 64, 10
    stride = 1 << 29
    buf = torch.full((9 * stride + 2 * Hkv * page * D,), float("nan"), dtype=torch.bfloat16, device="cuda")
    both = buf.as_strided((n_pages, 2, Hkv, page, D), (stride, Hkv * page * D, page * D, D, 1))
    cache = attention.PagedCache(both[:, 0], both[:, 1])
    g = gen(30)
    P, lens = 21, [18, 3, 0]
    k, v = randn(g, Hkv, P + 18 + 3, D).cuda(), randn(g, Hkv, P + 18 + 3, D).cuda()
    prefix = torch.tensor([9, 1], dtype=torch.int32).cuda()
    table = torch.tensor([[8, 7], [6, 0], [0, 0]], dtype=torch.int32).cuda()
    Setup._fill(both[:, 0], both[:, 1], prefix, k[:, :P], v[:, :P], page)
    Setup._fill(both[:, 0], both[:, 1], table[0], k[:, P:P + 18], v[:, P:P + 18], page)
    Setup._fill(both[:, 0], both[:, 1], table[1, :1], k[:, P + 18:], v[:, P + 18:], page)
    q = randn(g, 3, 8, D).cuda()
    out = cache.attend(q, table, torch.tensor(lens, dtype=torch.int32).cuda(), prefix, P)
    for b, part in enumerate((slice(P, P + 18), slice(P + 18, None), slice(0, 0))):
        kk, vv = (torch.cat((t[:, :P], t[:, part]), 1).double() for t in (k, v))
        want = attend64(q[b:b + 1].double(), kk[None], vv[None], 1 / 8)[0]
        assert ((out[b].double() - want).abs() <= attend_tol(want, vv)).all()


def test_attend_slices_of_tables_and_lengths():
    """Lengths and page lists that start at any int32, as slices do."""
    s = Setup(7, 8, 1, 128, 16, 100, [5, 30, 0, 1, 16, 17, 50], seed=31)
    full = s.run().clone()
    lens = torch.cat((torch.zeros(1, dtype=torch.int32, device="cuda"), s.seq_len))[1:]
    pages = torch.cat((torch.zeros(3, dtype=torch.int32, device="cuda"), s.prefix_pages))[3:]
    table = torch.cat((torch.zeros(1, dtype=torch.int32, device="cuda"), s.table.flatten()))[1:].view(7, -1)
    assert lens.data_ptr() % 16 and pages.data_ptr() % 16 and table.data_ptr() % 16
    out = s.cache.attend(s.q, table, lens, pages, 100)
    assert torch.equal(out, full)


def test_attend_many_calls_back_to_back():
    """Calls that follow one another without a pause, of changing shapes in one
    workspace: kernels of one overlap the end of the one before."""
    a = Setup(30, 16, 2, 128, 16, 500, [i for i in range(30)], seed=32)
    b = Setup(3, 16, 2, 128, 16, 0, [900, 20, 1], seed=33)
    c = Setup(8, 16, 2, 128, 16, 3000, [1] * 8, seed=34)
    ws = a.cache.workspace(30, 16, 3000)
    want = [s.run().clone() for s in (a, b, c)]
    outs = [[torch.zeros_like(w) for w in want] for _ in range(20)]
    for o in outs:
        for s, t in zip((a, b, c), o):
            s.run(out=t, ws=ws)
    torch.cuda.synchronize()
    for o in outs:
        for t, w in zip(o, want):
            assert torch.equal(t, w)
    assert _lib.moe_read_device_status(ws) == 0


def test_attend_on_a_side_stream_with_its_own_allocations():
    s = Setup(4, 16, 2, 128, 16, 200, [9, 90, 0, 33], seed=35)
    want = s.run().clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [s.run(stream=side) for _ in range(5)]
    side.synchronize()
    for o in outs:
        assert torch.equal(o, want)


def test_one_workspace_serves_smaller_calls_in_turn():
    big = Setup(40, 16, 2, 128, 16, 900, [i for i in range(40)], seed=11)
    small = Setup(2, 8, 1, 64, 16, 0, [50, 3], seed=12)
    ws = big.cache.workspace(40, 16, 900)
    for _ in range(2):
        big.check(big.run(ws=ws))
        small.check(small.run(ws=ws))
        few = big.run(ws=ws)
        big.check(few)


def test_attend_two_drafts_of_one_sequence():
    """Rows that name the same pages with growing lengths: draft tokens."""
    s = Setup(3, 16, 2, 128, 16, 50, [20, 21, 22], seed=13)
    s.table[0], s.table[1] = s.table[2], s.table[2]
    for b in range(2):
        s.k[b], s.v[b] = s.k[2][:, :50 + s.lens[b]], s.v[2][:, :50 + s.lens[b]]
    s.check(s.run())


# ----------------------------------------------------------------- together


def test_decoding_steps_of_a_batch_behind_a_prefix():
    """AttentionLayer over several steps: project, append, attend, project,
    then the MoE layer of the decoder block takes the result; against the same
    steps in 64 bits, fed with the layer's own bf16 values at each stage."""
    cfg = synthetic.CONFIGS["tiny"]
    H, Hq, Hkv, D, page, P = cfg.H, 6, 2, 64, 16, 45
    g = gen(21)
    wq, wq64 = make_int4(g, (Hq + 2 * Hkv) * D, H, 32)
    wo, wo64 = make_int4(g, H, Hq * D, 64)
    inv = (1e4 ** (-torch.arange(0, D, 2).double() / D)).float()
    layer = attention.AttentionLayer(wq, wo, Hq, Hkv, D, inv.cuda())
    B, n_pages = 5, 16
    cache = attention.PagedCache.empty(n_pages, Hkv, page, D)
    cache.k.fill_(float("nan"))
    cache.v.fill_(float("nan"))
    prefix_pages = torch.tensor([3, 9, 0], dtype=torch.int32).cuda()
    px = randn(g, P, H).cuda()
    _, k, v = layer.project(px)
    zeros = torch.zeros(P, dtype=torch.int32).cuda()
    cache.append(None, k, v, zeros, torch.arange(P, dtype=torch.int32).cuda(), prefix_pages[None], layer.inv_freq)
    table = torch.tensor([[1, 2], [4, 5], [6, 7], [8, 10], [11, 12]], dtype=torch.int32).cuda()
    index = torch.tensor([0, 0, 0, -1, 0], dtype=torch.int32).cuda()      # row 3 is padding
    seq_len = torch.tensor([1, 1, 1, -1, 1], dtype=torch.int32).cuda()
    seq = torch.arange(B, dtype=torch.int32).cuda()
    ws = cache.workspace(B, Hq, P)
    L = synthetic.make_layer(cfg)
    packed = moe.PackedLayer.from_fp32(cfg, L.router_w, L.router_bias, L.w_gate, L.w_up, L.w_down)
    mws = packed.workspace(8)
    norm_w = torch.ones(H, dtype=torch.float32).cuda()

    seen_k = [[] for _ in range(B)]
    seen_v = [[] for _ in range(B)]
    pk = rotate64(k.cpu(), torch.arange(P), inv, False)
    pv = v.cpu().double()
    for step in range(18):   # past the end of a page
        x = randn(g, B, H)
        attn = layer.decode(x.cuda(), cache, seq, index, table, seq_len, ws, prefix_pages, P)
        q1, k1, v1 = (t.cpu() for t in layer.project(x.cuda()))
        full = torch.cat((q1, k1, v1), 1).view(B, -1).double()
        want = x.double() @ wq64.t()
        assert ((full - want).abs() <= linear_bound(x, wq64, H) + want.abs() * BF16 * 1.01).all()
        pos = torch.full((B,), P + step)
        q64, k64 = rotate64(q1, pos, inv, False), rotate64(k1, pos, inv, False)
        for b in (0, 1, 2, 4):
            seen_k[b].append(k64[b])
            seen_v[b].append(v1[b].double())
            kk = torch.cat((pk.transpose(0, 1), torch.stack(seen_k[b], 1)), 1)
            vv = torch.cat((pv.transpose(0, 1), torch.stack(seen_v[b], 1)), 1)
            o = attend64(q64[b:b + 1], kk[None], vv[None], 1 / 8)[0].reshape(-1)
            a = o @ wo64.t()
            # q and k rounded to bf16 on the way (2^-8 of each: scores off by
            # up to 2 * 2^-8 |q| |k| / 8, weights by twice that), weights and
            # o to bf16
            slack = 2 * 2 * BF16 * float(q64[b].norm(dim=1).max() * kk.norm(dim=2).max()) / 8 + 3 * BF16
            tol = slack * float(vv.abs().max()) * wo64.abs().sum(1) + a.abs() * BF16 + 1e-3
            got = attn[b].cpu().double()
            assert ((got - a).abs() <= tol).all()
            # and on average far below that bound
            assert (got - a).abs().mean() <= 0.02 * a.abs().mean() + 1e-3
        h = packed.decode_batch_block(attn, x.cuda(), norm_w, mws)
        assert torch.isfinite(h[[0, 1, 2, 4]]).all()
        index += (index >= 0).int()
        seq_len += (seq_len >= 0).int()
    assert _lib.moe_read_device_status(ws) == 0 and int(cache.status[0]) == 0
    assert torch.isnan(cache.k[8].float()).all() and torch.isnan(cache.v[10].float()).all()   # row 3's pages


def test_refusals_on_the_device():
    """What the wrappers refuse before a launch (the C entries' own refusals
    are tested without a GPU)."""
    kp, vp = pools(4, 2, 16, 64, True, fill=0.0)
    cache = attention.PagedCache(kp, vp)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    t, n = torch.zeros(2, 1, dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    for bad in (lambda: cache.attend(q.float(), t, n), lambda: cache.attend(q, t.long(), n),
                lambda: cache.attend(q, t, n[:1]), lambda: cache.attend(q.cpu(), t, n),
                lambda: cache.attend(q, t, n, None, 5), lambda: cache.attend(q, t, n, t[0], 17),
                lambda: cache.attend(q[:, :, ::2].repeat(1, 1, 2)[:, :, ::2], t, n),
                lambda: cache.append(q, q[:, :2], q[:, :1], n, n, t, None),
                lambda: cache.append(q, q[:, :2], q[:, :2], n.float(), n, t, None),
                lambda: attention.PagedCache(kp, vp.transpose(1, 2).contiguous().transpose(1, 2)),
                lambda: attention.PagedCache(kp.float(), vp.float())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(_lib.MoEError) as e:
        cache.attend(q[:, :3], t, n)                                     # 3 heads over 2
    assert e.value.code == _lib.MOE_ERR_SHAPE
    with pytest.raises(_lib.MoEError) as e:
        cache.attend(q, t, n, ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == _lib.MOE_ERR_WORKSPACE
