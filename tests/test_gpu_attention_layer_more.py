"""More of the attention sub-layer on the GPU: the many-token linear where its token
sums do not all have a place, several tiles a block, two calls at once, and
device-side waits that run out."""
import pytest
import torch

from int4_grouped_gemm_gb300 import _lib, attention, moe

pytestmark = pytest.mark.gpu

BF16 = torch.finfo(torch.bfloat16).eps / 2
FP32 = torch.finfo(torch.float32).eps / 2


def case(B, K, N, G, seed):
    """Weights and tokens on the GPU, and the weights' exact values in fp64."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randint(0, 16, (N, K), generator=g, device="cuda", dtype=torch.int32)
    words = torch.zeros(N, K // 8, device="cuda", dtype=torch.int32)
    for e in range(8):
        words |= q[:, e::8] << (4 * (e // 2 + 4 * (e % 2)))
    pitch = moe.ld_groups(K, G)
    s = (torch.rand(N, K // G, generator=g, device="cuda") * 0.01 + 0.001).to(torch.bfloat16)
    z = (torch.randn(N, K // G, generator=g, device="cuda") * 0.03).to(torch.bfloat16)
    # what stands in the padding of the rows of scales does not matter to more than eight tokens
    sp = torch.full((N, pitch), float("nan"), dtype=torch.bfloat16, device="cuda")
    zp = torch.full((N, pitch), float("nan"), dtype=torch.bfloat16, device="cuda")
    sp[:, :K // G], zp[:, :K // G] = s, z
    w = q.double() * s.double().repeat_interleave(G, 1) + z.double().repeat_interleave(G, 1)
    x = torch.randn(B, K, generator=g, device="cuda").to(torch.bfloat16)
    return moe.QMatrix(words, sp.view(torch.int16), zp.view(torch.int16), N, K, G), w, x


def bound(x, w, K):
    """The fp32 error of y in the worst case: code products q x are summed per
    group (|s q x| <= 0.011 * 15 |x|), biases times the groups' token sums apart
    from them (|z x|, z below 0.2; the sums as three bf16 parts, off by 2^-25 of
    themselves), so |s q x| + |z x| <= |w x| + 2 |z x| enters K / 16 + 64
    rounded additions (products of 16, then groups, warps and blocks)."""
    mag = x.abs().double() @ w.abs().t() + 2 * 0.2 * x.abs().double().sum(1, keepdim=True)
    return mag * (K / 16 + 64) * FP32


@pytest.mark.parametrize("B, K, N, G", [
    (12, 4224, 19500, 32),    # 132 groups: more chunks of token sums than places, two tiles on some blocks
    (33, 4224, 19500, 32),
    (20, 16640, 8600, 128),   # 130 groups of 128
    (64, 8320, 8600, 64),     # 130 groups of 64
    (9, 256, 40000, 32),      # one chunk, three tiles a block
    (48, 4096, 20000, 64),    # four chunks, kept from the first tile on
    (16, 96, 20001, 32),      # half a step
])
def test_linear_many_tiles_and_chunks(B, K, N, G):
    m, w, x = case(B, K, N, G, B + K + N)
    want = x.double() @ w.t()
    err = bound(x, w, K)
    assert float(w.abs().max()) < 0.011 * 15 + 0.2
    y = moe.linear(m, x, dtype=torch.float32)
    assert ((y.double() - want).abs() <= err).all()
    y16 = moe.linear(m, x)
    assert ((y16.double() - want).abs() <= err * (1 + BF16) + want.abs() * BF16).all()
    # the same again, from a graph too
    graph = torch.cuda.CUDAGraph()
    z = torch.empty_like(y)
    with torch.cuda.graph(graph):
        moe.linear(m, x, z)
    graph.replay()
    assert torch.equal(y, z)


@pytest.mark.parametrize("B", [4, 40])
def test_linear_on_two_streams_at_once(B):
    cases = [case(B, 1024, 3000, 64, s) for s in (1, 2)]
    want = [moe.linear(m, x, dtype=torch.float32) for m, _, x in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (m, _, x) in enumerate(cases):
            got[i].append(moe.linear(m, x, dtype=torch.float32, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(want[i], y) for y in got[i])


def test_a_wait_that_runs_out_is_recorded_and_harmless():
    """With a limit of one cycle the kernels' waits may run out (a try has a time
    of its own, so they need not): then the status says so.  Either way the block
    ends, and the next call is right."""
    m, w, x = case(40, 2048, 3000, 64, 5)
    want = moe.linear(m, x, dtype=torch.float32)
    cache = attention.PagedCache.empty(64, 2, 64, 128)
    cache.k.normal_()
    cache.v.normal_()
    q = torch.randn(16, 16, 128, device="cuda").to(torch.bfloat16)
    table = torch.arange(32, device="cuda", dtype=torch.int32).view(16, 2)
    prefix = torch.arange(32, 64, device="cuda", dtype=torch.int32)
    lens = torch.full((16,), 100, device="cuda", dtype=torch.int32)
    ws = cache.workspace(16, 16, 2000)
    out = cache.attend(q, table, lens, prefix, 2000, ws=ws)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    old = _lib.moe_set_wait_limit(1)
    try:
        y = moe.linear(m, x, dtype=torch.float32, status=status)
        out1 = cache.attend(q, table, lens, prefix, 2000, ws=ws)
        torch.cuda.synchronize()
    finally:
        _lib.moe_set_wait_limit(old)
    code = int(status)
    assert code == 0 and torch.equal(y, want) or code <= _lib.MOE_ERR_TIMEOUT
    code = _lib.moe_read_device_status(ws)
    assert code == 0 and torch.equal(out1, out) or code <= _lib.MOE_ERR_TIMEOUT
    _lib.moe_workspace_init(ws)
    assert torch.equal(moe.linear(m, x, dtype=torch.float32), want)
    assert torch.equal(cache.attend(q, table, lens, prefix, 2000, ws=ws), out)


@pytest.mark.parametrize("B, K, N, G", [(9, 32, 40, 32), (64, 32, 3, 32), (17, 32, 1, 32), (33, 64, 7, 64), (64, 64, 200, 32),
                                        (12, 128, 5, 128), (64, 128, 1, 64), (25, 128, 129, 128), (16, 160, 64, 32),
                                        (10, 32768, 8, 128), (64, 32768, 130, 32)])
def test_linear_smallest_and_longest_k(B, K, N, G):
    """One group of k, rows fewer than a box of any load, the longest k."""
    m, w, x = case(B, K, N, G, 3 * B + K + N)
    want = x.double() @ w.t()
    y = moe.linear(m, x, dtype=torch.float32)
    assert ((y.double() - want).abs() <= bound(x, w, K)).all()


def test_append_ragged_numbers_of_heads():
    """Blocks whose items are not a multiple of the threads' two in flight, rotated
    in place: against the rotation in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(9)
    for T, Hq, Hkv, D, rot, inter in ((2500, 3, 1, 64, 48, False), (1300, 40, 5, 128, 128, True), (5000, 7, 7, 64, 16, True),
                                      (700, 255, 1, 64, 64, False)):
        n_pages = (T + 63) // 64
        cache = attention.PagedCache.empty(n_pages, Hkv, 64, D)
        cache.k.fill_(7.0)
        cache.v.fill_(7.0)
        q, k, v = (torch.randn(T, h, D, generator=g, device="cuda").to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
        table = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32).view(1, -1)
        index = torch.randperm(T, generator=g, device="cuda").to(torch.int32)
        freq = 10000.0 ** (-torch.arange(rot // 2, device="cuda") / (rot // 2))
        ang = (index.double() + 5)[:, None, None] * freq.double()

        def turned(x):
            x = x.double()
            a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
            c, s = a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()
            y = x.clone()
            if inter:
                y[..., 0:rot:2], y[..., 1:rot:2] = c, s
            else:
                y[..., :rot // 2], y[..., rot // 2:rot] = c, s
            return y
        want_q, want_k = turned(q), turned(k)
        out = cache.append(q, k, v, torch.zeros(T, dtype=torch.int32, device="cuda"), index, table, freq, 5, inter, q_out=q)
        assert out is q
        pages, off = table[0, index.long() // 64].long(), index.long() % 64
        # cos and sin off by 2^-22 at most (angle and function in fp32), two
        # products and a sum, then the rounding to bf16
        for got, want in ((q, want_q), (cache.k[pages, :, off], want_k)):
            mag = 12.0 * (2.0 ** -21 + 4 * FP32)       # of |a| + |b| <= 12: six deviations each
            assert ((got.double() - want).abs() <= want.abs() * BF16 * 1.01 + mag).all()
        assert torch.equal(cache.v[pages, :, off], v)


@pytest.mark.parametrize("B, K, N, G", [
    (1, 512, 6000, 64), (3, 512, 9700, 32), (8, 2048, 2500, 64), (8, 2080, 5000, 32),     # two tiles of rows a block
    (1, 256, 12000, 128), (5, 1024, 11111, 64), (7, 4096, 5100, 64),                      # four
    (8, 8192, 2000, 64), (3, 32768, 2600, 128), (8, 32768, 131, 64),                      # tokens in chunks; K in a cluster
    (6, 1056, 16, 32), (8, 128, 1, 128),
])
def test_linear_few_tokens_tiles_and_shares(B, K, N, G):
    m, w, x = case(B, K, N, G, B + K + N)
    # (the padding of the rows of scales holds zeros here, as pack_int4 leaves it)
    for t in (m.scale, m.bias):
        t[:, K // G:] = 0
    x[B // 2] *= 2.0 ** -60      # tokens of different magnitude, and one that grows along k
    x[-1] = (x[-1].double() * 2.0 ** torch.linspace(-20, 0, K, device="cuda").double()).to(torch.bfloat16)
    want = x.double() @ w.t()
    err = bound(x, w, K)
    # tokens as fp16: an element below 2^-31 of the largest is off by 2^-40 of that
    err = err + x.abs().double().max(1, keepdim=True).values * 2.0 ** -40 * w.abs().sum(1)
    y = moe.linear(m, x, dtype=torch.float32)
    assert ((y.double() - want).abs() <= err).all()
    assert torch.equal(y, moe.linear(m, x, dtype=torch.float32))


@pytest.mark.parametrize("B", [1, 2, 30, 31, 32, 33, 255, 256, 257, 1023, 1024])
@pytest.mark.parametrize("prefix", [0, 40])
def test_attend_numbers_of_rows(B, prefix):
    """Row counts at which the rows' tiles are counted another way, with rows that
    are empty, padding, or full."""
    g = torch.Generator(device="cuda").manual_seed(B + prefix)
    Hq, Hkv, D, page, ld = 4, 2, 64, 16, 3
    cache = attention.PagedCache.empty(B * ld + 3, Hkv, page, D)
    cache.k.copy_(torch.randn(cache.k.shape, generator=g, device="cuda"))
    cache.v.copy_(torch.randn(cache.v.shape, generator=g, device="cuda"))
    pages = torch.randperm(B * ld + 3, generator=g, device="cuda").to(torch.int32)
    table, shared = pages[:B * ld].view(B, ld), pages[B * ld:]
    lens = torch.randint(-1, ld * page + 1, (B,), generator=g, device="cuda").to(torch.int32)
    lens[-1] = ld * page if B % 2 else -1
    lens[0] = 0 if B % 3 else lens[0]
    q = torch.randn(B, Hq, D, generator=g, device="cuda").to(torch.bfloat16)
    out = torch.full_like(q, 9.0)
    cache.attend(q, table, lens, shared if prefix else None, prefix, out=out)
    assert int(cache.status[0]) == 0

    def gather(pool, t):  # [.., n pages] -> [.., Hkv, positions, D]
        return pool[t.long()].transpose(-4, -3).flatten(-3, -2).double()
    k, v = gather(cache.k, table), gather(cache.v, table)
    s = torch.einsum("bgrd,bgnd->bgrn", q.double().view(B, Hkv, 2, D), k) / D ** 0.5
    s = s.masked_fill(torch.arange(ld * page, device="cuda") >= lens.view(B, 1, 1, 1), -float("inf"))
    if prefix:
        pk, pv = gather(cache.k, shared)[:, :prefix], gather(cache.v, shared)[:, :prefix]
        sp = torch.einsum("bgrd,gnd->bgrn", q.double().view(B, Hkv, 2, D), pk) / D ** 0.5
        s, v = torch.cat((sp, s), -1), torch.cat((pv.expand(B, -1, -1, -1), v), 2)
    p = s.softmax(-1).nan_to_num(0.0)
    want = torch.einsum("bgrn,bgnd->bgrd", p, v).reshape(B, Hq, D)
    # weights rounded to bf16, each 2^-8 of itself at most, a hundredth more for the
    # fp32 arithmetic; then the output's rounding
    tol = BF16 * 1.01 * (torch.einsum("bgrn,bgnd->bgrd", p, v.abs()).reshape(B, Hq, D) * 2 + want.abs()) + 1e-6
    real = lens >= 0
    assert ((out.double() - want).abs() <= tol)[real].all()
    assert (out[~real] == 9.0).all()
    assert prefix or (out[lens == 0] == 0).all()


def test_the_c_calls_of_the_binding_agree_with_the_helpers():
    """The calls under their C names on raw descriptors, as for the other operators."""
    m, _, x = case(5, 512, 300, 64, 1)
    m.scale[:, 8:] = 0
    y = torch.empty(5, 300, device="cuda")
    _lib.int4_linear(m.as_c(), 300, 512, 64, x, y)
    assert torch.equal(y, moe.linear(m, x, dtype=torch.float32))
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = (torch.randn(4, h, 64, generator=g, device="cuda").to(torch.bfloat16) for h in (6, 2, 2))
    seq = torch.arange(4, dtype=torch.int32, device="cuda")
    index = torch.tensor([0, 5, 17, 31], dtype=torch.int32, device="cuda")
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2)
    shared = torch.tensor([8, 9], dtype=torch.int32, device="cuda")
    freq = 100.0 ** (-torch.arange(16, device="cuda") / 16)
    results = []
    for raw in (False, True):
        cache = attention.PagedCache.empty(10, 2, 16, 64)
        cache.k.copy_(torch.randn(cache.k.shape, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda"))
        cache.v.copy_(cache.k * 2)
        turned, out = torch.empty_like(q), torch.empty_like(q)
        if raw:
            _lib.gqa_append(cache.desc, q, k, v, seq, index, table, 20, freq, True, turned, cache.status)
            ws = torch.zeros(_lib.gqa_paged_workspace_bytes(4, 6, 2, 64, 20), dtype=torch.uint8, device="cuda")
            _lib.gqa_paged_attention(cache.desc, turned, shared, 20, table, index + 1, 0.125, out, ws)
        else:
            cache.append(q, k, v, seq, index, table, freq, 20, True, q_out=turned)
            cache.attend(turned, table, index + 1, shared, 20, out=out)
        results.append((turned, cache.k, cache.v, out))
    for a, b in zip(*results):
        assert torch.equal(a, b)
