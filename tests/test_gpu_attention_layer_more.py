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
