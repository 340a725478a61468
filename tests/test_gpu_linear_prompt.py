"""int4_linear_prompt (any number of tokens) against a plain implementation in 64
bits.

Tolerance.  Products of tokens and weights are exact; a result is a sum of them in
fp32.  Whichever way the weights s q + z are split into terms (codes and biases
apart, codes around their middle 8), the terms' magnitudes are at most |x| (16 s + |z|)
in all; additions in any order of depth K / 16 + 64, each off by up to 2^-23 of the
running magnitude (the tensor core cuts off where a rounding would be half of that),
and parts of biases and token sums of at least 22 bits."""
import pytest
import torch

from int4_grouped_gemm_gb300 import _lib, moe, synthetic
from test_gpu_attention_layer import gen, make_int4, randn

pytestmark = pytest.mark.gpu

BF16 = torch.finfo(torch.bfloat16).eps / 2


def bound(x, w, K, s_max=0.011):
    mag = x.abs().double().sum(1, keepdim=True) * 16 * s_max + x.abs().double() @ w.abs().t()
    return mag * ((K / 16 + 64) * 2.0 ** -23 + 2.0 ** -20)


CASES = [  # T, K, N, group
    (1, 32, 1, 32), (2, 64, 7, 64), (65, 128, 16, 128), (64, 96, 17, 32), (127, 2048, 160, 64), (128, 2080, 33, 32),
    (129, 192, 129, 64), (200, 1152, 250, 128), (255, 256, 64, 64), (256, 160, 515, 32), (257, 1024, 272, 64),
    (1000, 4224, 31, 128), (70, 32768, 24, 64), (90, 8192, 40, 32), (65, 2048, 2560, 64), (333, 4096, 20000, 128),
    (2500, 512, 700, 64), (20000, 64, 40, 32), (130, 128, 40000, 64), (4096, 32, 257, 32),
]


@pytest.mark.parametrize("fp32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,K,N,G", CASES)
def test_linear_prompt_against_64_bits(T, K, N, G, fp32):
    g = gen(T * 7 + K + N)
    m, w = make_int4(g, N, K, G)
    w = w.cuda()
    x = randn(g, T, K).cuda()
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = moe.linear_prompt_workspace(m, T)
    dtype = torch.float32 if fp32 else torch.bfloat16
    got = moe.linear_prompt(m, x, dtype=dtype, ws=ws, status=status)
    assert _lib.moe_read_device_status(status) == 0
    want = x.double() @ w.t()
    tol = bound(x, w, K) + (0 if fp32 else want.abs() * BF16 * 1.01)
    err = (got.double() - want).abs()
    assert (err <= tol).all(), float((err - tol).max())
    # in the norm of a token far below the worst case: 2^-24 sqrt(depth) a sum, and the rounding to bf16
    rel = (got.double() - want).norm() / want.norm()
    assert rel <= (2e-6 if fp32 else 2e-6 + BF16 / 3 ** 0.5)
    assert torch.equal(got, moe.linear_prompt(m, x, dtype=dtype, ws=ws))


def test_linear_prompt_strided_rows_and_untouched_neighbours():
    g = gen(5)
    m, w = make_int4(g, 77, 320, 64)
    xb = torch.full((150, 320 + 48), float("nan"), dtype=torch.bfloat16)
    xb[:, 16:336] = randn(g, 150, 320)
    want = xb[:, 16:336].double() @ w.t()
    for dtype in (torch.bfloat16, torch.float32):
        for width, at in ((100, 8), (101, 3), (85, 8)):
            yb = torch.full((150, width), 3.0, dtype=dtype, device="cuda")
            # (y starts on a 16-byte boundary: a whole number of them into its buffer)
            at = at // 8 * 8
            moe.linear_prompt(m, xb.cuda()[:, 16:336], yb[:, at:at + 77])
            got = yb.cpu().double()
            assert (got[:, :at] == 3).all() and (got[:, at + 77:] == 3).all()
            assert ((got[:, at:at + 77] - want).abs() <= bound(xb[:, 16:336], w, 320) + want.abs() * BF16 * 1.01).all()


@pytest.mark.parametrize("top", [1e-38, 1e-20, 1e15])
def test_linear_prompt_tokens_of_any_magnitude(top):
    """Tokens whose largest element is tiny, huge or subnormal, each row another,
    and rows that span 30 binary orders."""
    g = gen(50)
    m, w = make_int4(g, 40, 128, 32)
    x = randn(g, 140, 128).double()
    x = x / x.abs().max(1, keepdim=True).values * top
    x[:, ::3] *= 2.0 ** -15
    x[:, 1::3] *= 2.0 ** -30
    x[5] = 0
    x = x.to(torch.bfloat16)
    got = moe.linear_prompt(m, x.cuda(), dtype=torch.float32).cpu().double()
    want = x.double() @ w.t()
    tol = bound(x, w, 128) + x.abs().double().max(1, keepdim=True).values * 2.0 ** -39 * w.abs().sum(1) + 1e-43
    assert ((got - want).abs() <= tol).all()
    assert (got[5] == 0).all()


@pytest.mark.parametrize("size", [2.0 ** -80, 2.0 ** 80])
def test_linear_prompt_weights_of_any_magnitude(size):
    """Scales and biases far from one, each row another power, and groups of one
    row that span 20 binary orders."""
    g = gen(51)
    m, w = make_int4(g, 48, 256, 32)
    s, z = (t.view(torch.bfloat16).double().cpu() for t in (m.scale, m.bias))
    f = size * 2.0 ** (torch.arange(48) % 5 - 2).double()[:, None] * torch.ones(1, 8, dtype=torch.float64)
    f[:, 3] *= 2.0 ** -20
    s[:, :8] *= f
    z[:, :8] *= f
    m = moe.QMatrix(m.q, s.to(torch.bfloat16).view(torch.int16).cuda(), z.to(torch.bfloat16).view(torch.int16).cuda(), 48, 256, 32)
    w = w * f.repeat_interleave(32, 1)
    x = randn(g, 100, 256)
    got = moe.linear_prompt(m, x.cuda(), dtype=torch.float32).cpu().double()
    want = x.double() @ w.t()
    mag = x.abs().double() @ (16 * 0.011 * f.repeat_interleave(32, 1) + w.abs()).t()
    tol = mag * ((256 / 16 + 64) * 2.0 ** -23 + 2.0 ** -20) + x.abs().double().sum(1, keepdim=True) * f.max(1).values * 2.0 ** -30
    assert ((got - want).abs() <= tol).all()


@pytest.mark.parametrize("T", [3, 129, 300])
def test_linear_prompt_a_broken_token_stays_alone(T):
    g = gen(40 + T)
    m, w = make_int4(g, 150, 256, 64)
    x = randn(g, T, 256).cuda()
    want = moe.linear_prompt(m, x, dtype=torch.float32)
    for bad in (float("nan"), float("inf"), -float("inf")):
        broken = x.clone()
        broken[T // 2, 17] = bad
        got = moe.linear_prompt(m, broken, dtype=torch.float32)
        assert not torch.isfinite(got[T // 2]).any()
        keep = torch.arange(T, device="cuda") != T // 2
        assert torch.equal(got[keep], want[keep])


def test_linear_prompt_agrees_with_linear():
    """The calls for few and for many tokens give the same up to their sums."""
    g = gen(60)
    m, w = make_int4(g, 700, 1024, 64)
    x = randn(g, 64, 1024)
    a = moe.linear(m, x.cuda(), dtype=torch.float32).cpu().double()
    b = moe.linear_prompt(m, x.cuda(), dtype=torch.float32).cpu().double()
    assert ((a - b).abs() <= 2 * bound(x, w, 1024)).all()


def test_linear_prompt_of_packed_weights_on_streams_and_replayed():
    w = synthetic.make_weight_matrix(520, 512, seed=3, device="cuda")
    m = moe.pack_matrix(w, 64)
    x = synthetic.make_tokens(512, 300, seed=4, device="cuda")
    want = moe.linear_prompt(m, x)
    ref = x.double() @ w.double().t()
    # 15 steps over a group's range: |w - packed| <= half a step plus the bf16 rounding of scale and bias
    assert (want.double() - ref).abs().max() < 0.1 * ref.abs().max()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(want) for _ in range(2)]
    wss = [moe.linear_prompt_workspace(m, 300) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, ws, y in zip(streams, wss, outs):
            moe.linear_prompt(m, x, y, ws=ws, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.linear_prompt(m, x, outs[0], ws=wss[0])
    x2 = synthetic.make_tokens(512, 300, seed=5, device="cuda")
    x.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], moe.linear_prompt(m, x2))


def test_linear_prompt_smaller_call_in_a_larger_workspace():
    g = gen(61)
    m, w = make_int4(g, 130, 256, 64)
    ws = moe.linear_prompt_workspace(m, 1000)
    for T in (1000, 66, 513, 1):
        x = randn(g, T, 256)
        got = moe.linear_prompt(m, x.cuda(), dtype=torch.float32, ws=ws).cpu().double()
        assert ((got - x.double() @ w.t()).abs() <= bound(x, w, 256)).all()


@pytest.mark.parametrize("T,K,N,G", [(130, 96, 440000, 32), (257, 64, 330000, 64), (700, 1152, 40000, 128),
                                     (129, 2080, 20000, 32), (2048, 256, 131000, 64), (300, 4096, 10300, 128),
                                     (2049, 576, 70000, 64), (150, 32, 330100, 32)])
def test_linear_prompt_of_large_matrices(T, K, N, G):
    """More fp16 weights than are held at a time: unpacked by the product's kernel for
    up to 2048 tokens, in pieces of rows for more; few and odd numbers of steps."""
    g = torch.Generator(device="cuda").manual_seed(T + N)
    codes = torch.randint(-2 ** 31, 2 ** 31, (N, K // 8), generator=g, device="cuda", dtype=torch.int32)
    s = (torch.rand(N, K // G, generator=g, device="cuda") * 0.01 + 0.001).to(torch.bfloat16)
    z = (torch.randn(N, K // G, generator=g, device="cuda") * 0.03).to(torch.bfloat16)
    pad = (0, moe.ld_groups(K, G) - K // G)
    m = moe.QMatrix(codes, torch.nn.functional.pad(s, pad).view(torch.int16), torch.nn.functional.pad(z, pad).view(torch.int16),
                    N, K, G)
    x = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    got = moe.linear_prompt(m, x, dtype=torch.float32, status=status)
    assert _lib.moe_read_device_status(status) == 0
    assert torch.equal(got, moe.linear_prompt(m, x, dtype=torch.float32))
    # rows here and there, and the last ones
    rows = torch.cat((torch.arange(0, N, 997), torch.arange(max(0, N - 600), N))).cuda()
    words = codes[rows].long() & 0xFFFFFFFF
    q = torch.empty(len(rows), K, dtype=torch.float64, device="cuda")
    for e in range(8):
        q[:, e::8] = ((words >> (4 * (e // 2 + 4 * (e % 2)))) & 15).double()
    w = q * s[rows].double().repeat_interleave(G, 1) + z[rows].double().repeat_interleave(G, 1)
    want = x.double() @ w.t()
    assert ((got[:, rows].double() - want).abs() <= bound(x, w, K)).all()


@pytest.mark.parametrize("T,K,N,G", [(65, 2048, 8192, 64), (1024, 2048, 8192, 64), (1025, 2048, 8192, 64),
                                     (300, 1056, 16001, 32), (1281, 2048, 10000, 128)])
def test_linear_prompt_of_middling_matrices(T, K, N, G):
    """Around the number of tokens up to which the product's kernel unpacks."""
    test_linear_prompt_of_large_matrices(T, K, N, G)


def test_linear_prompt_workspace_of_more_tokens_serves_fewer():
    m, _ = make_int4(gen(71), 16384, 2048, 64)
    sizes = [moe.linear_prompt_workspace(m, T).numel() for T in (1, 64, 65, 1000, 1024, 1025, 2047, 2048, 2049, 5000)]
    assert sizes == sorted(sizes)
