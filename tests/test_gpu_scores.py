"""token_logprobs against a plain implementation in 64 bits.

Tolerance.  With d = x - max and S = sum e^d, e^d is off by |d| 2^-24 (the
difference's rounding) and 2^-21 (the exponential) of itself; |d| e^d <= 0.37, so that
this is below 2^-20 of S + 2^-24 V e^-1, the second again below 2^-24 (1 + the mean of
|d|) S.  The additions, in any order of depth V / 256 + 64, are off by that many 2^-24.
log S, x - max - log S and the entropy log S - (sum e^d d) / S then take a few
roundings of numbers up to |logprob|, log V and |mean d|."""
import math

import pytest
import torch

from int4_grouped_gemm_gb300 import _lib, scores

pytestmark = pytest.mark.gpu

FP32 = 2.0 ** -24


def reference(x, targets, n_top):
    x = x.double()
    lp = torch.log_softmax(x, -1)
    p = lp.exp()
    entropy = -torch.where(p > 0, p * lp, 0.0).sum(-1)
    ids = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :n_top]
    given = None if targets is None else lp.gather(1, targets.long()[:, None])[:, 0]
    return given, entropy, ids, lp.gather(1, ids)


def check(x, targets, n_top, r, rows=None):
    given, entropy, ids, top = reference(x, targets, n_top)
    V = x.shape[1]
    rows = slice(None) if rows is None else rows
    base = (V / 256 + 64 + 16) * FP32 * (2 + entropy)
    if targets is not None:
        tol = base + given.abs() * 4 * FP32
        assert ((r.logprob.double() - given).abs() <= tol)[rows].all()
    assert ((r.entropy.double() - entropy).abs() <= base + entropy.abs() * 4 * FP32)[rows].all()
    assert torch.equal(r.top_ids[rows].long(), ids[rows])
    assert ((r.top_logprobs.double() - top).abs() <= base[:, None] + top.abs() * 4 * FP32)[rows].all()


def make(T, V, seed=0, std=2.5, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty(T, V, device="cuda").normal_(0.0, std, generator=g).to(dtype)
    return x, torch.randint(0, V, (T,), generator=g, device="cuda").to(torch.int32)


SHAPES = [(1, 1, 1), (1, 2, 2), (3, 5, 5), (2, 31, 31), (4, 32, 32), (5, 33, 32), (7, 100, 0), (1, 255, 1), (2, 256, 7),
          (3, 257, 32), (9, 1000, 20), (1, 4096, 5), (1, 131072, 20), (2, 131073, 32), (65, 5003, 8), (300, 777, 3),
          (1000, 64, 2), (17, 50021, 0), (160, 20000, 1), (700, 8192, 10), (4, 1 << 20, 32)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("T,V,n_top", SHAPES)
def test_scores_against_64_bits(T, V, n_top, dtype):
    x, targets = make(T, V, T + V, dtype=dtype)
    ws = scores.workspace(T, V, n_top)
    r = scores.token_logprobs(x, targets, n_top, ws=ws)
    assert _lib.moe_read_device_status(ws) == 0
    check(x, targets, n_top, r)
    again = scores.token_logprobs(x, targets, n_top, ws=ws)
    assert all(torch.equal(a, b) for a, b in zip(r, again))


@pytest.mark.parametrize("offset,stride", [(0, 1003), (1, 1001), (2, 1002), (3, 1007), (1, 1024), (5, 1009)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_scores_of_strided_and_unaligned_rows(offset, stride, dtype):
    """Columns of a wider tensor; what lies either side is NaN."""
    V, T = 1000, 9
    wide = torch.full((T, stride + 8), float("nan"), device="cuda", dtype=dtype)
    x, targets = make(T, V, 3, dtype=dtype)
    wide.view(-1)[:T * stride + offset + V].as_strided((T, V), (stride, 1), offset).copy_(x)
    view = wide.view(-1).as_strided((T, V), (stride, 1), offset)
    check(x, targets, 12, scores.token_logprobs(view, targets, 12))


@pytest.mark.parametrize("order", ["up", "down", "equal", "two values"])
@pytest.mark.parametrize("T,V", [(3, 40000), (1, 131072), (400, 3000)])
def test_scores_in_order_and_equal(order, T, V):
    """Rising scores (every one a new alternative), falling ones, and ties,
    which go to the lower id."""
    i = torch.arange(V, device="cuda", dtype=torch.float32)
    row = {"up": i / V, "down": -i / V, "equal": torch.full_like(i, 0.5), "two values": (i % 7 == 3).float()}[order]
    x = row.expand(T, V).contiguous()
    targets = torch.full((T,), V // 2, dtype=torch.int32, device="cuda")
    check(x, targets, 32, scores.token_logprobs(x, targets, 32))


def test_scores_zeros_of_both_signs_are_equal():
    x = torch.zeros(1, 300, device="cuda")
    x[0, ::2] = -0.0
    r = scores.token_logprobs(x, None, 5)
    assert r.logprob is None and r.top_ids[0].tolist() == [0, 1, 2, 3, 4]


@pytest.mark.parametrize("T,V", [(1, 131072), (6, 5003), (300, 2000)])
def test_scores_of_masked_tokens(T, V):
    """Minus infinity weighs nothing; one token left: log probability 0, entropy 0;
    scores of the type's lowest value; none left: NaN, ids from the lowest on."""
    x, targets = make(T, V, 9)
    x[:, 1::2] = -math.inf
    r = scores.token_logprobs(x, targets, 4)
    check(x, None, 4, r._replace(logprob=None))
    odd = targets % 2 == 1
    assert (r.logprob[odd] == -math.inf).all() and torch.isfinite(r.logprob[~odd]).all()
    # fewer finite scores than alternatives
    x = torch.full((T, V), -math.inf, device="cuda")
    x[:, 17], x[:, 1003] = 3.0, 3.0
    r = scores.token_logprobs(x, torch.full_like(targets, 17), 6)
    assert r.top_ids.tolist() == [[17, 1003, 0, 1, 2, 3]] * T
    assert (r.top_logprobs[:, 2:] == -math.inf).all() and (r.logprob + math.log(2)).abs().max() < 1e-6
    x[:, 1003] = -math.inf
    r = scores.token_logprobs(x, torch.full_like(targets, 17), 1)
    assert (r.logprob == 0).all() and (r.entropy == 0).all()
    low = torch.finfo(torch.float32).min
    x = torch.full((T, V), low, device="cuda")
    x[:, 5] = 1.0
    r = scores.token_logprobs(x, torch.full_like(targets, 5), 2)
    assert (r.logprob == 0).all() and (r.entropy == 0).all() and r.top_ids.tolist() == [[5, 0]] * T
    x[:, 5] = low
    r = scores.token_logprobs(x, torch.full_like(targets, 5), 2)
    assert (r.logprob + math.log(V)).abs().max() < 1e-4 and (r.entropy - math.log(V)).abs().max() < 1e-4
    r = scores.token_logprobs(torch.full((T, V), -math.inf, device="cuda"), targets, 3)
    assert torch.isnan(r.logprob).all() and torch.isnan(r.entropy).all() and torch.isnan(r.top_logprobs).all()
    assert r.top_ids.tolist() == [[0, 1, 2]] * T


@pytest.mark.parametrize("T,V", [(2, 131072), (5, 700), (300, 2000)])
def test_scores_not_finite(T, V):
    """A NaN or an infinity leaves its row without numbers, and the others alone."""
    x, targets = make(T, V, 10)
    want = scores.token_logprobs(x, targets, 5)
    for bad in (math.nan, -math.nan, math.inf):
        y = x.clone()
        y[1, V - 3] = bad
        r = scores.token_logprobs(y, targets, 5)
        assert torch.isnan(r.logprob[1]) and torch.isnan(r.entropy[1]) and torch.isnan(r.top_logprobs[1]).all()
        assert int(r.top_ids[1, 0]) == V - 3 and torch.equal(r.top_ids[1, 1:], want.top_ids[1, :4])
        keep = torch.arange(T, device="cuda") != 1
        assert all(torch.equal(a[keep], b[keep]) for a, b in zip(r, want))


def test_scores_far_apart_and_large():
    x = torch.tensor([[1e30, -1e30, 0.0], [3e38, 3e38, -3e38], [-1e30, -1e30, -1e30], [1e-40, 0.0, -1e-40]], device="cuda")
    r = scores.token_logprobs(x, torch.tensor([0, 0, 2, 1], dtype=torch.int32, device="cuda"), 3)
    assert (r.logprob.cpu() - torch.tensor([0.0, -math.log(2), -math.log(3), -math.log(3)])).abs().max() < 1e-6
    assert (r.entropy.cpu() - torch.tensor([0.0, math.log(2), math.log(3), math.log(3)])).abs().max() < 1e-6
    assert r.top_ids.tolist() == [[0, 2, 1], [0, 1, 2], [0, 1, 2], [0, 1, 2]]


@pytest.mark.parametrize("T,V", [(6, 131072), (400, 1000)])
def test_scores_padding_and_targets_outside(T, V):
    x, targets = make(T, V, 11)
    want = scores.token_logprobs(x, targets, 4)
    targets[0], targets[3] = -1, -(2 ** 31)
    x[3] = math.nan
    out = scores.TokenScores.empty(T, 4)
    for t in out:
        t.fill_(7)
    ws = scores.workspace(T, V, 4)
    scores.token_logprobs(x, targets, 4, out=out, ws=ws)
    assert _lib.moe_read_device_status(ws) == 0
    pad = torch.zeros(T, dtype=torch.bool, device="cuda")
    pad[0] = pad[3] = True
    for a, b in zip(out, want):
        assert (a[pad] == 7).all() and torch.equal(a[~pad], b[~pad])
    for bad in (V, 2 ** 31 - 1):
        targets[1] = bad
        scores.token_logprobs(x, targets, 4, out=out, ws=ws)
        assert _lib.moe_read_device_status(ws) == _lib.MOE_ERR_TOKEN_ID
        assert torch.isnan(out.logprob[1]) and torch.equal(out.top_ids[1], want.top_ids[1])
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        scores.token_logprobs(x, targets, 4, out=out, status=status)
        assert int(status) == _lib.MOE_ERR_TOKEN_ID


def test_scores_on_streams_and_replayed():
    x, targets = make(3, 60000, 12)
    want = scores.token_logprobs(x, targets, 10)
    outs = [scores.TokenScores.empty(3, 10) for _ in range(2)]
    wss = [scores.workspace(3, 60000, 10) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, ws, out in zip(streams, wss, outs):
            scores.token_logprobs(x, targets, 10, out=out, ws=ws, stream=s)
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        scores.token_logprobs(x, targets, 10, out=outs[0], ws=wss[0])
    y, _ = make(3, 60000, 13)
    x.copy_(y)
    targets.add_(1).remainder_(60000)
    graph.replay()
    torch.cuda.synchronize()
    check(x, targets, 10, outs[0])
