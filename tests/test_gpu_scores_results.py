"""What token_logprobs and OutputHead return for padding rows where the caller gives
no results to write to."""
import pytest
import torch

from int4_grouped_gemm_gb300 import scores
from test_gpu_attention_layer import gen, make_int4, randn

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


def leave_sevens(*sizes):
    """Memory that the next allocations of these sizes get holds 7s."""
    held = [torch.full((n,), 7, **I32) for n in sizes for _ in range(4)]
    torch.cuda.synchronize()
    del held


def check_padding(r, pad):
    assert torch.isnan(r.logprob[pad]).all() and torch.isnan(r.entropy[pad]).all()
    assert (r.top_ids[pad] == -1).all() and torch.isnan(r.top_logprobs[pad]).all()


@pytest.mark.parametrize("n_top", [0, 6])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("T,V", [(1, 7), (2, 131072), (5, 5003), (300, 1000), (330, 3000), (400, 6000), (700, 20000)])
def test_padding_of_results_that_the_call_makes(T, V, dtype, n_top):
    x = torch.randn(T, V, generator=torch.Generator(device="cuda").manual_seed(T), device="cuda").to(dtype)
    targets = torch.randint(0, V, (T,), **I32)
    want = scores.token_logprobs(x, targets, n_top)
    pad = torch.arange(T, device="cuda") % 3 == 0
    targets[pad] = -5
    leave_sevens(T, T * n_top)
    for ws in (None, scores.workspace(T, V, n_top)):
        r = scores.token_logprobs(x, targets, n_top, ws=ws)
        check_padding(r, pad)
        assert all(torch.equal(a[~pad], b[~pad]) for a, b in zip(r, want))
    # results of the caller's own keep what they hold
    out = scores.TokenScores.empty(T, n_top)
    for t in out:
        t.fill_(7)
    scores.token_logprobs(x, targets, n_top, out=out)
    for a, b in zip(out, want):
        assert (a[pad] == 7).all() and torch.equal(a[~pad], b[~pad])


@pytest.mark.parametrize("rows", [1024, 30])
def test_padding_of_a_head(rows):
    m, _ = make_int4(gen(1), 700, 256, 64)
    head = scores.OutputHead(m, rows=rows)
    x = randn(gen(2), 100, 256).cuda()
    targets = torch.randint(0, 700, (100,), **I32)
    want = head.logprobs(x, targets, 4)
    pad = torch.arange(100, device="cuda") % 7 == 2
    targets[pad] = -1
    leave_sevens(100, 400)
    r = head.logprobs(x, targets, 4)
    check_padding(r, pad)
    assert all(torch.equal(a[~pad], b[~pad]) for a, b in zip(r, want))
