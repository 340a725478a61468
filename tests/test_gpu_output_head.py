"""OutputHead: its pieces share their scratch, its errors are kept."""
import math

import pytest
import torch

from int4_grouped_gemm_gb300 import _lib, moe, scores
from test_gpu_attention_layer import gen, make_int4, randn

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("T", [1, 70, 200, 401])
def test_a_head_makes_scratch_once(T):
    """... whatever is left for its last piece."""
    m, _ = make_int4(gen(4), 600, 256, 64)
    head = scores.OutputHead(m, rows=100)
    x = randn(gen(5), T, 256).cuda()
    targets = torch.randint(0, 600, (T,), dtype=torch.int32, device="cuda")
    want = scores.token_logprobs(moe.linear_prompt(m, x, dtype=torch.float32), targets, 3)

    def made():
        torch.cuda.synchronize()
        before = torch.cuda.memory_stats()["allocation.all.allocated"]
        got = head.logprobs(x, targets, 3)
        return torch.cuda.memory_stats()["allocation.all.allocated"] - before, got

    count, got = made()
    for a, b in zip(got, want):
        assert torch.allclose(a, b, rtol=0, atol=1e-3) if a.dtype == torch.float32 else a.shape == b.shape
    # four results, scores, the linear's scratch and that of the scores
    assert count <= 7


def test_errors_of_a_head_are_kept():
    """Without a status of the caller's they go to the head's own."""
    m, _ = make_int4(gen(3), 500, 256, 64)
    head = scores.OutputHead(m, rows=40)
    x = randn(gen(4), 90, 256).cuda()
    targets = torch.randint(0, 500, (90,), **I32)
    head.logprobs(x, targets, 2)
    assert _lib.moe_read_device_status(head.status) == 0
    targets[85] = 500
    given = torch.zeros(1, **I32)
    r = head.logprobs(x, targets, 2, status=given)
    assert int(given) == _lib.MOE_ERR_TOKEN_ID and _lib.moe_read_device_status(head.status) == 0
    assert math.isnan(float(r.logprob[85]))
    head.logprobs(x, targets, 2, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert _lib.moe_read_device_status(head.status) == _lib.MOE_ERR_TOKEN_ID
