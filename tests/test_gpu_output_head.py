"""OutputHead: its pieces share their scratch."""
import pytest
import torch

from int4_grouped_gemm_gb300 import moe, scores
from test_gpu_attention_layer import gen, make_int4, randn

pytestmark = pytest.mark.gpu


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
