"""int4_linear_prompt of 64 tokens and fewer needs no scratch."""
import pytest
import torch

from int4_grouped_gemm_gb300 import moe
from test_gpu_attention_layer import gen, make_int4, randn
from test_gpu_linear_prompt import bound

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 8, 9, 64])
def test_a_small_workspace_serves_few_tokens(T):
    g = gen(T)
    m, w = make_int4(g, 20000, 1024, 64)
    ws = moe.linear_prompt_workspace(m, T)
    assert 0 < ws.numel() <= 4096
    x = randn(g, T, 1024)
    got = moe.linear_prompt(m, x.cuda(), dtype=torch.float32, ws=ws).cpu().double()
    assert ((got - x.double() @ w.t()).abs() <= bound(x, w, 1024)).all()
    # scratch of more tokens serves as well
    large = moe.linear_prompt_workspace(m, 65)
    assert torch.equal(moe.linear_prompt(m, x.cuda(), dtype=torch.float32, ws=large).cpu().double(), got)


def test_memory_of_few_tokens():
    m, _ = make_int4(gen(2), 20000, 1024, 64)
    x = randn(gen(3), 64, 1024).cuda()
    y = torch.empty(64, 20000, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    moe.linear_prompt(m, x, y)
    assert torch.cuda.max_memory_allocated() - before <= 4096
