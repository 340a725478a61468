"""token_logprobs where a row's largest score so far moves often, or is no number."""
import math

import pytest
import torch

from int4_grouped_gemm_gb300 import scores
from test_gpu_scores import check

pytestmark = pytest.mark.gpu

SHAPES = [(2, 131072), (5, 700), (300, 2000), (200, 50021)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("T,V", SHAPES)
def test_rising_rows(T, V, dtype):
    """A larger score in nearly every batch, of a row's many lanes' own and of one lane's."""
    i = torch.arange(V, device="cuda", dtype=torch.float64)
    for row in (60 * i / V - 30, torch.where(i % 32 == 5, 40 * i / V, -3 * i / V), -60 * i / V):
        x = row.to(dtype).expand(T, V).contiguous()
        targets = torch.full((T,), V - 7, dtype=torch.int32, device="cuda")
        check(x, targets, 5, scores.token_logprobs(x, targets, 5))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("T,V", SHAPES)
def test_not_finite_wherever_it_stands(T, V, dtype):
    """One score that is no finite number, first, last or between; two of them."""
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, V, generator=g, device="cuda").to(dtype)
    targets = torch.randint(0, V, (T,), generator=g, device="cuda").to(torch.int32)
    want = scores.token_logprobs(x, targets, 3)
    keep = torch.arange(T, device="cuda") != 1
    for at in ((0,), (1,), (255,), (V // 2,), (V - 1,), (3, V - 2)):
        for bad in ((math.nan, math.inf), (math.inf, math.nan), (math.inf, math.inf)):
            y = x.clone()
            for p, b in zip(at, bad):
                y[1, p] = b
            r = scores.token_logprobs(y, targets, 3)
            assert torch.isnan(r.logprob[1]) and torch.isnan(r.entropy[1]) and torch.isnan(r.top_logprobs[1]).all()
            assert all(torch.equal(a[keep], b[keep]) for a, b in zip(r, want))
