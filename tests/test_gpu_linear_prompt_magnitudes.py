"""int4_linear_prompt with scales and biases at either end of bf16's range.  Tolerance:
as in test_gpu_linear_prompt_ranges."""
import pytest
import torch

from test_gpu_attention_layer import gen, randn
from test_gpu_linear_prompt_ranges import check, matrix

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [70, 300])
@pytest.mark.parametrize("N", [48, 17000])
def test_scales_and_biases_near_the_end_of_fp32(N, T):
    """Biases from 2^119 to 2^126, with c = z + 8 s beyond fp32 in some rows; small tokens, so
    that weights and results are within it."""
    g = gen(N + T)
    G, K = 64, 128 if N < 1000 else 1024
    # codes of 0 .. 3
    q = torch.randint(0, 4, (N, K), generator=g)
    e = 119 + torch.arange(N)[:, None] % 8
    z = ((1 + torch.rand(N, K // G, generator=g)) * 2.0 ** e * torch.where(torch.rand(N, K // G, generator=g) < 0.5, -0.5, 0.5))
    s = torch.rand(N, K // G, generator=g) * 2.0 ** (e - 8)
    s[::3] = (1 + torch.rand(N, K // G, generator=g)[::3] / 2) * 2.0 ** 125
    z[::3] = -z[::3].abs()
    s, z = s.to(torch.bfloat16), z.to(torch.bfloat16)
    x = randn(g, T, K, std=2.0 ** -60)
    check(x, *matrix(q, s, z, G), G)


@pytest.mark.parametrize("size", [2.0 ** -126, 2.0 ** -118])
def test_scales_and_biases_near_the_least_numbers(size):
    """Scales and biases among and just above bf16's subnormal numbers."""
    g = gen(7)
    q = torch.randint(0, 16, (40, 128), generator=g)
    s = (torch.rand(40, 4, generator=g) + 0.5).double().mul(size).to(torch.bfloat16)
    z = torch.randn(40, 4, generator=g).double().mul(size * 4).to(torch.bfloat16)
    x = randn(g, 100, 128, std=2.0 ** 60)
    check(x, *matrix(q, s, z, 32), 32)
