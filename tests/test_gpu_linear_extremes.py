"""int4_linear with scales and biases as large and as small as documented, and tokens
that bring the products back into range."""
import pytest
import torch

from int4_grouped_gemm_gb300 import moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [1, 3, 8, 9, 30, 64])
@pytest.mark.parametrize("weight, token", [(89, -60), (89, -100), (-100, 80), (60, -126), (-126, 120), (0, 120)])
def test_scales_of_any_documented_magnitude(B, weight, token):
    """Powers of two change no rounding: the result is that of the plain weights and
    tokens, times the two powers, to the fp32 bound of the norm tests."""
    K, N, G = 512, 300, 64
    g = torch.Generator(device="cuda").manual_seed(B)
    q = torch.randint(0, 16, (N, K), generator=g, device="cuda", dtype=torch.int32)
    words = torch.zeros(N, K // 8, device="cuda", dtype=torch.int32)
    for e in range(8):
        words |= q[:, e::8] << (4 * (e // 2 + 4 * (e % 2)))
    s = (torch.rand(N, K // G, generator=g, device="cuda").double() * 0.9 + 0.1).to(torch.bfloat16).double() * 2.0 ** weight
    z = torch.randn(N, K // G, generator=g, device="cuda").clamp(-3.9, 3.9).to(torch.bfloat16).double() / 4 * 2.0 ** weight
    x = torch.randn(B, K, generator=g, device="cuda").to(torch.bfloat16).double() * 2.0 ** token
    s16, z16, x16 = (t.to(torch.bfloat16) for t in (s, z, x))
    y = moe.linear(moe.QMatrix(words, s16.view(torch.int16), z16.view(torch.int16), N, K, G), x16, dtype=torch.float32)
    w = q.double() * s16.double().repeat_interleave(G, 1) + z16.double().repeat_interleave(G, 1)
    want = x16.double() @ w.t()
    rms = (x16.double() ** 2 @ (w ** 2).t()).sqrt()
    # (tokens of 2^120 and weights of 1 give results of 2^127 on average, many of them
    # past fp32's largest value: an element counts where no order of its sum passes that)
    sure = x16.double().abs() @ (w.abs() + 2 * z16.double().abs().repeat_interleave(G, 1)).t() < 3.4e38
    assert sure.all() or weight == 0
    assert torch.isfinite(y[sure]).all()
    # (and fp32's smallest step for the results that are subnormal; intermediate sums of
    # scaled tokens times weights likewise)
    assert ((y.double() - want).abs() <= 1e-5 * rms + 2.0 ** -140)[sure].all()
