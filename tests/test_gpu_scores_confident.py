"""token_logprobs of tokens that a row is nearly certain of, against 64 bits.

Tolerance.  All scores of a row but two weigh nothing (e^-100 is below fp32's
normal numbers).  With the larger one as the reference S = 1 + s, s = e^-h: the
one sum that is rounded is off by 2^-24, s by 2^-19 of itself (the exponential, and
the rounding of its argument, below 64), the logarithm and the quotient by an ulp of
themselves; what has to be added to the result is no larger than 1 + h s < 1.4."""
import math

import pytest
import torch

from int4_grouped_gemm_gb300 import scores

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rest", [-100.0, -math.inf])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("T,V,n_top", [(8, 131072, 3), (8, 131072, 0), (64, 20000, 2), (200, 50021, 0), (200, 50021, 4),
                                       (1000, 8192, 1), (3000, 4100, 0)])
def test_scores_far_above_the_first_of_their_lane(T, V, n_top, dtype, rest):
    """A score among a row's first, and one up to 7.9375 above it in a multiple of 2048 from
    there, which the same thread works on."""
    h = torch.tensor([0.25, 1.0, 2.5, 4.0, 6.0, 7.5, 7.875, 7.9375], device="cuda").repeat(T // 8)
    t = torch.arange(T, device="cuda")
    at = t * 37 % 256
    peak = at + 2048 * (1 + t % ((V - 256) // 2048))
    x = torch.full((T, V), rest, device="cuda", dtype=dtype)
    x[t, at] = 0.0
    x[t, peak] = h.to(dtype)
    s = (-h.double()).exp()
    tol = 2.0 ** -24 * 1.5 + s * (1 + h) * 2.0 ** -19
    for target, given in ((peak, -torch.log1p(s)), (at, -h.double() - torch.log1p(s))):
        r = scores.token_logprobs(x, target.to(torch.int32), n_top)
        # (the other one's log probability is a rounded number of up to 8)
        assert ((r.logprob.double() - given).abs() <= tol + given.abs() * 2.0 ** -23).all()
        entropy = torch.log1p(s) + h * s / (1 + s)
        assert ((r.entropy.double() - entropy).abs() <= tol + entropy * 2.0 ** -22).all()
        if n_top:
            assert torch.equal(r.top_ids[:, 0].long(), peak)
            assert ((r.top_logprobs[:, 0].double() + torch.log1p(s)).abs() <= tol).all()
