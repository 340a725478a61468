"""int4_linear_prompt where a token's groups are far from one another.

Tolerance.  As for any of its results: terms of magnitude |x| (16 |s| + |w|), a depth of
K / 16 + 64 additions of 2^-23 of them each, and parts of biases and group sums of 22 bits
(2^-20 covers those of both).  Besides, of the token's largest element: elements below
2^-31 of it are off by 2^-39 of it, group sums by 2^-42 of it times |c|, c = z + 8 s."""
import pytest
import torch

from int4_grouped_gemm_gb300 import _lib, moe
from test_gpu_attention_layer import gen, randn

pytestmark = pytest.mark.gpu


def matrix(q, s, z, G):
    """codes [N, K], scales and biases [N, K / G] (bf16): the packed matrix, and its
    weights, scales and |c| of each element in 64 bits."""
    N, K = q.shape
    words = torch.zeros(N, K // 8, dtype=torch.int64)
    for e in range(8):
        words |= q[:, e::8].long() << (4 * (e // 2 + 4 * (e % 2)))
    words = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
    pad = (0, moe.ld_groups(K, G) - K // G)
    sp, zp = (torch.nn.functional.pad(t, pad).contiguous().view(torch.int16).cuda() for t in (s, z))
    sd, zd = (t.double().repeat_interleave(G, 1) for t in (s, z))
    return moe.QMatrix(words.cuda(), sp, zp, N, K, G), q.double() * sd + zd, sd.abs(), (zd + 8 * sd).abs()


def check(x, m, w, s, c, G):
    K = x.shape[1]
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    for dtype, rounding in ((torch.float32, 2.0 ** -24), (torch.bfloat16, 2.0 ** -8)):
        got = moe.linear_prompt(m, x.cuda(), dtype=dtype, status=status).cpu().double()
        assert _lib.moe_read_device_status(status) == 0
        want = x.double() @ w.t()
        top = x.abs().double().max(1, keepdim=True).values
        tol = (x.abs().double() @ (16 * s + w.abs()).t()) * ((K / 16 + 64) * 2.0 ** -23 + 2.0 ** -20)
        tol += top * ((8 * s + w.abs()).sum(1) * 2.0 ** -39 + c[:, ::G].sum(1) * 2.0 ** -42) + want.abs() * rounding
        assert torch.isfinite(got).all()
        assert ((got - want).abs() <= tol).all(), float(((got - want).abs() / tol).max())


@pytest.mark.parametrize("N", [40, 20000])
@pytest.mark.parametrize("power", [-20, -24, -28])
@pytest.mark.parametrize("G", [32, 128])
def test_groups_far_below_the_largest_element(G, power, N):
    """The first group holds the token's large elements, where the row's weights are zero;
    the other groups, as wholes, are 2^power of them.  (N = 20000: codes that the product
    unpacks.)"""
    g = gen(G - power)
    K = 4 * G if N < 1000 else 1024
    q = torch.randint(0, 16, (N, K), generator=g)
    s = (torch.rand(N, K // G, generator=g) * 0.01 + 0.001).to(torch.bfloat16)
    z = (torch.randn(N, K // G, generator=g) * 0.03).to(torch.bfloat16)
    s[:, 0] = z[:, 0] = 0
    x = randn(g, 100, K)
    x[:, G:] *= 2.0 ** power
    check(x, *matrix(q, s, z, G), G)
