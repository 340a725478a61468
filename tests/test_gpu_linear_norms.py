"""How far int4_linear with fp32 output is from 64 bits, in the norm of each token's
row and for each element: the worst-case bounds of the other tests grow with K until a
whole group of weights could be missing unseen; these could not miss one."""
import pytest
import torch

from int4_grouped_gemm_gb300 import moe

pytestmark = pytest.mark.gpu

# Roundings of 2^-24 are independent: the running sum of K / G group sums, of at
# most R = sqrt(sum (x w)^2) each way, is off by sqrt(K / G / 2) 2^-24 R, at most
# 1.4e-6 R for the 1,024 groups of the longest K; a group's own eight additions by
# 8 2^-23 of it at most, 1e-6 R over the independent groups.  Per element five
# times the first and the second once: below 1e-5 R.
ROW, ELEMENT = 2e-6, 1e-5

CASES = [  # B, K, N, group
    (1, 32, 16, 32), (1, 2048, 2560, 64), (2, 96, 17, 32), (3, 4096, 20000, 128), (5, 32768, 24, 64), (8, 8192, 4100, 32),
    (8, 32768, 131, 128), (8, 2080, 33, 32), (1, 32768, 5000, 32), (6, 16384, 21000, 128), (8, 32768, 20000, 128),
    (9, 32, 40, 32), (12, 4224, 19500, 32), (16, 4096, 3001, 64), (20, 16640, 8600, 128), (33, 160, 515, 32),
    (37, 2080, 5003, 32), (40, 32768, 2000, 128), (48, 4096, 20000, 64), (64, 8320, 8600, 64), (64, 32768, 130, 32),
    (64, 2048, 24000, 64),
    # very many rows: tokens that fit at once, and in chunks (blocks of sixteen warps)
    (2, 8192, 78001, 64), (8, 14336, 78001, 32), (7, 16384, 77900, 64), (6, 20480, 77900, 128),
]


@pytest.mark.parametrize("B, K, N, G", CASES)
def test_linear_in_the_norm(B, K, N, G):
    g = torch.Generator(device="cuda").manual_seed(B + K + N + G)
    q = torch.randint(0, 16, (N, K), generator=g, device="cuda", dtype=torch.int32)
    words = torch.zeros(N, K // 8, device="cuda", dtype=torch.int32)
    for e in range(8):
        words |= q[:, e::8] << (4 * (e // 2 + 4 * (e % 2)))
    pitch = moe.ld_groups(K, G)
    s, z = (torch.zeros(N, pitch, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    s[:, :K // G] = torch.rand(N, K // G, generator=g, device="cuda") * 0.01 + 0.001
    z[:, :K // G] = torch.randn(N, K // G, generator=g, device="cuda") * 0.03
    x = torch.randn(B, K, generator=g, device="cuda").to(torch.bfloat16)
    y = moe.linear(moe.QMatrix(words, s.view(torch.int16), z.view(torch.int16), N, K, G), x, dtype=torch.float32)
    want = torch.empty(B, N, dtype=torch.float64, device="cuda")
    rms = torch.empty_like(want)
    for r in range(0, N, 4096):
        part = slice(r, min(N, r + 4096))
        w = q[part].double() * s[part, :K // G].double().repeat_interleave(G, 1) + z[part, :K // G].double().repeat_interleave(G, 1)
        want[:, part] = x.double() @ w.t()
        rms[:, part] = (x.double() ** 2 @ (w ** 2).t()).sqrt()
    err = y.double() - want
    assert (err.norm(dim=1) <= ROW * want.norm(dim=1)).all(), float((err.norm(dim=1) / want.norm(dim=1)).max())
    assert (err.abs() <= ELEMENT * rms).all(), float((err.abs() / rms).max())
