"""The softmax weights of the paged attention carry fp32 accuracy into the second
product, as the one-sequence call's do.

Values come in pairs of opposite sign at positions whose keys nearly agree, so
that the result is a difference of nearly equal weights: its own rounding to
bf16 is then far smaller than a rounding of the weights to bf16 would be."""
import math

import pytest
import torch

from int4_grouped_gemm_gb300 import _lib, attention

pytestmark = pytest.mark.gpu

BF16 = torch.finfo(torch.bfloat16).eps / 2
FP32 = torch.finfo(torch.float32).eps / 2


def pairs(g, Hkv, n, D):
    """Keys of 2 n positions in nearly equal pairs, values +-1 of opposite sign."""
    k = torch.randn(Hkv, n, 1, D, generator=g)
    k = (k + 0.02 * torch.randn(Hkv, n, 2, D, generator=g)).to(torch.bfloat16)
    v = torch.randint(0, 2, (Hkv, n, 1, D), generator=g) * 2.0 - 1.0
    v = torch.cat((v, -v), 2).to(torch.bfloat16)
    return k.flatten(1, 2).cuda(), v.flatten(1, 2).cuda()


def reference(q, k, v, scale):
    """In 64 bits, and how far off fp32 arithmetic may be before the output's rounding.

    A score is off by at most 2^-20 of scale sum |q_i k_i| (D <= 128 products, exact,
    in rounded additions), and by three roundings of itself and of its distance
    to the reference (scaling, subtraction, exponential); so a weight is off by
    that, by 2^-22 of the exponential's own, and by 2^-17 as two bf16 parts.
    Numerator and denominator add up n weights, 16 at a time, in roundings of 2^-23
    of the sum, and join at most 64 parts."""
    Hkv, n, D = k.shape
    group = q.shape[0] // Hkv
    qq = q.double().view(Hkv, group, D)
    s = qq @ k.double().transpose(1, 2) * scale
    p = torch.softmax(s, -1)
    want = p @ v.double()
    score = float((qq.abs() @ k.double().abs().transpose(1, 2)).max()) * scale
    spread = float(s.max() - s.min()) + float(s.abs().max())
    weight = score * 2.0 ** -20 + 3 * spread * 1.45 * FP32 + 2.0 ** -22
    rel = 2 * weight + 2.0 ** -17 + 2 * (n / 16 + 64) * 2.0 ** -23
    return want.view(-1, D), rel * (p @ v.double().abs()).view(-1, D)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B, Hq, Hkv, page, prefix, own", [
    (1, 8, 1, 16, 0, 16),        # one tile
    (3, 16, 2, 16, 0, 46),       # pieces by warp
    (1, 16, 2, 64, 0, 1100),     # by block
    (1, 16, 2, 16, 90, 30),      # one row reads the prefix as its own
    (5, 16, 2, 16, 130, 0),      # 128 rows of the prefix at most
    (40, 8, 1, 32, 300, 0),      # 256-row blocks
    (33, 16, 4, 16, 100, 20),    # both parts in one softmax
])
def test_weights_are_not_rounded_to_bf16(B, Hq, Hkv, page, prefix, own, D):
    g = torch.Generator().manual_seed(B + prefix + own + D)
    np_, no = -(-prefix // page), -(-own // page)
    cache = attention.PagedCache.empty(np_ + B * no + 1, Hkv, page, D)
    cache.k.fill_(float("nan"))
    cache.v.fill_(float("nan"))
    order = torch.randperm(cache.n_pages, generator=g).to(torch.int32)

    def put(pages, k, v):
        for i, p in enumerate(pages.tolist()):
            part = slice(i * page, min((i + 1) * page, k.shape[1]))
            cache.k[p, :, :part.stop - part.start] = k[:, part]
            cache.v[p, :, :part.stop - part.start] = v[:, part]
    pk, pv = pairs(g, Hkv, prefix // 2, D)
    put(order[:np_], pk, pv)
    table = order[np_:np_ + B * no].view(B, no) if no else torch.zeros(B, 1, dtype=torch.int32)
    rows = [pairs(g, Hkv, own // 2, D) for _ in range(B)]
    if no:
        for b in range(B):
            put(table[b], *rows[b])
    q = torch.randn(B, Hq, D, generator=g).to(torch.bfloat16).cuda()
    ws = cache.workspace(B, Hq, prefix)
    out = cache.attend(q, table.cuda(), torch.full((B,), own, dtype=torch.int32).cuda(),
                       order[:np_].cuda() if prefix else None, prefix, ws=ws)
    assert _lib.moe_read_device_status(ws) == 0
    for b in range(B):
        want, off = reference(q[b], torch.cat((pk, rows[b][0]), 1), torch.cat((pv, rows[b][1]), 1), 1 / math.sqrt(D))
        assert float(off.max()) < 2e-4          # the bound is far below 2^-9, a weight's rounding to bf16
        err = (out[b].double() - want).abs()
        assert (err <= off * (1 + BF16) + want.abs() * BF16).all(), (b, float((err - want.abs() * BF16).max()), float(off.max()))
