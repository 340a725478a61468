"""Values near the ends of bf16's range: what the reference of the softmax leaves above
or below 1 in the weights must not take the sums out of fp32."""
import pytest
import torch

from int4_grouped_gemm_gb300 import _lib, attention

pytestmark = pytest.mark.gpu

BF16 = torch.finfo(torch.bfloat16).eps / 2


@pytest.mark.parametrize("B, Hq, Hkv, D, prefix", [(2, 16, 2, 128, 900), (20, 8, 1, 64, 2000), (60, 16, 2, 128, 1300)])
@pytest.mark.parametrize("power", [104, -87])
@pytest.mark.parametrize("step", [6.0, 14.0, 28.0])
def test_values_up_to_2_to_the_105(B, Hq, Hkv, D, prefix, step, power):
    """Scores (log2 units) of 0 at first, then `step`, then step + 1, 900 to 2000 positions
    of values up to 2^105: no partial sum of weights of at most 2^9 passes 2^126.  And of
    values about 2^-87: with weights of 2^-24 their sums stay 2^15 above fp32's least."""
    page = 64
    g = torch.Generator(device="cuda").manual_seed(B)
    n = -(-prefix // page)
    cache = attention.PagedCache.empty(n + 1, Hkv, page, D)
    cache.k.zero_()
    v = torch.randn(cache.v.shape, generator=g, device="cuda").clamp(-2, 2) * 2.0 ** power
    cache.v.copy_(v)
    score = torch.zeros(prefix, device="cuda")
    score[100:prefix // 2] = step
    score[prefix // 2:] = step + 1
    ln2 = 0.6931471805599453
    for p in range(prefix):
        cache.k[p // page, :, p % page, 0] = score[p]
    q = torch.zeros(B, Hq, D, device="cuda", dtype=torch.bfloat16)
    q[..., 0] = 1.0
    ws = cache.workspace(B, Hq, prefix)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    out = cache.attend(q, torch.zeros(B, 1, dtype=torch.int32, device="cuda"), lens,
                       torch.arange(n, dtype=torch.int32, device="cuda"), prefix, ln2, ws=ws)
    assert _lib.moe_read_device_status(ws) == 0
    p = torch.softmax(score.double() * ln2, 0)
    vv = cache.v[:n].transpose(0, 1).flatten(1, 2)[:, :prefix].double()
    want = torch.einsum("n,hnd->hd", p, vv).repeat_interleave(Hq // Hkv, 0)
    mag = torch.einsum("n,hnd->hd", p, vv.abs()).repeat_interleave(Hq // Hkv, 0)
    # weights 2^-17, their exponent's rounding 2^-19, sums of up to 126 + 64 roundings of 2^-23
    assert ((out.double() - want).abs() <= mag * 2.0 ** -14 + want.abs() * BF16).all()
