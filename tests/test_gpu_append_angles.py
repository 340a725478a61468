"""The rotation's angle is the exact product of position and frequency, whatever
the frequency: seen where the two products of a turned element nearly cancel,
so that the result's own rounding does not hide the angle's error."""
import pytest
import torch

from int4_grouped_gemm_gb300 import attention

pytestmark = pytest.mark.gpu

BF16 = torch.finfo(torch.bfloat16).eps / 2


@pytest.mark.parametrize("f", [1.0, 3.0, 7.0, 100.0, -1000.0, 12345.678, 2.0 ** -20, 1e-5])
@pytest.mark.parametrize("offset", [0, 1 << 20, 1 << 30])
def test_angles_are_exact_far_out(f, offset):
    """Angle: 2^-32 of a turn twice in the 32-bit fraction, its rounding to fp32 2^-25 of
    half a turn: below 1.1e-7.  Cosine and sine 2^-23, products and sum 2^-24 each:
    below 2^-21 of |a| + |b| together; then the rounding to bf16."""
    g = torch.Generator(device="cuda").manual_seed(offset + int(abs(f)))
    page = 65536
    cache = attention.PagedCache.empty(1, 1, page, 64)
    k = torch.randn(page, 1, 64, generator=g, device="cuda").to(torch.bfloat16)
    index = torch.arange(page, dtype=torch.int32, device="cuda")
    zero = torch.zeros(page, dtype=torch.int32, device="cuda")
    inv = torch.full((32,), f, device="cuda")
    cache.append(None, k, k, zero, index, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), inv, pos_offset=offset)
    # position = high + low with 15 bits below: each product with the 24-bit
    # frequency is exact in 64 bits, and so is a 64-bit cosine of it (to 2^-52)
    pos = index.long() + offset
    low = pos % 32768
    f64 = inv.double()[0].item()
    a1, a2 = (pos - low).double() * f64, low.double() * f64
    c = (a1.cos() * a2.cos() - a1.sin() * a2.sin())[:, None]
    s = (a1.sin() * a2.cos() + a1.cos() * a2.sin())[:, None]
    x, y = k[:, 0, :32].double(), k[:, 0, 32:].double()
    want = torch.cat((x * c - y * s, y * c + x * s), 1)
    mag = (x.abs() + y.abs()).repeat(1, 2)
    err = (cache.k[0, 0].double() - want).abs()
    # (rounded after the error: the value rounded is off by the bound already)
    tol = mag * 2.0 ** -21 * (1 + BF16) + want.abs() * BF16
    assert (err <= tol).all(), float((err - tol).max())
    # and the test could tell: many results are so small that 2^-19 of |a| + |b| would show
    assert int((want.abs() * BF16 < mag * 2.0 ** -20).sum()) > 100
