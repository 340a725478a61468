"""Scores of the paged attention that are infinite, NaN or far from one another:
a score of minus infinity has weight zero, anything that the definition makes NaN
is NaN and stays with its row and head."""
import math

import pytest
import torch

from int4_grouped_gemm_gb300 import _lib, attention

pytestmark = pytest.mark.gpu

BF16 = torch.finfo(torch.bfloat16).eps / 2
INF, NAN = float("inf"), float("nan")


class Batch:
    """B rows of `own` positions behind `prefix` shared ones, all in order of page."""

    def __init__(self, B, Hq, Hkv, D, prefix, own, page=16, seed=1):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.Hq, self.Hkv, self.D, self.prefix, self.own, self.page = B, Hq, Hkv, D, prefix, own, page
        self.np, self.no = -(-prefix // page), -(-own // page)
        self.cache = attention.PagedCache.empty(self.np + B * self.no, Hkv, page, D)
        for t in (self.cache.k, self.cache.v):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        self.pages = torch.arange(self.np, dtype=torch.int32, device="cuda")
        self.table = (self.np + torch.arange(B * max(self.no, 0), dtype=torch.int32, device="cuda")).view(B, -1) \
            if self.no else torch.zeros(B, 1, dtype=torch.int32, device="cuda")
        self.lens = torch.full((B,), own, dtype=torch.int32, device="cuda")
        self.q = torch.randn(B, Hq, D, generator=g, device="cuda").to(torch.bfloat16)
        self.q[..., 0] = 1.0

    def set_keys(self, b, first, last, value, dim=0):
        """Dimension `dim` of the keys of positions [first, last), counted from the prefix's
        start, of row b (prefix positions: of all rows)."""
        for p in range(first, last):
            if p < self.prefix:
                self.cache.k[p // self.page, :, p % self.page, dim] = value
            else:
                o = p - self.prefix
                self.cache.k[int(self.table[b, o // self.page]), :, o % self.page, dim] = value

    def gathered(self, pool, b):
        shared = pool[:self.np].transpose(0, 1).flatten(1, 2)[:, :self.prefix]
        if not self.no:
            return shared.double()
        mine = pool[self.table[b].long()].transpose(0, 1).flatten(1, 2)[:, :self.own]
        return torch.cat((shared, mine), 1).double()

    def run(self, scale=None):
        ws = self.cache.workspace(self.B, self.Hq, self.prefix)
        out = self.cache.attend(self.q, self.table, self.lens, self.pages if self.prefix else None, self.prefix, scale, ws=ws)
        assert _lib.moe_read_device_status(ws) == 0
        return out

    def want(self, b, scale=None):
        k, v = self.gathered(self.cache.k, b), self.gathered(self.cache.v, b)
        q = self.q[b].double().view(self.Hkv, -1, self.D)
        s = q @ k.transpose(1, 2) * (scale or 1 / math.sqrt(self.D))
        return (torch.softmax(s, -1) @ v).reshape(self.Hq, self.D), float(v.abs().max())


# B, Hq, Hkv, D, prefix, own
SHAPES = [(3, 8, 1, 128, 0, 100), (1, 16, 2, 64, 0, 2500), (1, 8, 2, 128, 300, 50), (20, 8, 1, 64, 700, 5),
          (70, 16, 4, 128, 400, 20), (2, 16, 2, 128, 40000, 3)]
IDS = ["by warp", "by block", "one row's prefix", "prefix 160 rows", "prefix 256 rows", "long prefix"]


@pytest.mark.parametrize("value", [-INF, -3e38], ids=["infinite", "leaves fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_scores_of_minus_infinity_weigh_nothing(shape, value):
    """Whole tiles and whole pieces of such scores, at the start and between others."""
    s = Batch(*shape)
    n = s.prefix + s.own
    if value != -INF:
        s.q[..., 0] = 8.0                   # 8 * -3e38 is below fp32's range
    for b in range(s.B):
        s.set_keys(b, s.prefix if b and s.prefix else 0, n // 3, value)
        s.set_keys(b, n // 2, n // 2 + 17, value)
    out = s.run()
    for b in range(s.B):
        want, top = s.want(b)
        err = (out[b].double() - want).abs()
        # weights to 2^-8 each in numerator and denominator (fp32 scores of up to 20 in 2^-20 of them)
        assert (err <= top * (2 * BF16 + 2.0 ** -11) + want.abs() * BF16).all(), b


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_a_row_without_a_finite_score_is_nan(shape):
    """0 / 0 by the definition; the other rows do not change."""
    s = Batch(*shape)
    clean = s.run()
    s.q[0, 1] = 0.0
    s.q[0, 1, 0] = -INF
    for b in range(s.B if s.prefix else 1):
        s.set_keys(b, 0, s.prefix + s.own, 1.0)
    same = s.run()
    assert torch.isnan(same[0, 1]).all()
    if not s.prefix:
        assert torch.equal(same[1:], clean[1:])
    s.q[0, 1, 0] = 1.0
    again = s.run()
    others = torch.ones(s.B, s.Hq, dtype=torch.bool, device="cuda")
    others[0, 1] = False
    assert torch.equal(again[others], same[others]) and torch.isfinite(again).all()


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_a_nan_query_makes_its_own_head_nan(shape):
    s = Batch(*shape)
    clean = s.run()
    s.q[-1, 2, 7] = NAN
    out = s.run()
    assert torch.isnan(out[-1, 2]).all()
    out[-1, 2] = clean[-1, 2]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_nan_and_infinite_scores_are_not_dropped(shape, value):
    """A whole tile and more of NaN scores among finite ones, or one score of plus
    infinity (its weight is infinity less infinity): the row is NaN."""
    s = Batch(*shape)
    clean = s.run()
    n = s.prefix + s.own
    first = n // 2
    s.set_keys(0, first, first + (min(160, n - first) if value != value else 1), value)
    out = s.run()
    hit = s.B if first < s.prefix else 1        # the prefix is everybody's
    assert torch.isnan(out[:hit]).all()
    assert torch.equal(out[hit:], clean[hit:])


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_scores_far_below_others_in_front_of_them(shape):
    """The first half scores -8e11 (log2 units), the second 47,000 throughout: the
    mean of the second half's values."""
    s = Batch(*shape)
    n = s.prefix + s.own
    s.q.zero_()
    s.q[..., 0] = 2.0 ** 20
    for b in range(s.B):
        s.set_keys(b, s.prefix if b and s.prefix else 0, n // 2, -2.0 ** 22)
        s.set_keys(b, max(n // 2, s.prefix if b and s.prefix else 0), n, 0.25)
    out = s.run(0.125)
    for b in range(s.B):
        want, top = s.want(b, 0.125)
        err = (out[b].double() - want).abs()
        assert (err <= top * 2.0 ** -11 + want.abs() * BF16).all(), b


@pytest.mark.parametrize("L", [40, 1000, 30000])
def test_one_sequence_call_with_infinite_and_nan_scores(L):
    """gqa_decode_attention likewise."""
    Hq, Hkv, D = 16, 2, 128
    g = torch.Generator(device="cuda").manual_seed(L)
    q, k, v = (torch.randn(h, *n, D, generator=g, device="cuda").to(torch.bfloat16) for h, n in ((Hq, ()), (Hkv, (L,)), (Hkv, (L,))))
    q[:, 0] = 1.0
    out = torch.empty(Hq, D, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(_lib.gqa_attention_workspace_bytes(Hq, Hkv, D, L), dtype=torch.uint8, device="cuda")

    def run():
        _lib.gqa_decode_attention(q, k, v, L, 1 / math.sqrt(D), out, ws)
        return out.clone()
    clean = run()
    keep = k.clone()
    k[:, :L // 3, 0] = -INF
    got = run()
    p = torch.softmax(q.double().view(Hkv, 8, D) @ k.double().transpose(1, 2) / math.sqrt(D), -1)
    want = (p @ v.double()).view(Hq, D)
    assert ((got.double() - want).abs() <= float(v.abs().max()) * 2.0 ** -11 + want.abs() * BF16).all()
    k.copy_(keep)
    k[0, L // 2:L // 2 + 20] = NAN
    got = run()
    assert torch.isnan(got[:8]).all() and torch.equal(got[8:], clean[8:])
    k.copy_(keep)
    q[3, 5] = NAN
    got = run()
    assert torch.isnan(got[3]).all()
    got[3] = clean[3]
    assert torch.equal(got, clean)
