"""Causal attention of packed prompts over the paged cache against a plain
implementation in 64 bits, at the lengths, layouts and masks where it can go
wrong, and a prompt's whole sub-layer, layer and scores together.

Tolerance.  A score is off by its fp32 sums, at most 2^-20 of scale sum |q_i k_i|
(D <= 128 rounded additions), which stays below 512 here: a weight is off by 2^-11
of itself at most, in the numerator and in the denominator.  Weights enter the
second product as two bf16 parts, 2^-17 of themselves off, and the sums of up to
2^15 of them in fp32, tiles of 128 after another, are off by 2^-14 of the sum of the
magnitudes; then the output is rounded to bf16, half a step: 2^-8 of itself."""
import math

import pytest
import torch

from int4_grouped_gemm_gb300 import _lib, attention, moe, scores, synthetic

pytestmark = pytest.mark.gpu

BF16 = torch.finfo(torch.bfloat16).eps / 2


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16)


def tol_of(want, v):
    return float(v.abs().max()) * 2 * (2 ** -11 + 2 ** -17 + 2 ** -14) + want.abs() * BF16


class Prompt:
    """seqs: (rows, positions) of each sequence; positions -1: padding."""

    def __init__(self, seqs, Hq, Hkv, D, page, prefix=0, heads_first=True, seed=0, k_std=1.0, spare=2, lead=0, tail=0):
        g = gen(seed)
        self.seqs, self.prefix, self.D, self.Hq, self.Hkv, self.page = seqs, prefix, D, Hq, Hkv, page
        lens = [n for _, n in seqs]
        n_p = -(-prefix // page)
        own = [-(-max(n, 0) // page) for n in lens]
        total = n_p + sum(own) + spare
        perm = torch.randperm(total, generator=g).to(torch.int32)
        # what no sequence holds is NaN
        shape = (total, Hkv, page, D) if heads_first else (total, page, Hkv, D)
        kp, vp = (torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        if not heads_first:
            kp, vp = kp.transpose(1, 2), vp.transpose(1, 2)
        table = torch.zeros(len(seqs), max(1, max(own)), dtype=torch.int32)
        self.pk, self.pv = randn(g, Hkv, prefix, D, std=k_std).cuda(), randn(g, Hkv, prefix, D).cuda()
        self.fill(kp, vp, perm[:n_p], self.pk, self.pv)
        at, self.k, self.v = n_p, [], []
        for b, n in enumerate(lens):
            n = max(n, 0)
            table[b, :own[b]] = perm[at:at + own[b]]
            self.k.append(randn(g, Hkv, n, D, std=k_std).cuda())
            self.v.append(randn(g, Hkv, n, D).cuda())
            self.fill(kp, vp, perm[at:at + own[b]], self.k[b], self.v[b])
            at += own[b]
        self.cache = attention.PagedCache(kp, vp)
        self.table = table.cuda()
        self.prefix_pages = perm[:n_p].cuda() if n_p else None
        self.starts = [lead]
        for n, _ in seqs:
            self.starts.append(self.starts[-1] + n)
        self.T = self.starts[-1] + tail
        self.q_start = torch.tensor(self.starts, dtype=torch.int32).cuda()
        self.seq_len = torch.tensor(lens, dtype=torch.int32).cuda()
        self.q = randn(g, self.T, Hq, D).cuda()

    def fill(self, kp, vp, pages, k, v):
        n = k.shape[1]
        for i, p in enumerate(pages.tolist()):
            m = min(self.page, n - i * self.page)
            kp[p, :, :m], vp[p, :, :m] = k[:, i * self.page:i * self.page + m], v[:, i * self.page:i * self.page + m]

    def refill(self, b):
        n = self.k[b].shape[1]
        self.fill(self.cache.k, self.cache.v, self.table[b, :-(-n // self.page)], self.k[b], self.v[b])

    def run(self, **kw):
        return self.cache.attend_prompt(self.q, self.q_start, self.table, self.seq_len, self.prefix_pages, self.prefix,
                                        **kw)

    def want(self, b, scale):
        """Sequence b's rows in 64 bits."""
        nq, n = self.seqs[b]
        q = self.q[self.starts[b]:self.starts[b + 1]].double()
        k = torch.cat((self.pk, self.k[b]), 1).double()
        v = torch.cat((self.pv, self.v[b]), 1).double()
        G, N = self.Hq // self.Hkv, k.shape[1]
        out = torch.zeros(nq, self.Hq, self.D, dtype=torch.float64, device="cuda")
        if N == 0:
            return out
        sees = self.prefix + n - nq + torch.arange(nq, device="cuda") + 1     # positions a row sees
        sees = sees.clamp(min=self.prefix)
        hidden = torch.arange(N, device="cuda") >= sees[:, None]
        for h in range(self.Hq):
            s = (q[:, h] @ k[h // G].t() * scale).masked_fill(hidden, -math.inf)
            out[:, h] = torch.softmax(s, -1) @ v[h // G]
        return torch.where((sees > 0)[:, None, None], out, 0.0)

    def check(self, out, scale=None, only=None):
        scale = 1 / math.sqrt(self.D) if scale is None else scale
        for b, (nq, n) in enumerate(self.seqs):
            if nq == 0 or n < 0 or (only is not None and b not in only):
                continue
            want = self.want(b, scale)
            got = out[self.starts[b]:self.starts[b + 1]].double()
            assert torch.isfinite(got).all(), b
            v = torch.cat((self.pv, self.v[b]), 1)
            if v.shape[1] == 0:
                assert (got == 0).all()
                continue
            err, tol = (got - want).abs(), tol_of(want, v)
            assert (err <= tol).all(), (b, nq, n, float((err - tol).max()))
            # roundings are independent: far below the worst case on average
            assert err.mean() <= BF16 * want.abs().mean() + 2 ** -12 * float(v.abs().float().mean())


CASES = [  # (rows, positions) of the sequences, Hq, Hkv, D, page, prefix, heads_first
    ([(1, 1)], 1, 1, 64, 16, 0, True),
    ([(77, 77)], 16, 2, 128, 64, 0, True),
    ([(1, 1), (2, 2), (15, 15), (16, 16), (17, 17)], 16, 2, 128, 16, 0, False),
    ([(127, 127), (128, 128), (129, 129)], 4, 4, 64, 32, 0, True),
    ([(1, 129), (1, 128), (1, 127), (3, 400)], 8, 1, 128, 16, 0, True),
    ([(300, 300), (0, 0), (41, 700), (0, 5), (5, 5)], 24, 8, 64, 16, 0, False),
    ([(130, 130), (61, 200)], 10, 2, 128, 16, 0, True),          # five heads a key-value head
    ([(90, 90), (33, 33)], 14, 2, 64, 64, 0, True),              # seven
    ([(64, 64)], 6, 1, 128, 128, 0, True),                       # six
    ([(200, 200), (57, 57)], 8, 4, 128, 256, 0, False),          # two
    ([(100, 100), (28, 50)], 64, 64, 64, 16, 0, True),
    ([(33, 33)], 256, 32, 64, 16, 0, True),
    ([(1, 0), (4, 2), (20, 0), (130, 3)], 16, 2, 128, 16, 0, True),   # rows before the first position
    ([(4, 2), (30, 0), (7, 7)], 16, 2, 64, 16, 1, True),
    ([(50, 50), (1, 1), (17, 40)], 16, 2, 128, 16, 127, True),
    ([(50, 50), (1, 1)], 8, 1, 64, 32, 128, False),
    ([(9, 9)] * 20, 16, 2, 128, 16, 129, True),
    ([(40, 40), (300, 310)], 3, 3, 64, 256, 1000, True),
    ([(2, -1), (30, 30), (3, -1), (0, -1), (5, 9), (1, -7)], 16, 2, 128, 16, 64, True),   # padding
    ([(i % 4, 3 + i) for i in range(300)], 8, 1, 64, 16, 0, True),
    ([(1, 1 + i) for i in range(200)], 16, 2, 128, 16, 33, False),
    ([(7, 6000), (1, 5001)], 16, 2, 128, 64, 0, True),           # few rows behind many positions
    ([(1, 20000)], 8, 8, 64, 16, 0, True),
    ([(2000, 2000)], 8, 1, 128, 64, 0, True),
    ([(1100, 1100), (700, 900), (3, 3)], 4, 2, 64, 32, 300, False),
    ([(600, 900), (20, 20)], 2, 2, 128, 65536, 0, True),         # a page that holds a whole sequence
    ([(1500, 4000), (1, 3000), (90, 90)], 32, 4, 128, 128, 500, True),
]


@pytest.mark.parametrize("seqs,Hq,Hkv,D,page,prefix,hf", CASES)
def test_prompt_against_64_bits(seqs, Hq, Hkv, D, page, prefix, hf):
    p = Prompt(seqs, Hq, Hkv, D, page, prefix, hf, seed=len(seqs) + Hq + prefix, spare=2 if page < 4096 else 1)
    ws = p.cache.prompt_workspace(p.T, len(seqs), Hq)
    out = p.run(out=torch.full_like(p.q, 3.0), ws=ws)
    assert _lib.moe_read_device_status(ws) == 0
    p.check(out)
    for b, (nq, n) in enumerate(seqs):
        if n < 0:
            assert (out[p.starts[b]:p.starts[b + 1]] == 3).all()     # padding keeps what out held
    # the same bits again, in the workspace as it is now
    assert torch.equal(out, p.run(out=torch.full_like(p.q, 3.0), ws=ws))


def test_prompt_rows_of_no_sequence_stay_as_they_were():
    p = Prompt([(20, 20), (0, 9), (37, 100)], 16, 2, 128, 16, seed=2, lead=5, tail=40)
    out = p.run(out=torch.full_like(p.q, 3.0))
    p.check(out)
    assert (out[:5] == 3).all() and (out[p.starts[-1]:] == 3).all()


def test_prompt_strided_rows_and_in_place():
    p = Prompt([(140, 140), (3, 9)], 16, 2, 128, 16, seed=3)
    wide = torch.full((p.T, 20, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :16] = p.q
    p.q = wide[:, :16]
    out = torch.full((p.T, 24, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    p.run(out=out[:, 8:])
    p.check(out[:, 8:])
    assert (out[:, :8] == 7).all()
    p.run(out=p.q)
    assert torch.equal(p.q, out[:, 8:]) and (wide[:, 16:] == 9).all()


@pytest.mark.parametrize("k_std,scale", [(6.0, None), (1.0, 0.0), (1.0, -0.3), (30.0, None)])
def test_prompt_peaked_uniform_and_negative_scales(k_std, scale):
    p = Prompt([(150, 150), (40, 333)], 16, 2, 128, 32, 200, seed=4, k_std=k_std)
    p.check(p.run(scale=scale), scale)


@pytest.mark.parametrize("up", [True, False])
def test_prompt_rising_and_falling_scores(up):
    """Keys along a query, each larger (smaller) than the last: the running
    reference moves all the time, or never."""
    p = Prompt([(900, 900)], 8, 1, 128, 16, seed=5)
    ramp = torch.linspace(0.0, 4.0, 900).to(torch.bfloat16)
    p.k[0] = ((ramp if up else ramp.flip(0))[:, None].cuda() * p.q[450, 0].sign())[None].contiguous()
    p.refill(0)
    p.check(p.run())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("at", [0, 5, 128, 200, 255, 299])
def test_prompt_later_positions_have_no_influence(D, bad, what, at):
    """A broken key or value at one position leaves every earlier token's rows as
    they are, bit for bit, and those that see a value of NaN or infinity not finite."""
    p = Prompt([(300, 300), (20, 20)], 6, 2, D, 16, seed=6)
    good = p.run()
    (p.k if what == "k" else p.v)[0][1, at, 3] = bad
    p.refill(0)
    out = p.run()
    heads = slice(3, 6)                                   # those of key-value head 1
    assert torch.equal(out[:at], good[:at]) and torch.equal(out[300:], good[300:])
    assert torch.equal(out[:, :3], good[:, :3])
    if what == "v":
        assert not torch.isfinite(out[at:300, heads, 3]).any()
        rest = torch.arange(D, device="cuda") != 3
        assert torch.equal(out[:300, heads][:, :, rest], good[:300, heads][:, :, rest])
    elif math.isnan(bad):
        assert torch.isnan(out[at:300, heads]).all()


def test_prompt_scores_of_minus_infinity_weigh_nothing():
    """Keys that score minus infinity against a token (an infinite element of the
    sign that the query's is not) count as if they were not there; a token that
    has no other is NaN."""
    p = Prompt([(200, 200)], 1, 1, 64, 16, seed=7)
    p.q[:, 0, 0] = 1.0
    gone = torch.zeros(200, dtype=torch.bool)
    gone[:130] = True
    gone[150:160] = True
    p.k[0][0, gone, 0] = -math.inf
    p.refill(0)
    out = p.run()
    assert torch.isnan(out[:130]).all()
    q, k, v = p.q[:, 0].double(), p.k[0][0].double(), p.v[0][0].double()
    s = q @ k.t() / 8
    s = s.masked_fill(torch.arange(200, device="cuda") > torch.arange(200, device="cuda")[:, None], -math.inf)
    want = torch.softmax(s, -1) @ v
    assert ((out[130:, 0].double() - want[130:]).abs() <= tol_of(want[130:], v)).all()


@pytest.mark.parametrize("size", [2.0 ** 95, 2.0 ** -90])
def test_prompt_values_of_any_magnitude(size):
    p = Prompt([(150, 150), (5, 400)], 8, 1, 128, 16, seed=8)
    for b in range(2):
        p.v[b] = (p.v[b].float() * size).to(torch.bfloat16)
        p.refill(b)
    out = p.run()
    assert torch.isfinite(out).all()
    for b in range(2):
        want = p.want(b, 1 / math.sqrt(128))
        got = out[p.starts[b]:p.starts[b + 1]].double()
        assert ((got - want).abs() <= tol_of(want, p.v[b].double())).all()


def test_prompt_scores_far_apart():
    """Scores 2^40 below the following ones: the reference jumps, and what came
    before weighs nothing."""
    p = Prompt([(400, 400)], 1, 1, 64, 16, seed=9)
    p.q[:, 0] = 1.0
    p.k[0][0, :128] = -(2.0 ** 40)
    p.k[0][0, 128:256] = 0.0
    p.k[0][0, 256:] = 2.0 ** 30
    p.refill(0)
    out = p.run()[:, 0].double()
    v = p.v[0][0].double()
    for t, lo in ((100, 0), (200, 128), (300, 256), (399, 256)):
        want = v[lo:t + 1].mean(0)
        assert ((out[t] - want).abs() <= tol_of(want, v)).all(), t


def test_prompt_agrees_with_decoding_steps():
    """A token's rows are those of a decoding step at its position."""
    p = Prompt([(40, 200), (25, 25)], 16, 2, 128, 16, 100, seed=10)
    out = p.run()
    rows = [(b, i) for b in range(2) for i in (0, 7, p.seqs[b][0] - 1)]
    at = torch.tensor([p.starts[b] + i for b, i in rows], device="cuda")
    lens = torch.tensor([p.seqs[b][1] - p.seqs[b][0] + i + 1 for b, i in rows], dtype=torch.int32, device="cuda")
    table = p.table[torch.tensor([b for b, _ in rows], device="cuda")].contiguous()
    step = p.cache.attend(p.q[at].contiguous(), table, lens, p.prefix_pages, p.prefix)
    want = step.double()
    assert ((out[at].double() - want).abs() <= 2 * tol_of(want, torch.cat((p.pv, p.v[0]), 1))).all()


def test_prompt_in_pieces_gives_the_same():
    p = Prompt([(500, 500)], 16, 2, 128, 32, 70, seed=11)
    whole = p.run()
    for a, b in ((0, 130), (130, 131), (131, 500)):
        q_start = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        n = torch.tensor([b], dtype=torch.int32, device="cuda")
        part = p.cache.attend_prompt(p.q[a:b].contiguous(), q_start, p.table, n, p.prefix_pages, p.prefix)
        want = whole[a:b].double()
        assert ((part.double() - want).abs() <= 2 * tol_of(want, p.v[0])).all()


def test_prompt_bad_pages_starts_and_lengths_are_recorded_not_followed():
    p = Prompt([(40, 40), (33, 50), (21, 21)], 16, 2, 128, 16, 40, seed=12)
    ws = p.cache.prompt_workspace(p.T, 3, 16)
    good = p.run(ws=ws).clone()
    assert _lib.moe_read_device_status(ws) == 0
    rows = [slice(p.starts[b], p.starts[b + 1]) for b in range(3)]
    table, q_start, seq_len, pages = p.table.clone(), p.q_start.clone(), p.seq_len.clone(), p.prefix_pages.clone()
    for bad in (-1, p.cache.n_pages, 2 ** 31 - 1, -2 ** 31):
        p.table = table.clone()
        p.table[1, 1] = bad
        out = p.run(ws=ws)
        assert _lib.moe_read_device_status(ws) == _lib.MOE_ERR_PAGE
        assert torch.equal(out[rows[0]], good[rows[0]]) and torch.equal(out[rows[2]], good[rows[2]])
    p.table = table
    for bad in (p.table.shape[1] * 16 + 1, 2 ** 31 - 1):
        p.seq_len = seq_len.clone()
        p.seq_len[1] = bad
        out = p.run(ws=ws)
        assert _lib.moe_read_device_status(ws) == _lib.MOE_ERR_PAGE
        assert torch.equal(out[rows[0]], good[rows[0]]) and torch.equal(out[rows[2]], good[rows[2]])
    p.seq_len = seq_len
    for i, bad in ((3, p.T + 1), (3, 2 ** 31 - 1), (0, -1), (0, -2 ** 31)):
        p.q_start = q_start.clone()
        p.q_start[i] = bad
        out = p.run(ws=ws)
        assert _lib.moe_read_device_status(ws) == _lib.MOE_ERR_PAGE
        assert torch.equal(out[rows[1]], good[rows[1]])
    for bad in ([0, 40, 39, p.T], [0, 2 ** 31 - 1, -2 ** 31, 0], [5, 4, 3, 2], [p.T, p.T, p.T, 0]):
        p.q_start = torch.tensor(bad, dtype=torch.int32, device="cuda")
        p.run(ws=ws)
        assert _lib.moe_read_device_status(ws) == _lib.MOE_ERR_PAGE
    p.q_start = q_start
    p.prefix_pages = pages.clone()
    p.prefix_pages[1] = p.cache.n_pages
    p.run(ws=ws)
    assert _lib.moe_read_device_status(ws) == _lib.MOE_ERR_PAGE
    p.prefix_pages = pages
    assert torch.equal(p.run(ws=ws), good) and _lib.moe_read_device_status(ws) == 0
    # without a workspace the cache's status has it
    p.table = table.clone()
    p.table[0, 0] = -1
    p.run()
    assert _lib.moe_read_device_status(p.cache.status) == _lib.MOE_ERR_PAGE


def test_prompt_on_streams_and_replayed_with_other_lengths():
    """Two calls at once, and a captured one replayed after its lengths, tables and
    starts have changed."""
    p = Prompt([(70, 70), (100, 400), (1, 9)], 16, 2, 128, 16, seed=13)
    want = p.run().clone()
    streams = [torch.cuda.Stream() for _ in range(2)]
    wss = [p.cache.prompt_workspace(p.T, 3, 16) for _ in range(2)]
    outs = [torch.zeros_like(p.q) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, ws, out in zip(streams, wss, outs):
            p.run(out=out, ws=ws, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    own = p.run(stream=streams[0])
    torch.cuda.synchronize()
    assert torch.equal(own, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run(out=outs[0], ws=wss[0])
    outs[0].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want)
    # the middle sequence's rows become two single tokens and the last one's the rest
    p.seqs = [(70, 70), (2, 300), (9, 9)]
    p.starts = [0, 70, 72, 81]
    p.q_start.copy_(torch.tensor(p.starts, dtype=torch.int32))
    p.seq_len.copy_(torch.tensor([70, 300, 9], dtype=torch.int32))
    p.k[1], p.v[1] = p.k[1][:, :300], p.v[1][:, :300]
    outs[0].fill_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    p.check(outs[0])
    assert (outs[0][81:] == 3).all()
    assert _lib.moe_read_device_status(wss[0]) == 0


def test_prompt_of_a_position_beyond_32_bits_of_elements():
    """A pool of more than 2^32 elements: the last pages' offsets pass 32 bits."""
    page, Hkv, D = 65536, 2, 128
    n_pages = 2 ** 32 // (page * Hkv * D) + 3
    kp = torch.empty(n_pages, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
    g = gen(14)
    k, v = randn(g, Hkv, 200, D).cuda(), randn(g, Hkv, 200, D).cuda()
    kp[n_pages - 1, :, :200], kp[n_pages - 2, :, :200] = k, v
    # keys and values in one buffer: values a page before the keys
    cache = attention.PagedCache(kp[1:], kp[:-1])
    table = torch.tensor([[n_pages - 2]], dtype=torch.int32, device="cuda")
    q = randn(g, 200, 16, D).cuda()
    out = cache.attend_prompt(q, torch.tensor([0, 200], dtype=torch.int32, device="cuda"), table,
                              torch.tensor([200], dtype=torch.int32, device="cuda"))
    s = torch.einsum("thd,hjd->htj", q.double(), k.double().repeat_interleave(8, 0)) / math.sqrt(D)
    s = s.masked_fill(torch.arange(200, device="cuda") > torch.arange(200, device="cuda")[:, None], -math.inf)
    want = torch.einsum("htj,hjd->thd", torch.softmax(s, -1), v.double().repeat_interleave(8, 0))
    assert ((out.double() - want).abs() <= tol_of(want, v)).all()


def test_prompt_sublayer_layer_and_scores_together():
    """Two prompts through attention, MoE layer and output head: the same numbers
    as token by token through the decoding calls."""
    H, Hq, Hkv, D, V = 256, 8, 2, 64, 1000
    cfg = synthetic.CONFIGS["tiny"]
    assert cfg.H == H
    L = synthetic.make_layer(cfg, device="cuda")
    layer = moe.PackedLayer.from_fp32(cfg, L.router_w, L.router_bias, L.w_gate, L.w_up, L.w_down)
    g = gen(15)
    qkv = moe.pack_matrix(torch.randn((Hq + 2 * Hkv) * D, H, generator=g).cuda() / H ** 0.5, 64)
    proj = moe.pack_matrix(torch.randn(H, Hq * D, generator=g).cuda() / (Hq * D) ** 0.5, 64)
    head = moe.pack_matrix(torch.randn(V, H, generator=g).cuda() / H ** 0.5 * 3, 64)
    inv_freq = (10000.0 ** (-torch.arange(D // 2) / (D // 2))).cuda()
    att = attention.AttentionLayer(qkv, proj, Hq, Hkv, D, inv_freq)
    lens = [70, 33]
    T = sum(lens)
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(lens)]).to(torch.int32).cuda()
    index = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).cuda()
    q_start = torch.tensor([0, 70, T], dtype=torch.int32, device="cuda")
    seq_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    table = torch.arange(10, dtype=torch.int32, device="cuda").view(2, 5)
    x = randn(g, T, H).cuda()
    norm_w = torch.ones(H, device="cuda")

    cache = attention.PagedCache.empty(10, Hkv, 16, D)
    attn = att.prefill(x, cache, seq, index, q_start, table, seq_len)
    hidden = layer.prefill_block(attn, x, norm_w, layer.workspace(T))
    targets = torch.randint(0, V, (T,), generator=g).to(torch.int32).cuda()
    got = scores.OutputHead(head, rows=40).logprobs(hidden, targets, n_top=3)
    assert _lib.moe_read_device_status(cache.status) == 0

    steps = attention.PagedCache.empty(10, Hkv, 16, D)
    ws = steps.workspace(1, Hq)
    rows = []
    for t in range(T):
        b = int(seq[t])
        rows.append(att.decode(x[t:t + 1], steps, torch.zeros(1, dtype=torch.int32, device="cuda"), index[t:t + 1],
                               table[b:b + 1].contiguous(), index[t:t + 1] + 1, ws))
    step = torch.cat(rows)
    used = torch.arange(16, device="cuda")
    for b, n in enumerate(lens):
        for j, pg in enumerate(table[b].tolist()):
            m = (j * 16 + used < n)
            # (projections of both calls are within half a step of the exact ones: rotated keys a step apart)
            assert (cache.k[pg][:, m].float() - steps.k[pg][:, m].float()).abs().max() <= \
                4 * BF16 * float(steps.k[pg][:, m].abs().max()) if m.any() else True
    # bf16 roundings of queries, keys, values and attention, each half a step, through the projection
    assert (attn.float() - step.float()).norm() <= 8 * BF16 * step.float().norm()
    logits = moe.linear_prompt(head, hidden, dtype=torch.float32).double()
    lp = torch.log_softmax(logits, -1)
    want = lp.gather(1, targets.long()[:, None])[:, 0]
    assert (got.logprob.double() - want).abs().max() <= 2e-5
    assert (got.entropy.double() + (lp.exp() * lp).sum(-1)).abs().max() <= 2e-5
    top = lp.topk(3, -1)
    assert torch.equal(got.top_ids.long(), top.indices) and (got.top_logprobs.double() - top.values).abs().max() <= 2e-5


@pytest.mark.parametrize("n", [32, 33, 400, 1100])
def test_prompt_of_many_sequences(n):
    # sequences of one to some tokens, empty ones and padding between them, over more
    # than a warp's lanes and more than 32 of each
    g = gen(n)
    seqs = []
    for _ in range(n):
        rows = int(torch.randint(0, 6, (1,), generator=g))
        seqs.append((0, -1) if rows == 5 else (rows, rows + int(torch.randint(0, 40, (1,), generator=g))))
    c = Prompt(seqs + [(300, 700)], 2, 1, 64, 16, 0, True, seed=9, lead=3, tail=2)
    out = torch.full_like(c.q, 7.0)
    c.run(out=out)
    c.check(out)
    assert (out[:3] == 7.0).all() and (out[-2:] == 7.0).all()
