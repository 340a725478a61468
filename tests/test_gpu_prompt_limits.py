"""The prompt operators at the ends of their documented ranges, and calls that run
at the same time.  Tolerances as derived in the operators' own tests."""
import pytest
import torch

from int4_grouped_gemm_gb300 import _lib, attention, moe, scores
from test_gpu_attention_layer import gen, make_int4, randn
from test_gpu_linear_prompt import bound
from test_gpu_prompt import Prompt

pytestmark = pytest.mark.gpu


def test_prompt_of_the_most_sequences():
    # one position a sequence: the only weight is one, and the row is the value as it is
    n, D = 65536, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    kp, vp = (torch.randn(n, 1, 16, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    cache = attention.PagedCache(kp, vp)
    q = torch.randn(n, 2, D, generator=g, device="cuda").to(torch.bfloat16)
    table = torch.randperm(n, generator=g, device="cuda").to(torch.int32).view(n, 1)
    start = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    lens = torch.ones(n, dtype=torch.int32, device="cuda")
    out = cache.attend_prompt(q, start, table, lens)
    assert torch.equal(out, vp[table[:, 0].long(), 0, :1].expand(-1, 2, -1))
    assert _lib.moe_read_device_status(cache.status) == 0


def test_prompt_of_sequences_that_share_their_pages():
    c = Prompt([(40, 300), (40, 300), (7, 300)], 8, 2, 128, 64, seed=5)
    c.table[1], c.table[2] = c.table[0], c.table[0]
    c.k, c.v = [c.k[0]] * 3, [c.v[0]] * 3
    c.check(c.run())


def test_linear_prompt_of_the_most_tokens():
    g = gen(17)
    m, w = make_int4(g, 24, 32, 32)
    x = randn(g, 1 << 20, 32)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    got = moe.linear_prompt(m, x.cuda(), dtype=torch.float32, status=status)
    want = x.cuda().double() @ w.cuda().t()
    assert ((got.double() - want).abs() <= bound(x.cuda(), w.cuda(), 32)).all()
    assert _lib.moe_read_device_status(status) == 0
    with pytest.raises(_lib.MoEError):
        moe.linear_prompt(m, torch.empty((1 << 20) + 1, 32, dtype=torch.bfloat16, device="cuda"))


def test_scores_of_the_largest_vocabulary():
    # a row of this length is cut over more than 2^7 blocks of 2^8 threads, fewer than
    # 2^13 scores each: sums of fewer than 2^13 + 2^9 additions, each 2^-24 of itself
    # off, and as much again in the entropy's second one
    V = 1 << 28
    x = torch.zeros(1, V, device="cuda")
    at = torch.tensor([5, V - 1, 1 << 27, 77], device="cuda")
    x[0, at] = torch.tensor([3.0, 2.5, 2.0, 1.5], device="cuda")
    t = torch.tensor([V - 1], dtype=torch.int32, device="cuda")
    got = scores.token_logprobs(x, t, 5)
    lse = torch.logsumexp(x[0].double(), 0)
    assert got.top_ids[0].tolist() == at.tolist() + [0]
    assert abs(float(got.logprob[0].double() - (2.5 - lse))) <= 2.0 ** -10
    assert abs(float(got.entropy[0].double() - (lse - (torch.softmax(x[0].double(), 0) * x[0]).sum()))) <= 2.0 ** -9


def test_calls_on_two_streams_at_the_same_time():
    g = gen(23)
    m, w = make_int4(g, 5000, 512, 64)
    streams = [torch.cuda.Stream() for _ in range(2)]
    xs = [randn(g, T, 512).cuda() for T in (900, 300)]
    rows = [torch.randn(T, 50000, generator=g).cuda() for T in (3, 200)]
    ps = [Prompt([(90, 900), (300, 300)], 16, 2, 128, 64, seed=s) for s in (1, 2)]
    want_y = [moe.linear_prompt(m, x) for x in xs]
    want_s = [scores.token_logprobs(r, None, 9) for r in rows]
    want_o = [p.run() for p in ps]
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for i, s in enumerate(streams):
            got.append((moe.linear_prompt(m, xs[i], stream=s), scores.token_logprobs(rows[i], None, 9, stream=s),
                        ps[i].run(stream=s)))
        torch.cuda.synchronize()
        for i, (y, sc, o) in enumerate(got):
            assert torch.equal(y, want_y[i]) and torch.equal(o, want_o[i])
            assert torch.equal(sc.entropy, want_s[i].entropy) and torch.equal(sc.top_ids, want_s[i].top_ids)


@pytest.mark.parametrize("T,V", [(40, 9000), (700, 900), (700, 3000), (700, 20000), (2, 100000)])
def test_scores_of_rows_with_many_equal_largest(T, V):
    # more candidates than a warp keeps unsorted: the lists are merged the long way
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randint(0, 3, (T, V), generator=g, device="cuda").float()
    for dtype in (torch.float32, torch.bfloat16):
        got = scores.token_logprobs(x.to(dtype), None, 32)
        want = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :32]
        assert torch.equal(got.top_ids.long(), want)


def test_scores_workspace_serves_fewer_rows():
    V = 60000
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(400, V, generator=g, device="cuda")
    ws = scores.workspace(400, V, 4)
    for T in (400, 7, 1, 130, 304):
        a, b = scores.token_logprobs(x[:T], None, 4, ws=ws), scores.token_logprobs(x[:T], None, 4)
        assert torch.equal(a.entropy, b.entropy) and torch.equal(a.top_ids, b.top_ids)
