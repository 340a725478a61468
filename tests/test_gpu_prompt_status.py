"""Errors that the prompt's operators find on the device reach the caller: waits
that run out for certain are recorded, the block unwinds and the next call is as
before; a prefill's errors are in the cache's status."""
import pytest
import torch

from int4_grouped_gemm_gb300 import _lib, attention, moe, scores

pytestmark = pytest.mark.gpu


def matrix(N, K, G, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return moe.pack_matrix(torch.randn(N, K, generator=g, device="cuda") / K ** 0.5, G)


def timeout(code):
    return _lib.MOE_ERR_TIMEOUT - 100 < code <= _lib.MOE_ERR_TIMEOUT


def with_no_patience(run):
    torch.cuda.synchronize()
    old = _lib.moe_set_wait_limit(1)
    try:
        run()
        torch.cuda.synchronize()
    finally:
        _lib.moe_set_wait_limit(old)


@pytest.mark.parametrize("T, K, N, fp32", [(70, 256, 40, True), (300, 2048, 3000, False), (1000, 4096, 4000, True),
                                           (200, 1024, 60000, True)])
def test_linear_prompt_waits_that_run_out_are_recorded(T, K, N, fp32):
    """One tile, several, chunks of sums, codes unpacked by the product's kernel."""
    w = matrix(N, K, 64, 5)
    x = torch.randn(T, K, device="cuda").to(torch.bfloat16)
    dtype = torch.float32 if fp32 else torch.bfloat16
    want = moe.linear_prompt(w, x, dtype=dtype)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    with_no_patience(lambda: moe.linear_prompt(w, x, dtype=dtype, status=status))
    assert timeout(_lib.moe_read_device_status(status))
    assert torch.equal(moe.linear_prompt(w, x, dtype=dtype, status=status), want)
    assert _lib.moe_read_device_status(status) == 0


class Packed:
    def __init__(self, rows, Hq=8, D=64, page=16):
        self.H, self.rows = 256, rows
        n, T = len(rows), sum(rows)
        self.layer = attention.AttentionLayer(matrix((Hq + 4) * D, self.H, 64, 1), matrix(self.H, Hq * D, 64, 2), Hq, 2, D, None)
        per = -(-max(rows) // page)
        self.cache = attention.PagedCache.empty(n * per, 2, page, D)
        self.cache.k.normal_()
        self.cache.v.normal_()
        self.table = torch.arange(n * per, dtype=torch.int32, device="cuda").view(n, per)
        self.start = torch.tensor([sum(rows[:i]) for i in range(n + 1)], dtype=torch.int32, device="cuda")
        self.lens = torch.tensor(rows, dtype=torch.int32, device="cuda")
        self.seq = torch.cat([torch.full((r,), i) for i, r in enumerate(rows)]).to(torch.int32).cuda()
        self.index = torch.cat([torch.arange(r) for r in rows]).to(torch.int32).cuda()
        self.x = torch.randn(T, self.H, device="cuda").to(torch.bfloat16)
        self.q = torch.randn(T, Hq, D, device="cuda").to(torch.bfloat16)

    def attend(self, **kw):
        return self.cache.attend_prompt(self.q, self.start, self.table, self.lens, **kw)

    def prefill(self, **kw):
        return self.layer.prefill(self.x, self.cache, self.seq, self.index, self.start, self.table, self.lens, **kw)


@pytest.mark.parametrize("rows, Hq, D", [([5], 8, 64), ([300, 20], 16, 128), ([3000, 1, 700], 8, 64)])
def test_prompt_waits_that_run_out_are_recorded(rows, Hq, D):
    p = Packed(rows, Hq, D)
    ws = p.cache.prompt_workspace(sum(rows), len(rows), Hq)
    want = p.attend(ws=ws)
    with_no_patience(lambda: p.attend(ws=ws))
    assert timeout(_lib.moe_read_device_status(ws))
    assert torch.equal(p.attend(ws=ws), want) and _lib.moe_read_device_status(ws) == 0
    with_no_patience(p.attend)
    assert timeout(_lib.moe_read_device_status(p.cache.status))


def test_a_prefill_records_its_errors_and_recovers():
    p = Packed([140, 33])
    want = p.prefill()
    assert _lib.moe_read_device_status(p.cache.status) == 0
    with_no_patience(p.prefill)
    assert timeout(_lib.moe_read_device_status(p.cache.status))
    assert torch.equal(p.prefill(), want) and _lib.moe_read_device_status(p.cache.status) == 0
    table = p.table.clone()
    p.table[1, 1] = p.cache.n_pages
    out = p.prefill()
    assert _lib.moe_read_device_status(p.cache.status) == _lib.MOE_ERR_PAGE
    assert torch.equal(out[:140], want[:140])
    p.table.copy_(table)
    # on another stream, and from a graph replayed with other lengths
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = p.prefill(stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = p.prefill()
    out.zero_()
    graph.replay()
    assert torch.equal(out, want) and _lib.moe_read_device_status(p.cache.status) == 0
    p.lens[1] = p.table.shape[1] * 16 + 1
    graph.replay()
    assert _lib.moe_read_device_status(p.cache.status) == _lib.MOE_ERR_PAGE
    assert torch.equal(out[:140], want[:140])


def test_two_captured_graphs_may_share_a_workspace_in_turn():
    """Replays one after the other: what one leaves in the workspace is nothing to
    the other."""
    p, r = Packed([500, 3]), Packed([70, 900, 8])
    ws = p.cache.prompt_workspace(2000, 3, 8)
    wants = [p.attend(), r.attend()]
    graphs, outs = [], []
    for c in (p, r):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c.attend(ws=ws))
        graphs.append(g)
    for _ in range(3):
        for g, out, want in zip(graphs, outs, wants):
            out.zero_()
            g.replay()
            assert torch.equal(out, want)


def test_head_and_scores_record_a_token_outside_the_vocabulary():
    head = scores.OutputHead(matrix(500, 256, 64, 7), rows=30)
    x = torch.randn(70, 256, device="cuda").to(torch.bfloat16)
    targets = torch.arange(70, dtype=torch.int32, device="cuda")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    want = head.logprobs(x, targets, 4, status=status)
    assert _lib.moe_read_device_status(status) == 0
    targets[65] = 500
    got = head.logprobs(x, targets, 4, status=status)
    assert _lib.moe_read_device_status(status) == _lib.MOE_ERR_TOKEN_ID
    keep = torch.arange(70, device="cuda") != 65
    assert torch.isnan(got.logprob[65]) and torch.equal(got.logprob[keep], want.logprob[keep])
    assert all(torch.equal(a, b) for a, b in zip(got[1:], want[1:]))
    assert head.logprobs(x[:0], targets[:0], 4).entropy.shape == (0,)
