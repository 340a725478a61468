"""Errors that the attention sub-layer finds on the device reach the caller on every
path: a wait that runs out for certain, a bad page in a call without a workspace."""
import pytest
import torch

from int4_grouped_gemm_gb300 import _lib, attention, moe

pytestmark = pytest.mark.gpu


def matrix(N, K, G, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randn(N, K, generator=g, device="cuda") / K ** 0.5
    return moe.pack_matrix(w, G)


class Step:
    """12 rows behind a prefix (more than eight: the tensor-core projections)."""

    def __init__(self):
        self.B, self.H, Hq, Hkv, D, page = 12, 1024, 8, 2, 64, 16
        self.layer = attention.AttentionLayer(matrix((Hq + 2 * Hkv) * D, self.H, 64, 1), matrix(self.H, Hq * D, 64, 2), Hq, Hkv, D,
                                              (1e4 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float().cuda())
        self.cache = attention.PagedCache.empty(40, Hkv, page, D)
        g = torch.Generator(device="cuda").manual_seed(3)
        for t in (self.cache.k, self.cache.v):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        self.x = torch.randn(self.B, self.H, generator=g, device="cuda").to(torch.bfloat16)
        self.prefix, self.P = torch.arange(10, dtype=torch.int32, device="cuda"), 150
        self.table = torch.arange(10, 34, dtype=torch.int32, device="cuda").view(12, 2)
        self.seq = torch.arange(12, dtype=torch.int32, device="cuda")
        self.index = torch.full((12,), 20, dtype=torch.int32, device="cuda")
        self.ws = self.cache.workspace(self.B, Hq, self.P)

    def decode(self, **kw):
        return self.layer.decode(self.x, self.cache, self.seq, self.index, self.table, self.index + 1, self.ws, self.prefix, self.P,
                                 **kw)


def timeout(code):
    return _lib.MOE_ERR_TIMEOUT - 100 < code <= _lib.MOE_ERR_TIMEOUT


@pytest.mark.parametrize("B, K, N", [(9, 256, 40), (40, 2048, 3000), (64, 4096, 30000), (16, 8192, 300)])
def test_linear_waits_that_run_out_are_recorded(B, K, N):
    """One block of rows, several, several rounds of tiles, a cluster that shares K."""
    w = matrix(N, K, 64, 5)
    x = torch.randn(B, K, device="cuda").to(torch.bfloat16)
    want = moe.linear(w, x, dtype=torch.float32)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    old = _lib.moe_set_wait_limit(1)
    try:
        moe.linear(w, x, dtype=torch.float32, status=status)
        torch.cuda.synchronize()
    finally:
        _lib.moe_set_wait_limit(old)
    assert timeout(_lib.moe_read_device_status(status))
    assert torch.equal(moe.linear(w, x, dtype=torch.float32, status=status), want)
    assert _lib.moe_read_device_status(status) == 0


@pytest.mark.parametrize("B, Hq, D, P", [(2, 8, 128, 100), (16, 16, 128, 2000), (40, 8, 64, 40000)])
def test_attention_waits_that_run_out_are_recorded(B, Hq, D, P):
    cache = attention.PagedCache.empty(-(-P // 64) + B, 2, 64, D)
    cache.k.normal_()
    cache.v.normal_()
    q = torch.randn(B, Hq, D, device="cuda").to(torch.bfloat16)
    pages = torch.arange(cache.n_pages, dtype=torch.int32, device="cuda")
    lens = torch.full((B,), 30, dtype=torch.int32, device="cuda")
    ws = cache.workspace(B, Hq, P)

    def run():
        return cache.attend(q, pages[-B:].view(B, 1), lens, pages[:-B], P, ws=ws)
    want = run()
    old = _lib.moe_set_wait_limit(1)
    try:
        run()
        torch.cuda.synchronize()
    finally:
        _lib.moe_set_wait_limit(old)
    assert timeout(_lib.moe_read_device_status(ws))
    _lib.moe_workspace_init(ws)
    assert torch.equal(run(), want) and _lib.moe_read_device_status(ws) == 0


def test_a_step_records_the_projections_errors():
    s = Step()
    want = s.decode()
    assert _lib.moe_read_device_status(s.cache.status) == 0 and _lib.moe_read_device_status(s.ws) == 0
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    old = _lib.moe_set_wait_limit(1)
    try:
        s.decode()
        s.layer.project(s.x, status=status)
        torch.cuda.synchronize()
    finally:
        _lib.moe_set_wait_limit(old)
    assert timeout(_lib.moe_read_device_status(s.cache.status))
    assert timeout(_lib.moe_read_device_status(status))
    _lib.moe_workspace_init(s.ws)
    assert torch.equal(s.decode(), want)
    assert _lib.moe_read_device_status(s.cache.status) == 0 and _lib.moe_read_device_status(s.ws) == 0


@pytest.mark.parametrize("side", [False, True], ids=["current stream", "other stream"])
def test_attend_without_a_workspace_records_its_errors_with_the_cache(side):
    s = Step()
    q = torch.randn(12, 8, 64, device="cuda").to(torch.bfloat16)
    stream = torch.cuda.Stream() if side else None
    torch.cuda.synchronize()

    def run(table, prefix):
        # what the allocator hands out holds anything
        torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        out = s.cache.attend(q, table, s.index, prefix, s.P, stream=stream)
        torch.cuda.synchronize()
        return out
    good = s.cache.attend(q, s.table, s.index, s.prefix, s.P, ws=s.ws)
    assert torch.equal(run(s.table, s.prefix), good) and int(s.cache.status[0]) == 0
    bad = s.table.clone()
    bad[3, 1] = 40
    out = run(bad, s.prefix)
    assert _lib.moe_read_device_status(s.cache.status) == _lib.MOE_ERR_PAGE
    assert torch.equal(out[:3], good[:3]) and torch.equal(out[4:], good[4:])
    run(s.table, torch.full_like(s.prefix, -1))
    assert _lib.moe_read_device_status(s.cache.status) == _lib.MOE_ERR_PAGE
    assert torch.equal(run(s.table, s.prefix), good) and _lib.moe_read_device_status(s.cache.status) == 0


def test_the_first_error_of_a_cache_stays():
    """An append's error is not lost by an attend without a workspace that follows."""
    s = Step()
    k = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    s.cache.append(None, k, k, one, one + 99, s.table, None)
    s.cache.attend(torch.zeros(12, 8, 64, dtype=torch.bfloat16, device="cuda"), s.table, s.index)
    assert _lib.moe_read_device_status(s.cache.status) == _lib.MOE_ERR_PAGE


def test_attend_without_a_workspace_in_a_graph():
    """The scratch is the graph's own and cleared in each replay."""
    s = Step()
    q = torch.randn(12, 8, 64, device="cuda").to(torch.bfloat16)
    want = s.cache.attend(q, s.table, s.index, s.prefix, s.P, ws=s.ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = s.cache.attend(q, s.table, s.index, s.prefix, s.P)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
    s.table[5, 0] = -7
    graph.replay()
    assert _lib.moe_read_device_status(s.cache.status) == _lib.MOE_ERR_PAGE


@pytest.mark.parametrize("B", [1, 31, 32, 256, 257, 1024])
@pytest.mark.parametrize("prefix", [0, 40])
def test_attend_records_nothing_where_nothing_is_wrong(B, prefix):
    """At row counts that are counted another way, in a workspace of the test's own."""
    cache = attention.PagedCache.empty(2 * B + 3, 2, 16, 64)
    cache.k.normal_()
    cache.v.normal_()
    pages = torch.arange(2 * B + 3, dtype=torch.int32, device="cuda")
    lens = torch.arange(B, dtype=torch.int32, device="cuda") % 34 - 1
    ws = cache.workspace(B, 4, prefix)
    q = torch.randn(B, 4, 64, device="cuda").to(torch.bfloat16)
    cache.attend(q, pages[3:].view(B, 2), lens, pages[:3] if prefix else None, prefix, ws=ws)
    assert _lib.moe_read_device_status(ws) == 0
    lens[-1] = 33
    cache.attend(q, pages[3:].view(B, 2), lens, pages[:3] if prefix else None, prefix, ws=ws)
    assert _lib.moe_read_device_status(ws) == _lib.MOE_ERR_PAGE
