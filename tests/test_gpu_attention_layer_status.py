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
