"""Host-side refusals of the prompt's C entries and Python calls (no GPU needed):
every case is turned away before a device or a pointer is touched."""
import ctypes

import pytest
import torch

from int4_grouped_gemm_gb300 import _lib, attention, moe, scores
from test_attention_layer_abi import BAD_PAGES, pages
from test_attention_layer_binding import BF, cache, ints, matrix

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from int4_grouped_gemm_gb300 import build
    build.build()
    return _lib.load()


def test_linear_prompt_refusals(lib):
    w = _lib.moe_qweight(256, 512, 768)

    def call(w=w, N=64, K=128, group=64, x=P(1024), xs=128, T=400, y=P(2048), ys=64, fp32=0, ws=P(4096), n=1 << 40,
             status=None):
        return lib.int4_linear_prompt(None if w is None else ctypes.byref(w), N, K, group, x, xs, T, y, ys, fp32, ws, n,
                                      status, None)

    assert call(w=None) == _lib.MOE_ERR_NULL
    assert call(w=_lib.moe_qweight(256, 0, 768)) == _lib.MOE_ERR_NULL
    assert call(w=_lib.moe_qweight(256, 520, 768)) == _lib.MOE_ERR_ALIGN
    for name in ("x", "y", "ws"):
        assert call(**{name: None}) == _lib.MOE_ERR_NULL, name
        assert call(**{name: P(2056)}) == _lib.MOE_ERR_ALIGN, name
    assert call(status=P(6)) == _lib.MOE_ERR_ALIGN
    for bad in (dict(group=16), dict(group=48), dict(K=96), dict(K=0), dict(K=32832, xs=32832), dict(N=0), dict(N=-5),
                dict(N=(1 << 30) + 1, ys=1 << 31), dict(xs=127), dict(xs=129), dict(xs=120), dict(ys=63), dict(fp32=2),
                dict(xs=1 << 39), dict(ys=1 << 39)):
        assert call(**bad) == _lib.MOE_ERR_SHAPE, bad
    for T in (0, -1, (1 << 20) + 1):
        assert call(T=T) == _lib.MOE_ERR_TOKENS
    assert call(n=0) == _lib.MOE_ERR_WORKSPACE
    f = _lib.int4_linear_prompt_workspace_bytes
    assert call(n=f(64, 128, 64, 400) - 1) == _lib.MOE_ERR_WORKSPACE
    for bad in ((0, 128, 64, 1), (64, 96, 64, 1), (64, 128, 48, 1), (64, 128, 64, 0), (64, 128, 64, (1 << 20) + 1)):
        assert f(*bad) == 0, bad
    # a call of fewer tokens fits a workspace of more
    sizes = [f(5000, 2048, 64, T) for T in (1, 65, 128, 129, 1000, 4096, 20000, 1 << 20)]
    assert sizes == sorted(sizes) and sizes[0] > 0


def test_prompt_attention_refusals(lib):
    def call(c=None, q=P(16), qs=2048, T=30, Hq=16, start=P(32), n_seq=3, pp=P(32), plen=100, table=P(64), ld=4,
             lens=P(128), scale=0.1, out=P(1024), os=2048, ws=P(4096), n=1 << 40, status=None):
        c = pages(_lib) if c is None else c
        return lib.gqa_prompt_attention(ctypes.byref(c), q, qs, T, Hq, start, n_seq, pp, plen, table, ld, lens,
                                        ctypes.c_float(scale), out, os, ws, n, status, None)

    for bad in BAD_PAGES:
        assert call(c=pages(_lib, **bad)) == _lib.MOE_ERR_SHAPE, bad
    for name in ("q", "start", "pp", "table", "lens", "out", "ws"):
        assert call(**{name: None}) == _lib.MOE_ERR_NULL, name
    for name in ("q", "out", "ws"):
        assert call(**{name: P(40)}) == _lib.MOE_ERR_ALIGN, name
    for name in ("start", "pp", "table", "lens", "status"):
        assert call(**{name: P(42)}) == _lib.MOE_ERR_ALIGN, name
    for bad in (dict(Hq=15), dict(Hq=18), dict(Hq=1), dict(Hq=258), dict(c=pages(_lib, Hkv=129), Hq=258),
                dict(qs=2040), dict(qs=2052), dict(os=1024), dict(out=P(16), os=4096), dict(scale=float("nan")),
                dict(scale=float("inf"))):
        assert call(**bad) == _lib.MOE_ERR_SHAPE, bad
    for bad in (dict(T=0), dict(T=-3), dict(T=(1 << 22) + 1), dict(n_seq=0), dict(n_seq=65537), dict(plen=-1),
                dict(plen=(1 << 26) + 1), dict(ld=0), dict(ld=1 << 23)):
        assert call(**bad) == _lib.MOE_ERR_TOKENS, bad
    assert call(n=0) == _lib.MOE_ERR_WORKSPACE
    f = _lib.gqa_prompt_workspace_bytes
    assert f(1, 1, 16, 2, 128) >= 256
    for bad in ((0, 1, 16, 2, 128), (1, 0, 16, 2, 128), (1, 1, 15, 2, 128), (1, 1, 18, 2, 128), (1, 1, 16, 2, 96),
                ((1 << 22) + 1, 1, 16, 2, 128), (1, 65537, 16, 2, 128)):
        assert f(*bad) == 0, bad


def test_token_logprobs_refusals(lib):
    def call(x=P(16), stride=100, fp32=1, T=3, V=100, targets=P(64), lp=P(128), h=P(256), n_top=4, ids=P(512), top=P(768),
             ws=P(1024), n=1 << 40, status=None):
        return lib.token_logprobs(x, stride, fp32, T, V, targets, lp, h, n_top, ids, top, ws, n, status, None)

    for name in ("x", "targets", "lp", "ids", "top", "ws"):
        assert call(**{name: None}) == _lib.MOE_ERR_NULL, name
    for name in ("x", "targets", "lp", "h", "ids", "top", "status"):
        assert call(**{name: P(42)}) == _lib.MOE_ERR_ALIGN, name
    assert call(x=P(41), fp32=0) == _lib.MOE_ERR_ALIGN
    assert call(ws=P(1032)) == _lib.MOE_ERR_ALIGN
    for bad in (dict(fp32=2), dict(V=0), dict(V=(1 << 28) + 1, stride=1 << 29), dict(n_top=-1), dict(n_top=33),
                dict(V=3, stride=3), dict(stride=99), dict(stride=1 << 39)):
        assert call(**bad) == _lib.MOE_ERR_SHAPE, bad
    for T in (0, -1, (1 << 24) + 1):
        assert call(T=T) == _lib.MOE_ERR_TOKENS
    assert call(n=0) == _lib.MOE_ERR_WORKSPACE
    f = _lib.token_logprobs_workspace_bytes
    assert f(1, 1, 0) >= 256
    for bad in ((0, 5, 0), (1, 0, 0), (1, 5, 6), (1, 100, 33), (1, 100, -1), ((1 << 24) + 1, 5, 0)):
        assert f(*bad) == 0, bad
    assert "vocabulary" in _lib.status_string(_lib.MOE_ERR_TOKEN_ID)


def test_linear_prompt_refuses_tensors():
    ws = torch.zeros(8)
    for x, what in ((torch.zeros(90, 128), r"x \[B, 128\] in bf16"), (torch.zeros(128, 90, dtype=BF).t(), "its rows contiguous"),
                    (torch.zeros(90, 128, dtype=BF), "linear: x: on cpu, the current device is cuda:0")):
        with pytest.raises(ValueError, match=what):
            moe.linear_prompt(matrix(), x, y=torch.zeros(90, 64), ws=ws)
    with pytest.raises(ValueError, match=r"linear: y \[B, 64\]"):
        moe.linear_prompt(matrix(), torch.zeros(90, 128, dtype=BF), y=torch.zeros(90, 63), ws=ws)
    with pytest.raises(_lib.MoEError):
        moe.linear_prompt(matrix(), torch.zeros(0, 128, dtype=BF))
    with pytest.raises(_lib.MoEError):
        moe.linear_prompt_workspace(matrix(), 0)


def test_attend_prompt_refuses_tensors(monkeypatch):
    c = cache()
    q, ws = torch.zeros(9, 4, 64, dtype=BF), torch.zeros(8)
    with pytest.raises(ValueError, match="attend_prompt: the cache is on cuda:-1"):
        c.attend_prompt(q, ints(4), ints(3, 2), ints(3), out=q, ws=ws)
    monkeypatch.setattr(c, "_device", 0)
    for bad, what in ((torch.zeros(9, 4, 64), r"q: \[9, heads, 64\] in bf16"),
                      (torch.zeros(9, 4, 32, dtype=BF), r"q: \[9, heads, 64\]"),
                      (torch.zeros(9, 64, 4, dtype=BF).transpose(1, 2), "heads of a row must be contiguous"),
                      (q, "q: on cpu")):
        with pytest.raises(ValueError, match=what):
            c.attend_prompt(bad, ints(4), ints(3, 2), ints(3), out=q, ws=ws)
    with pytest.raises(_lib.MoEError):
        c.prompt_workspace(0, 1, 4)
    with pytest.raises(_lib.MoEError):
        c.prompt_workspace(1, 1, 5)


def test_token_logprobs_refuses_tensors():
    x = torch.zeros(3, 50)
    for bad, what in ((x.double(), r"logits: \[T, V\] in fp32 or bf16"), (x.half(), "in fp32 or bf16"),
                      (torch.zeros(50, 3).t(), "its rows contiguous"), (x, "logits: on cpu")):
        with pytest.raises(ValueError, match=what):
            scores.token_logprobs(bad, None, 2, out=scores.TokenScores.empty(3, 2, device="cpu"), ws=torch.zeros(8))
    with pytest.raises(ValueError, match=r"logits \[T, V\]"):
        scores.token_logprobs(torch.zeros(50))
    with pytest.raises(_lib.MoEError):
        scores.workspace(1, 10, 11)
    with pytest.raises(ValueError):
        scores.OutputHead(matrix(), rows=0)


def test_the_module_counts_arguments():
    n = _lib.native()
    for call in (n.linear_prompt, n.attend_prompt, n.scores):
        with pytest.raises(TypeError, match="arguments"):
            call()
