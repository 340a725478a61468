"""Host-side refusals of the attention sub-layer's C entries (no GPU needed):
every case must be turned away before a device or a pointer is touched."""
import ctypes

import pytest

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from int4_grouped_gemm_gb300 import _lib, build
    build.build()
    return _lib.load()


def test_linear_refusals(lib):
    from int4_grouped_gemm_gb300 import _lib
    w = _lib.moe_qweight(256, 512, 768)

    def call(w=w, N=64, K=128, group=64, x=P(1024), xs=128, B=4, y=P(2048), ys=64, fp32=0, status=None):
        return lib.int4_linear(None if w is None else ctypes.byref(w), N, K, group, x, xs, B, y, ys, fp32, status, None)

    assert call(w=None) == _lib.MOE_ERR_NULL
    assert call(w=_lib.moe_qweight(256, 0, 768)) == _lib.MOE_ERR_NULL
    assert call(w=_lib.moe_qweight(256, 520, 768)) == _lib.MOE_ERR_ALIGN
    assert call(x=None) == _lib.MOE_ERR_NULL
    assert call(y=P(2056)) == _lib.MOE_ERR_ALIGN
    assert call(status=P(6)) == _lib.MOE_ERR_ALIGN
    for bad in (dict(group=16), dict(group=48), dict(K=96), dict(K=0), dict(K=32832, xs=32832), dict(N=0), dict(N=-5),
                dict(xs=127), dict(xs=129), dict(xs=120), dict(ys=63), dict(fp32=2),
                dict(xs=1 << 39)):
        assert call(**bad) == _lib.MOE_ERR_SHAPE, bad
    for B in (0, -1, 65):
        assert call(B=B) == _lib.MOE_ERR_TOKENS


def pages(_lib, **kw):
    d = dict(k=4096, v=8192, n_pages=8, page_size=16, Hkv=2, D=128, page_stride=4096, head_stride=2048, pos_stride=128)
    d.update(kw)
    return _lib.gqa_pages(**d)


BAD_PAGES = [dict(D=96), dict(page_size=8), dict(page_size=24), dict(page_size=131072), dict(n_pages=0), dict(Hkv=0),
             dict(Hkv=257), dict(pos_stride=64), dict(pos_stride=132), dict(head_stride=100), dict(page_stride=0),
             dict(page_stride=1 << 39), dict(page_stride=-4096)]


def test_append_refusals(lib):
    from int4_grouped_gemm_gb300 import _lib

    def call(c=None, q=P(16), qs=512, k=P(32), ks=256, v=P(64), vs=256, T=3, Hq=4, seq=P(128), index=P(256),
             table=P(512), n_seq=2, ld=4, off=0, inv=P(1024), rot=64, inter=0, qo=P(2048), qos=512, status=None):
        c = pages(_lib) if c is None else c
        return lib.gqa_append(ctypes.byref(c), q, qs, k, ks, v, vs, T, Hq, seq, index, table, n_seq, ld, off, inv, rot,
                              inter, qo, qos, status, None)

    assert lib.gqa_append(None, *[None] * 1, 0, None, 0, None, 0, 1, 1, None, None, None, 1, 1, 0, None, 0, 0, None, 0,
                          None, None) == _lib.MOE_ERR_NULL
    for bad in BAD_PAGES:
        assert call(c=pages(_lib, **bad)) == _lib.MOE_ERR_SHAPE, bad
    assert call(c=pages(_lib, k=0)) == _lib.MOE_ERR_NULL
    assert call(c=pages(_lib, v=8200)) == _lib.MOE_ERR_ALIGN
    for name in ("k", "v", "seq", "index", "table", "q", "qo", "inv"):
        assert call(**{name: None}) == _lib.MOE_ERR_NULL, name
    for name in ("k", "v", "q", "qo"):
        assert call(**{name: P(40)}) == _lib.MOE_ERR_ALIGN, name
    for name in ("inv", "seq", "index", "table"):
        assert call(**{name: P(42)}) == _lib.MOE_ERR_ALIGN, name
    assert call(status=P(2)) == _lib.MOE_ERR_ALIGN
    for bad in (dict(rot=8), dict(rot=144), dict(rot=-16), dict(inter=2), dict(Hq=0), dict(Hq=257), dict(qs=504),
                dict(qs=516), dict(ks=248), dict(vs=260), dict(qos=0), dict(qo=P(16), qos=1024)):
        assert call(**bad) == _lib.MOE_ERR_SHAPE, bad
    for bad in (dict(T=0), dict(T=(1 << 24) + 1), dict(n_seq=0), dict(ld=0), dict(off=-1), dict(off=(1 << 30) + 1)):
        assert call(**bad) == _lib.MOE_ERR_TOKENS, bad


def test_attention_refusals_and_workspace(lib):
    from int4_grouped_gemm_gb300 import _lib

    def call(c=None, q=P(16), qs=2048, B=3, Hq=16, pp=P(32), plen=100, table=P(64), ld=4, lens=P(128), scale=0.1,
             out=P(1024), os=2048, ws=P(4096), n=1 << 40):
        c = pages(_lib) if c is None else c
        return lib.gqa_paged_attention(ctypes.byref(c), q, qs, B, Hq, pp, plen, table, ld, lens, ctypes.c_float(scale),
                                       out, os, ws, n, None)

    for bad in BAD_PAGES:
        assert call(c=pages(_lib, **bad)) == _lib.MOE_ERR_SHAPE, bad
    for name in ("q", "pp", "table", "lens", "out", "ws"):
        assert call(**{name: None}) == _lib.MOE_ERR_NULL, name
    for name in ("q", "out", "ws"):
        assert call(**{name: P(40)}) == _lib.MOE_ERR_ALIGN, name
    for name in ("pp", "table", "lens"):
        assert call(**{name: P(42)}) == _lib.MOE_ERR_ALIGN, name
    for bad in (dict(Hq=15), dict(Hq=18), dict(Hq=1), dict(Hq=258), dict(c=pages(_lib, Hkv=129), Hq=258),
                dict(qs=2040), dict(qs=2052), dict(os=1024), dict(out=P(16), os=4096), dict(scale=float("nan")),
                dict(scale=float("inf"))):
        assert call(**bad) == _lib.MOE_ERR_SHAPE, bad
    for bad in (dict(B=0), dict(B=1025), dict(plen=-1), dict(plen=(1 << 26) + 1), dict(ld=0), dict(ld=1 << 23)):
        assert call(**bad) == _lib.MOE_ERR_TOKENS, bad
    f = _lib.gqa_paged_workspace_bytes
    assert f(8, 16, 2, 128, 0) >= 256
    assert f(8, 16, 2, 128, 1000) >= f(8, 16, 2, 128, 0)
    for bad in ((0, 16, 2, 128, 0), (1025, 16, 2, 128, 0), (8, 15, 2, 128, 0), (8, 18, 2, 128, 0), (8, 16, 2, 96, 0),
                (8, 16, 2, 128, -1), (8, 257, 257, 64, 0)):
        assert f(*bad) == 0, bad


def test_status_text(lib):
    from int4_grouped_gemm_gb300 import _lib
    assert "page" in _lib.status_string(_lib.MOE_ERR_PAGE)
