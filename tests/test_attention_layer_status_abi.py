"""Refusals of gqa_paged_attention_status, before a device or a pointer is touched."""
import ctypes

import pytest

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from int4_grouped_gemm_gb300 import _lib, build
    build.build()
    return _lib.load()


def test_status_address(lib):
    from int4_grouped_gemm_gb300 import _lib
    cache = _lib.gqa_pages(k=4096, v=8192, n_pages=8, page_size=16, Hkv=2, D=128, page_stride=4096, head_stride=2048, pos_stride=128)

    def call(B=3, status=P(16)):
        return lib.gqa_paged_attention_status(ctypes.byref(cache), P(16), 2048, B, 16, None, 0, P(64), 4, P(128),
                                              ctypes.c_float(0.1), P(1024), 2048, P(4096), 1 << 40, status, None)
    assert call(status=None) == _lib.MOE_ERR_NULL
    assert call(status=P(18)) == _lib.MOE_ERR_ALIGN
    assert call(B=0) == _lib.MOE_ERR_TOKENS
