"""Sizes of the prompt calls' workspaces, on the host."""
import ctypes

import pytest

from int4_grouped_gemm_gb300 import _lib

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from int4_grouped_gemm_gb300 import build
    build.build()
    return _lib.load()


@pytest.mark.parametrize("N,K,group", [(131072, 2048, 64), (5000, 32768, 32), (1, 32, 32)])
def test_a_linear_of_few_tokens_asks_for_no_scratch(lib, N, K, group):
    """64 tokens and fewer are int4_linear's, which has none."""
    w = _lib.moe_qweight(256, 512, 768)
    f = _lib.int4_linear_prompt_workspace_bytes
    for T in (1, 8, 64):
        assert 0 < f(N, K, group, T) <= 4096

        def call(n):
            # (turned away after the workspace, for want of a device)
            return lib.int4_linear_prompt(ctypes.byref(w), N, K, group, P(1024), K, T, P(2048), N, 0, P(4096), n, None, None)

        assert call(f(N, K, group, T) - 1) == _lib.MOE_ERR_WORKSPACE
    sizes = [f(N, K, group, T) for T in (1, 64, 65, 66, 300, 2048, 2049)]
    assert sizes == sorted(sizes) and f(N, K, group, 65) > 4096
