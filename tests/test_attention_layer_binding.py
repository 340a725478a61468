"""Refusals of the Python calls of the attention sub-layer that need no GPU: what
is wrong with an argument is said before anything reaches the library."""
import ctypes
import os

import pytest
import torch

from int4_grouped_gemm_gb300 import _lib, attention, moe

BF = torch.bfloat16


def matrix(N=64, K=128, group=64):
    return moe.QMatrix(torch.zeros(N, K // 8, dtype=torch.int32), torch.zeros(N, 8, dtype=torch.int16),
                       torch.zeros(N, 8, dtype=torch.int16), N, K, group)


def cache(n_pages=4, Hkv=2, page=16, D=64):
    return attention.PagedCache.empty(n_pages, Hkv, page, D, device="cpu")


@pytest.fixture
def on_zero(monkeypatch):
    """A cache that counts as one of the current device, so that the checks of
    the other arguments are reached."""
    c = cache()
    monkeypatch.setattr(c, "_device", 0)
    return c


def ints(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


@pytest.mark.parametrize("x, what", [
    (torch.zeros(2, 128), r"x \[B, 128\] in bf16"),
    (torch.zeros(2, 64, dtype=BF), r"x \[B, 128\] in bf16"),
    (torch.zeros(128, dtype=BF), r"x \[B, 128\] in bf16"),
    (torch.zeros(128, 2, dtype=BF).t(), "its rows contiguous"),
    (torch.zeros(2, 128, dtype=BF), "linear: x: on cpu, the current device is cuda:0"),
])
def test_linear_refuses_tokens(x, what):
    with pytest.raises(ValueError, match=what):
        moe.linear(matrix(), x, y=torch.zeros(2, 64))


@pytest.mark.parametrize("y", [torch.zeros(2, 63), torch.zeros(3, 64), torch.zeros(2, 64, dtype=torch.float16),
                               torch.zeros(64, 2).t(), torch.zeros(64)])
def test_linear_refuses_outputs(y):
    with pytest.raises(ValueError, match=r"linear: y \[B, 64\]"):
        moe.linear(matrix(), torch.zeros(2, 128, dtype=BF), y=y)


def test_linear_refuses_a_stack_and_no_tensor():
    w = matrix()
    w.q = torch.zeros(2, 64, 16, dtype=torch.int32)
    with pytest.raises(ValueError, match="not a stack"):
        moe.linear(w, torch.zeros(2, 128, dtype=BF), y=torch.zeros(2, 64))
    for x in (None, 3, [[1.0]]):
        with pytest.raises(TypeError, match="a tensor"):
            moe.linear(matrix(), x, y=torch.zeros(2, 64))
    with pytest.raises(ValueError, match="a dense tensor"):
        moe.linear(matrix(), torch.zeros(2, 128, dtype=BF).to_sparse(), y=torch.zeros(2, 64))


@pytest.mark.parametrize("name, t", [
    ("scale", torch.zeros(64, 4, dtype=torch.int16)), ("bias", torch.zeros(32, 8, dtype=torch.int16)),
    ("bias", torch.zeros(64, 8)), ("scale", torch.zeros(8, 64, dtype=torch.int16).t()),
    ("q", torch.zeros(64, 8, dtype=torch.int64).repeat(1, 2)), ("q", torch.zeros(16, 64, dtype=torch.int32).t())])
def test_linear_refuses_weights_of_another_layout(name, t):
    """Fewer scales than the kernel reads would be a read past their end."""
    w = matrix()
    setattr(w, name, t)
    with pytest.raises(ValueError, match="linear: (scales and biases|codes)"):
        moe.linear(w, torch.zeros(2, 128, dtype=BF), y=torch.zeros(2, 64))


def test_linear_refuses_rows_and_strides_past_its_index():
    """Row numbers of the last tile and offsets of y would not fit their types."""
    lib, w = _lib.load(), _lib.moe_qweight(256, 512, 768)
    P = ctypes.c_void_p

    def call(N, ys):
        return lib.int4_linear(ctypes.byref(w), N, 128, 64, P(1024), 128, 4, P(2048), ys, 0, None, None)
    assert call((1 << 30) + 1, 1 << 31) == _lib.MOE_ERR_SHAPE
    assert call((1 << 31) - 1, 1 << 31) == _lib.MOE_ERR_SHAPE
    assert call(64, 1 << 39) == _lib.MOE_ERR_SHAPE


def test_a_cache_of_another_device():
    c = cache()
    k = torch.zeros(3, 2, 64, dtype=BF)
    with pytest.raises(ValueError, match="append: the cache is on cuda:-1"):
        c.append(None, k, k, ints(3), ints(3), ints(1, 4), None)
    with pytest.raises(ValueError, match="attend: the cache is on cuda:-1"):
        c.attend(torch.zeros(3, 4, 64, dtype=BF), ints(3, 4), ints(3), ws=torch.zeros(8))


@pytest.mark.parametrize("k, what", [
    (torch.zeros(3, 2, 64), r"k: \[3, 2, 64\] in bf16"),
    (torch.zeros(3, 1, 64, dtype=BF), r"k: \[3, 2, 64\]"),
    (torch.zeros(3, 2, 32, dtype=BF), r"k: \[3, 2, 64\]"),
    (torch.zeros(2, 64, dtype=BF), r"k: \[2, 2, 64\]"),
    (torch.zeros((), dtype=BF), r"k: \[0, 2, 64\]"),
    (torch.zeros(3, 64, 2, dtype=BF).transpose(1, 2), "heads of a row must be contiguous"),
    (torch.zeros(2, 3, 64, dtype=BF).transpose(0, 1), "heads of a row must be contiguous"),
    (torch.zeros(3, 2, 64, dtype=BF), "k: on cpu"),
])
def test_append_refuses_keys(on_zero, k, what):
    with pytest.raises(ValueError, match=what):
        on_zero.append(None, k, torch.zeros(3, 2, 64, dtype=BF), ints(3), ints(3), ints(1, 4), None)


@pytest.mark.parametrize("q, what", [
    (torch.zeros(3, 4, 64), r"q: \[3, heads, 64\] in bf16"),
    (torch.zeros(3, 4, 32, dtype=BF), r"q: \[3, heads, 64\]"),
    (torch.zeros(3, 4, 64, dtype=BF), "q: on cpu"),
])
def test_attend_refuses_queries(on_zero, q, what):
    with pytest.raises(ValueError, match=what):
        on_zero.attend(q, ints(3, 4), ints(3), out=torch.zeros(3, 4, 64, dtype=BF), ws=torch.zeros(8))


def test_the_module_checks_numbers_and_their_count():
    n = _lib.native()
    for call in (n.linear, n.append, n.attend):
        with pytest.raises(TypeError, match="arguments"):
            call()
    w, x = matrix(), torch.zeros(2, 128, dtype=BF)
    with pytest.raises(ValueError, match="K: outside 32 bits"):
        n.linear(w.q, w.scale, w.bias, 64, 1 << 31, 64, x, torch.zeros(2, 64), None, None)
    with pytest.raises(TypeError):
        n.linear(w.q, w.scale, w.bias, "64", 128, 64, x, torch.zeros(2, 64), None, None)
    with pytest.raises(OverflowError):
        n.linear(w.q, w.scale, w.bias, 1 << 70, 128, 64, x, torch.zeros(2, 64), None, None)


def test_the_module_takes_addresses_only():
    n, c = _lib.native(), cache()
    k = torch.zeros(3, 2, 64, dtype=BF)
    rest = (None, k, k, ints(3), ints(3), ints(1, 4), None, 0, False, None, None)
    for pages, status, error in ((0, 0, ValueError), (None, 0, TypeError), (c._at, "x", TypeError), (c.desc, 0, TypeError)):
        with pytest.raises(error):
            n.append(pages, 0, status, *rest)
    for pages, error in ((0, ValueError), ("x", TypeError)):
        with pytest.raises(error):
            n.attend(pages, 0, k, ints(3, 4), ints(3), None, 0, 1.0, k, k, None)
    with pytest.raises(TypeError):
        n.attend(c._at, "x", k, ints(3, 4), ints(3), None, 0, 1.0, k, k, None)


def test_the_module_and_the_binding_share_one_library():
    """The module is linked to the library beside it, which ctypes has loaded:
    one set of limits and device state in the process."""
    _lib.native()
    with open("/proc/self/maps") as f:
        libs = {line.split()[-1] for line in f if "libmoe_gb300" in line}
    assert libs == {os.path.realpath(_lib.LIB_PATH)}
    assert ctypes.CDLL(_lib.LIB_PATH)._handle == _lib.load()._handle
