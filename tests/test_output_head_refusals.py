"""What OutputHead refuses, without a GPU."""
import pytest
import torch

from int4_grouped_gemm_gb300 import _lib, scores
from test_attention_layer_binding import BF, matrix


@pytest.mark.parametrize("rows", [2, 100])
def test_targets_of_another_length(rows):
    """Ones that are too many would be left out without a word."""
    head = scores.OutputHead(matrix(), rows=rows)
    x = torch.zeros(5, 128, dtype=BF)
    for shape in ((6,), (4,), (0,), (5, 1), (1,)):
        with pytest.raises(ValueError, match=r"targets \[5\]"):
            head.logprobs(x, torch.zeros(shape, dtype=torch.int32), 2)


@pytest.mark.parametrize("T", [0, 5])
def test_alternatives_that_there_cannot_be(T):
    """... before memory for them is asked for."""
    head = scores.OutputHead(matrix())
    for n in (-1, 33, 65, 2 ** 31 - 1):
        with pytest.raises(_lib.MoEError):
            head.logprobs(torch.zeros(T, 128, dtype=BF), None, n)
