"""What OutputHead refuses, without a GPU."""
import pytest
import torch

from int4_grouped_gemm_gb300 import scores
from test_attention_layer_binding import BF, matrix


@pytest.mark.parametrize("rows", [2, 100])
def test_targets_of_another_length(rows):
    """Ones that are too many would be left out without a word."""
    head = scores.OutputHead(matrix(), rows=rows)
    x = torch.zeros(5, 128, dtype=BF)
    for shape in ((6,), (4,), (0,), (5, 1), (1,)):
        with pytest.raises(ValueError, match=r"targets \[5\]"):
            head.logprobs(x, torch.zeros(shape, dtype=torch.int32), 2)
