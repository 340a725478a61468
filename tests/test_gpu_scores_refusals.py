"""token_logprobs refuses more alternatives than there can be."""
import pytest
import torch

from int4_grouped_gemm_gb300 import _lib, scores

pytestmark = pytest.mark.gpu


def test_alternatives_are_refused_before_results_are_made():
    """More than there can be: no memory is asked for."""
    x = torch.zeros(4096, 50, device="cuda")
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    for n in (33, 51, 2 ** 31 - 1):
        with pytest.raises(_lib.MoEError):
            scores.token_logprobs(x, None, n)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before


def test_the_reason_of_a_refusal():
    for x, n, code in ((torch.zeros(3, 50), 33, _lib.MOE_ERR_SHAPE), (torch.zeros(3, 5), 6, _lib.MOE_ERR_SHAPE),
                       (torch.zeros(3, 0), 0, _lib.MOE_ERR_SHAPE), (torch.zeros(0, 50), 2, _lib.MOE_ERR_TOKENS)):
        with pytest.raises(_lib.MoEError) as e:
            scores.token_logprobs(x.cuda(), None, n)
        assert e.value.code == code
