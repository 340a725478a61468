"""int4_linear_prompt gives the same bits however often and beside whatever it is
called: what a stage or an accumulator held before has no say."""
import pytest
import torch

from int4_grouped_gemm_gb300 import _lib, moe
from test_gpu_attention_layer import gen, make_int4, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T", [100, 700])
def test_alternating_calls_repeat_their_bits(T, fp32):
    """Two matrices whose codes the product unpacks and one whose codes it does not,
    in turn, each with tokens of its own."""
    dtype = torch.float32 if fp32 else torch.bfloat16
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    calls = []
    for i, (N, K, G) in enumerate(((20000, 1024, 64), (20000, 1056, 32), (2560, 2048, 64))):
        m, _ = make_int4(gen(i), N, K, G)
        x = randn(gen(9 + i), T, K, std=2.0 ** (10 * i)).cuda()
        calls.append((m, x, torch.empty(T, N, dtype=dtype, device="cuda"), moe.linear_prompt_workspace(m, T)))
    want = [moe.linear_prompt(m, x, dtype=dtype, ws=ws) for m, x, _, ws in calls]
    torch.cuda.synchronize()
    for _ in range(15):
        for m, x, y, ws in calls:
            moe.linear_prompt(m, x, y.fill_(float("nan")), ws=ws, status=status)
        for (_, _, y, _), w in zip(calls, want):
            assert torch.equal(y, w)
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(15):
        for s, (m, x, y, ws) in zip(streams, calls):
            moe.linear_prompt(m, x, y, ws=ws, status=status, stream=s)
    torch.cuda.synchronize()
    assert _lib.moe_read_device_status(status) == 0
    for (_, _, y, _), w in zip(calls, want):
        assert torch.equal(y, w)
