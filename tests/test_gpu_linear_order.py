"""kda_linear_prefill's tensor-core kernel over many chunks: what one product reads, the next chunk's
products may not overwrite before it is done.

P, the weighted scores of a chunk, is an operand of P V in tensor memory, and the next chunk's scores go
into the same columns.  Unless they wait for P V, only the order in which the hardware happens to run
the products keeps a row of outputs from mixing two chunks' scores; where it does not, the error is far
outside the bounds and the results change from call to call.  So: many chunks, every pair of head widths (at d_v = 64 the two products differ in shape
too), whole and cut sequences, no decay that would hide an old chunk; each output within the bounds of
test_gpu_linear.py and the same bits every time.
"""
import pytest
import torch

import kimi_delta_attention_13_gb300 as kda
from test_gpu_linear import DEV, check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    yield
    assert kda.device_status() == 0
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("lengths,H,cut", [([1536, 1], 80, False), ([2816], 2, True)], ids=["whole", "cut"])
def test_chunks_wait_for_what_they_overwrite(lengths, H, cut, dk, dv):
    x = make(lengths, H, H // 2, dk, dv, "bf16", seed=dk + 2 * dv)
    x["g"].mul_(0.01)
    need = kda.load().kda_linear_prefill_workspace(len(lengths), sum(lengths), H, dk, dv, 0)
    assert (need > 0) == cut
    args = (x["q"], x["k"], x["v"], x["g"], x["cu"], x["init"])
    got = kda.linear_prefill(*args, scale=0.3)
    check(x, got, "bf16", "bf16", 0.3)
    for _ in range(20):
        again = kda.linear_prefill(*args, scale=0.3)
        assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])
