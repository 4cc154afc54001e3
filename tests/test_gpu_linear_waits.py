"""The waits of kda_linear_prefill's tensor-core kernel run out by the clock, are reported, and leave the
context as it was.  No kernel is broken for it: one warp waits for a phase that nothing completes.
"""
import time

import pytest
import torch

import kimi_delta_attention_13_gb300 as kda
from test_gpu_linear import check, make

pytestmark = pytest.mark.gpu
KDA_ERR_DEVICE_TIMEOUT = 5


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()


def test_expired_wait_is_reported_and_prefill_goes_on():
    assert kda.device_status() == 0
    kda.diag_linear_timeout(2_000_000)           # about 1 ms of SM clock
    torch.cuda.synchronize()
    assert kda.device_status() == KDA_ERR_DEVICE_TIMEOUT
    assert kda.device_status() == 0              # read and cleared
    x = make([300, 77], 2, 1, 128, 128, "bf16", seed=31)
    got = kda.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["cu"], x["init"])
    check(x, got, "bf16", "bf16", 1.0)
    assert kda.device_status() == 0


@pytest.mark.parametrize("cycles", [1_000_000, 100_000_000, 400_000_000])
def test_wait_takes_the_time_it_is_given(cycles):
    """Not sooner than at 2.1 GHz, which no clock exceeds; not later than at 0.5 GHz and a tenth of a
    second for the call and the sleep that was begun."""
    kda.diag_linear_timeout(1)
    torch.cuda.synchronize()
    t = time.perf_counter()
    kda.diag_linear_timeout(cycles)
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    assert cycles / 2.1e9 <= t <= cycles / 0.5e9 + 0.1
    assert kda.device_status() == KDA_ERR_DEVICE_TIMEOUT


def test_refuses():
    for cycles in (0, -1, 4_000_000_001):
        with pytest.raises(kda.KDAError, match="INVALID"):
            kda.diag_linear_timeout(cycles)
    assert kda.device_status() == 0
