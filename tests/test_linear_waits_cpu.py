"""kda_diag_linear_timeout's refusals, without a GPU."""
import pytest

from kimi_delta_attention_13_gb300 import _lib, build


@pytest.mark.parametrize("cycles", [0, -1, 4_000_000_001, 1 << 40])
def test_diag_linear_timeout_refuses_cycles_out_of_range(cycles):
    build.build()
    assert _lib.load().kda_diag_linear_timeout(cycles, None) == 1   # KDA_ERR_INVALID_ARG
