"""delta_prefill's outputs on the tensor cores, held to what its roundings leave: two bf16 parts of the state and of the new
values, one of the scores (delta_outputs.py).  tests/test_delta_bounds_cpu.py shows that one part less is seen."""
import pytest
import torch

import kimi_delta_attention_13_gb300 as kda
from delta_outputs import output_bounds, unit_keys, within
from delta_plain import inputs

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
SHAPES = [(2, 1, 128, 128), (4, 2, 64, 64), (2, 2, 96, 72), (2, 1, 64, 128)]
LENGTHS = [[128], [129], [300], [191, 260, 1, 0, 300]]


def run(x, lengths, scale=1.0, out_dtype=F32, **kw):
    out, state = kda.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], x["cu"], x["init"], scale=scale,
                                   out_dtype=out_dtype)
    want, bound = output_bounds(x, lengths, scale, **kw)
    assert out.dtype is out_dtype and bool((bound >= 0).all())
    assert within(out, want, bound) and bool(state.isfinite().all())
    assert kda.device_status() == 0


@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("shape", SHAPES)
def test_outputs(shape, lengths, out_dtype):
    h, hk, dk, dv = shape
    x = inputs(lengths, h, hk, dk, dv, BF16, seed=sum(lengths) + dk + dv, init=len(lengths) > 1, per_token=dv != 72)
    run(x, lengths, dk ** -0.5, out_dtype)


@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("shape", SHAPES)
def test_the_state_s_term(shape, lengths):
    """Closed gates: outputs are the state's alone, 2^-16 of their terms."""
    h, hk, dk, dv = shape
    x = inputs(lengths, h, hk, dk, dv, BF16, seed=sum(lengths) + dk, init=True)
    x["beta"].zero_()
    x["g"].mul_(0.05)
    run(x, lengths)


@pytest.mark.parametrize("init", [False, True])
@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("shape", SHAPES)
def test_the_scores_term(shape, lengths, init):
    """Scores of 2^-4, which no rounding touches: outputs are sums of the new values, off by what two parts leave."""
    h, hk, dk, dv = shape
    x = unit_keys(inputs(lengths, h, hk, dk, dv, BF16, seed=sum(lengths) + dv, init=init), sum(lengths))
    run(x, lengths, exact_scores=True)
