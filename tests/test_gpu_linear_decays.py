"""Constant slow decays: what a product of decays is off by may not grow with the tokens it spans as if
each had been rounded by itself.

exp(g) for g = -1/M lies just below 1, where fp32 is off by up to 2^-25.  For heads whose exp(g) is rounded
by nearly as much, always to the same side, a state made of products of rounded decays is off by
M x 0.47 x 2^-24 or so (its terms span M tokens on average).  Taken over blocks of eight tokens or more,
the exponential of a sum is off by an ulp (2 x 2^-24) and the state's product by a rounding, 3 x 2^-24 a
block: M x 0.375 x 2^-24 in all, with some 24 more for the sums within.  In the 2-norm of a head's state.
"""
import math

import numpy as np
import pytest
import torch

import kimi_delta_attention_13_gb300 as kda
from test_gpu_linear import DEV, make, recurrence

pytestmark = pytest.mark.gpu
MEMORY = 1024


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    yield
    assert kda.device_status() == 0
    torch.cuda.empty_cache()


def slow(heads):
    """Log decays near -1/MEMORY whose exponentials fp32 is off by 0.47 to 0.5 of 2^-24, by turns up and down."""
    gs, rng = [], np.random.default_rng(0)
    while len(gs) < heads:
        g = np.float32(-1.0 / MEMORY * rng.uniform(0.95, 1.05))
        off = (float(np.float32(math.exp(float(g)))) - math.exp(float(g))) * 2.0 ** 24
        if 0.47 <= abs(off) <= 0.5 and (off > 0) == (len(gs) % 2 == 0):
            gs.append(float(g))
    return torch.tensor(gs, device=DEV)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths,H,dk,dv", [([4 * MEMORY], 4, 64, 64), ([4 * MEMORY, 3000], 2, 128, 128),
                                             ([4 * MEMORY, 300] + [1] * 40, 16, 64, 128)], ids=["cut", "two", "many"])
def test_states_with_slow_decays(lengths, H, dk, dv, dtype):
    x = make(lengths, H, H // 2, dk, dv, dtype, seed=41, init=False)
    x["g"] = slow(H)
    _, fin = kda.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["cu"], None, scale=dk ** -0.5)
    _, want, _, _ = recurrence(x, 1.0)
    off = (fin.double() - want)[:2].flatten(2).norm(dim=2) / want[:2].flatten(2).norm(dim=2)
    bound = (0.375 * MEMORY + 24) * 2.0 ** -24
    assert float(off.max()) <= bound, float(off.max()) / bound
