"""The tensor-core prefill of the gated delta rule over many chunks of one slow decay: its rounding must not add up.

With closed gates (beta = 0) all that is left of a state is its decay, S_T = exp(T g) S_0.  A chunk of 64 tokens may be
off it by a rounding of each element, half an eps of it at most and as often up as down (eps = 2^-23, so 2^-24, rms
2^-24 / sqrt(3)), and by what its decay is off, the same way each time: the sum G = 64 g and exp(G) - 1 by an eps of
them each at most, which is 4 * 2^-24 |G| of the state.  Where G is far from 0 the decay itself may be off by 2 eps
(2^-22), and a state is forgotten within a few chunks.
"""
import pytest
import torch

import kimi_delta_attention_13_gb300 as kda
from delta_plain import inputs, recurrence

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
ULP = 2.0 ** -24


@pytest.mark.parametrize("d", [128, 64, 40])
@pytest.mark.parametrize("tokens,g", [(8192, -7.6e-4), (8192, -1e-4), (8191, -3e-3), (65536, -1e-4), (65537, -1e-5),
                                      (65536, 0.0), (1024, -7e-3), (512, -0.05)])
def test_closed_gates(tokens, g, d):
    gen = torch.Generator().manual_seed(tokens + d)
    x = {n: torch.randn(tokens, 2, d, generator=gen).mul_(0.05).to(BF16).cuda() for n in "qkv"}
    decay = torch.tensor([g, 1.01 * g], dtype=F32).cuda()
    init = torch.randn(1, 2, d, d, generator=gen).cuda()
    _, state = kda.delta_prefill(x["q"], x["k"], x["v"], decay, torch.zeros(tokens, 2, device="cuda"), None, init)
    want = init.double() * (tokens * decay.double()).exp()[:, None, None]
    assert bool(state.isfinite().all()) and kda.device_status() == 0
    off = state.double() - want
    chunks = -(-tokens // 64)
    total = tokens * abs(1.01 * g)
    same = ULP * (4 * total if 64 * abs(g) < 0.48 else 4 * chunks + 4 * total)
    # the mean over elements leaves the systematic part: 5 deviations of the rest
    bias = (off / want).mean(dim=(0, 2, 3)).abs()
    assert bool((bias <= same + ULP * 5 * (chunks / 3) ** 0.5 / d).all()), bias
    off, size = (x[0].flatten(1).norm(dim=1) for x in (off, want))
    assert bool((off <= (same + 1.2 * ULP * (chunks / 3) ** 0.5) * size).all()), off / size


@pytest.mark.parametrize("per_token", [False, True])
def test_written_states(per_token):
    """8192 tokens that write, of a decay near 1 that is constant, or that differs a little from token to token."""
    x = inputs([8192], 1, 1, 128, 128, BF16, seed=31, init=True, per_token=per_token)
    x["g"].mul_(1e-3)
    _, state = kda.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], x["cu"], x["init"])
    _, final, _, _ = recurrence(x["q"], x["k"], x["v"], x["g"], x["beta"], [8192], x["init"])
    # operands are exact and roundings of fp32 sums are as often up as down: near eps, far from their bound
    assert float((state.double() - final).norm() / final.norm()) < 16 * ULP
    assert kda.device_status() == 0
