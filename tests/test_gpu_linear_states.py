"""Final states of kda_linear_prefill from bf16 operands are good to fp32: products of two bf16 are exact in
it, so nothing but fp32's own roundings may show.

Bounds.  Element by element over a few tokens, where they are tight: a token's weight is an exponential
(an ulp, 2 x 2^-24) and a product with each of up to T others, or that of a sum of T logs of 0.2 or so
each (T in either case); its product with v is rounded once; three operand parts are added to a sum that
may cut off instead of rounding (2 x 2^-24 each) for each of T tokens; the state before them takes a
decay and an addition: n = 2 + T + 1 + 6 T + 2 T <= 9 T + 4 steps of 2^-24 of the sum of magnitudes.  Over
long sequences, in the 2-norm: roundings are as good as independent, so that some 9 a token over a memory
of 64 tokens add up to sqrt(9 x 64) = 24 of them.
"""
import pytest
import torch

import kimi_delta_attention_13_gb300 as kda
from test_gpu_linear import DEV, make, recurrence

pytestmark = pytest.mark.gpu
DIMS = [(128, 128), (64, 128), (128, 64), (64, 64), (96, 80), (8, 16)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    yield
    assert kda.device_status() == 0
    torch.cuda.empty_cache()


@pytest.mark.parametrize("init", [False, True])
@pytest.mark.parametrize("dk,dv", DIMS)
def test_states_of_a_few_tokens(dk, dv, init):
    lengths = [2, 1, 3, 8, 5, 0, 33]
    x = make(lengths, 4, 2, dk, dv, "bf16", seed=dk + dv, init=init)
    _, fin = kda.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["cu"], x["init"])
    _, want, _, mag = recurrence(x, 1.0)
    for i, n in enumerate(lengths):
        err, tol = (fin[i].double() - want[i]).abs(), (9 * n + 4) * 2.0 ** -24 * mag[i] + 1e-37
        assert bool((err <= tol).all()), (n, float((err / tol).max()))


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("lengths,H,cut", [([1700, 300, 129], 60, False), ([4000], 2, True)], ids=["whole", "cut"])
def test_states_of_long_sequences(lengths, H, cut, dk, dv):
    x = make(lengths, H, 2, dk, dv, "bf16", seed=dk * dv)
    gen = torch.Generator(device=DEV).manual_seed(1)             # memories of some 4 to 64 tokens and more
    x["g"] = -torch.nn.functional.softplus(torch.randn(sum(lengths), H, generator=gen, device=DEV) - 3)
    assert (kda.load().kda_linear_prefill_workspace(len(lengths), sum(lengths), H, dk, dv, 0) > 0) == cut
    _, fin = kda.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["cu"], x["init"])
    _, want, _, _ = recurrence(x, 1.0)
    off = ((fin.double() - want).flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)).max()
    assert float(off) <= 24 * 2.0 ** -24, float(off) * 2 ** 24
