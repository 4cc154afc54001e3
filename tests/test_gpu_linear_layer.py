"""The linear-attention layer from the library's calls: two stacked layers over packed prompts, then
single tokens, against the same layers over the whole sequences, and a state stored and restored.

Bound: between the two ways an output passes at most eight roundings to bf16 more (the recurrence's
operands, o, the gate, the projections and sums of two layers), each of at most 2^-8 of its tensor's
norm: 8 x 2^-8 in the 2-norm.
"""
import pytest
import torch

import kimi_delta_attention_13_gb300 as kda
from kimi_delta_attention_13_gb300.linear_layer import LinearLayer

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
BOUND = 8 * 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    yield
    assert kda.device_status() == 0
    torch.cuda.empty_cache()


def stack(width=256):
    return [LinearLayer(width, 4, kv, residual_scale=0.5, device=DEV, seed=i) for i, kv in enumerate((4, 2))]


def prefill(layers, x, cu):
    y, states = None, []
    for layer in layers:
        x, y, s = layer.prefill(x, y, cu)
        states.append(s)
    return x, y, states


def decode(layers, x, states):
    y = None
    for layer, s in zip(layers, states):
        x, y = layer.decode(x, y, s)
    return x, y


def off(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def test_single_tokens_continue_the_prompts():
    layers, lengths, extra = stack(), [150, 1, 300], 5
    gen = torch.Generator(device=DEV).manual_seed(1)
    whole = [torch.randn(n + extra, 256, generator=gen, device=DEV).bfloat16() for n in lengths]
    cu = lambda ns: torch.tensor([0] + ns, device=DEV).cumsum(0).to(torch.int32)  # noqa: E731
    _, want, want_states = prefill(layers, torch.cat(whole), cu([n + extra for n in lengths]))
    want = want.split([n + extra for n in lengths])
    _, y, states = prefill(layers, torch.cat([w[:n] for w, n in zip(whole, lengths)]), cu(lengths))
    for got, ref, n in zip(y.split(lengths), want, lengths):
        assert off(got, ref[:n]) <= BOUND
    for t in range(extra):
        _, y = decode(layers, torch.stack([w[n + t] for w, n in zip(whole, lengths)]), states)
        assert off(y, torch.stack([r[n + t] for r, n in zip(want, lengths)])) <= BOUND
    for got, ref in zip(states, want_states):
        assert off(got, ref) <= BOUND


def test_states_move_with_state_copy():
    layers = stack()
    x = torch.randn(64, 256, generator=torch.Generator(device=DEV).manual_seed(2), device=DEV).bfloat16()
    _, _, states = prefill(layers, x, None)
    pool = torch.empty(3, 4, 128, 128, device=DEV)
    kda.state_copy(pool, states[0], torch.tensor([2], device=DEV), torch.tensor([0], device=DEV))
    back = torch.empty_like(states[0])
    kda.state_copy(back, pool, torch.tensor([0], device=DEV), torch.tensor([2], device=DEV))
    a = layers[0].decode(x[:1].contiguous(), None, states[0].clone())[1]
    b = layers[0].decode(x[:1].contiguous(), None, back)[1]
    assert torch.equal(a, b)


def test_layer_refuses_uneven_heads():
    with pytest.raises(ValueError, match="share"):
        LinearLayer(64, 4, 3, device=DEV)
