"""The linear-attention layer against its formulas in 64 bits, from the layer's own weights: two stacked
layers over packed prompts, then single tokens, on residual streams of both types.

Bound, in the 2-norm: an output of one bf16 layer has passed at most twelve roundings to bf16, each of
2^-8 at most of its tensor's norm (its input norm; q, k, v, z and the decay's logit; the key's norm, its
inverse's product; the recurrence's operands; o; the gate; the projection; the residual stream), and a
second layer as many on top.  With fp32 weights the sums decide: n 2^-24 a step with n = 1024 terms at
most (256 channels, 512 of the output projection, up to 300 tokens), over the same steps, and a bf16
stream beside them is rounded once a layer.
"""
import pytest
import torch

import kimi_delta_attention_13_gb300 as kda
from kimi_delta_attention_13_gb300.linear_layer import LinearLayer

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
WIDTH, LENGTHS, EXTRA = 256, [150, 1, 300], 3


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    yield
    assert kda.device_status() == 0
    torch.cuda.empty_cache()


def norm(x, w, eps):
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()


def plain(layer, x, y, lengths):
    """(residual stream, output, states) of whole sequences, token by token."""
    if y is not None:
        x = x + layer.residual_scale * norm(y, layer.n_post, layer.eps)
    H, Hkv, dk, dv = layer.heads, layer.kv_heads, layer.d_k, layer.d_v
    p = norm(x, layer.n_in, layer.eps) @ layer.w_in.double()
    q, k, v, z, a = p.split([H * dk, Hkv * dk, Hkv * dv, H * dv, H], dim=1)
    rows = x.shape[0]
    q, z = q.reshape(rows, H, dk), z.reshape(rows, H, dv)
    k = k.reshape(rows, Hkv, dk)
    k = (k / k.norm(dim=-1, keepdim=True)).repeat_interleave(H // Hkv, 1)
    v = v.reshape(rows, Hkv, dv).repeat_interleave(H // Hkv, 1)
    keep = torch.sigmoid(-(a + layer.bias.double()))          # exp(-softplus(u)) = 1 / (1 + exp(u))
    o, states, at = torch.empty(rows, H, dv, device=DEV, dtype=torch.float64), [], 0
    for n in lengths:
        s = torch.zeros(H, dk, dv, device=DEV, dtype=torch.float64)
        for t in range(at, at + n):
            s = s * keep[t][:, None, None] + k[t][:, :, None] * v[t][:, None, :]
            o[t] = (q[t][:, None, :] @ s)[:, 0] * dk ** -0.5
        states.append(s)
        at += n
    o = norm(o, layer.n_head, layer.eps) * torch.sigmoid(z)
    return x, o.flatten(1) @ layer.w_out.double(), torch.stack(states)


def off(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("weights,stream", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
def test_layers_match_their_formulas(weights, stream):
    layers = [LinearLayer(WIDTH, 4, kv, residual_scale=0.5, device=DEV, dtype=TYPES[weights], seed=i)
              for i, kv in enumerate((4, 2))]
    gen = torch.Generator(device=DEV).manual_seed(3)
    for layer in layers:       # weights of norms that are not all alike
        for w in (layer.n_in, layer.n_post, layer.n_head):
            w.add_(0.2 * torch.randn(w.shape, generator=gen, device=DEV))
    step = 12 * 2.0 ** -8 if weights == "bf16" else 12 * 1024 * 2.0 ** -24
    if weights == "f32" and stream == "bf16":
        step += 2.0 ** -8
    whole = [torch.randn(n + EXTRA, WIDTH, generator=gen, device=DEV).to(TYPES[stream]) for n in LENGTHS]
    x, y, want, want_states = torch.cat(whole).double(), None, [], []
    for layer in layers:
        x, y, s = plain(layer, x, y, [n + EXTRA for n in LENGTHS])
        want.append([t.split([n + EXTRA for n in LENGTHS]) for t in (x, y)])
        want_states.append(s)
    cu = torch.tensor([0] + LENGTHS, device=DEV).cumsum(0).to(torch.int32)
    x, y, states = torch.cat([w[:n] for w, n in zip(whole, LENGTHS)]), None, []
    for i, layer in enumerate(layers):
        x, y, s = layer.prefill(x, y, cu)
        states.append(s)
        assert x.dtype == TYPES[stream] and y.dtype == TYPES[weights]
        for got, ref in ((x, want[i][0]), (y, want[i][1])):
            assert off(got, torch.cat([r[:n] for r, n in zip(ref, LENGTHS)])) <= (i + 1) * step
    for t in range(EXTRA):
        x, y = torch.stack([w[n + t] for w, n in zip(whole, LENGTHS)]), None
        for i, layer in enumerate(layers):
            x, y = layer.decode(x, y, states[i])
            assert x.dtype == TYPES[stream] and y.dtype == TYPES[weights]
            for got, ref in ((x, want[i][0]), (y, want[i][1])):
                assert off(got, torch.stack([r[n + t] for r, n in zip(ref, LENGTHS)])) <= (i + 1) * step
    for i in range(2):
        assert off(states[i], want_states[i]) <= (i + 1) * step
