"""Prefix reuse of the gated delta rule's layer: a prompt's final states are checkpoints at its length; a later prompt
that continues it takes its state from the store, as it is or in fewer bits."""
import pytest
import torch

import kimi_delta_attention_13_gb300 as kda
from kimi_delta_attention_13_gb300.delta_layer import DeltaLayer
from kimi_delta_attention_13_gb300.prefix_cache import CheckpointStore

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.int8])
def test_states_are_stored_and_restored(dtype):
    layer = DeltaLayer(256, 4, 2, 64, 128, seed=1)
    gen = torch.Generator(device="cuda").manual_seed(2)
    lengths, more = [190, 331], [40, 7]
    cu = lambda ns: torch.tensor([0] + ns, device="cuda").cumsum(0).to(torch.int32)  # noqa: E731
    x = torch.randn(sum(lengths), 256, generator=gen, device="cuda").bfloat16()
    _, _, states = layer.prefill(x, None, cu(lengths))
    store = CheckpointStore(4, 4, 64, 128, device="cuda", dtype=dtype)
    for i, n in enumerate(lengths):
        assert store.add_checkpoints([i], states[i:i + 1], n, [n]) == [(i, n, i)]
    found = [store.lookup(i, n + more[i]) for i, n in enumerate(lengths)]
    assert [covered for _, covered in found] == lengths
    back = torch.empty_like(states)
    store.read(back, torch.arange(2, device="cuda"), torch.tensor([s for s, _ in found], device="cuda"))
    if dtype is torch.float32:
        assert torch.equal(back, states)
    elif dtype is torch.bfloat16:
        assert torch.equal(back, states.to(dtype).float())
    else:   # half a step of the row's scale, and the roundings of the scale and of the product
        top = states.abs().amax(-1, keepdim=True)
        assert bool(((back - states).abs() <= top * (0.5 / 127 + 2.0 ** -22)).all())
    # continued from the store, bit for bit as from the values that it holds
    held = {torch.float32: lambda: states, torch.bfloat16: lambda: states.to(dtype).float(), torch.int8: back.clone}[dtype]()
    x = torch.randn(sum(more), 256, generator=gen, device="cuda").bfloat16()
    got, want = (layer.prefill(x, None, cu(more), s) for s in (back, held))
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and bool(got[1].isfinite().all())
    assert kda.device_status() == 0
