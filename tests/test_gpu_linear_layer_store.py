"""Final states of the linear-attention layer in the checkpoint store: a prompt's state is one checkpoint
at its length; a later prompt that continues it restores the state and gives the same bits as from the
state itself.
"""
import pytest
import torch

import kimi_delta_attention_13_gb300 as kda
from kimi_delta_attention_13_gb300.linear_layer import LinearLayer
from kimi_delta_attention_13_gb300.prefix_cache import CheckpointStore

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    yield
    assert kda.device_status() == 0


def test_states_are_stored_and_restored():
    layer = LinearLayer(256, 4, 2, 64, 128, device=DEV, seed=1)
    gen = torch.Generator(device=DEV).manual_seed(2)
    lengths, more = [90, 131], [40, 7]
    cu = lambda ns: torch.tensor([0] + ns, device=DEV).cumsum(0).to(torch.int32)  # noqa: E731
    x = torch.randn(sum(lengths), 256, generator=gen, device=DEV).bfloat16()
    _, _, states = layer.prefill(x, None, cu(lengths))
    store = CheckpointStore(4, 4, 64, 128, device=DEV)
    for i, n in enumerate(lengths):
        store.add_checkpoints([i], states[i:i + 1], n, [n])
    found = [store.lookup(i, n + more[i]) for i, n in enumerate(lengths)]
    assert [covered for _, covered in found] == lengths
    back = torch.empty_like(states)
    kda.state_copy(back, store.states, torch.arange(2, device=DEV), torch.tensor([s for s, _ in found], device=DEV))
    assert torch.equal(back, states)
    x = torch.randn(sum(more), 256, generator=gen, device=DEV).bfloat16()
    want = layer.prefill(x, None, cu(more), states)
    got = layer.prefill(x, None, cu(more), back)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
