"""Checkpoint stores that refuse: nothing is indexed that was not written, and no store is made that could not be
filled.  On the CPU, where every device copy is refused."""
import pytest
import torch

from kimi_delta_attention_13_gb300 import prefix_cache
from kimi_delta_attention_13_gb300.prefix_cache import CheckpointStore


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.int8])
def test_a_refused_write_leaves_the_index(monkeypatch, dtype):
    store = CheckpointStore(3, heads=1, d_k=4, d_v=4, device="cpu", dtype=dtype)
    with monkeypatch.context() as m:            # a first prompt, written
        for name in ("state_copy", "state_pack"):
            m.setattr(prefix_cache, name, lambda *a, **kw: None)
        store.add_checkpoints(["a"], torch.zeros(2, 1, 4, 4), 32, [64])
    with pytest.raises(ValueError):             # a second one, refused
        store.add_checkpoints(["b"], torch.zeros(2, 1, 4, 4), 32, [64])
    assert store.lookup("b", 100) == (None, 0)
    assert store.lookup("a", 100) == (1, 64) and store.lookup("a", 40) == (0, 32)
    with monkeypatch.context() as m:            # and again, written where the refused one would have been
        for name in ("state_copy", "state_pack"):
            m.setattr(prefix_cache, name, lambda *a, **kw: None)
        assert store.add_checkpoints(["b"], torch.zeros(2, 1, 4, 4), 32, [64]) == [("b", 32, 2), ("b", 64, 0)]
    assert store.lookup("a", 40) == (None, 0) and store.lookup("a", 100) == (1, 64)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.int8])
@pytest.mark.parametrize("d_k,d_v", [(8, 6), (8, 258), (8, 260), (264, 8), (257, 256)])
def test_head_sizes_that_cannot_be_packed(dtype, d_k, d_v):
    with pytest.raises(ValueError):
        CheckpointStore(2, 1, d_k, d_v, device="cpu", dtype=dtype)
    CheckpointStore(2, 1, d_k, d_v, device="cpu")        # as they are
    CheckpointStore(2, 1, 256, 256, device="cpu", dtype=dtype)
    CheckpointStore(2, 1, 9, 4, device="cpu", dtype=dtype)
