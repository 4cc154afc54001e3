"""Host-side checks of the gated delta rule's calls and of packed states, without a GPU."""
import pytest

from kimi_delta_attention_13_gb300 import _lib, build

A = 1 << 20  # a 16-byte aligned "device address" that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def prefill(lib, **over):
    a = dict(q=A, k=2 * A, v=3 * A, g=4 * A, per=1, beta=5 * A, cu=None, n=1, T=16, H=4, Hk=2, dk=128, dv=128, scale=1.0,
             dt=0, odt=1, init=None, out=6 * A, fin=7 * A)
    a.update(over)
    return lib.kda_delta_prefill(*a.values(), None)


@pytest.mark.parametrize("over,code", [
    (dict(H=0), 1), (dict(Hk=0), 1), (dict(Hk=3), 1), (dict(n=-1), 1), (dict(T=-1), 1), (dict(T=1 << 31), 1), (dict(n=0), 1),
    (dict(n=2), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(g=None), 1), (dict(beta=None), 1),
    (dict(out=None), 1), (dict(dt=2), 1), (dict(odt=-1), 1), (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1),
    (dict(dk=0), 1), (dict(dk=4), 2), (dict(dk=12), 2), (dict(dk=264), 2), (dict(dv=264), 2), (dict(dv=20), 2),
    (dict(q=A + 8), 3), (dict(beta=5 * A + 2), 3), (dict(g=4 * A + 1), 3), (dict(fin=7 * A + 8), 3), (dict(cu=A + 2, n=2), 3),
    (dict(out=A), 1), (dict(out=5 * A), 1), (dict(out=7 * A), 1), (dict(fin=5 * A), 1), (dict(fin=3 * A), 1),
    (dict(init=6 * A), 1), (dict(n=1 << 30, cu=A, T=0), 2)])
def test_prefill_rejects(lib, over, code):
    assert prefill(lib, **over) == code


# one byte into another's memory, and one behind it: [16, 4 or 2, 128] bf16 is 16 or 8 KB, out 32 KB, the state 256 KB
@pytest.mark.parametrize("over,code", [
    (dict(out=A + 8176), 1), (dict(out=3 * A + 16368), 1), (dict(out=4 * A + 240), 1), (dict(out=3 * A - 32752), 1),
    (dict(out=7 * A + 262128), 1), (dict(out=8 * A, init=7 * A + 16), 1), (dict(fin=2 * A + 8176), 1), (dict(fin=6 * A - 16), 1),
    (dict(cu=6 * A + 4), 1), (dict(cu=7 * A + 8), 1)])
def test_prefill_rejects_overlap(lib, over, code):
    assert prefill(lib, **over) == code


@pytest.mark.parametrize("over", [dict(out=3 * A + 3056), dict(out=6 * A + 16), dict(state=5 * A - 16), dict(state=7 * A - 16)])
def test_decode_rejects_overlap(lib, over):
    a = dict(q=A, k=2 * A, v=3 * A, g=4 * A, per=0, beta=5 * A, state=6 * A, out=7 * A, n=3, H=4, Hk=2, dk=128, dv=128,
             scale=1.0, dt=0, odt=0)
    a.update(over)
    assert lib.kda_delta_decode(*a.values(), None) == 1


@pytest.mark.parametrize("over", [dict(didx=2 * (1 << 40) + 64), dict(sidx=(1 << 40) + 64), dict(didx=1 << 20)])
def test_pack_rejects_indices_in_its_memory(lib, over):
    a = dict(dst=1 << 40, scales=1 << 20, fmt=1, didx=None, nd=8, src=2 << 40, sidx=None, ns=8, n=3, H=2, dk=128, dv=128)
    a.update(over)
    assert lib.kda_state_pack(*a.values(), None) == 1


def test_timeout_probe_rejects(lib):
    assert lib.kda_diag_delta_timeout(0, None) == 1 and lib.kda_diag_delta_timeout(4000000001, None) == 1


def test_nothing_to_do(lib):
    assert prefill(lib, T=0, n=0, q=None, k=None, v=None, g=None, beta=None, out=None, fin=None) == 0
    assert lib.kda_delta_decode(None, None, None, None, 1, None, None, None, 0, 4, 2, 128, 128, 1.0, 0, 1, None) == 0
    assert lib.kda_state_pack(None, None, 0, None, 0, None, None, 0, 0, 2, 128, 128, None) == 0
    assert lib.kda_state_unpack(None, None, 0, None, None, 1, None, 0, 0, 2, 128, 128, None) == 0


@pytest.mark.parametrize("over,code", [
    (dict(n=-1), 1), (dict(H=0), 1), (dict(Hk=3), 1), (dict(state=None), 1), (dict(out=None), 1), (dict(beta=None), 1),
    (dict(dt=5), 1), (dict(scale=float("nan")), 1), (dict(dk=260), 2), (dict(dv=4), 2), (dict(state=6 * A + 4), 3), (dict(g=4 * A + 2), 3), (dict(beta=5 * A + 1), 3),
    (dict(out=6 * A), 1), (dict(state=A), 1), (dict(n=1 << 30), 2)])
def test_decode_rejects(lib, over, code):
    a = dict(q=A, k=2 * A, v=3 * A, g=4 * A, per=0, beta=5 * A, state=6 * A, out=7 * A, n=3, H=4, Hk=2, dk=128, dv=128,
             scale=1.0, dt=0, odt=0)
    a.update(over)
    assert lib.kda_delta_decode(*a.values(), None) == code


HUGE = 1 << 40


@pytest.mark.parametrize("over,code", [
    (dict(n=-1), 1), (dict(H=0), 1), (dict(dk=0), 1), (dict(fmt=2), 1), (dict(fmt=-1), 1), (dict(dst=None), 1),
    (dict(src=None), 1), (dict(scales=None), 1), (dict(fmt=0), 1), (dict(n=9), 1), (dict(didx=A, n=9), 1),
    (dict(dv=6), 2), (dict(dv=260), 2), (dict(dk=257), 2), (dict(dst=HUGE + 4), 3), (dict(scales=A + 4), 3),
    (dict(didx=A + 8), 3), (dict(sidx=A + 8), 3),
    (dict(dst=2 * HUGE + 16), 1), (dict(scales=2 * HUGE), 1), (dict(scales=HUGE + 1024), 1)])
def test_pack_rejects(lib, over, code):
    a = dict(dst=HUGE, scales=A, fmt=1, didx=None, nd=8, src=2 * HUGE, sidx=None, ns=8, n=3, H=2, dk=128, dv=128)
    a.update(over)
    assert lib.kda_state_pack(*a.values(), None) == code
    back = [a[x] for x in ("src", "sidx", "ns", "dst", "scales", "fmt", "didx", "nd", "n", "H", "dk", "dv")]
    assert lib.kda_state_unpack(*back, None) == code


def test_store_refuses_other_types():
    import torch

    from kimi_delta_attention_13_gb300.prefix_cache import CheckpointStore

    with pytest.raises(ValueError):
        CheckpointStore(2, 1, device="cpu", dtype=torch.float16)
    store = CheckpointStore(2, 1, 8, 8, device="cpu", dtype=torch.int8)
    assert store.states.dtype is torch.int8 and tuple(store.scales.shape) == (2, 1, 8)
    assert CheckpointStore(2, 1, 8, 8, device="cpu").scales is None
