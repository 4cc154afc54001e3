"""kda_linear_prefill where sequences are cut into segments, against the recurrence in 64 bits (bounds of
test_gpu_linear.py), and tensors of more than 2^31 elements on each of its paths and in decode.

That a case is cut is checked by its workspace, so that another rule cannot empty the tests unseen.
"""
import pytest
import torch

import kimi_delta_attention_13_gb300 as kda
from test_gpu_linear import DEV, TYPES, check, make, recurrence

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    yield
    assert kda.device_status() == 0
    torch.cuda.empty_cache()


SEVERAL = [0, 1900, 1, 128, 0, 2171, 300]   # empty ones first and between, one of a token, one of a chunk


@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("lengths,H,Hkv,dk,dv,decay,init", [
    (SEVERAL, 2, 1, 128, 128, "token", True),
    (SEVERAL, 2, 2, 64, 128, "head", True),
    (SEVERAL, 2, 1, 128, 64, "token", False),
    (SEVERAL, 3, 1, 64, 64, "head", False),
    (SEVERAL, 2, 1, 96, 80, "token", True),
    ([2049], 4, 2, 8, 120, "token", True),
    ([2561, 1], 2, 1, 40, 24, "head", False),
    ([1300, 0], 1, 1, 120, 128, "token", True),
], ids=str)
def test_cut_sequences(lengths, H, Hkv, dk, dv, decay, init, dtype, out_dtype):
    x = make(lengths, H, Hkv, dk, dv, dtype, seed=H + dk + dv, decay=decay, init=init)
    x["g"].mul_(0.05)      # segments that depend on those before them
    assert kda.load().kda_linear_prefill_workspace(len(lengths), sum(lengths), H, dk, dv, 0 if dtype == "bf16" else 1) > 0
    got = kda.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["cu"], x["init"], scale=0.3, out_dtype=TYPES[out_dtype])
    check(x, got, dtype, out_dtype, 0.3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cut_sequences_in_place(dtype):
    """final_state = init_state for several cut sequences with shared heads: the same bits."""
    x = make(SEVERAL, 2, 1, 64, 128, dtype, seed=17)
    args = (x["q"], x["k"], x["v"], x["g"], x["cu"])
    want = kda.linear_prefill(*args, x["init"])
    state = x["init"].clone()
    out, fin = kda.linear_prefill(*args, state, final_state=state)
    assert fin is state and torch.equal(out, want[0]) and torch.equal(state, want[1])


def _tail(q, k, v, g, tail):
    return dict(q=q[-tail:].contiguous(), k=k[-tail:].contiguous(), v=v[-tail:].contiguous(), g=g,
                cu=torch.tensor([0, tail], device=DEV, dtype=torch.int32), lengths=[tail], init=None)


@pytest.mark.parametrize("dtype,T,H,Hkv", [("bf16", 2_200_000, 8, 8), ("f32", 132_000, 128, 128), ("f32", 140_000, 128, 1)])
def test_cut_offsets_past_32_bits(dtype, T, H, Hkv):
    """The last tokens, which by their decays depend on the last few hundred alone, against those."""
    d, tail, dt = 128, 640, TYPES[dtype]
    gen = torch.Generator(device=DEV).manual_seed(18)
    q = torch.randn(T, H, d, generator=gen, device=DEV, dtype=dt)
    k, v = (torch.randn(T, Hkv, d, generator=gen, device=DEV, dtype=dt) for _ in range(2))
    assert q.numel() > 2 ** 31
    assert kda.load().kda_linear_prefill_workspace(1, T, H, d, d, 0 if dtype == "bf16" else 1) > 0
    g = torch.full((H,), -1.0, device=DEV)
    out, fin = kda.linear_prefill(q, k, v, g, scale=0.01)
    x = _tail(q, k, v, g, tail)
    late = out[-256:].double()
    del q, k, v, out
    ref, rfin, mag, smag = recurrence(x, 0.01)
    operand = (2.0 ** -8, 2.0 ** -16) if dtype == "bf16" else (0.0, 0.0)
    n = (d + 2 * tail + 8) * 2.0 ** -24
    tol = (operand[0] + n) * mag[-256:] + 1e-30        # exp(-384) of what came before
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * (ref[-256:].abs() + tol)
    assert bool(((late - ref[-256:]).abs() <= tol).all())
    assert bool(((fin.double() - rfin).abs() <= (operand[1] + n) * smag).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_offsets_past_32_bits(dtype):
    N, H, d = 700, 192, 128
    gen = torch.Generator(device=DEV).manual_seed(19)
    state = torch.randn(N, H, d, d, generator=gen, device=DEV)
    assert state.numel() > 2 ** 31
    q, k, v = (torch.randn(N, H, d, generator=gen, device=DEV).to(TYPES[dtype]) for _ in range(3))
    g = -torch.rand(N, H, generator=gen, device=DEV)
    last = dict(q=q[-3:], k=k[-3:], v=v[-3:], g=g[-3:], cu=torch.arange(4, device=DEV, dtype=torch.int32),
                lengths=[1, 1, 1], init=state[-3:].clone())
    out = kda.linear_decode(q, k, v, g, state, scale=0.5)
    check(last, (out[-3:], state[-3:]), "f32", dtype, 0.5)
