"""The delta calls where rows, offsets and streams are other than usual."""
import pytest
import torch

import kimi_delta_attention_13_gb300 as kda
from delta_plain import chunked_bounds, inputs, recurrence
from test_gpu_delta_tc import check as chunk_check

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("first,end", [(0, 100), (5, 100), (60, 60)])
def test_one_sequence_in_a_padded_batch(dtype, first, end):
    """A table of one sequence that does not cover the rows: the others are neither read nor written."""
    x = inputs([100], 2, 2, 128, 128, dtype, seed=20, init=True, tail=28)
    part = {n: x[n][first:end].contiguous() for n in ("q", "k", "v", "g", "beta")}
    want, final = kda.delta_prefill(**part, init_state=x["init"])
    for n in part:
        x[n][:first] = float("nan")
        x[n][end:] = float("nan")
    out = torch.full((128, 2, 128), 7.0, dtype=dtype, device="cuda")
    cu = torch.tensor([first, end], dtype=torch.int32, device="cuda")
    _, state = kda.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], cu, x["init"], out=out)
    assert bool((out[:first] == 7).all()) and bool((out[end:] == 7).all())
    assert torch.equal(out[first:end], want) and torch.equal(state, final)
    assert kda.device_status() == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prefill_past_32_bits(dtype):
    """Operands and outputs of more than 2^31 elements, the last sequence behind them."""
    t, h, d, n = 175_000, 96, 128, 100
    part = inputs([n], h, h, d, d, dtype, seed=21)
    want, final = kda.delta_prefill(part["q"], part["k"], part["v"], part["g"], part["beta"])
    x = {}
    for name in ("q", "k", "v", "g", "beta"):
        x[name] = torch.zeros(t, *part[name].shape[1:], dtype=part[name].dtype, device="cuda")
        x[name][t - n:] = part[name]
    cu = torch.tensor([0, t - n, t], dtype=torch.int32, device="cuda")
    out, state = kda.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], cu)
    assert torch.equal(out[t - n:], want) and torch.equal(state[1:], final)
    assert bool((out[:t - n] == 0).all()) and bool((state[0] == 0).all())
    assert kda.device_status() == 0


@pytest.mark.parametrize("n,d", [(1400, 128), (5500, 64)])
def test_decode_past_32_bits(n, d):
    """States of more than 2^31 elements; the last two sequences against 64 bits."""
    x = inputs([1, 1], 96, 48, d, d, F32, seed=22, init=True)
    big = {name: torch.zeros(n, *x[name].shape[1:], device="cuda") for name in ("q", "k", "v", "g", "beta")}
    state = torch.zeros(n, 96, d, d, device="cuda")
    for name, y in big.items():
        y[n - 2:] = x[name]
    state[n - 2:] = x["init"]
    out = kda.delta_decode(*big.values(), state)
    want, final, err, bound = recurrence(x["q"], x["k"], x["v"], x["g"], x["beta"], [1, 1], x["init"])
    assert bool(((out[n - 2:].double() - want).abs() <= bound + 2.0 ** -24 * (want.abs() + bound)).all())
    assert bool(((state[n - 2:].double() - final).norm(dim=-2) <= err).all())
    assert bool((out[:n - 2] == 0).all()) and bool((state[:n - 2] == 0).all())


def test_layer_on_tensor_cores():
    """A bf16 layer: its prompt's states against 64 bits, cut in two and resumed through a store of bf16 states."""
    from kimi_delta_attention_13_gb300.delta_layer import DeltaLayer
    from kimi_delta_attention_13_gb300.prefix_cache import CheckpointStore

    layer = DeltaLayer(256, heads=4, key_heads=2, seed=5)
    x = torch.randn(192, 256, generator=torch.Generator().manual_seed(6)).cuda()
    _, y, state = layer.prefill(x)
    _, mixer, _ = layer._enter(x, None)
    q, k, v, g, beta = mixer
    want, final, err, _ = chunked_bounds(q, k * 1.0, v, g, beta, [192])
    # a key's norm is off 1 by its rounding, 2^-8 at most: a step may lengthen an error by beta 2^-7, of which
    # sum(beta) are made, instead of shortening it
    grown = (beta.double().sum(0) * 2.0 ** -7).exp()[:, None]
    assert bool(((state.double() - final).norm(dim=-2) <= grown * err).all())
    _, _, first = layer.prefill(x[:128])
    store = CheckpointStore(2, 4, device="cuda", dtype=BF16)
    at = torch.tensor([1], device="cuda")
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    store.write(at, first, zero)
    back = torch.empty_like(first)
    store.read(back, zero, at)
    assert torch.equal(back, first.to(BF16).float())
    _, y2, resumed = layer.prefill(x[128:], state=back)
    # the stored state's rounding (2^-8 of each value) is carried on as an error is
    assert bool(((resumed - state).norm(dim=-2) <= grown * (2.0 ** -8 * first.norm(dim=-2) + 2 * err)).all())
    _, y3 = layer.decode(x[:1], None, resumed)
    assert y.shape == (192, 256) and y2.shape == (64, 256) and y3.shape == (1, 256)
    assert bool(torch.isfinite(y3).all()) and kda.device_status() == 0


def test_resume_on_another_stream():
    """The store's copies and the zeros of fresh requests run in order on the stream that is given."""
    from kimi_delta_attention_13_gb300 import synth
    from kimi_delta_attention_13_gb300.prefix_cache import CheckpointStore, resume_prefill

    lengths = [96, 64]
    s = synth.make_inputs(lengths, heads=2, dtype="bf16", seed=5, device="cuda")
    args = (s["q"], s["k"], s["v"], s["g"], s["beta"], s["cu_seqlens"])
    _, _, ckpts = kda.prefill(*args, ckpt_stride=32, lengths=lengths)
    part = [t[64:160].contiguous() for t in args[:5]]
    cu = torch.tensor([0, 32, 96], dtype=torch.int32, device="cuda")
    got = []
    for side in (None, torch.cuda.Stream()):
        store = CheckpointStore(8, 2, device="cuda", dtype=torch.int8)
        if side is not None:
            side.wait_stream(torch.cuda.current_stream())
            torch.cuda._sleep(2_000_000)                # the current stream is busy; `side` must not need it
        store.add_checkpoints(["a", "b"], ckpts, 32, lengths, stream=side)
        slot, _ = store.lookup("a", 70)
        got.append(resume_prefill(store, [slot, None], *part, cu, [32, 64], stream=side))
    torch.cuda.synchronize()
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dk,dv", [(8, 8), (16, 128), (24, 40), (64, 64), (64, 96), (40, 120)])
@pytest.mark.parametrize("lengths", [[150, 130], [260, 1, 0, 300]])
def test_small_heads_in_chunks(dk, dv, lengths):
    """Head sizes up to 64 with sequences long enough for chunks of 64 tokens."""
    x = inputs(lengths, 2, 1, dk, dv, BF16, seed=dk + dv, init=True, per_token=dv != 40)
    out, state = kda.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], x["cu"], x["init"], scale=0.5)
    chunk_check(out, state, x, lengths, 0.5)


@pytest.mark.parametrize("dtype,shape", [(F32, (3, 1, 128, 128)), (BF16, (4, 2, 64, 72)), (BF16, (2, 2, 128, 128)),
                                         (BF16, (2, 1, 248, 200))])
@pytest.mark.parametrize("lengths", [[9], [16, 1, 7, 0, 8], [25, 24, 23]])
def test_blocks_of_eight_tokens(dtype, shape, lengths):
    """Sequences that end within a block of eight tokens, at one and behind one."""
    h, hk, dk, dv = shape
    x = inputs(lengths, h, hk, dk, dv, dtype, seed=sum(lengths) + dk, init=True)
    out, state = kda.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], x["cu"], x["init"], out_dtype=F32)
    want, final, err, bound = recurrence(x["q"], x["k"], x["v"], x["g"], x["beta"], lengths, x["init"])
    assert bool(((out.double() - want).abs() <= bound + 2.0 ** -24 * (want.abs() + bound)).all())
    assert bool(((state.double() - final).norm(dim=-2) <= err).all())
    assert kda.device_status() == 0


@pytest.mark.parametrize("power", [-60, 60])
def test_magnitudes_of_fp32_values(power):
    """Values and states times a power of two: the same results times it, bit for bit."""
    x = inputs([50, 21], 2, 2, 64, 64, F32, seed=23, init=True)
    out, state = kda.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], x["cu"], x["init"])
    y, z = kda.delta_prefill(x["q"], x["k"], x["v"] * 2.0 ** power, x["g"], x["beta"], x["cu"], x["init"] * 2.0 ** power)
    assert torch.equal(y, out * 2.0 ** power) and torch.equal(z, state * 2.0 ** power)
