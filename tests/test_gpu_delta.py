"""delta_prefill and delta_decode on fp32 arithmetic against the recurrence in 64 bits, column by column."""
import pytest
import torch

import kimi_delta_attention_13_gb300 as kda
from delta_plain import inputs, recurrence

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def check(out, state, x, lengths, scale, q=None):
    want, final, err, bound = recurrence(x["q"], x["k"], x["v"], x["g"], x["beta"], lengths, x["init"], scale)
    rows = sum(lengths)
    half = torch.finfo(out.dtype).eps / 2
    got = out[:rows].double()
    # (what is rounded is off already)
    assert bool(((got - want[:rows]).abs() <= bound[:rows] + half * (want[:rows].abs() + bound[:rows]) + 1e-37).all())
    if state is not None:
        off = (state.double() - final).norm(dim=-2)
        assert bool((off <= err + 1e-37).all()), float((off / err.clamp(min=1e-300)).max())
    assert kda.device_status() == 0


SHAPES = [  # heads, keys, d_k, d_v
    (2, 2, 128, 128), (4, 2, 64, 128), (3, 1, 128, 64), (2, 2, 8, 8), (2, 1, 40, 72), (2, 2, 256, 256), (1, 1, 136, 24)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("lengths", [[1], [2, 0, 5], [0], [63, 64, 65], [130, 1, 7]])
def test_prefill_f32(shape, lengths):
    h, hk, dk, dv = shape
    x = inputs(lengths, h, hk, dk, dv, F32, seed=sum(lengths) + dk, init=len(lengths) > 1)
    out, state = kda.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], x["cu"], x["init"], scale=0.7)
    assert out.dtype is F32
    check(out, state, x, lengths, 0.7)


@pytest.mark.parametrize("shape", [(2, 2, 256, 128), (2, 1, 136, 136), (2, 2, 64, 256)])
@pytest.mark.parametrize("out_dtype", [F32, BF16])
def test_prefill_bf16_large_heads(shape, out_dtype):
    h, hk, dk, dv = shape
    x = inputs([70, 3], h, hk, dk, dv, BF16, seed=dv, init=True)
    out, state = kda.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], x["cu"], x["init"], out_dtype=out_dtype)
    assert out.dtype is out_dtype
    check(out, state, x, [70, 3], 1.0)


@pytest.mark.parametrize("dtype,out_dtype", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("shape", SHAPES + [(5, 5, 128, 256), (2, 2, 200, 128)])
@pytest.mark.parametrize("n", [1, 3, 90])
def test_decode(dtype, out_dtype, shape, n):
    h, hk, dk, dv = shape
    x = inputs([1] * n, h, hk, dk, dv, dtype, seed=n + dk, init=True, per_token=n != 3)
    state = x["init"].clone()
    out = kda.delta_decode(x["q"], x["k"], x["v"], x["g"], x["beta"], state, scale=dk ** -0.5, out_dtype=out_dtype)
    check(out, state, x, [1] * n, dk ** -0.5)


@pytest.mark.parametrize("n,shape", [(40, (96, 48, 128, 128)), (130, (4, 2, 120, 104)), (260, (2, 2, 256, 64)),
                                     (128, (4, 1, 64, 256)), (171, (3, 3, 72, 120)), (520, (1, 1, 128, 72))])
def test_decode_many_states(n, shape):
    """Sizes at which states go through shared memory whole."""
    h, hk, dk, dv = shape
    x = inputs([1] * n, h, hk, dk, dv, BF16, seed=3, init=True)
    state = x["init"].clone()
    out = kda.delta_decode(x["q"], x["k"], x["v"], x["g"], x["beta"], state, out_dtype=F32)
    check(out, state, x, [1] * n, 1.0)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_decode_of_a_constant_slow_decay(dtype):
    """2000 tokens of one decay near 1: its rounding must not add up."""
    x = inputs([1], 2, 2, 64, 64, F32, seed=21, init=True, per_token=False)
    x["g"].fill_(-1 / 300)
    x["beta"].fill_(0.0)                 # nothing is written, all that is left is the decay
    state = x["init"].clone()
    args = [x[n].to(dtype) if n in "qkv" else x[n] for n in ("q", "k", "v", "g", "beta")]
    for _ in range(2000):
        kda.delta_decode(*args, state)
    want = x["init"].double() * torch.exp(2000 * x["g"].double())[0]
    # a step rounds once, half an eps at most, as often up as down (5 deviations of the sum), and its decay is off by
    # eps / 300 or so
    off = ((state.double() - want) / want).abs().max()
    assert float(off) <= 2.0 ** -24 * (5 * 2000 ** 0.5 + 2 * 2000 / 300)


def test_prefill_of_a_constant_slow_decay():
    x = inputs([2000], 2, 2, 64, 64, F32, seed=22, init=True, per_token=False)
    x["g"].fill_(-1 / 300)
    x["beta"].fill_(0.0)
    _, state = kda.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], None, x["init"])
    want = x["init"].double() * torch.exp(2000 * x["g"].double())[0]
    # 250 blocks of eight tokens round once each, and their decays are off by 2 eps of the block's sum (8 / 300)
    off = ((state.double() - want) / want).abs().max()
    assert float(off) <= 2.0 ** -24 * (5 * 250 ** 0.5 + 4 * 2000 / 300)


@pytest.mark.parametrize("call", ["prefill", "decode"])
def test_decays_and_gates(call):
    """Decays from none to all, gates from 0 to 2; a token that forgets starts from nothing."""
    lengths = [90] if call == "prefill" else [1] * 90
    x = inputs(lengths, 2, 2, 64, 64, F32, seed=5, init=True)
    x["g"][::7] = -float("inf")
    x["g"][1::7] = 0.0
    x["g"][2::7] = -200.0
    x["g"][3::7] = -1e-6
    x["beta"][::5] = 0.0
    x["beta"][1::5] = 2.0
    x["beta"][2::5] = 1.0
    if call == "prefill":
        out, state = kda.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], x["cu"], x["init"])
    else:
        state = x["init"].clone()
        out = kda.delta_decode(x["q"], x["k"], x["v"], x["g"], x["beta"], state)
    check(out, state, x, lengths, 1.0)


def test_in_place_resume_and_given_outputs():
    x = inputs([33, 40], 2, 1, 64, 64, F32, seed=8, init=True)
    want, final = kda.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], x["cu"], x["init"])
    state, out = x["init"].clone(), torch.empty_like(want)
    got, same = kda.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], x["cu"], state, out=out, final_state=state)
    assert got is out and same is state
    assert torch.equal(out, want) and torch.equal(state, final)
    none = kda.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], x["cu"], x["init"], final_state=None)
    assert none[1] is None and torch.equal(none[0], want)


def test_cut_calls_give_the_whole():
    """A prompt in two calls, the second from the first one's state, against the definition."""
    x = inputs([100], 2, 2, 128, 128, F32, seed=9)
    parts = []
    state = None
    for b, e in ((0, 37), (37, 100)):
        o, state = kda.delta_prefill(*(x[n][b:e].contiguous() for n in ("q", "k", "v", "g", "beta")), None, state)
        parts.append(o)
    check(torch.cat(parts), state, x, [100], 1.0)


def test_refusals_of_the_binding():
    x = inputs([6], 4, 2, 64, 64, F32, seed=1)
    args = [x[n] for n in ("q", "k", "v", "g", "beta")]

    def bad(i, y, kind=ValueError, **kw):
        with pytest.raises(kind):
            kda.delta_prefill(*args[:i], y, *args[i + 1:], **kw)

    bad(0, x["q"].half())
    bad(0, x["q"].cpu())
    bad(0, x["q"].transpose(0, 1))
    bad(1, x["k"][:, :1].contiguous())
    bad(2, x["v"][:, :3].contiguous())
    bad(2, x["v"][:5].contiguous())
    bad(3, x["g"].double())
    bad(3, x["g"][:5].contiguous())
    bad(4, x["beta"].bfloat16())
    bad(4, x["beta"][0].contiguous())
    with pytest.raises(ValueError):
        kda.delta_prefill(*args, None, torch.zeros(2, 4, 64, 64, device="cuda"))
    with pytest.raises(ValueError):
        kda.delta_prefill(*args, out=torch.empty(6, 4, 32, device="cuda"))
    with pytest.raises(ValueError):
        kda.delta_prefill(*args, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        kda.delta_prefill(*args, torch.zeros(0, dtype=torch.int32, device="cuda"))
    with pytest.raises(kda.KDAError):
        kda.delta_prefill(*args, scale=float("nan"))
    with pytest.raises(kda.KDAError):
        kda.delta_prefill(*args, out=x["v"])
    with pytest.raises(ValueError):
        kda.delta_decode(*args, torch.zeros(6, 4, 64, 32, device="cuda"))
    with pytest.raises(kda.KDAError):
        y = inputs([2], 1, 1, 12, 8, F32, seed=1)
        kda.delta_prefill(y["q"], y["k"], y["v"], y["g"], y["beta"])


def test_graph_and_other_stream():
    """A prompt's call and a token's, captured together and replayed on new inputs; a call on a stream of its own."""
    x = inputs([50, 20], 2, 1, 64, 64, F32, seed=12, init=True)
    y = inputs([1, 1], 2, 1, 64, 64, F32, seed=13)
    state = x["init"].clone()
    out = torch.empty_like(x["v"])
    one = torch.empty_like(y["v"])

    def both():
        kda.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], x["cu"], x["init"], out=out, final_state=state)
        kda.delta_decode(y["q"], y["k"], y["v"], y["g"], y["beta"], state, out=one)

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    fresh = inputs([50, 20], 2, 1, 64, 64, F32, seed=14, init=True)
    for n in ("q", "k", "v", "g", "beta", "init"):
        x[n].copy_(fresh[n])
    graph.replay()
    torch.cuda.synchronize()
    got = out.clone(), state.clone(), one.clone()
    both()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, (out, state, one)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, s = kda.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], x["cu"], x["init"], stream=side)
    side.synchronize()
    assert torch.equal(o, out)


def test_rows_behind_the_last_sequence_and_nan():
    """Rows that no sequence has stay as they were; a NaN stays in its sequence."""
    lengths = [20, 30, 9]
    x = inputs(lengths, 2, 2, 64, 64, F32, seed=15, tail=5)
    out = torch.full_like(x["v"], 7.0)
    kda.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], x["cu"], out=out)
    assert bool((out[59:] == 7).all())
    want, final = kda.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], x["cu"])
    for n in ("q", "k", "v", "g", "beta"):
        x[n][20:50] = float("nan")
    out, state = kda.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], x["cu"])
    for part in (slice(0, 20), slice(50, 59)):
        assert torch.equal(out[part], want[part])
    assert torch.equal(state[0], final[0]) and torch.equal(state[2], final[2]) and bool(state[1].isnan().all())


def test_layer_with_a_packed_store():
    """The operators as they are used together: a prompt through the layer, its state packed into a store, read
    back, and tokens generated from it, against the layer's own formula in 64 bits on the same state."""
    from kimi_delta_attention_13_gb300.delta_layer import DeltaLayer
    from kimi_delta_attention_13_gb300.prefix_cache import CheckpointStore

    layer = DeltaLayer(256, heads=4, key_heads=2, d_k=64, d_v=64, dtype=F32, seed=3)
    gen = torch.Generator().manual_seed(4)
    x = torch.randn(41, 256, generator=gen).cuda()
    cu = torch.tensor([0, 30, 41], dtype=torch.int32, device="cuda")
    _, y, state = layer.prefill(x, cu_seqlens=cu)
    _, mixer, z = layer._enter(x, None)
    want, final, err, _ = recurrence(*mixer, [30, 11], None, layer.scale)
    assert bool(((state.double() - final).norm(dim=-2) <= err).all())
    store = CheckpointStore(3, 4, 64, 64, device="cuda", dtype=torch.int8)
    slots = torch.tensor([2, 0], device="cuda")
    rows = torch.arange(2, device="cuda")
    store.write(slots, state, rows)
    back = torch.empty_like(state)
    store.read(back, rows, slots)
    top = state.abs().amax(-1, keepdim=True)
    assert bool(((back - state).abs() <= top * (0.5 / 127 + 2.0 ** -22)).all())
    x1 = torch.randn(2, 256, generator=gen).cuda()
    _, mixer, z = layer._enter(x1, None)
    start = back.clone()
    _, y1 = layer.decode(x1, None, back)
    want, final, err, bound = recurrence(*mixer, [1, 1], start, layer.scale)
    assert bool(((back.double() - final).norm(dim=-2) <= err).all())
    gated = want / (want.square().mean(-1, keepdim=True) + layer.eps).sqrt() * torch.sigmoid(z.double())
    ref = gated.flatten(1) @ layer.w_out.double()
    # the norm divides an output's error by its row's size; the product adds 256 terms' roundings
    rms = (want.square().mean(-1, keepdim=True) + layer.eps).sqrt()
    rel = 2 * (bound / rms).amax() + 400 * 2.0 ** -24
    assert bool(((y1.double() - ref).abs() <= rel * (gated.abs().flatten(1) @ layer.w_out.double().abs()
                                                     + layer.w_out.double().abs().sum(0))).all())
