"""delta_prefill on the tensor cores (bf16 operands, head sizes up to 128) against the recurrence in 64 bits."""
import pytest
import torch

import kimi_delta_attention_13_gb300 as kda
from delta_plain import chunked_bounds, inputs, recurrence

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def call(x, **kw):
    return kda.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], x["cu"], x["init"], **kw)


def check(out, state, x, lengths, scale=1.0, slack=1e-30):
    want, final, err, bound = chunked_bounds(x["q"], x["k"], x["v"], x["g"], x["beta"], lengths, x["init"], scale)
    assert kda.device_status() == 0
    rows, half = sum(lengths), torch.finfo(out.dtype).eps / 2
    off = (out[:rows].double() - want[:rows]).abs()
    over = off > bound[:rows] + half * (want[:rows].abs() + bound[:rows]) + slack   # (what is rounded is off already)
    assert not bool(over.any()), (int(over.sum()), over.numel(), float(off[over].max()))
    off = (state.double() - final).norm(dim=-2)
    assert bool((off <= err + slack).all()), float((off / err.clamp(min=1e-300)).max())


@pytest.mark.parametrize("lengths", [[64], [8], [63], [65], [128], [200], [17, 0, 64, 130, 5]])
@pytest.mark.parametrize("shape", [(1, 1, 128, 128), (4, 2, 128, 128), (3, 1, 64, 64)])
def test_lengths(lengths, shape):
    h, hk, dk, dv = shape
    x = inputs(lengths, h, hk, dk, dv, BF16, seed=sum(lengths) + h, init=len(lengths) > 1 or lengths == [65])
    out, state = call(x, scale=dk ** -0.5)
    assert out.dtype is BF16
    check(out, state, x, lengths, dk ** -0.5)


@pytest.mark.parametrize("dk,dv", [(8, 8), (16, 128), (128, 8), (24, 40), (72, 96), (80, 120), (96, 64), (120, 104)])
@pytest.mark.parametrize("out_dtype", [F32, BF16])
def test_head_sizes(dk, dv, out_dtype):
    x = inputs([70, 90], 2, 1, dk, dv, BF16, seed=dk + dv, init=True, per_token=dv != 40)
    out, state = call(x, scale=0.5, out_dtype=out_dtype)
    check(out, state, x, [70, 90], 0.5)


def test_long_and_without_decay():
    """A thousand tokens that forget nothing, and a thousand of a constant slow decay."""
    for seed, g in ((1, 0.0), (2, -1 / 256)):
        x = inputs([1000], 2, 2, 128, 128, BF16, seed=seed)
        x["g"].fill_(g)
        out, state = call(x)
        check(out, state, x, [1000])
        _, final, _, _ = recurrence(x["q"], x["k"], x["v"], x["g"], x["beta"], [1000], None)
        # operands are exact, and roundings of fp32 sums are as often up as down: far from their bound, near eps
        assert float((state.double() - final).norm() / final.norm()) < 16 * 2.0 ** -24


def test_decays_and_gates():
    lengths = [150, 40]
    x = inputs(lengths, 2, 2, 128, 128, BF16, seed=5, init=True)
    x["g"][::7] = -float("inf")
    x["g"][1::7] = 0.0
    x["g"][2::7] = -200.0
    x["g"][3::7] = -1e-6
    x["g"][4::7] = -90.0
    x["beta"][::5] = 0.0
    x["beta"][1::5] = 2.0
    x["beta"][2::5] = 1.0
    out, state = call(x)
    check(out, state, x, lengths)


def test_strong_and_unlike_decays():
    """Sums of log decays far from 0, whose differences still have to be good."""
    x = inputs([130], 2, 1, 64, 128, BF16, seed=6)
    x["g"][:, 0] = -7.77
    x["g"][:, 1] = -0.001
    x["g"][::16, 1] = -100.0
    out, state = call(x, out_dtype=F32)
    check(out, state, x, [130])


def test_keys_all_alike():
    """The triangular matrix is then full of ones: beta 1 overwrites what the last token wrote."""
    x = inputs([128], 2, 2, 128, 128, BF16, seed=7)
    x["k"][:] = x["k"][:1]
    x["g"].zero_()
    x["beta"].fill_(1.0)
    out, state = call(x)
    check(out, state, x, [128])


def test_scales_of_values():
    """States and values far from 1 in magnitude."""
    for power in (-60, 60):
        x = inputs([100], 1, 1, 128, 128, BF16, seed=8, init=True)
        x["v"] *= 2.0 ** power
        x["init"] *= 2.0 ** power
        out, state = call(x)
        check(out, state, x, [100], slack=0.0)


def test_rows_behind_and_nan():
    """Rows that no sequence has stay as they were; a NaN, and any bits behind a sequence, stay out of the others."""
    lengths = [70, 64, 39]
    x = inputs(lengths, 2, 2, 128, 128, BF16, seed=9, tail=21)
    want, final = call(x)
    for n in ("q", "k", "v", "g", "beta"):
        x[n][70:134] = float("nan")
        x[n][173:] = float("nan")
    out = torch.full_like(want, 7.0)
    _, state = call(x, out=out)
    assert bool((out[173:] == 7).all())
    for part in (slice(0, 70), slice(134, 173)):
        assert torch.equal(out[part], want[part])
    assert torch.equal(state[0], final[0]) and torch.equal(state[2], final[2]) and bool(state[1].isnan().all())
    assert kda.device_status() == 0


def test_a_nan_reaches_back_to_its_chunk_at_most():
    x = inputs([192], 1, 1, 128, 128, BF16, seed=10)
    want, _ = call(x)
    x["v"][101] = float("nan")
    out, _ = call(x)
    assert torch.equal(out[:64], want[:64]) and bool(out[101:].isnan().all())


def test_in_place_graph_streams():
    lengths = [100, 200]
    x = inputs(lengths, 4, 2, 128, 128, BF16, seed=11, init=True)
    want, final = call(x)
    state = x["init"].clone()
    out = torch.empty_like(want)

    def one():
        kda.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], x["cu"], state, out=out, final_state=state)

    one()
    assert torch.equal(out, want) and torch.equal(state, final)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one()
    state.copy_(x["init"])
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(state, final)
    y = inputs(lengths, 4, 2, 128, 128, BF16, seed=12, init=True)
    ref = call(y)
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s, z in zip(sides, (x, y)):   # two calls at once
        s.wait_stream(torch.cuda.current_stream())
        got.append(call(z, stream=s))
    torch.cuda.synchronize()
    for (o, f), (a, b) in zip(got, ((want, final), ref)):
        assert torch.equal(o, a) and torch.equal(f, b)
    assert kda.device_status() == 0


def test_many_ctas():
    """More (sequence, head) pairs than the GPU holds at once."""
    lengths = [80] * 20
    x = inputs(lengths, 32, 8, 64, 64, BF16, seed=13, init=True)
    out, state = call(x)
    _, final, err, _ = chunked_bounds(*(x[n][:160] for n in ("q", "k", "v", "g", "beta")), lengths[:2], x["init"][:2])
    assert bool(((state[:2].double() - final).norm(dim=-2) <= err).all())
    for s in (7, 19):   # each as in a call of its own
        part = slice(80 * s, 80 * s + 80)
        o, f = kda.delta_prefill(*(x[n][part] for n in ("q", "k", "v", "g", "beta")), None, x["init"][s:s + 1].contiguous())
        assert torch.equal(o, out[part]) and torch.equal(f[0], state[s])


def test_bad_table_stays_inside():
    """A table that does not rise, or points past the tensors, reads and writes inside them."""
    x = inputs([100], 2, 1, 128, 128, BF16, seed=14)
    out = torch.full((132, 2, 128), 5.0, device="cuda", dtype=BF16)
    cu = torch.tensor([0, 64, 30, 1000], dtype=torch.int32, device="cuda")
    kda.delta_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], cu, out=out[:100])
    torch.cuda.synchronize()
    assert bool((out[100:] == 5).all()) and kda.device_status() == 0


def test_waits_run_out():
    kda.diag_delta_timeout(2_000_000)
    torch.cuda.synchronize()
    assert kda.device_status() == 5 and kda.device_status() == 0
    x = inputs([70], 1, 1, 128, 128, BF16, seed=15)
    check(*call(x), x, [70])
    for cycles in (0, -1, 4_000_000_001):
        with pytest.raises(kda.KDAError, match="INVALID"):
            kda.diag_delta_timeout(cycles)
