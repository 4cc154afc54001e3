"""kda_linear_prefill and kda_linear_decode on the GPU against the recurrence in 64 bits.

Bounds, element by element.  Let M be the recurrence run on absolute values (|q|, |k|, |v|), which
bounds the sum of the magnitudes of the terms of an output, and S_abs the same for the state.
  - fp32 inputs, and the state: every product and sum of an n-step chain is rounded once, by at most
    2^-24 of the magnitudes: n 2^-24 M, with n = d_k + 2 T + 8 for outputs, 2 T + 8 for states.
  - bf16 inputs: besides that, an output's terms have one bf16 operand that was rounded (a score, or
    an element of the state), by at most 2^-8 of it; a state's terms one operand that was split into
    two bf16 parts, of which the second is rounded: 2^-16.
  - a bf16 output is rounded once more: 2^-8 of its value.
"""
import pytest
import torch

import kimi_delta_attention_13_gb300 as kda

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    yield
    assert kda.device_status() == 0
    torch.cuda.empty_cache()


def make(lengths, H, Hkv, dk, dv, dtype, seed, decay="token", init=True):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    T, dt = sum(lengths), TYPES[dtype]
    g = -torch.nn.functional.softplus(n(T, H) - 2) if decay == "token" else -torch.rand(H, generator=gen, device=DEV)
    cu = torch.tensor([0] + lengths, device=DEV).cumsum(0).to(torch.int32)
    return dict(q=n(T, H, dk).to(dt), k=(n(T, Hkv, dk) * dk ** -0.5).to(dt), v=n(T, Hkv, dv).to(dt), g=g, cu=cu,
                lengths=lengths, init=0.1 * n(len(lengths), H, dk, dv) if init else None)


def recurrence(x, scale):
    """(out, final, out_abs, final_abs) in 64 bits, token by token, sequences side by side."""
    share = x["q"].shape[1] // x["k"].shape[1]
    q, k, v = x["q"].double(), x["k"].double().repeat_interleave(share, 1), x["v"].double().repeat_interleave(share, 1)
    T, H, dk = q.shape
    dv, N, cu = v.shape[-1], len(x["lengths"]), x["cu"].long()
    a = x["g"].double().exp().expand(T, H)
    s = x["init"].double().clone() if x["init"] is not None else torch.zeros(N, H, dk, dv, device=DEV).double()
    sa = s.abs()
    out, outa = torch.zeros(T, H, dv, device=DEV).double(), torch.zeros(T, H, dv, device=DEV).double()
    for t in range(max(x["lengths"], default=0)):
        live = torch.tensor([i for i, L in enumerate(x["lengths"]) if L > t], device=DEV)
        at = cu[live] + t
        kt, vt, at_a = k[at][..., :, None], v[at][..., None, :], a[at][..., None, None]
        s[live] = s[live] * at_a + kt * vt
        sa[live] = sa[live] * at_a + kt.abs() * vt.abs()
        out[at] = (q[at][..., None, :] @ s[live])[..., 0, :]
        outa[at] = (q[at].abs()[..., None, :] @ sa[live])[..., 0, :]
    return out * scale, s, outa * abs(scale), sa


def check(x, got, dtype, out_dtype, scale):
    out, fin = got
    ref, rfin, mag, smag = recurrence(x, scale)
    T = max(x["lengths"], default=0)
    dk = x["q"].shape[-1]
    operand = (2.0 ** -8, 2.0 ** -16) if dtype == "bf16" else (0.0, 0.0)
    tol = (operand[0] + (dk + 2 * T + 8) * 2.0 ** -24) * mag
    if out_dtype == "bf16":
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    err = (out.double() - ref).abs()
    assert bool((err <= tol + 1e-30).all()), f"outputs: {float((err / (tol + 1e-30)).max()):.3g} of the bound"
    if fin is not None:
        serr, stol = (fin.double() - rfin).abs(), (operand[1] + (2 * T + 8) * 2.0 ** -24) * smag + 1e-30
        assert bool((serr <= stol).all()), f"states: {float((serr / stol).max()):.3g} of the bound"


SHAPES = [   # lengths, H, H_kv, d_k, d_v
    ([1], 1, 1, 64, 64),
    ([127], 2, 2, 128, 128),
    ([128], 3, 1, 128, 128),
    ([129, 0, 1, 255, 257], 4, 2, 128, 128),
    ([0, 0, 5, 0, 64, 0], 2, 2, 128, 128),
    ([300, 3], 2, 1, 64, 128),
    ([40, 400], 2, 2, 128, 64),
    ([130], 6, 3, 64, 64),
    ([33, 200], 2, 2, 8, 8),
    ([150], 2, 2, 96, 80),
    ([70, 131], 1, 1, 120, 16),
    ([90], 2, 1, 256, 40),
    ([65, 2], 2, 2, 136, 256),
    ([1] * 70, 2, 2, 128, 128),
    ([1500, 700], 1, 1, 128, 128),       # cut into segments
    ([0, 900, 1, 128, 1100], 2, 1, 64, 64),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0][:5]}x{s[1:]}".replace(" ", ""))
def test_prefill(shape, dtype):
    lengths, H, Hkv, dk, dv = shape
    x = make(lengths, H, Hkv, dk, dv, dtype, seed=sum(lengths) + H + dk)
    got = kda.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["cu"], x["init"], scale=0.3)
    assert got[0].dtype == TYPES[dtype]
    check(x, got, dtype, dtype, 0.3)


@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("init", [False, True])
def test_prefill_types_and_decays(dtype, out_dtype, decay, init):
    x = make([260, 77], 4, 2, 128, 128, dtype, seed=5, decay=decay, init=init)
    got = kda.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["cu"], x["init"], out_dtype=TYPES[out_dtype])
    assert got[0].dtype == TYPES[out_dtype]
    check(x, got, dtype, out_dtype, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_forgets_and_keeps(dtype):
    """Log decays of -inf (nothing before is left), 0 (all of it is) and far below fp32's range."""
    x = make([200, 500], 4, 4, 128, 128, dtype, seed=6)
    x["g"][::7, 0] = float("-inf")
    x["g"][:, 1] = 0
    x["g"][5::31, 2] = -200.0
    x["g"][:, 3] = float("-inf")
    got = kda.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["cu"], x["init"])
    check(x, got, dtype, dtype, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths", [[100, 300], [4000]])
def test_prefill_in_place_resume(lengths, dtype):
    """final_state = init_state, sequences cut into segments among them."""
    x = make(lengths, 2, 2, 64, 64, dtype, seed=7)
    want = kda.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["cu"], x["init"])
    state = x["init"].clone()
    out, fin = kda.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["cu"], state, final_state=state)
    assert fin is state and torch.equal(out, want[0]) and torch.equal(state, want[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_continues_where_it_stopped(dtype):
    """Two prefills, the second from the first's state, against one."""
    x = make([512], 2, 2, 128, 128, dtype, seed=8, init=False)
    c, f = 200, lambda t, s: t[s].contiguous()  # noqa: E731
    parts, state = [], None
    for s in (slice(0, c), slice(c, None)):
        o, state = kda.linear_prefill(f(x["q"], s), f(x["k"], s), f(x["v"], s), f(x["g"], s), None, state)
        parts.append(o)
    check(x, (torch.cat(parts), state), dtype, dtype, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_other_sequences_stay_clean(dtype):
    """NaN and infinity in one sequence leave its neighbours as they are, bit for bit."""
    lengths = [60, 75, 190]
    x = make(lengths, 2, 2, 128, 128, dtype, seed=9)
    want = kda.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["cu"], x["init"])
    bad = {n: x[n].clone() for n in ("q", "k", "v", "g", "init")}
    for i, n in enumerate(("q", "k", "v")):
        bad[n][60:135] = float("nan") if i % 2 else float("inf")
    bad["init"][1] = float("nan")
    out, fin = kda.linear_prefill(bad["q"], bad["k"], bad["v"], bad["g"], x["cu"], bad["init"])
    keep = [*range(60), *range(135, 325)]
    assert torch.equal(out[keep], want[0][keep]) and torch.equal(fin[[0, 2]], want[1][[0, 2]])


def test_prefill_nothing_to_do():
    x = make([0, 0], 2, 2, 128, 128, "bf16", seed=10)
    out, fin = kda.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["cu"], x["init"])
    assert out.shape == (0, 2, 128) and torch.equal(fin, x["init"])
    out, fin = kda.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["cu"])
    assert not fin.any()
    out, fin = kda.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["cu"], final_state=False)
    assert fin is None


def test_prefill_own_buffers_and_stream():
    """Outputs, state and workspace of the caller's, on another stream; the same bits each time."""
    x = make([3000, 50], 2, 1, 128, 128, "bf16", seed=11)
    args = (x["q"], x["k"], x["v"], x["g"], x["cu"], x["init"])
    want = kda.linear_prefill(*args)
    ws = torch.empty(kda.load().kda_linear_prefill_workspace(2, 3050, 2, 128, 128, 0), device=DEV, dtype=torch.uint8)
    side = torch.cuda.Stream()
    out, fin = torch.empty_like(want[0]), torch.empty_like(want[1])
    side.wait_stream(torch.cuda.current_stream())
    for w in (ws, None):
        out.zero_()
        side.wait_stream(torch.cuda.current_stream())
        kda.linear_prefill(*args, out=out, final_state=fin, workspace=w, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, want[0]) and torch.equal(fin, want[1])


def test_prefill_refuses():
    x = make([30], 4, 2, 64, 64, "bf16", seed=12)
    q, k, v, g = (x[n] for n in "qkvg")
    with pytest.raises(ValueError, match="contiguous"):
        kda.linear_prefill(q.transpose(0, 1).contiguous().transpose(0, 1), k, v, g)
    with pytest.raises(ValueError, match="shape"):
        kda.linear_prefill(q, k[:20], v, g)
    with pytest.raises(ValueError, match="float32"):
        kda.linear_prefill(q, k, v, g.bfloat16())
    with pytest.raises(ValueError, match="int32"):
        kda.linear_prefill(q, k, v, g, torch.tensor([0, 30], device=DEV))
    with pytest.raises(ValueError, match="shape"):
        kda.linear_prefill(q, k, v, g, None, torch.zeros(1, 2, 64, 64, device=DEV))
    with pytest.raises(kda.KDAError, match="UNSUPPORTED"):
        kda.linear_prefill(q[..., :20].contiguous(), k[..., :20].contiguous(), v, g)
    y = make([200000], 1, 1, 64, 64, "bf16", seed=13)
    with pytest.raises(ValueError, match="workspace"):
        kda.linear_prefill(y["q"], y["k"], y["v"], y["g"], workspace=torch.empty(16, device=DEV, dtype=torch.uint8))


def test_prefill_offsets_past_32_bits():
    """More than 2^31 elements a tensor: the last tokens, which by their decays depend on the last
    few hundred only, against a call on those alone."""
    T, H, d, tail = 180000, 96, 128, 640
    gen = torch.Generator(device=DEV).manual_seed(14)
    q, k, v = (torch.randn(T, H, d, generator=gen, device=DEV, dtype=torch.bfloat16) for _ in range(3))
    g = torch.full((H,), -1.0, device=DEV)
    out, fin = kda.linear_prefill(q, k, v, g, scale=0.01)
    x = dict(q=q[-tail:].contiguous(), k=k[-tail:].contiguous(), v=v[-tail:].contiguous(), g=g,
             cu=torch.tensor([0, tail], device=DEV, dtype=torch.int32), lengths=[tail], init=None)
    ref, rfin, mag, smag = recurrence(x, 0.01)
    late = slice(tail - 256, tail)   # exp(-384) of what came before
    err = (out[-256:].double() - ref[late]).abs()
    assert bool((err <= 2.0 ** -8 * (ref[late].abs() * 1.01 + mag[late]) * 1.01).all())
    assert bool(((fin.double() - rfin).abs() <= (2.0 ** -16 + 1400 * 2.0 ** -24) * smag).all())


# ---------------------------------------------------------------------------------------------
# one token per sequence

@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("N,H,Hkv,dk,dv,decay", [
    (1, 1, 1, 128, 128, "token"), (3, 4, 2, 128, 128, "head"), (200, 2, 2, 128, 128, "token"),
    (5, 6, 1, 64, 64, "token"), (400, 1, 1, 64, 64, "head"), (2, 2, 2, 8, 8, "token"), (7, 2, 1, 256, 40, "token"),
    (180, 2, 2, 96, 200, "token"), (170, 2, 2, 136, 24, "head"), (160, 2, 2, 256, 256, "token"),
])
def test_decode(N, H, Hkv, dk, dv, decay, dtype, out_dtype):
    x = make([1] * N, H, Hkv, dk, dv, dtype, seed=N + dk, decay=decay)
    if decay == "token":
        x["g"][0, 0] = float("-inf")
    state = x["init"].clone()
    out = kda.linear_decode(x["q"], x["k"], x["v"], x["g"], state, scale=-0.4, out_dtype=TYPES[out_dtype])
    assert out.dtype == TYPES[out_dtype]
    check(x, (out, state), "f32", out_dtype, -0.4)   # no operand is rounded here, whatever its type


def test_decode_continues_prefill():
    """A prompt, then single tokens from its state, against one recurrence over all of them."""
    x = make([140], 4, 2, 128, 128, "bf16", seed=20, init=False)
    n = 132
    head = [x[t][:n].contiguous() for t in "qkvg"]
    out, state = kda.linear_prefill(*head)
    outs = [out]
    for t in range(n, 140):
        outs.append(kda.linear_decode(*[x[c][t:t + 1].contiguous() for c in "qkvg"], state))
    check(x, (torch.cat(outs), state), "bf16", "bf16", 1.0)


def test_decode_nothing_to_do():
    z = torch.zeros(0, 2, 64, device=DEV)
    out = kda.linear_decode(z, z, z, torch.zeros(0, 2, device=DEV), torch.zeros(0, 2, 64, 64, device=DEV))
    assert out.shape == (0, 2, 64)


def test_decode_refuses():
    x = make([1] * 3, 4, 2, 64, 64, "bf16", seed=21)
    with pytest.raises(ValueError, match="state"):
        kda.linear_decode(x["q"], x["k"], x["v"], x["g"], x["init"].bfloat16())
    with pytest.raises(ValueError, match="state"):
        kda.linear_decode(x["q"], x["k"], x["v"], x["g"], x["init"][:2])
    with pytest.raises(ValueError, match="out"):
        kda.linear_decode(x["q"], x["k"], x["v"], x["g"], x["init"], out=torch.empty(3, 4, 32, device=DEV))
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        kda.linear_decode(x["q"], x["k"], x["v"], x["g"], x["init"], out_dtype=torch.float16)


def test_prefill_and_decode_in_a_graph():
    """Captured and replayed on changed inputs."""
    x = make([2500, 40], 2, 1, 128, 128, "bf16", seed=22)
    d = make([1] * 2, 2, 1, 128, 128, "bf16", seed=23)
    fin = torch.empty(2, 2, 128, 128, device=DEV)

    def step():
        out, _ = kda.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["cu"], x["init"], final_state=fin)
        return out, kda.linear_decode(d["q"], d["k"], d["v"], d["g"], fin)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, one = step()
    x["v"].mul_(0.5)
    x["g"].mul_(2)
    graph.replay()
    got = out.clone(), one.clone(), fin.clone()
    want = step()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2], fin)
