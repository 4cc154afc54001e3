"""The gates of kda_residual_norm and kda_norm_gate, element by element against 64 bits.

Bounds.  A gate is exp(-|z|) (an ulp), a sum with 1 (half of one), its reciprocal (one) and a product
(half); with the product of the gate 3.5 x 2^-23, within 2^-21 of the gated value.  Where every result is
rounded to bf16 the exponential is a fast one, by the documented error of such (2 + floor(1.173 |z|))
2^-23: (2 |z| + 6) 2^-23 with the rest, and 2^-8 for each rounding.  A gate below the smallest normal
number is off by half of the smallest subnormal one besides, and so is its product: 2^-149.
"""
import pytest
import torch

import kimi_delta_attention_13_gb300 as kda

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    yield
    torch.cuda.empty_cache()


def sigmoid(z):
    z = z.double()
    return torch.where(z < 0, z.exp(), torch.ones_like(z)) / (1 + (-z.abs()).exp())


def normal(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)


@pytest.mark.parametrize("D", [512, 1001])   # rows of whole 16-byte units, and not
@pytest.mark.parametrize("types", [("f32", "bf16"), ("f32", "f32")], ids="-".join)
def test_fp32_streams_get_the_full_gate(types, D):
    """Nothing but the gated part in the stream: x = 0, no norm, gates from the far left to the right."""
    tr, tb = (TYPES[t] for t in types)
    y, z = normal(1, 8, D).to(tb), torch.linspace(-60, 20, 8 * D, device=DEV).view(8, D).to(tb)
    res, _ = kda.residual_norm(torch.zeros(8, D, device=DEV, dtype=tr), y, torch.ones(D, device=DEV), z=z,
                               scale=0.5, eps=EPS)
    want = 0.5 * y.double() * sigmoid(z)
    err = (res.double() - want).abs()
    assert bool((err <= 2.0 ** -21 * want.abs()).all()), float((err / want.abs()).max() * 2 ** 21)


@pytest.mark.parametrize("D", [512, 1001])
def test_bf16_streams_get_the_fast_gate(D):
    y, z = normal(2, 8, D).bfloat16(), torch.linspace(-60, 20, 8 * D, device=DEV).view(8, D).bfloat16()
    res, _ = kda.residual_norm(torch.zeros(8, D, device=DEV, dtype=torch.bfloat16), y, torch.ones(D, device=DEV),
                               z=z, scale=0.5, eps=EPS)
    want = 0.5 * y.double() * sigmoid(z)
    tol = (2.0 ** -8 + (2 * z.double().abs() + 6) * 2.0 ** -23 * (1 + 2.0 ** -8)) * want.abs()
    assert bool(((res.double() - want).abs() <= tol).all())


# z around the points where exp(-z) passes 2^126 and 2^128, and well past them
FAR = [-80.0, -87.0, -87.5, -88.0, -88.5, -89.0, -92.0, -95.0]


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32"), ("bf16", "f32")], ids="-".join)
def test_residual_norm_gates_far_out(types):
    """Gates of 1e-35 to 1e-42 on parts large enough for them to count."""
    tr, tb = (TYPES[t] for t in types)
    z = torch.tensor(FAR, device=DEV).to(tb).repeat(4, 1)
    y = torch.full((4, 8), 2.0 ** 120, device=DEV).to(tb)
    res, out = kda.residual_norm(torch.zeros(4, 8, device=DEV, dtype=tr), y, torch.ones(8, device=DEV), z=z, eps=EPS)
    want = y.double() * sigmoid(z)
    gate = ((2 * z.double().abs() + 6) * 2.0 ** -23) if types == ("bf16", "bf16") else 2.0 ** -21
    tol = gate * want + y.double() * 2.0 ** -149
    tol = tol + (2.0 ** -8 * (want + tol) if tr is torch.bfloat16 else 0)
    assert bool(((res.double() - want).abs() <= tol).all()), (res[0], want[0])


@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
def test_norm_gate_gates_far_out(out_dtype):
    z = torch.tensor(FAR, device=DEV).repeat(3, 2, 1)
    o, w = torch.ones(3, 2, 8, device=DEV), torch.full((8,), 2.0 ** 120, device=DEV)
    out = kda.norm_gate(o, z, w, eps=EPS, out_dtype=TYPES[out_dtype])
    want = w.double() * sigmoid(z) / (1 + EPS) ** 0.5
    gate = (2 * z.double().abs() + 6) * 2.0 ** -23 if out_dtype == "bf16" else 2.0 ** -21
    # the mean of ones and its inverse root: sixteen roundings and function values of 2^-22 at most
    tol = (gate + 16 * 2.0 ** -22) * want + w.double() * 2.0 ** -149
    tol = tol + (2.0 ** -8 * (want + tol) if out_dtype == "bf16" else 0)
    assert bool(((out.double() - want).abs() <= tol).all()), (out[0, 0], want[0, 0])


@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
def test_norm_gate_at_the_edges(out_dtype):
    """Rows of zeros, tiny and large rows, gates far out, infinite gates, NaN: the other elements stay
    as they are, bit for bit."""
    o, z, w = normal(4, 6, 2, 128), normal(5, 6, 2, 128), torch.ones(128, device=DEV)
    o[0], o[1], o[2] = 0, o[1] * 1e-18, o[2] * 1e15
    z[3] = torch.linspace(-80, 80, 128, device=DEV)
    dt = TYPES[out_dtype]
    out = kda.norm_gate(o, z, w, eps=EPS, out_dtype=dt)
    want = o.double() / (o.double().square().mean(-1, keepdim=True) + EPS).sqrt() * sigmoid(z)
    gate = (2 * z.double().abs() + 6) * 2.0 ** -23 if out_dtype == "bf16" else 2.0 ** -21
    tol = (gate + 132 * 2.0 ** -24 + 16 * 2.0 ** -22) * want.abs()
    tol = tol + (2.0 ** -8 * (want.abs() + tol) if out_dtype == "bf16" else 0) + 1e-45
    assert bool(((out.double() - want).abs() <= tol).all())
    z[5, 0, 0], z[5, 1, 3], z[5, 1, 4] = float("nan"), float("inf"), float("-inf")
    o[4, 0, 7] = float("nan")
    again = kda.norm_gate(o, z, w, eps=EPS, out_dtype=dt)
    assert torch.equal(again[:4], out[:4]) and again[4, 0].isnan().all() and torch.equal(again[4, 1], out[4, 1])
    assert again[5, 0, 0].isnan() and torch.equal(again[5, 0, 1:], out[5, 0, 1:])
    assert again[5, 1, 4] == 0 and bool(again[5, 1].isfinite().all())
    assert abs(float(again[5, 1, 3]) - float(want[5, 1, 3] / sigmoid(normal(5, 6, 2, 128)[5, 1, 3]))) \
        <= 2.0 ** -7 * abs(float(again[5, 1, 3]))
