"""kda_norm_gate and kda_residual_norm on the GPU against the formulas in 64 bits.

Bounds, from the arithmetic (sums of squares of n terms and a handful of products in fp32): the mean
is off by at most (n + 4) 2^-24 of itself, its inverse square root by half of that, and each of the
some 16 further roundings and function values by 2^-22 at most.  A gate rounded to bf16 may take the
fast exponential: |z| 2^-22 + 2^-20.  A bf16 result is rounded once more, by 2^-8 of its value.  An
add of x to the block's part is off by these shares of the part's magnitude, not of the sum.
"""
import pytest
import torch

import kimi_delta_attention_13_gb300 as kda

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    yield
    torch.cuda.empty_cache()


def normal(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)


def share(n, z=None):
    s = (n + 4) * 2.0 ** -24 + 16 * 2.0 ** -22
    return s if z is None else s + z.abs() * 2.0 ** -22 + 2.0 ** -20


def step(t):
    return 2.0 ** -8 if t is torch.bfloat16 else 0.0


def close(got, want, tol):
    tol = tol + step(got.dtype) * (want.abs() + tol) + 1e-37
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), f"{float((err / tol).max()):.3g} of the bound"


def gate_ref(o, z, w):
    o, z = o.double(), z.double()
    return o / (o.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double() * torch.sigmoid(z)


@pytest.mark.parametrize("types", [("bf16", "bf16", "bf16"), ("f32", "bf16", "bf16"), ("f32", "f32", "f32"),
                                   ("bf16", "f32", "f32"), ("f32", "bf16", "f32"), ("bf16", "bf16", "f32"),
                                   ("bf16", "f32", "bf16"), ("f32", "f32", "bf16")], ids="-".join)
@pytest.mark.parametrize("T,H,d,per_head", [(1, 1, 128, False), (3, 5, 128, True), (17, 3, 64, False), (700, 31, 128, True),
                                            (9, 2, 8, True), (5, 7, 72, False), (33, 2, 256, True), (2, 3, 200, False)])
def test_norm_gate(T, H, d, per_head, types):
    to, tz, ty = (TYPES[t] for t in types)
    o, z = normal(1, T, H, d).to(to), (3 * normal(2, T, H, d)).to(tz)
    w = 1 + 0.2 * (normal(3, H, d) if per_head else normal(3, d))
    out = kda.norm_gate(o, z, w, eps=EPS, out_dtype=ty)
    assert out.dtype == ty
    want = gate_ref(o, z, w)
    close(out, want, share(d, z.double()) * want.abs())


def test_norm_gate_rows_at_the_edges():
    """All zeros, tiny and large rows, gates far out, NaN and infinity in a row of their own."""
    o, z = normal(4, 6, 2, 128), normal(5, 6, 2, 128)
    o[0] = 0
    o[1] *= 1e-18
    o[2] *= 1e15
    z[3] = torch.linspace(-80, 80, 128, device=DEV)
    w = torch.ones(128, device=DEV)
    want = gate_ref(o, z, w)
    out = kda.norm_gate(o, z, w, eps=EPS)
    close(out, want, share(128, z.double()) * want.abs())
    o[4, 0, 7], o[4, 1, 9], z[5, 0, 0] = float("nan"), float("inf"), float("nan")
    again = kda.norm_gate(o, z, w, eps=EPS)
    assert torch.equal(again[:4], out[:4]) and again[4, 0].isnan().all() and torch.equal(again[5, 1], out[5, 1])
    assert again[5, 0, 0].isnan() and torch.equal(again[5, 0, 1:], out[5, 0, 1:])
    z.fill_(float("-inf"))
    assert not kda.norm_gate(normal(4, 6, 2, 128), z, w, eps=EPS).any()


@pytest.mark.parametrize("over", ["o", "z"])
def test_norm_gate_in_place(over):
    o, z, w = normal(6, 300, 8, 128).bfloat16(), normal(7, 300, 8, 128).bfloat16(), normal(8, 128)
    want = kda.norm_gate(o, z, w)
    into = o if over == "o" else z
    out = kda.norm_gate(o, z, w, out=into)
    assert out is into and torch.equal(out, want)


def residual_ref(x, y, z, w_post, w, scale):
    """(r, n, magnitude of the block's part)."""
    u = y.double()
    if w_post is not None:
        u = u / (u.square().mean(-1, keepdim=True) + EPS).sqrt() * w_post.double()
    if z is not None:
        u = u * torch.sigmoid(z.double())
    r = x.double() + scale * u
    return r, r / (r.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double(), abs(scale) * u.abs()


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32"), ("bf16", "f32")], ids="-".join)
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,D", [(1, 1), (3, 7), (2, 8), (5, 100), (70, 256), (33, 1000), (4, 1024), (6, 1032), (3, 2304),
                                 (2, 4096), (3, 4104), (2, 8192), (2, 12288), (3, 16384), (2, 16392), (2, 20001)])
def test_residual_norm(T, D, gated, post, types):
    tr, tb = (TYPES[t] for t in types)
    x, y = normal(1, T, D).to(tr), (2 * normal(2, T, D)).to(tb)
    z = (2 * normal(3, T, D)).to(tb) if gated else None
    w, w_post = 1 + 0.1 * normal(4, D), 1 + 0.1 * normal(5, D) if post else None
    res, out = kda.residual_norm(x, y, w, w_post=w_post, z=z, scale=-0.7, eps=EPS)
    assert res.dtype == tr and out.dtype == tb
    r, n, mag = residual_ref(x, y, z, w_post, w, -0.7)
    part = share(D, None if z is None else z.double()) * mag + 2.0 ** -24 * r.abs()
    close(res, r, part)
    rms = (r.square().mean(-1, keepdim=True) + EPS).sqrt()
    inv = w.double().abs() / rms
    # the part's error moves the norm too: by its share of the rms at most
    close(out, n, inv * part + n.abs() * (share(D) + part.square().mean(-1, keepdim=True).sqrt() / rms))


@pytest.mark.parametrize("D", [128, 1001, 12288])
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")], ids="-".join)
def test_norm_without_an_add(D, types):
    tr, tb = (TYPES[t] for t in types)
    x, w = normal(6, 5, D).to(tr), normal(7, D)
    res, out = kda.residual_norm(x, None, w, eps=EPS, out_dtype=tb)
    assert res is x and out.dtype == tb
    n = x.double() / (x.double().square().mean(-1, keepdim=True) + EPS).sqrt() * w.double()
    close(out, n, share(D) * n.abs())


@pytest.mark.parametrize("D", [1001, 2048])
def test_residual_norm_in_place(D):
    """res over x, out over y."""
    x, y, z, w = normal(8, 40, D).bfloat16(), normal(9, 40, D).bfloat16(), normal(10, 40, D).bfloat16(), normal(11, D)
    want = kda.residual_norm(x, y, w, w_post=w, z=z)
    got = kda.residual_norm(x, y, w, w_post=w, z=z, res=x, out=y)
    assert got[0] is x and got[1] is y and torch.equal(x, want[0]) and torch.equal(y, want[1])


def test_residual_norm_rows_at_the_edges():
    x, y, w = normal(12, 5, 512), normal(13, 5, 512), torch.ones(512, device=DEV)
    x[0], y[0] = 0, 0
    y[1] *= 1e-20
    res, out = kda.residual_norm(x, y, w, w_post=w, eps=EPS)
    assert not res[0].any() and not out[0].any()
    r, n, mag = residual_ref(x, y, None, w, w, 1.0)
    close(res, r, share(512) * mag + 2.0 ** -24 * r.abs())
    x[2, 3], y[3, 4] = float("inf"), float("nan")
    again = kda.residual_norm(x, y, w, w_post=w, eps=EPS)
    for i in (0, 1, 4):
        assert torch.equal(again[0][i], res[i]) and torch.equal(again[1][i], out[i])
    assert again[1][2].isnan().any() and again[0][3].isnan().all() and again[1][3].isnan().all()


def test_norms_with_no_tokens_and_on_another_stream():
    w = torch.ones(128, device=DEV)
    assert kda.norm_gate(torch.zeros(0, 2, 128, device=DEV), torch.zeros(0, 2, 128, device=DEV), w).shape == (0, 2, 128)
    assert kda.residual_norm(torch.zeros(0, 128, device=DEV), torch.zeros(0, 128, device=DEV), w)[1].shape == (0, 128)
    o, z = normal(14, 50, 4, 128).bfloat16(), normal(15, 50, 4, 128).bfloat16()
    want = kda.norm_gate(o, z, w)
    out, side = torch.zeros_like(want), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kda.norm_gate(o, z, w, out=out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)


def test_norms_refuse():
    o, w = normal(16, 4, 2, 64), torch.ones(64, device=DEV)
    with pytest.raises(ValueError, match="shape"):
        kda.norm_gate(o, o[:3], w)
    with pytest.raises(ValueError, match="w "):
        kda.norm_gate(o, o, torch.ones(3, 64, device=DEV))
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        kda.norm_gate(o.half(), o, w)
    with pytest.raises(kda.KDAError, match="UNSUPPORTED"):
        kda.norm_gate(o[..., :20].contiguous(), o[..., :20].contiguous(), torch.ones(20, device=DEV))
    with pytest.raises(kda.KDAError, match="INVALID"):
        kda.norm_gate(o, o, w, eps=0.0)
    x = normal(17, 4, 64)
    with pytest.raises(ValueError, match="pass y"):
        kda.residual_norm(x, None, w, z=x)
    with pytest.raises(ValueError, match="shape"):
        kda.residual_norm(x, x[:2], w)
    with pytest.raises(ValueError, match="of its type"):
        kda.residual_norm(x, x, w, out_dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="float32"):
        kda.residual_norm(x, x, w.bfloat16())
