"""kda_norm_gate and kda_residual_norm at sizes that take their kernels for many rows, with rows that do
not fill the last block, and past 2^31 elements.  References and bounds as in test_gpu_norms.py.
"""
import pytest
import torch

import kimi_delta_attention_13_gb300 as kda
from test_gpu_norms import EPS, TYPES, close, gate_ref, normal, residual_ref, share

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    yield
    torch.cuda.empty_cache()


# Rows a thread group takes four at a time from 152 x 32 blocks' worth on: 4 x 32, 16 or 8 rows a block
# for up to 64, 128 or 256 channels.
MANY = {64: 152 * 32 * 128, 128: 152 * 32 * 64, 256: 152 * 32 * 32}


@pytest.mark.parametrize("types", [("bf16", "bf16", "bf16"), ("f32", "bf16", "f32"), ("f32", "f32", "bf16")], ids="-".join)
@pytest.mark.parametrize("d,H,per_head", [(8, 3, True), (64, 1, False), (72, 3, True), (128, 2, True), (128, 1, False),
                                          (200, 3, False), (256, 5, True)])
def test_norm_gate_many_rows(d, H, per_head, types):
    to, tz, ty = (TYPES[t] for t in types)
    many = MANY[64 if d <= 64 else 128 if d <= 128 else 256]
    for T in (-(-many // H) - 1, -(-many // H) + 7):    # one token short of the rule, and past it
        o, z = normal(1, T, H, d).to(to), (3 * normal(2, T, H, d)).to(tz)
        w = 1 + 0.2 * (normal(3, H, d) if per_head else normal(3, d))
        out = kda.norm_gate(o, z, w, eps=EPS, out_dtype=ty)
        want = gate_ref(o, z, w)
        close(out, want, share(d, z.double()) * want.abs())


@pytest.mark.parametrize("over", ["o", "z"])
@pytest.mark.parametrize("d", [72, 256])
def test_norm_gate_many_rows_in_place(d, over):
    T = MANY[128 if d <= 128 else 256] // 2 + 5
    o, z, w = normal(4, T, 2, d).bfloat16(), normal(5, T, 2, d).bfloat16(), normal(6, 2, d)
    want = kda.norm_gate(o, z, w)
    into = o if over == "o" else z
    assert kda.norm_gate(o, z, w, out=into) is into and torch.equal(into, want)


def test_norm_gate_past_32_bits():
    T, H, d = 180_001, 96, 128
    gen = torch.Generator(device=DEV).manual_seed(7)
    o, z = (torch.randn(T, H, d, generator=gen, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    assert o.numel() > 2 ** 31
    w = 1 + 0.2 * normal(8, H, d)
    out = kda.norm_gate(o, z, w, eps=EPS)
    for at in (slice(0, 50), slice(174_700, 174_800), slice(T - 50, T)):   # 2^31 elements lie at token 174,762
        want = gate_ref(o[at], z[at], w)
        close(out[at], want, share(d, z[at].double()) * want.abs())


@pytest.mark.parametrize("T,D", [(180_001, 12_288), (2_150_001, 1001)])
def test_residual_norm_past_32_bits(T, D):
    gen = torch.Generator(device=DEV).manual_seed(9)
    x, y, z = (torch.randn(T, D, generator=gen, device=DEV, dtype=torch.bfloat16) for _ in range(3))
    assert x.numel() > 2 ** 31
    w = 1 + 0.1 * normal(10, D)
    res, out = kda.residual_norm(x, y, w, w_post=w, z=z, scale=-0.7, eps=EPS)
    border = 2 ** 31 // D
    for at in (slice(0, 20), slice(border - 20, border + 20), slice(T - 20, T)):
        r, n, mag = residual_ref(x[at], y[at], z[at], w, w, -0.7)
        part = share(D, z[at].double()) * mag + 2.0 ** -24 * r.abs()
        close(res[at], r, part)
        rms = (r.square().mean(-1, keepdim=True) + EPS).sqrt()
        close(out[at], n, w.double().abs() / rms * part
              + n.abs() * (share(D) + part.square().mean(-1, keepdim=True).sqrt() / rms))
