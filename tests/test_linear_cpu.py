"""Refusals of the linear-attention and norm calls, without a GPU: the library's host-side checks
on made-up addresses, in a process that sees no GPU, and the binding's on CPU tensors."""
import os
import subprocess
import sys

import pytest
import torch

import kimi_delta_attention_13_gb300 as kda
from kimi_delta_attention_13_gb300 import _lib, build

A = 1 << 20   # a 16-byte aligned address that nothing dereferences
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


PREFILL = dict(q=A, k=A + 16, v=A + 32, g=A + 48, pt=1, cu=None, n=1, T=64, H=4, Hkv=2, dk=128, dv=128,
               scale=1.0, dtype=0, odt=0, init=None, out=A + 4096, fin=None, ws=None, wsb=0, stream=None)
DECODE = dict(q=A, k=A + 16, v=A + 32, g=A + 48, pt=1, state=A + 64, out=A + 4096, n=2, H=4, Hkv=2, dk=128,
              dv=128, scale=1.0, dtype=0, odt=0, stream=None)
GATE = dict(o=A, odt=0, z=A + 16, zdt=0, w=A + 32, wh=1, out=A + 4096, outdt=0, T=8, H=4, d=128, eps=1e-6,
            stream=None)
RESIDUAL = dict(x=A, rdt=0, y=A + 16, z=A + 32, dtype=0, wp=A + 48, w=A + 64, scale=1.0, eps=1e-6,
                res=A + 4096, out=A + 8192, T=8, D=256, stream=None)
INF, NAN = float("inf"), float("nan")

CASES = [("kda_linear_prefill", PREFILL, over, code) for over, code in [
    (dict(H=0), 1), (dict(Hkv=0), 1), (dict(Hkv=3), 1), (dict(n=-1), 1), (dict(T=-1), 1), (dict(dtype=2), 1),
    (dict(odt=2), 1), (dict(scale=NAN), 1), (dict(scale=INF), 1), (dict(q=None), 1), (dict(k=None), 1),
    (dict(v=None), 1), (dict(g=None), 1), (dict(out=None), 1), (dict(n=0), 1), (dict(n=2), 1),
    (dict(T=1 << 31), 1), (dict(dk=0), 1), (dict(dk=4), 2), (dict(dk=132), 2), (dict(dk=264), 2),
    (dict(dv=12), 2), (dict(dv=512), 2), (dict(q=A + 8), 3), (dict(g=A + 4), 3), (dict(init=A + 4), 3),
    (dict(fin=A + 2), 3), (dict(ws=A + 4), 3), (dict(cu=A + 2), 3), (dict(out=A), 1), (dict(out=A + 48), 1),
    (dict(T=200000), 1),                                  # cut into segments: needs a workspace
    (dict(T=200000, ws=A + 65536, wsb=16), 1),            # ... of the size asked for
]] + [("kda_linear_decode", DECODE, over, code) for over, code in [
    (dict(H=0), 1), (dict(Hkv=3), 1), (dict(n=-1), 1), (dict(dtype=5), 1), (dict(odt=-1), 1),
    (dict(scale=NAN), 1), (dict(q=None), 1), (dict(g=None), 1), (dict(state=None), 1), (dict(out=None), 1),
    (dict(dk=12), 2), (dict(dv=264), 2), (dict(state=A + 68), 3), (dict(out=A + 64), 1), (dict(out=A), 1),
]] + [("kda_norm_gate", GATE, over, code) for over, code in [
    (dict(T=-1), 1), (dict(H=0), 1), (dict(wh=2), 1), (dict(odt=3), 1), (dict(zdt=3), 1), (dict(outdt=3), 1),
    (dict(eps=0.0), 1), (dict(eps=NAN), 1), (dict(eps=INF), 1), (dict(o=None), 1), (dict(w=None), 1),
    (dict(d=12), 2), (dict(d=264), 2), (dict(z=A + 24), 3), (dict(w=A + 36), 3), (dict(out=A, outdt=1), 1),
    (dict(out=A + 16, outdt=1), 1), (dict(out=A + 32), 1),
]] + [("kda_residual_norm", RESIDUAL, over, code) for over, code in [
    (dict(T=-1), 1), (dict(D=0), 1), (dict(rdt=2), 1), (dict(dtype=2), 1), (dict(scale=INF), 1),
    (dict(eps=0.0), 1), (dict(x=None), 1), (dict(w=None), 1), (dict(out=None), 1), (dict(res=None), 1),
    (dict(y=None), 1),                                    # z, w_post and res without y
    (dict(y=None, z=None, wp=None), 1), (dict(x=A + 8), 3), (dict(wp=A + 52), 3), (dict(out=A), 1),
    (dict(out=A + 4096), 1), (dict(res=A + 32), 1), (dict(res=A + 16, rdt=1), 1),
]]


def test_library_refuses(lib):
    """Every case in one child process without a GPU, so that no address can reach a device even if
    a check were lost (such a call would then return another code)."""
    script = ("import json, sys\nfrom kimi_delta_attention_13_gb300 import _lib\nlib = _lib.load()\n"
              "for name, args in json.load(sys.stdin):\n    print(getattr(lib, name)(*args))\n")
    import json

    calls = [(name, list(dict(base, **over).values())) for name, base, over, _ in CASES]
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-c", script], cwd=ROOT, env=env, input=json.dumps(calls),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    got = [int(x) for x in r.stdout.split()]
    bad = [(name, over, code, rc) for (name, _, over, code), rc in zip(CASES, got) if rc != code]
    assert len(got) == len(CASES) and not bad, bad


def test_workspace_sizes(lib):
    f = lib.kda_linear_prefill_workspace
    assert f(1, 64, 4, 128, 128, 0) == 0          # a short prompt is not cut
    assert f(2000, 2000, 32, 128, 128, 0) == 0    # many sequences fill the machine
    assert f(1, 200000, 4, 128, 128, 0) > 0
    assert f(-1, 64, 4, 128, 128, 0) == f(1, -1, 4, 128, 128, 0) == f(1, 64, 0, 128, 128, 0) == -1
    assert f(1, 64, 4, 12, 128, 0) == f(1, 64, 4, 128, 128, 7) == -1


def _cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refuses_cpu_tensors(lib):
    q, g = _cpu(4, 2, 64), _cpu(4, 2, dtype=torch.float32)
    with pytest.raises(ValueError, match="CUDA"):
        kda.linear_prefill(q, q, q, g)
    with pytest.raises(ValueError, match="CUDA"):
        kda.linear_decode(q, q, q, g, _cpu(4, 2, 64, 64, dtype=torch.float32))
    with pytest.raises(ValueError, match="CUDA"):
        kda.norm_gate(q, q, _cpu(64, dtype=torch.float32))
    with pytest.raises(ValueError, match="CUDA"):
        kda.residual_norm(_cpu(4, 64), _cpu(4, 64), _cpu(64, dtype=torch.float32))


def test_binding_refuses_head_counts_and_types(lib):
    q, g = _cpu(4, 3, 64), _cpu(4, 3, dtype=torch.float32)
    with pytest.raises(ValueError, match="share"):
        kda.linear_prefill(q, _cpu(4, 2, 64), _cpu(4, 2, 64), g)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        kda.linear_prefill(q.half(), q.half(), q.half(), g)
    with pytest.raises(ValueError, match=r"\[T, heads, d\]"):
        kda.linear_prefill(q[0], q[0], q[0], g)
