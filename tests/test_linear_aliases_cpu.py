"""The linear-attention and norm calls refuse outputs that share an address with what they read or with
each other, without a GPU: made-up addresses, in a process that sees none."""
import json
import os
import subprocess
import sys

from test_linear_cpu import A, DECODE, PREFILL, RESIDUAL, ROOT

WS = dict(ws=A + 65536, wsb=1 << 40)
INIT, FIN, CU = A + (1 << 30), A + (1 << 31), A + (1 << 32)
CASES = [("kda_linear_prefill", dict(PREFILL, **WS, init=INIT, fin=FIN, cu=CU), over) for over in [
    dict(out=INIT), dict(out=FIN), dict(out=WS["ws"]), dict(out=CU), dict(out=A + 16),
    dict(fin=A), dict(fin=A + 16), dict(fin=A + 32), dict(fin=A + 48), dict(fin=WS["ws"]), dict(fin=CU),
    dict(ws=A), dict(ws=A + 48), dict(ws=INIT), dict(ws=CU),
]] + [("kda_linear_decode", DECODE, over) for over in [
    dict(state=A), dict(state=A + 16), dict(state=A + 32), dict(state=A + 48),
]] + [("kda_residual_norm", RESIDUAL, over) for over in [
    dict(res=A + 48), dict(res=A + 64), dict(out=A + 48), dict(out=A + 64),
]]


def test_shared_addresses_are_refused():
    script = ("import json, sys\nfrom kimi_delta_attention_13_gb300 import _lib, build\nbuild.build()\nlib = _lib.load()\n"
              "for name, args in json.load(sys.stdin):\n    print(getattr(lib, name)(*args))\n")
    calls = [(name, list(dict(base, **over).values())) for name, base, over in CASES]
    r = subprocess.run([sys.executable, "-c", script], cwd=ROOT, env=dict(os.environ, CUDA_VISIBLE_DEVICES=""),
                       input=json.dumps(calls), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr
    got = [int(x) for x in r.stdout.split()]
    bad = [(name, over, rc) for (name, _, over), rc in zip(CASES, got) if rc != 1]   # KDA_ERR_INVALID_ARG
    assert len(got) == len(CASES) and not bad, bad
