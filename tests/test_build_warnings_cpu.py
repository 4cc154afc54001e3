"""build(): what the compiler warns of (spilled registers among it) is shown, and nothing else unless asked for."""
import os
import stat

import pytest

from kimi_delta_attention_13_gb300 import build as kbuild

NVCC = """#!/bin/sh
out=; say=
for a in "$@"; do
  [ "$last" = -o ] && out=$a
  case "$a" in *.cu) say=1;; esac
  last=$a
done
if [ -n "$say" ]; then
  echo "ptxas info    : Used 80 registers" >&2
  echo "ptxas warning : Registers are spilled to local memory in function 'f', 360 bytes spill stores" >&2
fi
: > "$out"
"""


@pytest.mark.parametrize("verbose", [False, True])
def test_warnings_are_shown(tmp_path, monkeypatch, capfd, verbose):
    cc = tmp_path / "nvcc"
    cc.write_text(NVCC)
    os.chmod(cc, cc.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setattr(kbuild, "nvcc", lambda: str(cc))
    monkeypatch.setattr(kbuild, "BUILD_DIR", str(tmp_path / "build"))
    monkeypatch.setattr(kbuild, "LIB_PATH", str(tmp_path / "build" / "lib.so"))
    assert kbuild.build(force=True, verbose=verbose) == str(tmp_path / "build" / "lib.so")
    out, err = capfd.readouterr()
    said = out + err
    assert said.count("360 bytes spill stores") == len(kbuild.sources())
    assert said.count("Used 80 registers") == (len(kbuild.sources()) if verbose else 0)
