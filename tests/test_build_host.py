"""The layer is built and called where the compiled marshalling of the newer calls cannot be (no GPU)."""
import os
import subprocess
import sys

import pytest

from moe_expert_layer_permute_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = r"""
import os, sys
from moe_expert_layer_permute_gb300 import build
if sys.argv[1] == "missing":
    build.MARSHAL = os.path.join(build.OUT_DIR, "not_there.so")
else:
    build.MARSHAL = sys.argv[1]
from moe_expert_layer_permute_gb300 import binding as bd
assert bd.moe_scratch_bytes(bd.make_desc(64, 256, 128, 8, 2)) > 0
assert bd.moe_balance_workspace_bytes(64, 8) > 0
import torch
t = torch.zeros(1, 4, 4)
class Holder: address = 0
for call in (lambda: bd.moe_orthogonalise(t, t, Holder, stream=0), lambda: bd.moe_balance_fwd(t, t, t, t, t, Holder, stream=0),
             lambda: bd.moe_balance_bwd(t, t, None, None, t, t, t, t, stream=0)):
    try:
        call()
    except (RuntimeError, ImportError) as e:
        assert not isinstance(e, bd.MoeError), e
    else:
        raise AssertionError("no error")
"""


@pytest.mark.parametrize("kind", ["missing", "broken"])
def test_the_layer_needs_no_marshalling(tmp_path, kind):
    build.build()
    at = "missing"
    if kind == "broken":                         # such as one of another torch
        at = str(tmp_path / "_marshal.so")
        with open(at, "wb") as f:
            f.write(b"no library")
    r = subprocess.run([sys.executable, "-c", SCRIPT, at], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("error", [RuntimeError("no Python.h"), FileNotFoundError("g++"), ImportError("torch")])
def test_the_library_is_built_without_the_marshalling(monkeypatch, error):
    build.build()

    def fail():
        raise error
    monkeypatch.setattr(build, "_marshal_flags", fail)
    with pytest.warns(UserWarning, match="cannot be called"):
        assert os.path.exists(build.build())
