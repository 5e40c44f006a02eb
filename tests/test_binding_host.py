"""The extension that calls the large products: the package without it, and what it was built for (no GPU needed)."""
import os
import shutil
import subprocess
import sys

import pytest

from segmented_gather_gemm_expand_b200 import _abi, build

PACKAGE = os.path.dirname(os.path.abspath(_abi.__file__))

WITHOUT = """
import torch
import segmented_gather_gemm_expand_b200 as sg
x, w, m = torch.zeros(4, 8), torch.zeros(2, 8, 8), [torch.zeros(2, dtype=torch.int32)] * 3
try:
    sg.sgmv_expand(x, w, x, *m, 2, 4)
except ValueError as e:
    print("expand:", e)
for call in (lambda: sg.sgmv_grouped_gemm(x, w, x, *m, 2, 4), lambda: sg.sgmv_grouped_wgrad(x, x, w, *m, 2, 4),
             lambda: sg.sgmv_lora_linear(x, w[0], w, w, x, *m, 2, 4)):
    try:
        call()
    except ImportError as e:
        print("large:", e)
"""


def test_the_other_calls_do_without_the_extension(tmp_path):
    here = tmp_path / "segmented_gather_gemm_expand_b200"
    here.mkdir()
    for name in os.listdir(PACKAGE):
        if name.endswith(".py") or name == "libsgmv.so":
            shutil.copy(os.path.join(PACKAGE, name), here / name)
    r = subprocess.run([sys.executable, "-c", WITHOUT], cwd=tmp_path, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    lines = r.stdout.splitlines()
    assert lines[0].startswith("expand:") and len(lines) == 4 and all(v.startswith("large: _binding.so not found") for v in lines[1:])


def test_the_extension_is_for_this_python_and_torch(monkeypatch):
    binding = _abi.load_binding(_abi.load())
    assert binding.built_for == build.binding_target() and build.binding_is_current()
    monkeypatch.setattr(build, "binding_target", lambda: "python 3.99, torch 9.9")
    assert not build.binding_is_current()          # the next build compiles it again
    with pytest.raises(ImportError, match="was built for python 3"):
        _abi.load_binding(_abi.load())
