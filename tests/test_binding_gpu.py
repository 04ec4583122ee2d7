"""The binding under another name than the one that it is developed with (a copy inside
another package): its errors are its own MalaError."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import importlib.util, os, sys
spec = importlib.util.spec_from_file_location("elsewhere", os.path.join({root!r}, "mass_gated_causal_b200", "__init__.py"))
lib = importlib.util.module_from_spec(spec)
sys.modules["elsewhere"] = lib
spec.loader.exec_module(lib)
import torch
m = torch.rand(1, 2, 100, device="cuda")
n = torch.ones(1, dtype=torch.int32, device="cuda")
try:
    lib.evict_select(m, n, 5, n_sink=6)
except lib.MalaError as e:
    assert e.code == lib.MALA_ERR_INVALID_ARG, e
    assert "mass_gated_causal_b200" not in sys.modules
    print("ok")
"""


def test_errors_of_a_package_of_another_name(cuda_lib):
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(root=ROOT)], cwd="/", capture_output=True, text=True,
                       timeout=300, env={k: v for k, v in os.environ.items() if k != "PYTHONPATH"})
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
