"""The binding can be imported where torch has none of the CUDA build's own functions."""
import subprocess
import sys

from conftest import ROOT

WITHOUT = """
import torch
del torch._C._cuda_getCurrentRawStream
from sparse_top_landmark_gb300 import mita
assert "mita_forward" in mita.declared_functions()
print("fine")
"""


def test_import_without_cuda():
    r = subprocess.run([sys.executable, "-c", WITHOUT], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout + r.stderr
