"""The binding can be imported, and looks its library up, under a torch that was built without CUDA."""
import subprocess
import sys

from conftest import ROOT

WITHOUT = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
from sparse_top_landmark_gb300 import mita
assert "mita_forward" in mita.declared_functions()
try:
    mita.mita_forward(*[torch.zeros(1, 1, 4, 16)] * 3, 1, 4, 2, 2)
except ValueError as e:
    assert "CUDA" in str(e)
    print("fine")
"""


def test_import_without_cuda():
    r = subprocess.run([sys.executable, "-c", WITHOUT], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout + r.stderr
