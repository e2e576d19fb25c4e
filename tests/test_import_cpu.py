"""The package imports on a torch that was built without CUDA: what is missing there is
refused by the calls that need it, not by the import."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Torch's names for the current device and its raw stream handle exist only in a build with
# CUDA; the child takes away every name of that kind before the package is imported.
CHILD = r"""
import torch

for name in [n for n in dir(torch._C) if n.startswith("_cuda_getDevice") or n.startswith("_cuda_getCurrent")]:
    delattr(torch._C, name)

import rmsnorm_fwd_bwd_03_gb300 as gb
import rmsnorm_fwd_bwd_03_gb300.autograd
from rmsnorm_fwd_bwd_03_gb300 import workload

assert workload.WORKLOADS
x = torch.zeros(4, 8)
for call in (lambda: gb.rmsnorm_fwd(x, torch.ones(8), 1e-5), lambda: gb.glu_fwd_fp8(x, x),
             lambda: gb.rmsnorm_fwd_ckpt8(x, torch.ones(8), 1e-5)):
    try:
        call()
    except ValueError as e:
        assert "CUDA" in str(e), e
    else:
        raise AssertionError("a CPU tensor was taken")
print("imported")
"""


def test_import_without_cuda_names():
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "imported", r.stderr[-2000:]


def test_the_public_functions_stand_in(monkeypatch):
    import torch

    import rmsnorm_fwd_bwd_03_gb300 as gb

    class Stream:
        cuda_stream = 1234

    seen = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: seen.append(d) or Stream)
    device, stream = gb._device_and_stream(object())  # an object without torch's private names
    assert device() == 3 and stream(2) == 1234 and seen == [2]
    device, stream = gb._device_and_stream(torch._C)
    if hasattr(torch._C, "_cuda_getDevice"):
        assert device is torch._C._cuda_getDevice and stream is torch._C._cuda_getCurrentRawStream
