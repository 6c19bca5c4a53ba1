"""Importing the package asks nothing of the CUDA driver: a program may import
it, fork its workers or choose their devices, and use the GPU only then."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

IMPORTS = """
import torch

def asked(*args, **kw):
    raise AssertionError("the import asked the CUDA driver")

for module, names in ((torch._C, ("_cuda_getDeviceCount", "_cuda_getDevice", "_cuda_init",
                                  "_cuda_getCurrentRawStream")),
                      (torch.cuda, ("is_available", "device_count", "current_device", "_lazy_init",
                                    "get_device_properties"))):
    for name in names:
        if hasattr(module, name):
            setattr(module, name, asked)
from bit_group_quantized_flexq_b200 import build, flexq, inputs, stack
assert not torch.cuda.is_initialized()
print("imported")
"""


def test_imports_leave_the_driver_alone():
    r = subprocess.run([sys.executable, "-c", IMPORTS], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "imported" in r.stdout, r.stderr[-2000:]


FORKS = """
import multiprocessing as mp
from bit_group_quantized_flexq_b200 import flexq
import torch

def work(q):
    q.put(torch.cuda._is_in_bad_fork())

ctx = mp.get_context("fork")
q = ctx.Queue()
p = ctx.Process(target=work, args=(q,))
p.start()
print("bad fork:", q.get(timeout=60))
p.join()
"""


def test_a_forked_worker_may_still_use_cuda():
    r = subprocess.run([sys.executable, "-c", FORKS], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "bad fork: False" in r.stdout, r.stdout + r.stderr[-2000:]
