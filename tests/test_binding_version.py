"""The C++ binding of the small operators uses torch's inline tensor members: it is loaded only by the torch and Python
that it was built for."""
import os
import subprocess
import sys
import sysconfig

import torch

from prefix_shared_kv_ra_gb300 import _build

CALL = """
import torch
{before}
import prefix_shared_kv_ra_gb300 as ra
t = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
try:
    ra.ra_kv8_store(torch.zeros(4, 4), t, t, None)
except (ImportError, TypeError) as e:
    print(type(e).__name__, e)
"""


def call(before):
    r = subprocess.run([sys.executable, "-c", CALL.format(before=before)], cwd=_build.ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return r.stdout


def test_the_file_names_its_torch_and_python():
    name = os.path.basename(_build.BINDING)
    assert torch.__version__ in name and sysconfig.get_config_var("SOABI") in name


def test_another_torch_does_not_load_it():
    _build.build()
    assert call("").startswith("TypeError")                  # loaded: the arguments are checked
    out = call("torch.__version__ = '0.0.1'")
    assert out.startswith("ImportError") and "torch0.0.1" in out and "build()" in out
