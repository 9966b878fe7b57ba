"""The binding's shortcuts through torch's private names are not needed: without them it takes the public ones."""
import subprocess
import sys

import pytest

SCRIPT = """
import sys, types
import torch
import torch._C
for name in sys.argv[1].split(","):
    delattr(torch._C, name)
import filtered_int8_ann_b200 as st
torch.cuda.is_initialized = torch.cuda.is_available = lambda: True
torch.cuda.current_stream = lambda *a: types.SimpleNamespace(cuda_stream=77)
assert st._stream(None) == 77 and st._stream(5) == 5
"""


@pytest.mark.parametrize("names", ["_cuda_getCurrentRawStream", "_cuda_getDevice", "_cuda_getCurrentRawStream,_cuda_getDevice"])
def test_stream_without_private_names(names):
    import os
    root = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..")
    done = subprocess.run([sys.executable, "-c", SCRIPT, names], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]
