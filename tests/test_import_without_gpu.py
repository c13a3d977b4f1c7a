"""The binding imports on a build of torch without a GPU backend (CPU): the
names that such a build lacks are taken away in a process of their own."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CODE = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from int4_output_head_amd import binding
try:
    binding.rms_norm(torch.zeros(2, 64), torch.ones(64))
except TypeError as e:
    print("refused:", e)
import types
torch.cuda.current_stream = lambda d=None: types.SimpleNamespace(cuda_stream=1000 + d)
torch.cuda.current_device = lambda: 3
print(binding._raw_stream(2), binding._current_device())
"""


def test_import_and_refuse():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.splitlines() == ["refused: x must be a CUDA (HIP) tensor of float16, bfloat16 or float32", "1002 3"]
