"""The package imports, and answers its host-side queries, on a torch whose C layer has no CUDA."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CODE = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import nvfp4_block_scaled_bf16_gb300 as nv
assert nv.sf_bytes(128, 256) == 128 * 16
assert nv.nvfp4_gemm_plan(1, 4096, 7168)["ctas"] > 0
class Stream:
    cuda_stream = 7
torch.cuda.current_device = nv._current_device = lambda: 0
torch.cuda.current_stream = lambda device: Stream
assert nv._stream(None) == 7 and nv._stream(5) == 5 and nv._stream(Stream) == 7
"""


def test_without_the_private_functions():
    import __graft_entry__
    __graft_entry__.build()
    run = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True)
    assert run.returncode == 0, run.stderr
