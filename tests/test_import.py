"""The package on a PyTorch built without CUDA (no GPU): it can be imported, its
size functions answer, and its calls refuse host tensors."""
import subprocess
import sys

from int8_quantized_linear_i8lt_gb300.build import build

CODE = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_") or n.startswith("_Cuda")]:
    delattr(torch._C, name)
import int8_quantized_linear_i8lt_gb300 as I
from int8_quantized_linear_i8lt_gb300 import _lib
assert I.weight_ld(1000) >= 1000 and _lib.i8lt_fp8_ld(17) == 32
layer = I.LinearFP8(300, 200)
t = torch.ones(4, 300)
for call in (lambda: layer(t.half()), lambda: I.grad_norm([t]), lambda: I.scale_grads_([t], torch.ones(1)),
             lambda: I.fp8_quantize_weight(t), lambda: I.quantize_weight(t)):
    try:
        call()
    except I.I8LTError:
        continue
    raise SystemExit("a host tensor was taken")
print("done")
"""


def test_import_without_cuda_names():
    build()
    r = subprocess.run([sys.executable, "-c", CODE], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, r.stderr[-2000:]
