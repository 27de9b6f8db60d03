"""The block-scaled FP8 layers on a GB300 where they are easily wrong."""
import pytest
import torch

import _fp8 as R
import int8_quantized_linear_i8lt_gb300 as I
from int8_quantized_linear_i8lt_gb300 import _lib

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def normal(*shape, seed, dtype=F32, std=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


def test_layers_after_a_conversion():
    """A model's dtype is converted around its FP8 layers, which keep their results."""
    layer = I.LinearFP8.from_float(normal(200, 300, seed=1).cuda(), normal(200, seed=2, dtype=BF16).cuda())
    experts = I.ExpertsFP8.from_float(normal(2, 72, 200, seed=3).cuda())
    x = normal(20, 300, seed=4, dtype=BF16).cuda()
    off = torch.tensor([0, 9, 20], dtype=torch.int32, device="cuda")
    expect = experts(layer(x), off)
    for convert in (lambda m: m.bfloat16(), lambda m: m.half().bfloat16(), lambda m: m.to(F32).to("cuda", BF16),
                    lambda m: m.cpu().cuda()):
        model = convert(torch.nn.ModuleList([layer, experts]))
        assert torch.equal(model[1](model[0](x), off), expect)
