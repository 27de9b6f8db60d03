"""The FP8 modules' buffers under conversions and moves (no GPU)."""
import copy

import pytest
import torch

import int8_quantized_linear_i8lt_gb300 as I
from int8_quantized_linear_i8lt_gb300.build import build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def layers():
    g = torch.Generator().manual_seed(1)
    for layer in (I.LinearFP8(300, 200), I.LinearFP8(17, 5, bias=False), I.ExpertsFP8(3, 130, 40)):
        layer.codes.view(torch.uint8).copy_(torch.randint(0, 120, layer.codes.shape, generator=g))
        layer.scales.copy_(torch.rand(layer.scales.shape, generator=g))
        yield layer


CONVERSIONS = [lambda m: m.half(), lambda m: m.bfloat16(), lambda m: m.double(), lambda m: m.float(),
               lambda m: m.to(torch.bfloat16), lambda m: m.to("cpu", torch.float16), lambda m: m.to(torch.ones(1).half()),
               lambda m: m.cpu(), lambda m: m.share_memory(), copy.deepcopy]


@pytest.mark.parametrize("convert", range(len(CONVERSIONS)))
def test_codes_and_scales_keep_their_types_and_values(convert):
    for layer in layers():
        codes, scales = layer.codes.view(torch.uint8).clone(), layer.scales.clone()
        model = torch.nn.Sequential(torch.nn.Linear(4, 4), torch.nn.ModuleDict({"inner": layer}))
        model = CONVERSIONS[convert](model)
        got = model[1]["inner"]
        assert got.codes.dtype == torch.float8_e4m3fn and got.scales.dtype == torch.float32
        assert torch.equal(got.codes.view(torch.uint8), codes) and torch.equal(got.scales, scales)
        assert dict(got.named_buffers()).keys() == {"codes", "scales"}
        if getattr(got, "bias", None) is not None and convert in (0, 5, 6):
            assert got.bias.dtype == torch.float16 and model[0].weight.dtype == torch.float16
        state = got.state_dict()
        assert state["codes"].dtype == torch.float8_e4m3fn and state["scales"].dtype == torch.float32


def test_moves_without_values():
    for layer in layers():
        shapes = layer.codes.shape, layer.scales.shape
        meta = copy.deepcopy(layer).to("meta")
        back = copy.deepcopy(meta).to_empty(device="cpu")
        for m in (meta, back):
            assert (m.codes.shape, m.scales.shape) == shapes
            assert m.codes.dtype == torch.float8_e4m3fn and m.scales.dtype == torch.float32
        assert meta.codes.is_meta and not back.codes.is_meta
        back.load_state_dict(layer.state_dict())
        assert torch.equal(back.codes.view(torch.uint8), layer.codes.view(torch.uint8))


def test_a_move_that_fails_leaves_the_layer_as_it_was():
    for layer in layers():
        with pytest.raises(ZeroDivisionError):
            layer._apply(lambda t: 1 // 0)
        assert layer.codes.dtype == torch.float8_e4m3fn and layer.scales.dtype == torch.float32
