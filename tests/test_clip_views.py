"""Which views ``scale_grads_`` takes for sharing memory, against the bytes
themselves (no GPU)."""
import random

import pytest
import torch

import int8_quantized_linear_i8lt_gb300.functional as F


def touched(t):
    """The offsets of t's elements in its storage, each of its bytes."""
    at = torch.zeros((), dtype=torch.int64) + t.storage_offset()
    for size, stride in zip(t.shape, t.stride()):
        at = at.unsqueeze(-1) + torch.arange(size) * stride
    e = t.element_size()
    return {i * e + k for i in at.flatten().tolist() for k in range(e)}


def refused(views):
    try:
        F._require_apart("views", views)
    except F.I8LTError:
        return True
    return False


def test_no_shared_byte_is_overlooked():
    rng = random.Random(1)
    base = torch.zeros(400, dtype=torch.uint8)
    found = 0
    for _ in range(4000):
        views = []
        for dtype in (rng.choice((torch.float16, torch.float32)), rng.choice((torch.float16, torch.float32))):
            f = base.view(dtype)
            dims = [(rng.randint(1, 4), rng.randint(1, 12)) for _ in range(rng.randint(1, 3))]
            span = sum((n - 1) * s for n, s in dims)
            if span < f.numel():
                views.append(f.as_strided([n for n, _ in dims], [s for _, s in dims], rng.randint(0, f.numel() - span - 1)))
        if len(views) == 2 and not all(v.is_contiguous() for v in views) and touched(views[0]) & touched(views[1]):
            found += 1
            assert refused(views) and refused(views[::-1]), [(v.shape, v.stride(), v.storage_offset()) for v in views]
    assert found > 500


@pytest.mark.parametrize("shape", [(6, 8), (6, 7), (4, 5, 6)])
def test_parts_of_one_tensor_are_told_apart(shape):
    m = torch.zeros(shape)
    for parts in (m.split(1, -1), m.split(2, -1), [m[..., ::2], m[..., 1::2]], [m[..., ::3], m[..., 1::3], m[..., 2::3]],
                  [m[::2], m[1::2, ..., :2], m[1::2, ..., 2:]], m.transpose(0, -1).unbind(0)):
        assert not refused(list(parts))
        assert refused(list(parts) + [m[..., :1, -1:]])
