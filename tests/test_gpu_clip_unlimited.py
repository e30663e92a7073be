"""Clipping with an infinite max_norm: the norm, and every gradient as it is, whatever the norm."""
import math

import pytest
import torch

from differentiable_gaussian_splat_amd import optim as O

from .test_gpu_clip import tensors
from .test_gpu_labels import BF16, F32, gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [False, True], ids=["out", "in place"])
@pytest.mark.parametrize("sizes", [[50, 300], [500, 40_000], [1000] * 200], ids=["small", "two", "many"])
@pytest.mark.parametrize("value", [float("inf"), float("nan"), 1e38])
def test_nothing_is_clipped(value, sizes, in_place):
    g = gen(len(sizes))
    ts = tensors(g, sizes, [F32, BF16] * 100)
    ts[1][sizes[1] - 7] = value
    ts[0][3] = -value
    kept = [t.clone() for t in ts]
    outs = None if in_place else [torch.zeros_like(t) for t in ts]
    norm = float(O.GradClip(ts, outs)(math.inf))
    assert math.isnan(norm) if math.isnan(value) else norm >= 1e38
    for before, after in zip(kept, ts if in_place else outs):
        assert ((after == before) | (after.isnan() & before.isnan())).all()
