"""Clipping on a stream beside the current one, against 64 bits (tolerances as in test_gpu_clip)."""
import math

import pytest
import torch

from differentiable_gaussian_splat_amd import optim as O

from .test_gpu_clip import expected, tensors
from .test_gpu_labels import BF16, DEV, F32, U, gen, half_step, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("count", [4, 300])
@pytest.mark.parametrize("handle", [False, True], ids=["call", "handle"])
def test_buffers_last_until_the_stream_is_through(count, handle):
    """The call returns long before its kernels run, behind other work of their stream; what is allocated on the current
    stream meanwhile, and written, is none of theirs."""
    g = gen(count)
    params = [torch.nn.Parameter(t) for t in tensors(g, [20_000] * count, [F32, BF16])]
    for p in params:
        p.grad = torch.randn(p.shape, generator=g, device=DEV).to(p.dtype)
    kept = [p.grad.clone() for p in params]
    norm, c = expected(kept, 1.0)
    a = torch.randn((4096, 4096), generator=g, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(20):
            a = a @ a * 1e-3
    if handle:
        got = O.GradClip([p.grad for p in params])(1.0, stream=side)
    else:
        got = O.clip_grads(params, 1.0, stream=side)
    size = O.gs_clip_grads_workspace_size(count)
    for k in (size, size, 4, 4, 512, 1 << 20):
        torch.full((k,), 0xFF, dtype=torch.uint8, device=DEV)
    torch.cuda.current_stream().wait_stream(side)
    assert abs(float(got) - norm) <= norm * 2 * U and not math.isnan(float(got))
    for p, k in zip(params, kept):
        ref = k.double() * c
        within("grad", p.grad, ref, ref.abs() * (2 * U + half_step(k.dtype)))
