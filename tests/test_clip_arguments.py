"""What clip_grads takes as parameters (no GPU): the handle is a stand-in."""
import torch

from differentiable_gaussian_splat_amd import optim as O


def test_a_single_tensor_is_one_parameter(monkeypatch):
    """And not a sequence of its rows, which have no gradients of their own."""
    seen = []

    class Clip:
        def __init__(self, grads):
            seen.extend(grads)

        def __call__(self, max_norm):
            return max_norm

    monkeypatch.setattr(O, "GradClip", Clip)
    p = torch.nn.Parameter(torch.zeros(3, 4))
    assert O.clip_grads(p, 2.0) is None  # without a gradient
    p.grad = torch.ones(3, 4)
    assert O.clip_grads(p, 2.0) == 2.0
    assert len(seen) == 1 and seen[0] is p.grad
