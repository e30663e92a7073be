"""A residual head at its edges: no rows, one row, a captured scoring; and gradients that share an input."""
import pytest
import torch

from differentiable_gaussian_splat_amd import labels as L
from differentiable_gaussian_splat_amd import optim as O

from .test_gpu_labels import BF16, DEV, F32, IDS, TYPES, gen, randn
from .test_gpu_residual import head_of

pytestmark = pytest.mark.gpu

SIZES = [60, 30, 20, 10]


def codes_of(g, n):
    return torch.stack([torch.randint(-1, k, (n,), generator=g, device=DEV) for k in SIZES])


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("stages", [1, 2, 3, 4])
def test_scores_of_some_rows_are_those_of_all(stages, dtype):
    """The same sums, rounded stage by stage, whatever the number of rows; none give no scores."""
    head = head_of(SIZES, 100, 90, dtype)
    whole, kept = codes_of(gen(stages), 700), head.vocabulary_q8()
    codes = whole[:stages]
    every = head.scores(codes, kept)
    assert head.scores(codes[:, :0], kept).shape == (0, 90)
    if dtype is F32:  # the features' values are those that the norm's kernel puts into 8 bits
        with torch.no_grad():
            rows = L.quantize_q8(head.features(whole)[stages - 1])
        assert torch.equal(L.label_scores(rows, kept), every)
    # another number of rows goes another way through the products: the order of float32 sums
    one = head.scores(codes[:, 5:6], kept)
    assert (one - every[5:6]).abs().max() <= 1e-5 * every.abs().max()


def test_captured_head_scores_replay():
    head = head_of(SIZES, 100, 90, BF16)
    g = gen(9)
    codes, kept = codes_of(g, 300), head.vocabulary_q8()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        head.scores(codes, kept)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = head.scores(codes, kept)
    for _ in range(4):
        codes.copy_(codes_of(g, 300))
        want = head.scores(codes, kept)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("use", ["y", "sum", "both"])
def test_the_two_inputs_gradients_are_tensors_of_their_own(use):
    """x and the residual have the same gradient, not the same memory: clipping it in place clips it once."""
    g = gen(10)
    x, r = (randn(g, 50, 40).clone().requires_grad_() for _ in range(2))
    y, h = L.rms_norm(x, None, r)
    up = randn(g, 50, 40)
    loss = (y * up).sum() * (use != "sum") + (h * up).sum() * (use != "y")
    loss.backward()
    assert torch.equal(x.grad, r.grad) and x.grad.data_ptr() != r.grad.data_ptr()
    before = x.grad.clone()
    norm = float(O.clip_grads([x, r], 1.0))
    assert torch.equal(x.grad, r.grad)
    assert (x.grad - before / norm).abs().max() <= 1e-6 * before.abs().max()


def test_an_input_that_is_its_own_residual():
    g = gen(11)
    x = randn(g, 50, 40).clone().requires_grad_()
    up = randn(g, 50, 40)
    y, h = L.rms_norm(x, None, x)
    ((y + 0.5 * h) * up).sum().backward()
    full = x.detach().double().requires_grad_()
    s = 2 * full
    ((s / (s.square().mean(1, keepdim=True) + 1e-6).sqrt() + 0.5 * s) * up.double()).sum().backward()
    assert float((x.grad.double() - full.grad).norm()) <= 1e-5 * float(full.grad.norm())
