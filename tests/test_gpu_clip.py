"""Clipping by the global norm against 64 bits.

The squares and their sums are float64: the norm is off by its rounding to float32 (2^-24 of itself) and a few steps
of float64. A clipped value is the product with a factor that is rounded to float32: off by 2 x 2^-24 of itself, and
the half step of its type.
"""
import math

import pytest
import torch

from differentiable_gaussian_splat_amd import labels as L
from differentiable_gaussian_splat_amd import optim as O
from differentiable_gaussian_splat_amd import raster

from .test_gpu_labels import BF16, DEV, F32, U, gen, half_step, within

pytestmark = pytest.mark.gpu


def tensors(g, sizes, kinds, offset=0, size=1.0):
    """Gradients of the given sizes, as slices of larger buffers that start `offset` elements in."""
    return [(torch.randn(k + offset, generator=g, device=DEV) * size).to(t)[offset:] for k, t in zip(sizes, kinds)]


def expected(grads, max_norm):
    norm = math.sqrt(math.fsum(float(t.double().square().sum()) for t in grads))
    return norm, 1.0 if math.isinf(max_norm) else min(1.0, max_norm / (norm + 1e-6))


def check(grads, max_norm, in_place=False):
    norm, c = expected(grads, max_norm)
    kept = [t.clone() for t in grads]
    outs = grads if in_place else [torch.full_like(t, float("nan")) for t in grads]
    got = O.GradClip(grads, None if in_place else outs)(max_norm)
    assert abs(float(got) - norm) <= norm * (U + 1e-14) + 1e-45
    for i, (before, o) in enumerate(zip(kept, outs)):
        ref = before.double() * c
        within(f"out {i}", o, ref, ref.abs() * (2 * U + half_step(o.dtype)) + (0 if c == 1 else 1e-40))
        if c == 1.0:
            assert torch.equal(o, before)
        if not in_place:
            assert torch.equal(grads[i], before)


KINDS = {"f32": [F32], "bf16": [BF16], "both": [F32, BF16]}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("sizes", [[1], [0, 1, 0], [3, 5], [8191, 8192, 8193, 16_383, 16_384, 16_385], [113_280],
                                   [1000] * 96, [777] * 97, [7] * 64, [130] * 64, [5] * 65, [16_384, 1],
                                   [40_000] * 160, [99] * 161, [20_000, 1] * 170, [33, 0] * 150, [5_000_001, 3, 70_000]],
                         ids=lambda s: f"{len(s)}x{max(s)}")
def test_clip(sizes, kind):
    kinds = [KINDS[kind][i % len(KINDS[kind])] for i in range(len(sizes))]
    g = gen(sum(sizes))
    for offset, ratio, in_place in ((0, 0.25, False), (3, 0.25, True), (1, 4.0, False), (0, 4.0, True)):
        ts = tensors(g, sizes, kinds, offset)
        check(ts, ratio * math.sqrt(sum(sizes)), in_place)


def test_norm_alone_and_no_tensors():
    g = gen(2)
    ts = tensors(g, [1000, 77], [F32, BF16])
    kept = [t.clone() for t in ts]
    norm = torch.full((1,), float("nan"), device=DEV)
    ws = torch.full((O.gs_clip_grads_workspace_size(2),), 0xFF, dtype=torch.uint8, device=DEV)
    O.gs_clip_grads(ts, None, norm, 0.1, ws)
    assert abs(float(norm) - expected(ts, 1)[0]) <= float(norm) * U * 2
    assert all(torch.equal(a, b) for a, b in zip(ts, kept))
    O.gs_clip_grads([], [], norm, 0.1, ws)
    assert float(norm) == 0
    check(ts, float("inf"))
    check(ts, 0.0)


def test_magnitudes_that_float32_squares_lose():
    g = gen(3)
    check(tensors(g, [5000, 300], [F32, F32], size=1e30), 1.0)
    check(tensors(g, [5000, 300], [F32, F32], size=1e-30), 1.0)
    # the factor, 1e-6 or less of the norm's, would be a subnormal number: none here
    check(tensors(g, [5000, 300], [F32, BF16], size=1e-3), 1e-5)


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_not_finite(value):
    g = gen(4)
    ts = tensors(g, [500, 40_000], [F32, BF16])
    ts[1][39_000] = value
    norm = O.GradClip(ts)(1.0)
    assert float(norm) == value or math.isnan(value) and math.isnan(float(norm))
    if math.isnan(value):
        assert all(t.isnan().all() for t in ts)
    else:
        assert (ts[0] == 0).all() and ts[1][39_000].isnan() and int(ts[1].isnan().sum()) == 1
        assert float(ts[1].nan_to_num().abs().sum()) == 0


def test_past_32_bits():
    """A tensor of more than 2^32 bytes and 2^31 elements."""
    n = (1 << 31) + 12_345
    g = torch.full((n,), 0.5, dtype=BF16, device=DEV)
    g[-3:] = 64.0
    norm = math.sqrt(0.25 * (n - 3) + 3 * 4096)
    got = O.GradClip([g])(norm / 2)
    assert abs(float(got) - norm) <= norm * 2 * U
    assert (g[-3:] == 32).all() and (g[:5] == 0.25).all() and (g[n // 2:n // 2 + 100_000] == 0.25).all()
    assert (g[:-3].view(torch.int16) == g[0].view(torch.int16)).all()


def test_neighbours_stay():
    buf = torch.full((50_000,), 2.0, device=DEV)
    O.GradClip([buf[101:33_001], buf[40_000:40_001]])(1.0)
    inside = torch.zeros(50_000, dtype=torch.bool, device=DEV)
    inside[101:33_001] = True
    inside[40_000] = True
    assert (buf[~inside] == 2).all() and (buf[inside] < 0.02).all()


def test_refuses_what_does_not_match():
    a, b = torch.ones(5, device=DEV), torch.ones(6, device=DEV)
    with pytest.raises(ValueError):
        O.GradClip([a], [b])
    with pytest.raises(ValueError):
        O.GradClip([a, b], [a])
    with pytest.raises(ValueError):
        O.GradClip([a], [torch.ones(10, device=DEV)[::2]])
    with pytest.raises(ValueError):
        O.GradClip([torch.ones((4, 4), device=DEV)[:, :2]])
    with pytest.raises(ValueError):
        O.GradClip([torch.ones((1, 4), device=DEV).expand(4, 4)])
    with pytest.raises(ValueError):
        O.GradClip([a, a])  # would be clipped twice
    with pytest.raises(ValueError):
        O.GradClip([torch.ones((3, 4), device=DEV)], [torch.ones((4, 3), device=DEV).t()])
    with pytest.raises(raster.GsError):
        O.GradClip([a])(-1.0)


def test_any_order_of_dimensions_and_shared_parameters():
    """Gradients follow their parameters' strides; a parameter that two modules share counts once."""
    g = gen(7)
    w = torch.nn.Parameter(torch.randn((30, 50), generator=g, device=DEV).t())
    v = torch.nn.Parameter(torch.randn(7, generator=g, device=DEV))
    w.grad = torch.randn((30, 50), generator=g, device=DEV).t()
    v.grad = torch.randn(7, generator=g, device=DEV)
    before = w.grad.clone()
    norm, c = expected([w.grad, v.grad], 3.0)
    assert not w.grad.is_contiguous()
    got = O.clip_grads([w, v, w], 3.0)
    assert abs(float(got) - norm) <= norm * U * 2
    within("grad", w.grad, before.double() * c, before.double().abs() * 3 * U)


def test_same_results_every_time_and_on_a_side_stream():
    g = gen(5)
    ts = tensors(g, [300_000, 41, 1_000_000], [F32, BF16, BF16])
    outs = [[torch.empty_like(t) for t in ts] for _ in range(3)]
    norms = [O.GradClip(ts, o)(10.0).clone() for o in outs[:2]]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        norms.append(O.GradClip(ts, outs[2])(10.0))
    s.synchronize()
    for k in (1, 2):
        assert torch.equal(norms[0], norms[k]) and all(torch.equal(a, b) for a, b in zip(outs[0], outs[k]))


@pytest.mark.parametrize("count", [3, 200])
def test_captured_clip_replays(count):
    g = gen(6)
    ts = tensors(g, [5000] * count, [F32, BF16] * count)
    clip = O.GradClip(ts, [torch.empty_like(t) for t in ts])
    eager = O.GradClip(ts, [torch.empty_like(t) for t in ts])
    graph = torch.cuda.CUDAGraph()
    clip(1.0)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        clip(1.0)
    for k in range(4):
        for t in ts:
            t.copy_(torch.randn(t.shape, generator=g, device=DEV) * (10.0 ** -k))
        want = eager(1.0).clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(clip.norm, want)
        assert all(torch.equal(a, b) for a, b in zip(clip._t.outs, eager._t.outs))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_label_head_and_scene_clipped(dtype):
    """A step of a residual label head's parameters, and a scene's five gradients, as they are clipped in training."""
    torch.manual_seed(1)
    head = L.ResidualLabelHead([50, 20], 32, 30, dtype=dtype)
    codes = torch.stack([torch.randint(0, k, (900,), device=DEV) for k in (50, 20)])
    head(codes, torch.randint(-1, 30, (900,), device=DEV)).backward()
    params = list(head.parameters())
    kept = [p.grad.clone() for p in params]
    norm, c = expected(kept, 1e-2)
    got = O.clip_grads(params, 1e-2)
    assert abs(float(got) - norm) <= norm * U * 2 and c < 1
    for p, k in zip(params, kept):
        ref = k.double() * c
        within("grad", p.grad, ref, ref.abs() * (2 * U + half_step(dtype)))
    means, sh = torch.zeros((1000, 3), device=DEV), torch.zeros((1000, 16, 3), device=DEV)
    grads = raster.zero_grads(means, sh)
    for v in grads.values():
        v.normal_()
    check(list(grads.values()), 5.0, in_place=True)


def test_captured_training_step_replays():
    """Forward, backward and clipping of a residual head recorded into a graph: replayed on changed inputs, against the
    same step run eagerly on a copy of the head."""
    torch.manual_seed(2)
    heads = [L.ResidualLabelHead([50, 20], 32, 30) for _ in range(2)]
    heads[1].load_state_dict(heads[0].state_dict())
    codes = torch.stack([torch.randint(0, k, (900,), device=DEV) for k in (50, 20)])
    labels = torch.randint(-1, 30, (900,), device=DEV)
    for head in heads:
        for p in head.parameters():
            p.grad = torch.zeros_like(p)
    clips = [O.GradClip([p.grad for p in head.parameters()]) for head in heads]

    def step(k):
        for p in heads[k].parameters():
            p.grad.zero_()
        loss = heads[k](codes, labels)
        loss.backward()
        clips[k](1e-2)
        return loss.detach()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(0)  # no eager graph of this head's parameters lives on when the step is recorded
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = step(0)
    for k in range(4):
        codes.copy_(torch.stack([torch.randint(0, c, (900,), device=DEV) for c in (50, 20)]))
        labels.copy_(torch.randint(-1, 30, (900,), device=DEV))
        want = step(1).clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, want) and torch.equal(clips[0].norm, clips[1].norm)
        for a, b in zip(heads[0].parameters(), heads[1].parameters()):
            assert torch.equal(a.grad, b.grad)
