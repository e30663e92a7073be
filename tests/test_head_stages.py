"""How a residual head's stages are added for its scores (no GPU): the kernels are stand-ins."""
import pytest
import torch

from differentiable_gaussian_splat_amd import labels as L


@pytest.mark.parametrize("stages", [1, 2, 3, 4])
def test_sums_come_from_the_norm_kernel(stages, monkeypatch):
    """Every addition is the kernel's, in the stages' order, and the last stage's sum, which nobody reads, is not
    written."""
    head = L.ResidualLabelHead([5] * 4, 8, 6, device="cpu")
    calls, adds = [], []

    class Adds(torch.utils._python_dispatch.TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            if "add" in func.__name__:
                adds.append(func)
            return func(*args, **(kwargs or {}))

    def norm(x, weight, q, scales, residual, total, eps):
        calls.append((weight, residual is not None, total is not None))
        if total is not None:
            total.numpy()[:] = x.numpy() + residual.numpy()
        q.view(torch.uint8).numpy()[:, 0] = len(calls)
        norm.sum = x.numpy() + (residual.numpy() if residual is not None else 0)

    monkeypatch.setattr(L, "embed", lambda table, ids, scale: (table * scale)[ids])
    monkeypatch.setattr(L, "gs_rms_norm_q8", norm)
    monkeypatch.setattr(L, "quantize_q8", lambda v: L.rows_q8(*v.shape, "cpu"))
    monkeypatch.setattr(L, "label_scores", lambda rows, words, dtype: rows[0].view(torch.uint8)[:, 0].clone())
    codes = torch.arange(stages * 3).reshape(stages, 3) % 5
    with Adds():
        out = head.scores(codes)
    assert not adds and (out == len(calls)).all()
    first = 0 if stages == 1 else 1
    assert [c[0].data_ptr() for c in calls] == [head.weights[k].data_ptr() for k in range(first, stages)]
    assert [c[1:] for c in calls] == [(k > 0, k < stages - 1) for k in range(first, stages)]
    want = sum(head.codebooks[k].detach()[codes[k]] * head.scales[k] for k in range(stages))
    assert (torch.from_numpy(norm.sum) - want).abs().max() <= 1e-5
