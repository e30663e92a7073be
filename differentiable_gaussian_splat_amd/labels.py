"""Learning labels of a scene: feature codebook, layer normalisation, vocabulary loss.

A scene's Gaussians (or the pixels of a view) carry features that are scored
against a vocabulary of labels. Three operators do that, each with its
gradients, in float32 or bfloat16:

- :func:`embed` looks a feature codebook up by each Gaussian's code;
- :func:`layer_norm` normalises feature rows;
- :func:`label_loss` is the softmax cross entropy of feature rows against the
  vocabulary's rows; the logits are never stored.

The ``gs_*`` functions marshal tensors into the C calls of the same names
(``include/gsplat.h``) and leave buffers to the caller; the three functions
above are autograd wrappers that allocate them. An index outside the table
(use -1) marks a row without a code or label: it takes no part.
:class:`LabelHead` chains the three.
"""
from __future__ import annotations

import torch

from .raster import _check, _nbytes, _p, _stream, load_library

__all__ = ["gs_embed_fwd", "gs_embed_bwd_workspace_size", "gs_embed_bwd", "gs_layer_norm_fwd",
           "gs_layer_norm_bwd_workspace_size", "gs_layer_norm_bwd", "gs_label_loss_workspace_size",
           "gs_label_loss_fwd", "gs_label_loss_bwd", "embed", "layer_norm", "label_loss", "LabelHead"]

_DTYPES = {torch.float32: 0, torch.bfloat16: 1}
_INDEX_TYPES = {torch.int32: 0, torch.int64: 1}


# ------------------------------------------------------------------ argument checks

def _dtype(dtype) -> int:
    if dtype not in _DTYPES:
        raise TypeError(f"rows must be float32 or bfloat16, got {dtype}")
    return _DTYPES[dtype]


def _matrix(name, t, like=None, rows=None, cols=None):
    """Checks a matrix of rows and returns its row stride."""
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, got {t.dim()}")
    if (rows is not None and t.shape[0] != rows) or (cols is not None and t.shape[1] != cols):
        raise ValueError(f"{name} must have shape ({'*' if rows is None else rows}, {'*' if cols is None else cols}), "
                         f"got {tuple(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}'s columns must be consecutive, got strides {t.stride()}")
    _dtype(t.dtype)
    _same(name, t, like)
    # one row has no stride of its own; torch may give it any
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _same(name, t, like):
    if like is None and t.device.type != "cuda":
        raise TypeError(f"{name} must be on the GPU, got {t.device}")
    if like is not None and (t.dtype != like.dtype or t.device != like.device):
        raise TypeError(f"{name} must be {like.dtype} on {like.device}, got {t.dtype} on {t.device}")


def _vector(name, t, n, dtype, device):
    if t is None:
        return
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector of {n}, got shape {tuple(t.shape)}")
    if t.dtype != dtype or t.device != device:
        raise TypeError(f"{name} must be {dtype} on {device}, got {t.dtype} on {t.device}")


def _index(name, t, n, device) -> int:
    if t.dtype not in _INDEX_TYPES:
        raise TypeError(f"{name} must be int32 or int64, got {t.dtype}")
    _vector(name, t, n, t.dtype, device)
    return _INDEX_TYPES[t.dtype]


# ------------------------------------------------------------------ thin C-ABI wrappers

def gs_embed_fwd(table, ids, out, scale=1.0, stream=None):
    """out[i] = scale * table[ids[i]]; zero rows where ids[i] names no row."""
    vocab, dim = table.shape
    n = ids.shape[0]
    ts, os_ = _matrix("table", table), _matrix("out", out, table, n, dim)
    it = _index("ids", ids, n, table.device)
    st = load_library().gs_embed_fwd(n, dim, vocab, _dtype(table.dtype), _p(table), ts, _p(ids), it, float(scale),
                                     _p(out), os_, _stream(stream))
    _check(st, "gs_embed_fwd")


def gs_embed_bwd_workspace_size(n, dim, vocab, dtype) -> int:
    return int(load_library().gs_embed_bwd_workspace_size(n, dim, vocab, _dtype(dtype)))


def gs_embed_bwd(ids, dout, dtable, workspace, scale=1.0, stream=None):
    """dtable[v] = scale * sum of dout over the rows whose index is v (every row of dtable is written)."""
    n, dim = dout.shape
    ds, ts = _matrix("dout", dout), _matrix("dtable", dtable, dout, None, dim)
    it = _index("ids", ids, n, dout.device)
    st = load_library().gs_embed_bwd(n, dim, dtable.shape[0], _dtype(dout.dtype), _p(ids), it, float(scale), _p(dout),
                                     ds, _p(dtable), ts, _p(workspace), _nbytes(workspace), _stream(stream))
    _check(st, "gs_embed_bwd")


def gs_layer_norm_fwd(x, weight, bias, y, mean=None, rstd=None, eps=1e-5, stream=None):
    """y = (x - mean) * rstd * weight + bias per row; weight and bias may be None."""
    n, dim = x.shape
    xs, ys = _matrix("x", x), _matrix("y", y, x, n, dim)
    for name, t in (("weight", weight), ("bias", bias)):
        _vector(name, t, dim, x.dtype, x.device)
    for name, t in (("mean", mean), ("rstd", rstd)):
        _vector(name, t, n, torch.float32, x.device)
    st = load_library().gs_layer_norm_fwd(n, dim, _dtype(x.dtype), _p(x), xs, _p(weight), _p(bias), float(eps), _p(y),
                                          ys, _p(mean), _p(rstd), _stream(stream))
    _check(st, "gs_layer_norm_fwd")


def gs_layer_norm_bwd_workspace_size(n, dim, dtype) -> int:
    return int(load_library().gs_layer_norm_bwd_workspace_size(n, dim, _dtype(dtype)))


def gs_layer_norm_bwd(x, weight, mean, rstd, dy, dx, dweight, dbias, workspace, stream=None):
    """Gradients of gs_layer_norm_fwd into dx, dweight and dbias (each may be None)."""
    n, dim = x.shape
    xs, dys = _matrix("x", x), _matrix("dy", dy, x, n, dim)
    dxs = _matrix("dx", dx, x, n, dim) if dx is not None else dim
    for name, t in (("weight", weight), ("dweight", dweight), ("dbias", dbias)):
        _vector(name, t, dim, x.dtype, x.device)
    for name, t in (("mean", mean), ("rstd", rstd)):
        _vector(name, t, n, torch.float32, x.device)
    st = load_library().gs_layer_norm_bwd(n, dim, _dtype(x.dtype), _p(x), xs, _p(weight), _p(mean), _p(rstd), _p(dy),
                                          dys, _p(dx), dxs, _p(dweight), _p(dbias), _p(workspace),
                                          _nbytes(workspace), _stream(stream))
    _check(st, "gs_layer_norm_bwd")


def gs_label_loss_workspace_size(n, dim, vocab, dtype, backward) -> int:
    return int(load_library().gs_label_loss_workspace_size(n, dim, vocab, _dtype(dtype), 1 if backward else 0))


def gs_label_loss_fwd(x, w, labels, loss, lse, mean, count, workspace, stream=None):
    """Per row lse = log sum_v exp(x . w[v]) and loss = lse - x . w[label] (0 without a label); the mean loss and
    the number of labelled rows."""
    n, dim = x.shape
    xs, ws = _matrix("x", x), _matrix("w", w, x, None, dim)
    it = _index("labels", labels, n, x.device)
    for name, t, k, dt in (("loss", loss, n, torch.float32), ("lse", lse, n, torch.float32),
                           ("mean", mean, 1, torch.float32), ("count", count, 1, torch.int32)):
        _vector(name, t, k, dt, x.device)
    st = load_library().gs_label_loss_fwd(n, dim, w.shape[0], _dtype(x.dtype), _p(x), xs, _p(w), ws, _p(labels), it,
                                          _p(loss), _p(lse), _p(mean), _p(count), _p(workspace), _nbytes(workspace),
                                          _stream(stream))
    _check(st, "gs_label_loss_fwd")


def gs_label_loss_bwd(x, w, labels, lse, dx, dw, workspace, dmean=None, dloss=None, stream=None):
    """Gradients into dx and dw (each may be None) from the upstream gradients of the mean loss and of the rows'
    losses."""
    n, dim = x.shape
    xs, ws = _matrix("x", x), _matrix("w", w, x, None, dim)
    it = _index("labels", labels, n, x.device)
    for name, t, k in (("lse", lse, n), ("dmean", dmean, 1), ("dloss", dloss, n)):
        _vector(name, t, k, torch.float32, x.device)
    dxs = _matrix("dx", dx, x, n, dim) if dx is not None else dim
    dws = _matrix("dw", dw, w, w.shape[0], dim) if dw is not None else dim
    st = load_library().gs_label_loss_bwd(n, dim, w.shape[0], _dtype(x.dtype), _p(x), xs, _p(w), ws, _p(labels), it,
                                          _p(lse), _p(dmean), _p(dloss), _p(dx), dxs, _p(dw), dws, _p(workspace),
                                          _nbytes(workspace), _stream(stream))
    _check(st, "gs_label_loss_bwd")


# ------------------------------------------------------------------ autograd

def _rows(t):
    """t with consecutive columns and rows that do not overlap, or are one row for all."""
    if t.dim() != 2:
        raise ValueError(f"expected a matrix of rows, got {t.dim()} dimensions")
    ok = (t.shape[1] <= 1 or t.stride(1) == 1) and (t.shape[0] <= 1 or t.stride(0) == 0 or t.stride(0) >= t.shape[1])
    return t if ok else t.contiguous()


def _workspace(size, device):
    return torch.empty(size, dtype=torch.uint8, device=device)


class _EmbedFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, ids, scale):
        table, ids = _rows(table), ids.contiguous()
        out = torch.empty((ids.shape[0], table.shape[1]), dtype=table.dtype, device=table.device)
        gs_embed_fwd(table, ids, out, scale)
        ctx.save_for_backward(ids)
        ctx.scale, ctx.vocab = scale, table.shape[0]
        return out

    @staticmethod
    def backward(ctx, dout):
        (ids,) = ctx.saved_tensors
        dout = _rows(dout)
        n, dim = dout.shape
        dtable = torch.empty((ctx.vocab, dim), dtype=dout.dtype, device=dout.device)
        ws = _workspace(gs_embed_bwd_workspace_size(n, dim, ctx.vocab, dout.dtype), dout.device)
        gs_embed_bwd(ids, dout, dtable, ws, ctx.scale)
        return dtable, None, None


def embed(table, ids, scale=1.0):
    """scale * table[ids] for ids [n]; differentiable in the table [vocab, dim]."""
    return _EmbedFn.apply(table, ids, float(scale))


class _LayerNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        x = _rows(x)
        weight = weight.contiguous() if weight is not None else None
        bias = bias.contiguous() if bias is not None else None
        n, dim = x.shape
        y = torch.empty((n, dim), dtype=x.dtype, device=x.device)
        mean = torch.empty(n, dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
        gs_layer_norm_fwd(x, weight, bias, y, mean, rstd, eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        dy = _rows(dy)
        n, dim = x.shape
        new = lambda want, *shape: torch.empty(shape, dtype=x.dtype, device=x.device) if want else None
        dx = new(ctx.needs_input_grad[0], n, dim)
        dweight, dbias = new(ctx.needs_input_grad[1], dim), new(ctx.needs_input_grad[2], dim)
        ws = _workspace(gs_layer_norm_bwd_workspace_size(n, dim, x.dtype), x.device)
        gs_layer_norm_bwd(x, weight, mean, rstd, dy, dx, dweight, dbias, ws)
        return dx, dweight, dbias, None


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """Rows of x [n, dim] normalised to mean 0 and variance 1, times weight [dim] plus bias [dim]."""
    return _LayerNormFn.apply(x, weight, bias, float(eps))


class _LabelLossFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, labels):
        x, w, labels = _rows(x), _rows(w), labels.contiguous()
        n, dim = x.shape
        vec = lambda k, dt=torch.float32: torch.empty(k, dtype=dt, device=x.device)
        loss, lse, mean, count = vec(n), vec(n), vec(1), vec(1, torch.int32)
        ws = _workspace(gs_label_loss_workspace_size(n, dim, w.shape[0], x.dtype, False), x.device)
        gs_label_loss_fwd(x, w, labels, loss, lse, mean, count, ws)
        ctx.save_for_backward(x, w, labels, lse)
        ctx.mark_non_differentiable(count)
        ctx.set_materialize_grads(False)
        return mean.reshape(()), loss, count

    @staticmethod
    def backward(ctx, dmean, dloss, _):
        x, w, labels, lse = ctx.saved_tensors
        if dmean is None and dloss is None:
            return None, None, None
        n, dim = x.shape
        dmean = dmean.reshape(1).float() if dmean is not None else None
        dloss = dloss.contiguous() if dloss is not None else None
        dx = torch.empty((n, dim), dtype=x.dtype, device=x.device) if ctx.needs_input_grad[0] else None
        dw = torch.empty((w.shape[0], dim), dtype=x.dtype, device=x.device) if ctx.needs_input_grad[1] else None
        ws = _workspace(gs_label_loss_workspace_size(n, dim, w.shape[0], x.dtype, True), x.device)
        gs_label_loss_bwd(x, w, labels, lse, dx, dw, ws, dmean, dloss)
        return dx, dw, None


def label_loss(x, w, labels, reduction="mean"):
    """Softmax cross entropy of x [n, dim] against the vocabulary's rows w [vocab, dim].

    reduction: "mean" over the labelled rows (0 if there is none), "sum", or "none" (a loss per row, 0 without a
    label).
    """
    if reduction not in ("mean", "sum", "none"):
        raise ValueError(f"reduction must be 'mean', 'sum' or 'none', got {reduction!r}")
    mean, loss, _ = _LabelLossFn.apply(x, w, labels)
    return mean if reduction == "mean" else loss.sum() if reduction == "sum" else loss


class LabelHead(torch.nn.Module):
    """Labels from codes: codebook lookup, layer normalisation, vocabulary rows.

    ``codebook`` [codes, dim], ``weight`` and ``bias`` [dim], ``vocabulary`` [labels, dim]. The lookup is scaled by
    sqrt(dim), so that a codebook of variance 1 / dim gives features of variance 1.
    """

    def __init__(self, codes, dim, labels, device="cuda", dtype=torch.float32, eps=1e-5):
        super().__init__()
        new = lambda *shape: torch.randn(shape, device=device, dtype=dtype) / dim ** 0.5
        self.codebook = torch.nn.Parameter(new(codes, dim))
        self.weight = torch.nn.Parameter(torch.ones(dim, device=device, dtype=dtype))
        self.bias = torch.nn.Parameter(torch.zeros(dim, device=device, dtype=dtype))
        self.vocabulary = torch.nn.Parameter(new(labels, dim))
        self.scale, self.eps = float(dim) ** 0.5, float(eps)

    def features(self, codes):
        """Normalised features [n, dim] of codes [n]."""
        return layer_norm(embed(self.codebook, codes, self.scale), self.weight, self.bias, self.eps)

    def forward(self, codes, labels, reduction="mean"):
        """The loss of labels [n] for the Gaussians with the given codes [n]."""
        return label_loss(self.features(codes), self.vocabulary, labels, reduction)
