"""Learning labels of a scene: feature codebook, layer normalisation, vocabulary loss.

A scene's Gaussians (or any other rows) carry features that are scored against a
vocabulary of labels. Three operators do that, each with its
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
from torch.autograd.function import once_differentiable

from .raster import _check, load_library

__all__ = ["gs_embed_fwd", "gs_embed_bwd_workspace_size", "gs_embed_bwd", "gs_layer_norm_fwd",
           "gs_layer_norm_bwd_workspace_size", "gs_layer_norm_bwd", "gs_label_loss_workspace_size",
           "gs_label_loss_fwd", "gs_label_loss_bwd", "embed", "layer_norm", "label_loss", "LabelHead"]

_DTYPES = {torch.float32: 0, torch.bfloat16: 1}
_INDEX_TYPES = {torch.int32: 0, torch.int64: 1}


# ------------------------------------------------------------------ argument checks
#
# The smallest calls are bound by the launch, so each check has a fast way
# through for a good argument; what fails it is looked at again for the message.

def _dtype(dtype) -> int:
    if dtype not in _DTYPES:
        raise TypeError(f"rows must be float32 or bfloat16, got {dtype}")
    return _DTYPES[dtype]


def _matrix(name, t, like=None, rows=None, cols=None):
    """Checks a matrix of rows (of the type and device of `like`, if given) and returns its row stride."""
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, got {t.dim()}")
    n, dim = t.shape
    st = t.stride()
    if (rows is not None and n != rows) or (cols is not None and dim != cols):
        raise ValueError(f"{name} must have shape ({'*' if rows is None else rows}, {'*' if cols is None else cols}), "
                         f"got {tuple(t.shape)}")
    if dim > 1 and st[1] != 1:
        raise ValueError(f"{name}'s columns must be consecutive, got strides {st}")
    if like is not None:
        if t.dtype != like.dtype or t.get_device() != like.get_device():
            raise TypeError(f"{name} must be {like.dtype} on {like.device}, got {t.dtype} on {t.device}")
    else:
        _dtype(t.dtype)
        if not t.is_cuda:
            raise TypeError(f"{name} must be on the GPU, got {t.device}")
    # one row has no stride of its own; torch may give it any
    return st[0] if n > 1 else max(dim, 1)


def _vector(name, t, n, dtype, device):
    """Checks a contiguous vector of n (device: an index, as get_device() gives it) and returns its address."""
    if t is None:
        return None
    if t.dtype is dtype and t.get_device() == device and t.dim() == 1 and t.numel() == n and t.is_contiguous():
        return t.data_ptr()
    if t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n}, got shape {tuple(t.shape)}")
    raise TypeError(f"{name} must be {dtype} on device {device}, got {t.dtype} on {t.device}")


def _index(name, t, n, device) -> int:
    """Checks an index vector; its address and type."""
    if t.dtype not in _INDEX_TYPES:
        raise TypeError(f"{name} must be int32 or int64, got {t.dtype}")
    return _vector(name, t, n, t.dtype, device), _INDEX_TYPES[t.dtype]


def _opt(t):
    return None if t is None else t.data_ptr()


def _workspace_of(t):
    """A workspace's address and bytes (None: none)."""
    if t is None:
        return None, 0
    if not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"a workspace must be a contiguous buffer on the GPU, got one on {t.device}")
    return t.data_ptr(), t.numel() * t.element_size()


def _stream(stream, device):
    """The stream's handle; the device's current stream if None (asked for by number: the object costs 2.5 us)."""
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream


# ------------------------------------------------------------------ thin C-ABI wrappers

def gs_embed_fwd(table, ids, out, scale=1.0, stream=None):
    """out[i] = scale * table[ids[i]]; zero rows where ids[i] names no row."""
    ts = _matrix("table", table)
    vocab, dim = table.shape
    n = ids.numel()  # of one dimension, as _index sees to
    os_ = _matrix("out", out, table, n, dim)
    dev = table.get_device()
    ip, it = _index("ids", ids, n, dev)
    st = load_library().gs_embed_fwd(n, dim, vocab, _DTYPES[table.dtype], table.data_ptr(), ts, ip, it, scale,
                                     out.data_ptr(), os_, _stream(stream, dev))
    _check(st, "gs_embed_fwd")


def gs_embed_bwd_workspace_size(n, dim, vocab, dtype) -> int:
    return int(load_library().gs_embed_bwd_workspace_size(n, dim, vocab, _dtype(dtype)))


def gs_embed_bwd(ids, dout, dtable, workspace, scale=1.0, stream=None):
    """dtable[v] = scale * sum of dout over the rows whose index is v (every row of dtable is written)."""
    ds = _matrix("dout", dout)
    n, dim = dout.shape
    ts = _matrix("dtable", dtable, dout, None, dim)
    dev = dout.get_device()
    ip, it = _index("ids", ids, n, dev)
    st = load_library().gs_embed_bwd(n, dim, dtable.shape[0], _DTYPES[dout.dtype], ip, it, scale, dout.data_ptr(), ds,
                                     dtable.data_ptr(), ts, *_workspace_of(workspace), _stream(stream, dev))
    _check(st, "gs_embed_bwd")


def gs_layer_norm_fwd(x, weight, bias, y, mean=None, rstd=None, eps=1e-5, stream=None):
    """y = (x - mean) * rstd * weight + bias per row; weight and bias may be None."""
    xs = _matrix("x", x)
    n, dim = x.shape
    ys = _matrix("y", y, x, n, dim)
    dt, dev = x.dtype, x.get_device()
    st = load_library().gs_layer_norm_fwd(n, dim, _DTYPES[dt], x.data_ptr(), xs,
                                          _vector("weight", weight, dim, dt, dev), _vector("bias", bias, dim, dt, dev),
                                          eps, y.data_ptr(), ys, _vector("mean", mean, n, torch.float32, dev),
                                          _vector("rstd", rstd, n, torch.float32, dev), _stream(stream, dev))
    _check(st, "gs_layer_norm_fwd")


def gs_layer_norm_bwd_workspace_size(n, dim, dtype) -> int:
    return int(load_library().gs_layer_norm_bwd_workspace_size(n, dim, _dtype(dtype)))


def gs_layer_norm_bwd(x, weight, mean, rstd, dy, dx, dweight, dbias, workspace, stream=None):
    """Gradients of gs_layer_norm_fwd into dx, dweight and dbias (each may be None)."""
    xs = _matrix("x", x)
    n, dim = x.shape
    dys = _matrix("dy", dy, x, n, dim)
    dxs = _matrix("dx", dx, x, n, dim) if dx is not None else dim
    dt, dev, f32 = x.dtype, x.get_device(), torch.float32
    st = load_library().gs_layer_norm_bwd(n, dim, _DTYPES[dt], x.data_ptr(), xs,
                                          _vector("weight", weight, dim, dt, dev), _vector("mean", mean, n, f32, dev),
                                          _vector("rstd", rstd, n, f32, dev), dy.data_ptr(), dys, _opt(dx), dxs,
                                          _vector("dweight", dweight, dim, dt, dev),
                                          _vector("dbias", dbias, dim, dt, dev), *_workspace_of(workspace),
                                          _stream(stream, dev))
    _check(st, "gs_layer_norm_bwd")


def gs_label_loss_workspace_size(n, dim, vocab, dtype, backward) -> int:
    return int(load_library().gs_label_loss_workspace_size(n, dim, vocab, _dtype(dtype), 1 if backward else 0))


def gs_label_loss_fwd(x, w, labels, loss, lse, mean, count, workspace, stream=None):
    """Per row lse = log sum_v exp(x . w[v]) and loss = lse - x . w[label] (0 without a label); the mean loss and
    the number of labelled rows."""
    xs = _matrix("x", x)
    n, dim = x.shape
    ws = _matrix("w", w, x, None, dim)
    dev, f32 = x.get_device(), torch.float32
    ip, it = _index("labels", labels, n, dev)
    st = load_library().gs_label_loss_fwd(n, dim, w.shape[0], _DTYPES[x.dtype], x.data_ptr(), xs, w.data_ptr(), ws, ip,
                                          it, _vector("loss", loss, n, f32, dev), _vector("lse", lse, n, f32, dev),
                                          _vector("mean", mean, 1, f32, dev),
                                          _vector("count", count, 1, torch.int32, dev), *_workspace_of(workspace),
                                          _stream(stream, dev))
    _check(st, "gs_label_loss_fwd")


def gs_label_loss_bwd(x, w, labels, lse, dx, dw, workspace, dmean=None, dloss=None, stream=None):
    """Gradients into dx and dw (each may be None) from the upstream gradients of the mean loss and of the rows'
    losses."""
    xs = _matrix("x", x)
    n, dim = x.shape
    ws = _matrix("w", w, x, None, dim)
    dev, f32 = x.get_device(), torch.float32
    ip, it = _index("labels", labels, n, dev)
    dxs = _matrix("dx", dx, x, n, dim) if dx is not None else dim
    dws = _matrix("dw", dw, w, w.shape[0], dim) if dw is not None else dim
    st = load_library().gs_label_loss_bwd(n, dim, w.shape[0], _DTYPES[x.dtype], x.data_ptr(), xs, w.data_ptr(), ws, ip,
                                          it, _vector("lse", lse, n, f32, dev), _vector("dmean", dmean, 1, f32, dev),
                                          _vector("dloss", dloss, n, f32, dev), _opt(dx), dxs, _opt(dw), dws,
                                          *_workspace_of(workspace), _stream(stream, dev))
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
        out = torch.empty((ids.numel(), table.shape[1]), dtype=table.dtype, device=table.device)
        gs_embed_fwd(table, ids, out, scale)
        ctx.save_for_backward(ids)
        ctx.scale, ctx.vocab = scale, table.shape[0]
        return out

    @staticmethod
    @once_differentiable
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
    @once_differentiable
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
    @once_differentiable
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
