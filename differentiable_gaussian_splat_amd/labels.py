"""Learning labels of a scene: feature codebook, layer normalisation, vocabulary loss.

A scene's Gaussians (or any other rows) carry features that are scored against a
vocabulary of labels. Three operators train that, each with its
gradients, in float32 or bfloat16:

- :func:`embed` looks a feature codebook up by each Gaussian's code;
- :func:`layer_norm` normalises feature rows;
- :func:`label_loss` is the softmax cross entropy of feature rows against the
  vocabulary's rows; the logits are never stored.

Two more are for features that are sums over several codebooks (residual
quantisation), and for naming labels by scores:

- :func:`rms_norm` adds a residual and normalises by the root mean square, with
  its gradients; :func:`rms_norm_q8` gives the result in 8 bits;
- :func:`label_scores` multiplies rows in 8 bits (of :func:`rms_norm_q8` or
  :func:`quantize_q8`) with a vocabulary in 8 bits: inference only.

The ``gs_*`` functions marshal tensors into the C calls of the same names
(``include/gsplat.h``) and leave buffers to the caller; the functions
above are wrappers that allocate them (autograd ones where there is a
gradient). An index outside the table
(use -1) marks a row without a code or label: it takes no part.
:class:`LabelHead` and :class:`ResidualLabelHead` chain them.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from .raster import _check, load_library

__all__ = ["gs_embed_fwd", "gs_embed_bwd_workspace_size", "gs_embed_bwd", "gs_layer_norm_fwd",
           "gs_layer_norm_bwd_workspace_size", "gs_layer_norm_bwd", "gs_label_loss_workspace_size",
           "gs_label_loss_fwd", "gs_label_loss_bwd", "gs_rms_norm_fwd", "gs_rms_norm_bwd_workspace_size",
           "gs_rms_norm_bwd", "gs_rms_norm_q8", "gs_quantize_q8", "gs_label_scores_q8", "embed", "layer_norm",
           "label_loss", "rms_norm", "rms_norm_q8", "rows_q8", "quantize_q8", "label_scores", "LabelHead",
           "ResidualLabelHead"]

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
    if dim > 1 and st[1] != 1 and n > 0:  # a matrix without rows may have any strides
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


def _rows8(name, q, scales, rows=None, cols=None):
    """Checks rows in 8 bits; the addresses and strides of the values and the scales."""
    if q.dim() != 2 or scales.dim() != 2:
        raise ValueError(f"{name} and its scales must have two dimensions, got {q.dim()} and {scales.dim()}")
    if q.dtype is not torch.float8_e4m3fn or scales.dtype is not torch.float8_e8m0fnu:
        raise TypeError(f"{name} must be float8_e4m3fn with float8_e8m0fnu scales, got {q.dtype} and {scales.dtype}")
    n, c = q.shape
    groups = (c // 128 + 3) // 4 * 4
    if c % 128 or c == 0 or (rows is not None and n != rows) or (cols is not None and c != cols):
        raise ValueError(f"{name} must have shape ({'*' if rows is None else rows}, "
                         f"{'a multiple of 128' if cols is None else cols}), got {tuple(q.shape)}")
    if scales.shape != (n, groups):
        raise ValueError(f"{name}'s scales must have shape ({n}, {groups}), got {tuple(scales.shape)}")
    if q.stride(1) != 1 or scales.stride(1) != 1:
        raise ValueError(f"{name}'s and its scales' columns must be consecutive")
    if not q.is_cuda or scales.get_device() != q.get_device():
        raise TypeError(f"{name} and its scales must be on one GPU, got {q.device} and {scales.device}")
    # one row has no stride of its own; torch may give it any
    return (q.data_ptr(), q.stride(0) if n > 1 else c, scales.data_ptr(), scales.stride(0) if n > 1 else groups)


def _same_device(name, t, device):
    if t.get_device() != device:
        raise TypeError(f"{name} must be on device {device}, got {t.device}")


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


def _call(name, device, *args):
    """A call on the tensors' device: the default stream's handle is the same on every device."""
    fn = getattr(load_library(), name)
    if device == torch._C._cuda_getDevice():
        st = fn(*args)
    else:
        with torch.cuda.device(device):
            st = fn(*args)
    _check(st, name)


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


def _rms_inputs(x, weight, residual, sum):
    """The arguments that both forms of the normalisation share: sizes, type, x to weight, sum."""
    xs = _matrix("x", x)
    n, dim = x.shape
    rs = _matrix("residual", residual, x, n, dim) if residual is not None else dim
    ss = _matrix("sum", sum, x, n, dim) if sum is not None else dim
    return ((n, dim, _DTYPES[x.dtype], x.data_ptr(), xs, _opt(residual), rs,
             _vector("weight", weight, dim, x.dtype, x.get_device())), (_opt(sum), ss))


def gs_rms_norm_fwd(x, weight, y, residual=None, sum=None, rstd=None, eps=1e-6, stream=None):
    """h = x + residual, y = h * rstd * weight with rstd = 1 / sqrt(mean(h^2) + eps) per row; residual and weight may
    be None. sum receives h."""
    first, kept = _rms_inputs(x, weight, residual, sum)
    n, dim = x.shape
    ys = _matrix("y", y, x, n, dim)
    dev = x.get_device()
    _call("gs_rms_norm_fwd", dev, *first, eps, *kept, y.data_ptr(), ys,
          _vector("rstd", rstd, n, torch.float32, dev), _stream(stream, dev))


def gs_rms_norm_bwd_workspace_size(n, dim, dtype) -> int:
    return int(load_library().gs_rms_norm_bwd_workspace_size(n, dim, _dtype(dtype)))


def gs_rms_norm_bwd(h, weight, rstd, dy, dx, dweight, workspace, dsum=None, stream=None):
    """Gradients of gs_rms_norm_fwd into dx (the residual's too) and dweight (each may be None); h: the forward's sum;
    dsum: the gradient of it as it was handed on, or None."""
    hs = _matrix("h", h)
    n, dim = h.shape
    dys = _matrix("dy", dy, h, n, dim)
    dss = _matrix("dsum", dsum, h, n, dim) if dsum is not None else dim
    dxs = _matrix("dx", dx, h, n, dim) if dx is not None else dim
    dt, dev = h.dtype, h.get_device()
    if workspace is not None:
        _same_device("the workspace", workspace, dev)
    _call("gs_rms_norm_bwd", dev, n, dim, _DTYPES[dt], h.data_ptr(), hs, _vector("weight", weight, dim, dt, dev),
          _vector("rstd", rstd, n, torch.float32, dev), dy.data_ptr(), dys, _opt(dsum),
          dss, _opt(dx), dxs, _vector("dweight", dweight, dim, dt, dev),
          *_workspace_of(workspace), _stream(stream, dev))


def gs_rms_norm_q8(x, weight, q, scales, residual=None, sum=None, eps=1e-6, stream=None):
    """gs_rms_norm_fwd with y as rows in 8 bits (q and scales: see rows_q8)."""
    first, kept = _rms_inputs(x, weight, residual, sum)
    n, dim = x.shape
    qp, qs, sp, scs = _rows8("q", q, scales, n, (dim + 127) // 128 * 128)
    dev = x.get_device()
    _same_device("q", q, dev)
    _call("gs_rms_norm_q8", dev, *first, eps, *kept, qp, qs, sp, scs, _stream(stream, dev))


def gs_quantize_q8(x, q, scales, stream=None):
    """Rows of x in 8 bits (q and scales: see rows_q8)."""
    xs = _matrix("x", x)
    n, dim = x.shape
    qp, qs, sp, scs = _rows8("q", q, scales, n, (dim + 127) // 128 * 128)
    dev = x.get_device()
    _same_device("q", q, dev)
    _call("gs_quantize_q8", dev, n, dim, _DTYPES[x.dtype], x.data_ptr(), xs, qp, qs, sp, scs,
          _stream(stream, dev))


def gs_label_scores_q8(q, q_scales, w, w_scales, out, stream=None):
    """out[i][v] = row i of q times row v of w, both in 8 bits; out is float32 or bfloat16, and its type says how the
    products are summed (see label_scores)."""
    qa = _rows8("q", q, q_scales)
    n, cols = q.shape
    wa = _rows8("w", w, w_scales, None, cols)
    vocab = w.shape[0]
    os_ = _matrix("out", out, None, n, vocab)
    dev = out.get_device()
    _same_device("q", q, dev)
    _same_device("w", w, dev)
    _call("gs_label_scores_q8", dev, n, cols, vocab, _DTYPES[out.dtype], *qa, *wa, out.data_ptr(), os_,
          _stream(stream, dev))


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


class _RmsNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        x = _rows(x)
        residual = _rows(residual) if residual is not None else None
        weight = weight.contiguous() if weight is not None else None
        n, dim = x.shape
        y = torch.empty((n, dim), dtype=x.dtype, device=x.device)
        h = torch.empty_like(y) if residual is not None else None
        rstd = torch.empty(n, dtype=torch.float32, device=x.device)
        gs_rms_norm_fwd(x, weight, y, residual, h, rstd, eps)
        ctx.save_for_backward(x if h is None else h, weight, rstd)
        ctx.set_materialize_grads(False)
        return y, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dsum):
        h, weight, rstd = ctx.saved_tensors
        if dy is None and dsum is None:
            return None, None, None, None
        want_x = ctx.needs_input_grad[0] or ctx.needs_input_grad[2]
        if dy is None:  # the sum alone was used
            return (dsum if ctx.needs_input_grad[0] else None, None, dsum if ctx.needs_input_grad[2] else None, None)
        n, dim = h.shape
        dy = _rows(dy)
        dsum = _rows(dsum) if dsum is not None else None
        dx = torch.empty((n, dim), dtype=h.dtype, device=h.device) if want_x else None
        dweight = torch.empty(dim, dtype=h.dtype, device=h.device) if ctx.needs_input_grad[1] else None
        ws = _workspace(gs_rms_norm_bwd_workspace_size(n, dim, h.dtype), h.device)
        gs_rms_norm_bwd(h, weight, rstd, dy, dx, dweight, ws, dsum)
        return (dx if ctx.needs_input_grad[0] else None, dweight, dx if ctx.needs_input_grad[2] else None, None)


def rms_norm(x, weight=None, residual=None, eps=1e-6):
    """Rows of x [n, dim], plus those of residual [n, dim], over their root mean square, times weight [dim].

    Returns the result; with a residual, the result and the sum (both differentiable).
    """
    y, h = _RmsNormFn.apply(x, weight, residual, float(eps))
    return y if residual is None else (y, h)


def rows_q8(n, dim, device="cuda"):
    """Empty rows in 8 bits: values [n, dim rounded up to 128] (float8_e4m3fn), scales (float8_e8m0fnu) one for each
    128 columns, rounded up to four to a row."""
    cols = (dim + 127) // 128 * 128
    return (torch.empty((n, cols), dtype=torch.float8_e4m3fn, device=device),
            torch.empty((n, (cols // 128 + 3) // 4 * 4), dtype=torch.float8_e8m0fnu, device=device))


def _no_gradient(name, *tensors):
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        raise RuntimeError(f"{name} has no gradient: call it under torch.no_grad(), or on detached tensors")


def rms_norm_q8(x, weight=None, residual=None, eps=1e-6):
    """rms_norm with its result in 8 bits: (values, scales), with a residual ((values, scales), sum). No gradient."""
    _no_gradient("rms_norm_q8", x, weight, residual)
    x = _rows(x)
    residual = _rows(residual) if residual is not None else None
    q, scales = rows_q8(*x.shape, x.device)
    h = torch.empty(x.shape, dtype=x.dtype, device=x.device) if residual is not None else None
    gs_rms_norm_q8(x, weight.contiguous() if weight is not None else None, q, scales, residual, h, eps)
    return (q, scales) if residual is None else ((q, scales), h)


def quantize_q8(x):
    """Rows of x [n, dim] in 8 bits: (values, scales). No gradient."""
    _no_gradient("quantize_q8", x)
    x = _rows(x)
    q, scales = rows_q8(*x.shape, x.device)
    gs_quantize_q8(x, q, scales)
    return q, scales


def label_scores(rows, vocabulary, dtype=torch.float32):
    """Scores [n, labels] of rows in 8 bits against a vocabulary in 8 bits, each a pair (values, scales).

    dtype chooses the sums with the result's type. float32: whole products, summed in float32. bfloat16: the matrix
    units' 8-bit products, up to 1.8 times as fast, which cut each of eight columns' products beside each other off at
    2^-13 of the largest one's power of two before they add them. On normal data that is 1.4e-5 of a score's size, far
    below bfloat16's own rounding; where large products cancel, small ones among the same eight columns are lost.
    """
    (q, q_scales), (w, w_scales) = rows, vocabulary
    _dtype(dtype)
    out = torch.empty((q.shape[0], w.shape[0]), dtype=dtype, device=q.device)
    gs_label_scores_q8(q, q_scales, w, w_scales, out)
    return out


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

    @torch.no_grad()
    def vocabulary_q8(self):
        """The vocabulary in 8 bits, for :meth:`scores`: made once after training."""
        return quantize_q8(self.vocabulary)

    @torch.no_grad()
    def scores(self, codes, vocabulary=None, dtype=torch.float32):
        """Scores [n, labels] of codes [n], features and vocabulary in 8 bits (dtype: see label_scores)."""
        return label_scores(quantize_q8(self.features(codes)),
                            self.vocabulary_q8() if vocabulary is None else vocabulary, dtype)


class ResidualLabelHead(torch.nn.Module):
    """Labels from several codes a row (residual quantisation): each stage's codebook row is added to the sum of the
    stages before it, and every stage's sum is normalised by its root mean square and scored.

    ``codebooks`` (one [codes[k], dim] for each stage), ``weights`` (one [dim] for each stage), ``vocabulary``
    [labels, dim]. The first stage's rows are scaled by sqrt(dim), so that codebooks of variance 1 / dim give features
    of variance 1, and each later one's by half of the one before: it refines.
    """

    def __init__(self, codes, dim, labels, device="cuda", dtype=torch.float32, eps=1e-6):
        super().__init__()
        new = lambda *shape: torch.nn.Parameter(torch.randn(shape, device=device, dtype=dtype) / dim ** 0.5)
        self.codebooks = torch.nn.ParameterList([new(k, dim) for k in codes])
        self.weights = torch.nn.ParameterList([torch.nn.Parameter(torch.ones(dim, device=device, dtype=dtype))
                                               for _ in codes])
        self.vocabulary = new(labels, dim)
        self.scales, self.eps = [float(dim) ** 0.5 / 2 ** k for k in range(len(codes))], float(eps)

    def features(self, codes):
        """Normalised features [n, dim] after each stage, of codes [stages, n]."""
        found, h = [], None
        for table, weight, scale, code in zip(self.codebooks, self.weights, self.scales, codes, strict=True):
            x = embed(table, code, scale)
            if h is None:
                y, h = rms_norm(x, weight, eps=self.eps), x
            else:
                y, h = rms_norm(x, weight, h, self.eps)
            found.append(y)
        return found

    def forward(self, codes, labels):
        """The mean over the stages of the loss of labels [n] for rows of the given codes [stages, n]: any first
        stages alone are trained to name the label."""
        losses = [label_loss(y, self.vocabulary, labels) for y in self.features(codes)]
        return torch.stack(losses).mean()

    @torch.no_grad()
    def vocabulary_q8(self):
        """The vocabulary in 8 bits, for :meth:`scores`: made once after training."""
        return quantize_q8(self.vocabulary)

    @torch.no_grad()
    def scores(self, codes, vocabulary=None, dtype=torch.float32):
        """Scores [n, labels] after the last of the given stages (codes [stages, n], as many stages as wanted; dtype:
        see label_scores)."""
        if not 0 < len(codes) <= len(self.codebooks):
            raise ValueError(f"codes must be of 1 to {len(self.codebooks)} stages, got {len(codes)}")
        h, rows, last = None, None, len(codes) - 1
        for k, code in enumerate(codes):
            x = embed(self.codebooks[k], code, self.scales[k])
            if k == 0 < last:
                h = x
                continue
            # the norm's kernel adds; a stage before the last is there for its sum, and its rows are overwritten
            rows = rows_q8(*x.shape, x.device) if rows is None else rows
            total = torch.empty_like(x) if k < last else None
            gs_rms_norm_q8(x, self.weights[k].contiguous(), *rows, h, total, self.eps)
            h = total
        return label_scores(rows, self.vocabulary_q8() if vocabulary is None else vocabulary, dtype)
