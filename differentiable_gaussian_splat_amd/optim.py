"""Clipping of gradients by their global norm, between the backward and the update.

:func:`clip_grads` clips a list of gradients (a scene's, as
:func:`.raster.gs_adam_step` takes them, or a label head's) in one call;
:class:`GradClip` keeps the addresses of gradients that stay in their buffers
from step to step. Both take all tensors together, float32 and bfloat16 side by
side, and neither waits for the device: one kernel for a small call (up to 64
tensors, 64 KB), else one for the norm and one for the scaling, and for more than
160 tensors one more for each 160, which puts their addresses into the workspace.
"""
from __future__ import annotations

import ctypes as C
from array import array

import torch

from .labels import _call, _stream
from .raster import load_library

__all__ = ["gs_clip_grads_workspace_size", "gs_clip_grads", "clip_grads", "GradClip"]

_DTYPES = {torch.float32: 0, torch.bfloat16: 1}


def _addresses(values):
    """A host array of 64-bit values, as the C call takes it."""
    a = array("q", values)
    return (C.c_int64 * len(a)).from_buffer(a) if a else None


def _dense(t):
    """Whether the tensor's elements fill one piece of memory, in any order of the dimensions."""
    if t.is_contiguous():
        return True
    if t.layout is not torch.strided:
        return False
    step = 1
    for stride, size in sorted((st, k) for st, k in zip(t.stride(), t.shape) if k != 1):
        if stride != step:
            return False
        step *= size
    return True


class _Tensors:
    """The host arrays of a call: checked once, and usable as long as the tensors keep their memory."""

    def __init__(self, grads, outs):
        self.grads = list(grads)
        self.outs = None if outs is None else list(outs)
        for name, ts in (("gradients", self.grads), ("outs", self.outs)):
            if ts is None:
                continue
            for t in ts:
                if t.dtype not in _DTYPES:
                    raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
            if not all([t.is_cuda for t in ts]):
                raise TypeError(f"{name} must be on the GPU")
            if not all([_dense(t) for t in ts]):
                raise ValueError(f"{name} must each fill one piece of memory")
        devices = {t.get_device() for t in self.grads + (self.outs or [])}
        if len(devices) > 1:
            raise ValueError(f"gradients and outs must be on one device, got {sorted(devices)}")
        self.device = devices.pop() if devices else None
        sizes = [t.numel() for t in self.grads]
        if outs is not None and outs is not grads and [(t.shape, t.stride(), t.dtype) for t in self.outs] != \
                [(t.shape, t.stride(), t.dtype) for t in self.grads]:
            raise ValueError("outs must have the gradients' number, shapes, strides and types")
        self.count = len(sizes)
        self.g = _addresses([t.data_ptr() for t in self.grads])
        places = None if outs is None else [t.data_ptr() for t in self.outs]
        if places is not None and len({p for p, k in zip(places, sizes) if k}) != sum([k > 0 for k in sizes]):
            raise ValueError("each tensor of outs must be there once")
        self.o = None if outs is None else _addresses(places) or C.c_void_p(1)
        self.n = _addresses(sizes)
        self.t = (C.c_int32 * self.count)(*[_DTYPES[t.dtype] for t in self.grads]) if self.count else None

    def call(self, max_norm, norm, workspace, stream):
        dev = norm.get_device()
        _call("gs_clip_grads", dev, self.count, self.g, self.o, self.n, self.t, max_norm, norm.data_ptr(),
              workspace.data_ptr(), workspace.numel(), _stream(stream, dev))


def gs_clip_grads_workspace_size(tensors) -> int:
    """Workspace bytes for a number of tensors."""
    return int(load_library().gs_clip_grads_workspace_size(int(tensors)))


def gs_clip_grads(grads, outs, norm, max_norm, workspace, stream=None):
    """norm[0] = sqrt(sum of all g^2); outs = min(1, max_norm / (norm + 1e-6)) grads (outs: the gradients themselves,
    tensors like them, or None for the norm only)."""
    t = _Tensors(grads, outs)
    if norm.dtype != torch.float32 or norm.numel() != 1 or not norm.is_cuda:
        raise TypeError(f"norm must be one float32 on the GPU, got {tuple(norm.shape)} {norm.dtype} on {norm.device}")
    if not workspace.is_cuda or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise TypeError("the workspace must be a contiguous uint8 buffer on the GPU")
    if {t.device, norm.get_device(), workspace.get_device()} - {None, norm.get_device()}:
        raise ValueError("gradients, norm and workspace must be on one device")
    t.call(max_norm, norm, workspace, stream)


class GradClip:
    """Clips gradients that stay in their buffers: ``clip = GradClip(grads)`` once, ``norm = clip(max_norm)`` per step.

    The tensors are checked, and their addresses kept, when the handle is made; it keeps them alive. A gradient that
    is replaced (``grad = None`` and a new one) needs a new handle. The norm (float32 [1], before clipping) and the
    workspace are the handle's own, written again by the next call: a handle is for one stream at a time, and a
    captured graph needs one of its own, which is kept as long as it. The first call on another stream than the one
    that was current when the handle was made waits for what that one has been given. outs: where the clipped
    gradients go (default: in place).
    """

    def __init__(self, grads, outs=None):
        grads = list(grads)
        if not grads:
            raise ValueError("there are no gradients to clip")
        self._t = _Tensors(grads, grads if outs is None else outs)
        self.norm = torch.empty(1, dtype=torch.float32, device=grads[0].device)
        self._ws = torch.empty(gs_clip_grads_workspace_size(len(grads)), dtype=torch.uint8, device=grads[0].device)
        self._made = _stream(None, self._t.device)
        self._tied = {self._made}

    def _tie(self, stream):
        """Makes the buffers, which are memory of the stream that was current when the handle was made, fit for use on
        another: work that had them before is done first, and none gets them before this stream is through."""
        device = self._t.device
        if stream is None:
            stream = torch.cuda.current_stream(device)
        with torch.cuda.stream(stream):
            if torch.cuda.is_current_stream_capturing():
                return  # a graph's calls run when it is replayed, with the handle kept beside it
        made = torch.cuda.ExternalStream(self._made, device) if self._made else torch.cuda.default_stream(device)
        stream.wait_stream(made)
        for t in [self.norm, self._ws] + self._t.grads + self._t.outs:
            t.record_stream(stream)
        self._tied.add(stream.cuda_stream)

    def __call__(self, max_norm, stream=None):
        if _stream(stream, self._t.device) not in self._tied:
            self._tie(stream)
        self._t.call(max_norm, self.norm, self._ws, stream)
        return self.norm


def clip_grads(params, max_norm, stream=None):
    """Clips the gradients of the parameters (those that have one; a single tensor is one parameter) in place by their
    global norm; returns it (float32 [1], before clipping), or None if there is no gradient. max_norm infinite: only
    the norm, the gradients stay as they are even where it is no number. stream: where this runs (default: the current
    one); its order with what writes and reads the gradients is the caller's."""
    if isinstance(params, torch.Tensor):
        params = [params]
    grads = list({id(p): p.grad for p in params if p.grad is not None}.values())  # a parameter named twice counts once
    if not grads:
        return None
    if stream is None:
        return GradClip(grads)(max_norm)
    # the handle is gone when this returns: its buffers are the stream's own, so that their next user comes after it
    with torch.cuda.stream(stream):
        norm = GradClip(grads)(max_norm, stream)  # named, so that another device's is refused
    norm.record_stream(torch.cuda.current_stream(norm.device))
    for t in grads:
        t.record_stream(stream)
    return norm
