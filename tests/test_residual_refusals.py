"""Refusals of the residual norm's, the 8-bit rows' and the clipping's calls (no GPU)."""
import ctypes as C

import pytest
import torch

from differentiable_gaussian_splat_amd import labels as L
from differentiable_gaussian_splat_amd import optim as O
from differentiable_gaussian_splat_amd import raster

INVALID, UNSUPPORTED, OK = raster.GS_ERR_INVALID_ARG, raster.GS_ERR_UNSUPPORTED, raster.GS_OK
D = C.c_void_p(4096)  # never dereferenced: validation fails first
P1, P2, P4, P8 = (C.c_void_p(4096 + k) for k in (1, 2, 4, 8))
BIG = 1 << 60


def lib():
    return raster.load_library()


FWD = dict(n=4, dim=8, dtype=0, x=D, xs=8, residual=D, rs=8, w=D, eps=1e-6, sum=D, ss=8, y=D, ys=8, rstd=D,
           stream=None)
BWD = dict(n=4, dim=8, dtype=1, h=D, hs=8, w=D, rstd=D, dy=D, dys=8, dsum=D, dss=8, dx=D, dxs=8, dw=D, ws=D, wb=BIG,
           stream=None)
Q8 = dict(n=4, dim=200, dtype=1, x=D, xs=200, residual=D, rs=200, w=D, eps=1e-6, sum=D, ss=200, q=D, qs=256, scales=D,
          scs=4, stream=None)
QUANT = dict(n=4, dim=200, dtype=0, x=D, xs=200, q=D, qs=256, scales=D, scs=4, stream=None)
SCORES = dict(n=4, cols=640, vocab=7, dtype=0, q=D, qs=640, qsc=D, qss=8, w=D, ws=640, wsc=D, wss=8, out=D, os=7,
              stream=None)

REFUSED = [
    ("gs_rms_norm_fwd", FWD, dict(n=-1), INVALID, "n must be"),
    ("gs_rms_norm_fwd", FWD, dict(dim=65537), INVALID, "dim"),
    ("gs_rms_norm_fwd", FWD, dict(dtype=2), UNSUPPORTED, "dtype"),
    ("gs_rms_norm_fwd", FWD, dict(eps=-1e-6), INVALID, "eps"),
    ("gs_rms_norm_fwd", FWD, dict(eps=float("inf")), INVALID, "eps"),
    ("gs_rms_norm_fwd", FWD, dict(x=None), INVALID, "x must"),
    ("gs_rms_norm_fwd", FWD, dict(residual=P1), INVALID, "misaligned residual"),
    ("gs_rms_norm_fwd", FWD, dict(rs=7), INVALID, "residual's row stride"),
    ("gs_rms_norm_fwd", FWD, dict(residual=None), INVALID, "sum needs a residual"),
    ("gs_rms_norm_fwd", FWD, dict(ss=0), INVALID, "sum's row stride"),
    ("gs_rms_norm_fwd", FWD, dict(y=None), INVALID, "y must"),
    ("gs_rms_norm_fwd", FWD, dict(rstd=P2), INVALID, "misaligned rstd"),
    ("gs_rms_norm_bwd", BWD, dict(rstd=None), INVALID, "rstd"),
    ("gs_rms_norm_bwd", BWD, dict(dy=None), INVALID, "dy"),
    ("gs_rms_norm_bwd", BWD, dict(dss=4), INVALID, "dsum's row stride"),
    ("gs_rms_norm_bwd", BWD, dict(dxs=0), INVALID, "dx's row stride"),
    ("gs_rms_norm_bwd", BWD, dict(wb=16), INVALID, "workspace too small"),
    ("gs_rms_norm_bwd", BWD, dict(ws=P4), INVALID, "256-byte"),
    ("gs_rms_norm_q8", Q8, dict(q=None), INVALID, "q and its scales"),
    ("gs_rms_norm_q8", Q8, dict(q=P8), INVALID, "16-byte"),
    ("gs_rms_norm_q8", Q8, dict(qs=200), INVALID, "16-byte"),
    ("gs_rms_norm_q8", Q8, dict(qs=240), INVALID, "q's row stride"),
    ("gs_rms_norm_q8", Q8, dict(qs=0), INVALID, "q's row stride"),
    ("gs_rms_norm_q8", Q8, dict(scales=P2), INVALID, "4-byte"),
    ("gs_rms_norm_q8", Q8, dict(scs=2), INVALID, "4-byte"),
    ("gs_rms_norm_q8", Q8, dict(scs=0), INVALID, "scales' row stride"),
    ("gs_quantize_q8", QUANT, dict(dim=0), INVALID, "dim"),
    ("gs_quantize_q8", QUANT, dict(x=P2), INVALID, "misaligned x"),
    ("gs_quantize_q8", QUANT, dict(scales=None), INVALID, "q and its scales"),
    ("gs_quantize_q8", QUANT, dict(qs=(1 << 22) + 16), INVALID, "q's row stride"),
    ("gs_label_scores_q8", SCORES, dict(cols=600), INVALID, "multiple of 128"),
    ("gs_label_scores_q8", SCORES, dict(cols=0), INVALID, "dim"),
    ("gs_label_scores_q8", SCORES, dict(vocab=0), INVALID, "vocab"),
    ("gs_label_scores_q8", SCORES, dict(dtype=7), UNSUPPORTED, "dtype"),
    ("gs_label_scores_q8", SCORES, dict(qs=512), INVALID, "q's row stride"),
    ("gs_label_scores_q8", SCORES, dict(qss=4), INVALID, "q's scales"),
    ("gs_label_scores_q8", SCORES, dict(w=None), INVALID, "w and its scales"),
    ("gs_label_scores_q8", SCORES, dict(wss=(1 << 22) + 4), INVALID, "w's scales"),
    ("gs_label_scores_q8", SCORES, dict(out=None), INVALID, "out"),
    ("gs_label_scores_q8", SCORES, dict(os=6), INVALID, "out's row stride"),
    ("gs_label_scores_q8", SCORES, dict(out=P2), INVALID, "misaligned out"),
]


@pytest.mark.parametrize("fn,base,change,code,text", REFUSED, ids=[f"{r[0]}-{'-'.join(r[2])}" for r in REFUSED])
def test_c_call_refuses(fn, base, change, code, text):
    assert getattr(lib(), fn)(*dict(base, **change).values()) == code
    message = lib().gs_last_error().decode()
    assert text in message and fn in message


def clip(n=2, grads=(4096, 8192), outs=(4096, 8192), numels=(5, 7), dtypes=(0, 1), max_norm=1.0, norm=D, ws=D, wb=BIG):
    p = lambda v: None if v is None else (C.c_int64 * len(v))(*v)
    t = None if dtypes is None else (C.c_int32 * len(dtypes))(*dtypes)
    return lib().gs_clip_grads(n, p(grads), p(outs), p(numels), t, max_norm, norm, ws, wb, None)


@pytest.mark.parametrize("change,code,text", [
    (dict(n=-1), INVALID, "tensors"),
    (dict(n=65537), INVALID, "tensors"),
    (dict(max_norm=-1.0), INVALID, "max_norm"),
    (dict(max_norm=float("nan")), INVALID, "max_norm"),
    (dict(grads=None), INVALID, "NULL"),
    (dict(numels=None), INVALID, "NULL"),
    (dict(dtypes=None), INVALID, "NULL"),
    (dict(numels=(5, -1)), INVALID, "tensor 1's size"),
    (dict(numels=(1 << 41, 1)), INVALID, "tensor 0's size"),
    (dict(numels=(1 << 40, 1)), INVALID, "2^40 elements"),
    (dict(dtypes=(0, 2)), UNSUPPORTED, "tensor 1's dtype"),
    (dict(grads=(0, 8192)), INVALID, "tensor 0 is NULL"),
    (dict(outs=(4096, 0)), INVALID, "tensor 1 is NULL"),
    (dict(grads=(4098, 8192)), INVALID, "tensor 0 is misaligned"),
    (dict(outs=(4096, 8193)), INVALID, "tensor 1 is misaligned"),
    (dict(norm=None), INVALID, "norm"),
    (dict(norm=P2), INVALID, "norm"),
    (dict(wb=100), INVALID, "workspace too small"),
    (dict(ws=P8), INVALID, "256-byte"),
])
def test_clip_refuses(change, code, text):
    assert clip(**change) == code
    message = lib().gs_last_error().decode()
    assert text in message and "gs_clip_grads" in message


def test_empty_calls_need_no_arrays():
    """n = 0: the calls return before any HIP call."""
    assert lib().gs_rms_norm_fwd(*dict(FWD, n=0, x=None, residual=None, sum=None, y=None, rstd=None).values()) == OK
    assert lib().gs_rms_norm_q8(*dict(Q8, n=0, x=None, residual=None, sum=None, q=None, scales=None).values()) == OK
    assert lib().gs_quantize_q8(*dict(QUANT, n=0, x=None, q=None, scales=None).values()) == OK
    assert lib().gs_label_scores_q8(*dict(SCORES, n=0, q=None, qsc=None, out=None).values()) == OK
    assert lib().gs_rms_norm_bwd(*dict(BWD, dx=None, dw=None).values()) == OK


def test_workspace_sizes():
    assert L.gs_rms_norm_bwd_workspace_size(1 << 20, 64, torch.bfloat16) >= 64 * 4
    assert L.gs_rms_norm_bwd_workspace_size(-1, 64, torch.float32) == 0
    a, b = O.gs_clip_grads_workspace_size(1), O.gs_clip_grads_workspace_size(5000)
    assert 0 < a < b
    assert O.gs_clip_grads_workspace_size(-1) == O.gs_clip_grads_workspace_size(65537) == 0


def _t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def _q(n, cols, groups):
    return torch.zeros((n, cols), dtype=torch.float8_e4m3fn), torch.ones((n, groups)).to(torch.float8_e8m0fnu)


@pytest.mark.parametrize("call,kind", [
    (lambda: L.gs_rms_norm_fwd(_t(3, 4), None, _t(3, 4)), TypeError),                         # not on the GPU
    (lambda: L.gs_rms_norm_fwd(_t(3, 4, dtype=torch.float16), None, _t(3, 4)), TypeError),
    (lambda: L.gs_rms_norm_fwd(_t(4, 3).t(), None, _t(3, 4)), ValueError),                     # columns apart
    (lambda: L.rms_norm(_t(5)), ValueError),
    (lambda: L.rms_norm_q8(_t(3, 4).requires_grad_()), RuntimeError),                          # no gradient
    (lambda: L.quantize_q8(_t(3, 4).requires_grad_()), RuntimeError),
    (lambda: L.quantize_q8(_t(3, 4)), TypeError),
    (lambda: L.label_scores(_q(3, 128, 4), _q(5, 128, 4)), TypeError),
    (lambda: L.label_scores(_q(3, 128, 4), _q(5, 128, 4), torch.float16), TypeError),
    (lambda: L._rows8("q", *_q(3, 128, 4), 2), ValueError),                                    # rows
    (lambda: L._rows8("q", *_q(3, 100, 4)), ValueError),                                       # columns
    (lambda: L._rows8("q", *_q(3, 0, 0)), ValueError),
    (lambda: L._rows8("q", *_q(3, 640, 4)), ValueError),                                       # scales
    (lambda: L._rows8("q", _t(3, 128), _q(3, 128, 4)[1]), TypeError),
    (lambda: L._rows8("q", _q(3, 128, 4)[0][0], _q(3, 128, 4)[1]), ValueError),
    (lambda: L._rows8("q", _q(128, 128, 4)[0].t(), _q(128, 128, 4)[1]), ValueError),
    (lambda: O.GradClip([]), ValueError),
    (lambda: O.GradClip([_t(3)]), TypeError),
    (lambda: O.GradClip([_t(3, dtype=torch.float16)]), TypeError),
    (lambda: O.gs_clip_grads([], None, _t(1), 1.0, _t(1, dtype=torch.uint8)), TypeError),
])
def test_binding_refuses(call, kind):
    with pytest.raises(kind):
        call()


def test_no_gradients_is_no_call():
    assert O.clip_grads([torch.nn.Parameter(_t(3))], 1.0) is None


def test_rows_q8_shapes():
    for dim, cols, groups in ((1, 128, 4), (128, 128, 4), (129, 256, 4), (512, 512, 4), (513, 640, 8)):
        q, scales = L.rows_q8(3, dim, "cpu")
        assert q.shape == (3, cols) and scales.shape == (3, groups)


def test_calls_switch_to_the_tensors_device(monkeypatch):
    """The default stream's handle is the same on every device: a call on another one than the current is made there."""
    seen = []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            seen.append(("enter", self.index))

        def __exit__(self, *_):
            seen.append(("leave", self.index))

    class Library:
        @staticmethod
        def gs_quantize_q8(*args):
            seen.append(args)
            return raster.GS_OK

    monkeypatch.setattr(L, "load_library", Library)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)
    L._call("gs_quantize_q8", 0, 1, 2)
    L._call("gs_quantize_q8", 1, 3, 4)
    assert seen == [(1, 2), ("enter", 1), (3, 4), ("leave", 1)]
