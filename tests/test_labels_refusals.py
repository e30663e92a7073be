"""Refusals of the label-learning calls (no GPU): the C ABI checks its
arguments before any HIP call, the binding checks shapes, types and devices."""
import ctypes as C

import pytest
import torch

from differentiable_gaussian_splat_amd import labels as L
from differentiable_gaussian_splat_amd import raster

INVALID, UNSUPPORTED, OK = raster.GS_ERR_INVALID_ARG, raster.GS_ERR_UNSUPPORTED, raster.GS_OK
D = C.c_void_p(4096)  # never dereferenced: validation fails first
BIG = 1 << 60


def lib():
    return raster.load_library()


def err():
    return lib().gs_last_error().decode()


EMBED_FWD = dict(n=4, dim=8, vocab=10, dtype=0, table=D, ts=8, ids=D, it=0, scale=1.0, out=D, os=8, stream=None)
EMBED_BWD = dict(n=4, dim=8, vocab=10, dtype=0, ids=D, it=1, scale=1.0, dout=D, ds=8, dtable=D, ts=8, ws=D, wb=BIG,
                 stream=None)
NORM_FWD = dict(n=4, dim=8, dtype=1, x=D, xs=8, w=D, b=D, eps=1e-5, y=D, ys=8, mean=D, rstd=D, stream=None)
NORM_BWD = dict(n=4, dim=8, dtype=1, x=D, xs=8, w=D, mean=D, rstd=D, dy=D, dys=8, dx=D, dxs=8, dw=D, db=D, ws=D,
                wb=BIG, stream=None)
LOSS_FWD = dict(n=4, dim=8, vocab=10, dtype=0, x=D, xs=8, w=D, ws_=8, labels=D, it=0, loss=D, lse=D, mean=D, count=D,
                ws=D, wb=BIG, stream=None)
LOSS_BWD = dict(n=4, dim=8, vocab=10, dtype=0, x=D, xs=8, w=D, ws_=8, labels=D, it=0, lse=D, dmean=D, dloss=D, dx=D,
                dxs=8, dw=D, dws=8, ws=D, wb=BIG, stream=None)
P1 = C.c_void_p(4097)
P4 = C.c_void_p(4100)

REFUSED = [
    ("gs_embed_fwd", EMBED_FWD, dict(n=-1), INVALID, "n must be"),
    ("gs_embed_fwd", EMBED_FWD, dict(n=(1 << 30) + 1), INVALID, "n must be"),
    ("gs_embed_fwd", EMBED_FWD, dict(dim=0), INVALID, "dim"),
    ("gs_embed_fwd", EMBED_FWD, dict(dim=65537), INVALID, "dim"),
    ("gs_embed_fwd", EMBED_FWD, dict(vocab=0), INVALID, "vocab"),
    ("gs_embed_fwd", EMBED_FWD, dict(dtype=2), UNSUPPORTED, "dtype"),
    ("gs_embed_fwd", EMBED_FWD, dict(it=2), UNSUPPORTED, "index_type"),
    ("gs_embed_fwd", EMBED_FWD, dict(ids=None), INVALID, "index array"),
    ("gs_embed_fwd", EMBED_FWD, dict(ids=P4, it=1), INVALID, "misaligned index"),
    ("gs_embed_fwd", EMBED_FWD, dict(table=None), INVALID, "table"),
    ("gs_embed_fwd", EMBED_FWD, dict(table=P1), INVALID, "misaligned table"),
    ("gs_embed_fwd", EMBED_FWD, dict(ts=7), INVALID, "stride"),
    ("gs_embed_fwd", EMBED_FWD, dict(ts=-8), INVALID, "stride"),
    ("gs_embed_fwd", EMBED_FWD, dict(out=None), INVALID, "out"),
    ("gs_embed_fwd", EMBED_FWD, dict(os=0), INVALID, "stride"),
    ("gs_embed_bwd", EMBED_BWD, dict(dout=None), INVALID, "dout"),
    ("gs_embed_bwd", EMBED_BWD, dict(dtable=None), INVALID, "dtable"),
    ("gs_embed_bwd", EMBED_BWD, dict(ts=0), INVALID, "stride"),
    ("gs_embed_bwd", EMBED_BWD, dict(wb=8), INVALID, "workspace too small"),
    ("gs_embed_bwd", EMBED_BWD, dict(ws=None), INVALID, "workspace"),
    ("gs_embed_bwd", EMBED_BWD, dict(ws=P4), INVALID, "256-byte"),
    ("gs_layer_norm_fwd", NORM_FWD, dict(eps=-1e-5), INVALID, "eps"),
    ("gs_layer_norm_fwd", NORM_FWD, dict(eps=float("nan")), INVALID, "eps"),
    ("gs_layer_norm_fwd", NORM_FWD, dict(x=None), INVALID, "x must"),
    ("gs_layer_norm_fwd", NORM_FWD, dict(y=None), INVALID, "y must"),
    ("gs_layer_norm_fwd", NORM_FWD, dict(x=P1), INVALID, "misaligned x"),
    ("gs_layer_norm_fwd", NORM_FWD, dict(mean=P1), INVALID, "misaligned mean"),
    ("gs_layer_norm_fwd", NORM_FWD, dict(dtype=-1), UNSUPPORTED, "dtype"),
    ("gs_layer_norm_bwd", NORM_BWD, dict(mean=None), INVALID, "mean and rstd"),
    ("gs_layer_norm_bwd", NORM_BWD, dict(dy=None), INVALID, "dy"),
    ("gs_layer_norm_bwd", NORM_BWD, dict(dxs=4), INVALID, "stride"),
    ("gs_layer_norm_bwd", NORM_BWD, dict(wb=16), INVALID, "workspace too small"),
    ("gs_label_loss_fwd", LOSS_FWD, dict(w=None), INVALID, "w must"),
    ("gs_label_loss_fwd", LOSS_FWD, dict(labels=None), INVALID, "index array"),
    ("gs_label_loss_fwd", LOSS_FWD, dict(loss=None), INVALID, "loss and lse"),
    ("gs_label_loss_fwd", LOSS_FWD, dict(mean=None), INVALID, "mean and count"),
    ("gs_label_loss_fwd", LOSS_FWD, dict(wb=0), INVALID, "workspace too small"),
    ("gs_label_loss_fwd", LOSS_FWD, dict(vocab=(1 << 30) + 1), INVALID, "vocab"),
    ("gs_label_loss_bwd", LOSS_BWD, dict(dmean=None, dloss=None), INVALID, "dmean and dloss"),
    ("gs_label_loss_bwd", LOSS_BWD, dict(lse=None), INVALID, "lse"),
    ("gs_label_loss_bwd", LOSS_BWD, dict(dws=7), INVALID, "stride"),
    ("gs_label_loss_bwd", LOSS_BWD, dict(wb=1024), INVALID, "workspace too small"),
]


@pytest.mark.parametrize("fn,base,change,code,text", REFUSED, ids=[f"{r[0]}-{'-'.join(r[2])}" for r in REFUSED])
def test_c_call_refuses(fn, base, change, code, text):
    assert getattr(lib(), fn)(*dict(base, **change).values()) == code
    assert text in err() and fn in err()


def test_empty_calls_need_no_arrays():
    """n = 0: nothing to look up or normalise (the calls return before any HIP call)."""
    a = dict(EMBED_FWD, n=0, ids=None, out=None)
    assert lib().gs_embed_fwd(*a.values()) == OK
    a = dict(NORM_FWD, n=0, x=None, y=None, mean=None, rstd=None)
    assert lib().gs_layer_norm_fwd(*a.values()) == OK
    a = dict(LOSS_BWD, dx=None, dw=None)
    assert lib().gs_label_loss_bwd(*a.values()) == OK


def test_workspace_sizes():
    f32, bf = torch.float32, torch.bfloat16
    assert L.gs_embed_bwd_workspace_size(0, 8, 10, f32) == 0
    assert L.gs_embed_bwd_workspace_size(1000, 8, 10, f32) >= 4 * 4 * 1000
    assert L.gs_layer_norm_bwd_workspace_size(1 << 20, 64, bf) >= 2 * 64 * 4
    small, large = (L.gs_label_loss_workspace_size(n, 64, 1000, bf, True) for n in (100, 100_000))
    assert 0 < small < large and small % 256 == 0
    # the pieces of the vocabulary bound the workspace far below a matrix of logits
    assert L.gs_label_loss_workspace_size(1 << 16, 64, 1 << 20, bf, True) < (1 << 36) // 16
    for bad in ((-1, 8, 10), (5, 0, 10), (5, 8, 0)):
        assert L.gs_embed_bwd_workspace_size(*bad, f32) == 0
        assert L.gs_label_loss_workspace_size(*bad, f32, True) == 0
    with pytest.raises(TypeError):
        L.gs_embed_bwd_workspace_size(10, 8, 10, torch.float16)


def _t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def _i(n, dtype=torch.int64):
    return torch.zeros(n, dtype=dtype)


@pytest.mark.parametrize("call,kind", [
    (lambda: L.gs_embed_fwd(_t(5, 4), _i(3), _t(3, 4)), TypeError),                       # not on the GPU
    (lambda: L.gs_embed_fwd(_t(5, 4, dtype=torch.float16), _i(3), _t(3, 4)), TypeError),
    (lambda: L.gs_embed_fwd(_t(4, 5).t(), _i(3), _t(3, 4)), ValueError),                   # columns apart
    (lambda: L.embed(_t(5, 4), _t(3), 1.0), TypeError),
    (lambda: L.layer_norm(_t(5)), ValueError),
    (lambda: L.gs_layer_norm_fwd(_t(3, 4), None, None, _t(3, 4)), TypeError),
    (lambda: L.label_loss(_t(3, 4), _t(5, 4), _i(3), reduction="max"), ValueError),
    (lambda: L.label_loss(_t(3, 4), _t(5, 4), _i(3)), TypeError),
])
def test_binding_refuses(call, kind):
    with pytest.raises(kind):
        call()


def test_binding_refuses_mismatched_shapes():
    assert L._matrix.__doc__
    with pytest.raises(ValueError):
        L._matrix("out", _t(3, 4), _t(2, 4), 2, 4)
    with pytest.raises(TypeError):
        L._matrix("out", _t(3, 4), _t(3, 4, dtype=torch.bfloat16), 3, 4)
    with pytest.raises(ValueError):
        L._vector("weight", _t(3), 4, torch.float32, -1)
    with pytest.raises(TypeError):
        L._index("ids", _i(3, torch.int16), 3, -1)
    with pytest.raises(ValueError):
        L._index("ids", _i(4), 3, -1)
