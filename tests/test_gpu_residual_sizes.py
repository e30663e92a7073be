"""The residual norm's column sums stay within the workspace that is asked for: long rows, more of them than blocks."""
import pytest
import torch

from differentiable_gaussian_splat_amd import labels as L

from .test_gpu_labels import BF16, DEV, F32, empty, gen, randn
from .test_gpu_residual import check_rms, run_rms

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,dim,dtype", [(1500, 4096, F32), (700, 4097, F32), (300, 20_001, F32), (258, 65_536, F32),
                                         (1200, 8192, BF16), (600, 8193, BF16), (259, 65_536, BF16)], ids=str)
def test_sums_stay_in_the_workspace(n, dim, dtype):
    g = gen(n + dim)
    x, w, dy = randn(g, n, dim, dtype=dtype), randn(g, 1, dim, dtype=dtype)[0], randn(g, n, dim, dtype=dtype)
    want = run_rms(x, w, None, dy, None, 1e-6)
    size = L.gs_rms_norm_bwd_workspace_size(n, dim, dtype)
    room = torch.full((2 * size,), 0x5A, dtype=torch.uint8, device=DEV)
    dx, dw = empty(n, dim, dtype=dtype), empty(dim, dtype=dtype)
    L.gs_rms_norm_bwd(x, w, want["rstd"], dy, dx, dw, room[:size])
    assert torch.equal(dw, want["dw"]) and torch.equal(dx, want["dx"])
    assert (room[size:] == 0x5A).all()
    check_rms(x, w, None, dy, None, 1e-6)
