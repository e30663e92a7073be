"""The residual norm over the range of its types, against 64 bits (tolerances as in test_gpu_residual)."""
import pytest
import torch

from differentiable_gaussian_splat_amd import labels as L

from .test_gpu_labels import BF16, DEV, F32, IDS, TYPES, U, empty, gen, half_step, randn, within
from .test_gpu_residual import CHAIN, check_rms, dequantize, filled_q8, rms_ref

pytestmark = pytest.mark.gpu

DIMS = [3, 64, 100, 771, 1024, 4096, 8200, 20_001, 65_536]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("power", [100, 64, 60, -38, -50, -66, -75, -100])
@pytest.mark.parametrize("dim", DIMS)
def test_large_and_small_rows(dim, power, dtype):
    """Rows whose squares float32 does not hold, between others, with their gradients."""
    g = gen(dim + power)
    n = 37
    x, res = randn(g, n, dim, dtype=dtype), randn(g, n, dim, dtype=dtype)
    size = torch.where(torch.arange(n, device=DEV) % 3 == 1, 1.0, 2.0 ** power)[:, None].to(dtype)
    w, dy = randn(g, 1, dim, dtype=dtype)[0], randn(g, n, dim, dtype=dtype)
    check_rms(x * size, w, res * size, dy, None, 0.0)
    check_rms(x * size, None, None, dy, None, 0.0 if power < 0 else 1e-6)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("power", [125, -126, -140])
@pytest.mark.parametrize("dim", DIMS)
def test_results_at_the_ends_of_the_type(dim, power, dtype):
    """Rows of almost the largest numbers, and of subnormal ones: the result, in its type and in 8 bits."""
    g = gen(dim - power)
    n, power = 21, power if dtype is F32 else max(power, -128)  # bfloat16 has no smaller rows
    v = randn(g, n, dim).clamp(-3.9, 3.9).double() * 2.0 ** power
    x = torch.where(torch.arange(n, device=DEV)[:, None] % 5 == 2, v * 2.0 ** -power, v).to(dtype)
    x[:, 0] = torch.where(x[:, 0] == 0, x[2, 0] * 2.0 ** power, x[:, 0])  # no row of zeros
    w = randn(g, 1, dim, dtype=dtype)[0]
    y = empty(n, dim, dtype=dtype)
    L.gs_rms_norm_fwd(x, w, y, eps=0.0)
    _, _, ref = rms_ref(x, w, None, 0.0)
    e = (CHAIN / 2 + 4) * U
    within("y", y, ref, ref.abs() * (e + 2 * U + half_step(dtype)))
    q, scales = filled_q8(n, dim)
    L.gs_rms_norm_q8(x, w, q, scales, eps=0.0)
    cols = q.shape[1]
    blocks = torch.nn.functional.pad(ref, (0, cols - dim)).reshape(n, -1, 128)
    s = scales.double()[:, :cols // 128]
    assert (blocks.abs().amax(2) <= 448 * s * (1 + e + 2 * U)).all()
    tol = (blocks.abs() * (2.0 ** -4 + e + 2 * U) + s[..., None] * 2.0 ** -10).reshape(n, cols)
    within("values", dequantize(q, scales), blocks.reshape(n, cols), tol)


def test_what_is_no_number_stays_in_its_row():
    """Infinite values, NaN and rows of zeros without eps, beside rows that are summed again."""
    x = torch.ones((6, 700), device=DEV) * 1e30
    x[1, 3] = float("inf")
    x[2, 5] = float("nan")
    x[3] = 0
    x[4] = 1e-30
    y, rstd = empty(6, 700), empty(6)
    L.gs_rms_norm_fwd(x, None, y, None, None, rstd, 0.0)
    for r in (0, 4, 5):
        assert (y[r] - 1).abs().max() <= (CHAIN / 2 + 6) * U
    assert y[1, 3].isnan() and (y[1, 4:] == 0).all() and rstd[1] == 0
    assert y[2].isnan().all() and y[3].isnan().all()
