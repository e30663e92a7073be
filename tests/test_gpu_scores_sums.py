"""How the 8-bit scores are summed where large products cancel, against 64 bits (tolerances as in test_gpu_residual)."""
import pytest
import torch

from .test_gpu_labels import BF16, DEV, F32
from .test_gpu_residual import E8, Q8, check_scores

pytestmark = pytest.mark.gpu

ONE = 127  # the byte of a scale of 1


def pairs(n, cols, small):
    """448 * 448 and -448 * 448 in the first two columns of every eight, `small` * 1 in the other six."""
    a, b = torch.full((n, cols), 1.0, device=DEV), torch.full((n, cols), float(small), device=DEV)
    for k in (0, 1):
        a[:, k::8], b[:, k::8] = 448, 448 * (-1) ** k
    one = torch.full((n, (cols // 128 + 3) // 4 * 4), ONE, dtype=torch.uint8, device=DEV).view(E8)
    return (a.to(Q8), one), (b.to(Q8), one)


@pytest.mark.parametrize("n,cols", [(3, 128), (64, 256), (300, 1024), (3000, 256)])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_sums_that_cancel(n, cols, dtype):
    """Within the bound that the type's sums have. In float32 the units add whole products, and the sum of at most 768
    ones is a number of it; in bfloat16 448 * 448, of 2^17 to 2^18, leaves what is above 2^4 of the others."""
    rows, words = pairs(n, cols, 1)
    out = check_scores(rows, words, dtype)
    if dtype is BF16:
        assert (out == 0).all()
        rows, words = pairs(n, cols, 64)
        assert (check_scores(rows, words, dtype) == 64 * cols / 8 * 6).all()
