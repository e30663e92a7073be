"""The residual norm's workspace (no GPU): a row of float32 sums for each block there can be, and no more."""
import pytest
import torch

from differentiable_gaussian_splat_amd import labels as L

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dim,dtype,blocks", [(1, F32, 1024), (64, BF16, 1024), (4096, F32, 1024), (4097, F32, 256),
                                              (8192, BF16, 1024), (8193, BF16, 256), (65_536, F32, 256),
                                              (65_536, BF16, 256)], ids=str)
def test_workspace_holds_the_blocks_sums(dim, dtype, blocks):
    whole = lambda n: (n * dim * 4 + 255) // 256 * 256
    for n in (0, 1, 7, blocks, blocks + 1, 1 << 20):
        assert L.gs_rms_norm_bwd_workspace_size(n, dim, dtype) == whole(min(n, blocks))
