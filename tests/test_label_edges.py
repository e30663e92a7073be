"""Arguments of the label-learning calls that once passed or failed otherwise (no GPU)."""
import pytest
import torch

from differentiable_gaussian_splat_amd import labels as L
from tests.test_labels_refusals import EMBED_BWD, EMBED_FWD, INVALID, err, lib


@pytest.mark.parametrize("scale", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("fn,base", [("gs_embed_fwd", EMBED_FWD), ("gs_embed_bwd", EMBED_BWD)])
def test_lookup_refuses_a_scale_that_is_no_finite_number(fn, base, scale):
    """Zero rows (no code, or a row that no code names) would be zero or no number, by the size of the call."""
    assert getattr(lib(), fn)(*dict(base, scale=scale).values()) == INVALID
    assert "scale" in err() and fn in err()


@pytest.mark.parametrize("ids", [torch.tensor(3), torch.zeros((3, 1), dtype=torch.int64)], ids=["no dimension", "two"])
def test_lookup_refuses_indices_that_are_no_vector(ids):
    table = torch.zeros((5, 4))
    with pytest.raises(ValueError, match="ids must be a contiguous vector"):
        L._index("ids", ids, ids.numel(), -1)
    with pytest.raises((ValueError, TypeError)):  # here the table's device comes first
        L.embed(table, ids)
