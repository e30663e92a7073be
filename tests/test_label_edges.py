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
