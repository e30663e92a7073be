"""What the 8-bit scores refuse beside test_residual_refusals (no GPU)."""
import pytest

from .test_residual_refusals import INVALID, SCORES, lib


@pytest.mark.parametrize("n,vocab", [(1 << 30, 1025), (1 << 20, (1 << 20) + 1), (1 << 30, 1 << 30)])
def test_more_scores_than_a_launch_numbers(n, vocab):
    """Tiles are numbered in 32 bits: sizes that no memory holds are refused, not split."""
    assert lib().gs_label_scores_q8(*dict(SCORES, n=n, vocab=vocab, os=vocab).values()) == INVALID
    assert "2^40 scores" in lib().gs_last_error().decode()
