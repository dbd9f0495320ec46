"""Joins of results that were split along the keys, where the parts' weights are
hard to hold: logits in steps of up to 256 (test_gpu_attention_large_logits has
the construction and its bound), so that a part's sum counts for nothing beside
its reference."""
import pytest

from test_gpu_attention_large_logits import fa, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("e", [10, 14, 17, 20, 22, 23, 24, 25, 26, 27, 28, 30])
def test_large_logits(fa, e, sign):  # noqa: F811
    """All logits level, so that a part counts by its number of keys; a few steps
    apart; rising from part to part.  Even shares of few and of many parts,
    chunks of few and of many."""
    for n, L, H, Hq, D, bs in ((1, 2000, 1, 2, 64, 64), (2, 1700, 1, 16, 128, 64), (2, 1700, 60, 60, 64, 32),
                               (40, 700, 1, 1, 64, 64), (34, 4500, 1, 1, 64, 32)):
        for rise in ((0, 1), None, (1, 8)):
            if rise != (1, 8) or L <= 8 * 64 * 16:
                run(fa, e, sign, n, L, H, Hq, D, bs, rise=rise)
