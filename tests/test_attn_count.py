"""The cases that count tokens do see one that is lost (CPU)."""
import pytest
import torch

from tests import _attn_count as count


@pytest.mark.parametrize("D,n,spread", [(128, 60001, 0), (64, 70001, 8), (256, 30001, 8), (128, 17, 8), (64, 5000, 0)])
def test_a_lost_token_is_more_than_the_bound(D, n, spread):
    for lost in (0, 15, 16, 4095, 8191, 8192, 16384, n // 2, n - 1):
        if lost >= n:
            continue
        at = lost // count.chunk(D) * count.chunk(D)
        want, _ = count.counts(n, 0, at, 1, D, spread)
        less, _ = count.counts(n, 0, at, 1, D, spread, lost=lost)
        assert bool(((want - less).abs() > 3 * count.bound(want)).any()), lost
    assert int(torch.bincount(count.column(torch.arange(count.chunk(D)), 3, D)).max()) == count.SHARED
