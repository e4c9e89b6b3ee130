"""Shared prefixes over batches of more requests than the partitioner has threads (1024)."""
import pytest

from prefix_case import PrefixCase


@pytest.mark.gpu
@pytest.mark.parametrize("kind,p", [("bf16", dict(p_bits=8, p_floor=0.0)), ("e4m3", {}), ("fp4", {})])
@pytest.mark.parametrize("sizes,shared,own,qs,gap", [([1300], [260], [1, 40, 70], [1], 0), ([700, 3, 900], [200, 500, 130], [3, 90], [1, 2], 9)])
def test_many_requests(kind, p, sizes, shared, own, qs, gap):
    c = PrefixCase(kind, 64, sizes, shared, own, qs, 16, gap=gap, seed=sum(sizes)).run()
    c.check(**p)
    assert c.shares()
