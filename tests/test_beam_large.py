"""Selection over the largest vocabulary, 2^28 tokens, cut into parts and in one."""
import math

import pytest
import torch

import paged_mla_decode_03_gb300 as mla

V = 1 << 28


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 640])  # (640 rows are a part each: 2^20 values a thread; one row, repeated)
def test_the_largest_vocabulary(rows):
    x = torch.full((V,), -5.0, dtype=torch.bfloat16, device="cuda")
    places = [V - 1, 12345, V // 2 + 1]
    x[places] = torch.tensor([1.0, 0.5, 0.25], dtype=torch.bfloat16, device="cuda")
    c = -torch.arange(rows, dtype=torch.float32, device="cuda")[:, None] / 1024
    s, t, p = mla.beam_select(x.expand(rows, 1, V), c, k=5)
    lse = math.log((V - 3) * math.exp(-5.0) + sum(math.exp(v) for v in (1.0, 0.5, 0.25)))
    assert (p == 0).all() and (t == torch.tensor(places + [0, 1], device="cuda")).all()
    for j, v in enumerate((1.0, 0.5, 0.25, -5.0, -5.0)):
        want = c.double()[:, 0] + v - lse
        # lse 2^-18 (tests/test_beam_order.py), and a score's rounding to fp32
        assert ((s[:, j].double() - want).abs() <= 2.0 ** -18 + want.abs() * 2.0 ** -24).all()
    # all the same: 2^20 terms of a thread are each the largest
    x.fill_(3.0)
    s, t, p = mla.beam_select(x.expand(rows, 1, V), c, k=5)
    assert (t == torch.arange(5, device="cuda")).all()
    want = c.double()[:, 0] - math.log(V)
    assert ((s.double() - want[:, None]).abs() <= 2.0 ** -18 + want.abs()[:, None] * 2.0 ** -24).all()
