"""What a request's own rows hold reaches no other request of its group: a NaN or an infinity there
leaves the others' outputs as they are, to the bit."""
import math

import pytest
import torch

from prefix_case import PrefixCase


def poison(c, b, j, how):
    """Row j of request b, which is on a page of its own."""
    page, row = int(c.tables[b, j // c.ps]), j % c.ps
    if c.kind == "fp4":
        raw = c.cache.view(c.cache.shape[0], -1)
        at = c.ps * 288 + row * 36
        raw[page, at + {"nan": 3, "rope": 33}[how]] = 0x7F  # a scale, so 16 dims
    elif c.kind == "e4m3":
        c.cache.view(torch.uint8)[page, row, {"nan": 100, "rope": 540}[how]] = 0xFF
    else:
        c.cache[page, row, 540 if how == "rope" else 301] = {"nan": math.nan, "rope": math.nan, "inf": math.inf, "-inf": -math.inf}[how]


CASES = [  # page, group sizes, shared rows, own rows, query lengths, heads, options
    (64, [40], [1000], [1, 70, 33], [1], 16, {}),
    (32, [20, 30], [1500, 2100], [5, 400], [1], 32, {}),
    (64, [30], [2000], [70, 8, 100], [3], 64, {}),                      # they straddle row groups
    (32, [12, 0, 9, 1], [2500, 500, 4001, 300], [4, 1, 300], [1, 2, 3], 64, dict(gap=2, pad=1)),
    (64, [8], [30000], [300, 1200], [1], 16, {}),                       # cut over the workers
    (64, [40], [1300], [20, 130], [2], 16, dict(causal=False, q_fp8=True)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("kind,how", [("bf16", "nan"), ("bf16", "inf"), ("bf16", "-inf"), ("bf16", "rope"), ("e4m3", "nan"),
                                      ("e4m3", "rope"), ("fp4", "nan"), ("fp4", "rope")])
@pytest.mark.parametrize("ps,sizes,shared,own,qs,heads,kw", CASES)
def test_own_rows_reach_no_other_request(kind, how, ps, sizes, shared, own, qs, heads, kw):
    c = PrefixCase(kind, ps, sizes, shared, own, qs, heads, seed=heads + sum(sizes), **kw).run()
    assert c.shares()
    first, lse = c.out.clone(), c.lse.clone()
    bad = [b for b, g in enumerate(c.group_of) if g >= 0 and b % 5 == 1 and c.ls[b] > shared[g] + max(c.qs)]
    assert bad
    for b in bad:
        poison(c, b, shared[c.group_of[b]], how)                # its first own row, which all its tokens see
        if c.ls[b] - c.qs[b] > shared[c.group_of[b]] + 200:
            poison(c, b, c.ls[b] - c.qs[b], how)
    for _ in range(2):
        c.run()
        torch.cuda.synchronize()
        starts = [sum(c.qs[:b]) for b in range(len(c.qs))]
        out, old = c.out.view(-1, heads, 512), first.view(-1, heads, 512)
        now, was = c.lse.view(-1, heads), lse.view(-1, heads)
        for b, q in enumerate(c.qs):
            rows = slice(starts[b], starts[b] + q)
            if b not in bad:
                assert torch.equal(out[rows].view(torch.int16), old[rows].view(torch.int16)), b
                assert torch.equal(now[rows], was[rows]), b
            elif "inf" not in how:
                assert out[rows].isnan().all() and now[rows].isnan().all(), b
            else:
                # a score of +infinity leaves no softmax; one of -infinity is a weight of 0, whose product
                # with the infinity may be a NaN to the request itself, as without sharing
                lost = now[rows].isnan()
                assert lost.any() and out[rows][lost].isnan().all()
                assert out[rows][..., [*range(301), *range(302, 512)]][~lost].isfinite().all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp4"])
def test_shared_rows_reach_all_that_see_them(kind):
    c = PrefixCase(kind, 64, [40, 20], [1000, 700], [1, 70, 33], [1], 16, seed=4).run()
    first = c.out.clone()
    poison(c, 0, 130, "nan")
    c.run()
    torch.cuda.synchronize()
    assert c.out.view(60, 16, 512)[:40].isnan().all() and c.lse.view(60, 16)[:40].isnan().all()
    assert torch.equal(c.out.view(60, -1)[40:], first.view(60, -1)[40:])
