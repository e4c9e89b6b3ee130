"""Shared rows that are widened: long enough ones behind enough query rows, so that the partitioner
does widen them (its work list is looked at), against the plain 64-bit form."""
import math

import pytest
import torch

import paged_mla_decode_03_gb300 as mla
from prefix_case import PrefixCase

CASES = [  # page, group sizes, shared rows, own rows, query lengths, heads, options
    (64, [32], [20000], [5, 100], [1], 128, dict(uniform=True)),
    (32, [32], [20033], [0], [1], 128, {}),                                        # none has a row of its own
    (32, [40, 2, 50], [9000, 4000, 7000], [3, 140], [3, 1, 2], 64, dict(gap=2, pad=1)),  # one group is not widened
    (64, [40], [16384], [64, 3], [2], 64, dict(causal=False, q_fp8=True)),
    (64, [128], [9000], [64, 3], [1], 32, dict(same_pages=False)),
]


def widened(c):
    """Whether the first list leaves shared rows out: what the largest group's row groups would walk."""
    items = c.items()
    walked = max(sum(q for q, of in zip(c.qs, c.group_of) if of == g) * c.heads // 128 * p for g, p in enumerate(c.shared))
    return int((items[:, 3] - items[:, 2]).sum()) < walked // 2


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["e4m3", "fp4"])
@pytest.mark.parametrize("ps,sizes,shared,own,qs,heads,kw", CASES)
def test_widened_rows(kind, ps, sizes, shared, own, qs, heads, kw):
    c = PrefixCase(kind, ps, sizes, shared, own, qs, heads, seed=heads + sum(sizes), **kw)
    c.workspace.fill_(0xFF)
    c.run().check()
    assert widened(c)
    first = c.out.clone(), c.lse.clone()
    c.workspace.fill_(0x7F)
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(first[0].view(torch.int16), c.out.view(torch.int16)) and torch.equal(first[1], c.lse)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["e4m3", "fp4"])
def test_a_graph_whose_lengths_change(kind):
    c = PrefixCase(kind, 64, [32], [20000], [5, 100], [1], 128, uniform=True, seed=40)
    c.run().check()
    assert widened(c)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for lens, wide in (([19000], True), ([0], False), ([700], False), ([19999], True)):
        c.prefix_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        c.workspace.fill_(0xFF)
        c.out.fill_(3.0)
        g.replay()
        c.check()
        assert widened(c) == wide
    # a page of the widened rows that is none: zeros, and flagged
    page = int(c.tables[0, 3])
    c.tables[:, 3] = -1
    g.replay()
    c.tables[:, 3] = page
    c.cache[page].zero_()
    c.check(status=16)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["e4m3", "fp4"])
def test_values_that_are_none(kind):
    """A NaN in a widened row reaches all that share it; in a request's own row that request alone."""
    c = PrefixCase(kind, 64, [64], [20000], [70, 100], [1], 64, uniform=True, seed=3)
    c.run().check()
    assert widened(c)
    first = c.out.view(64, 64, 512).clone()
    raw = c.cache.view(torch.uint8).view(c.cache.shape[0], -1)

    def spoil(b, j):
        page, row = int(c.tables[b, j // 64]), j % 64
        at, value = (64 * 288 + row * 36 + 5, 0x7F) if kind == "fp4" else (row * 576 + 77, 0xFF)
        old = int(raw[page, at])
        raw[page, at] = value
        return page, at, old

    page, at, old = spoil(7, 20003)
    c.run()
    torch.cuda.synchronize()
    out = c.out.view(64, 64, 512)
    rest = [b for b in range(64) if b != 7]
    assert torch.equal(out[rest].view(torch.int16), first[rest].view(torch.int16)) and out[7].isnan().all()
    raw[page, at] = old
    spoil(0, 9999)
    c.run()
    torch.cuda.synchronize()
    assert out.isnan().all() and c.lse.isnan().all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["e4m3", "fp4"])
def test_two_runs_at_once(kind):
    a = PrefixCase(kind, 64, [32], [20000], [5, 100], [1], 128, uniform=True, seed=21)
    b = PrefixCase(kind, 32, [40], [16384], [64, 3], [2], 64, seed=22)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        with torch.cuda.stream(s):
            a.run()
        with torch.cuda.stream(t):
            b.run()
    torch.cuda.synchronize()
    a.check()
    b.check()
    assert widened(a) and widened(b)


@pytest.mark.gpu
def test_scales_and_no_lse():
    c = PrefixCase("fp4", 64, [32], [20000], [5], [1], 128, uniform=True, seed=9)
    c.run(bmm1_scale=torch.tensor([c.bmm1], device="cuda"), bmm2_scale=torch.tensor([c.bmm2], device="cuda")).check()
    assert widened(c)
    out = mla.decode(c.query.view(32, 1, 128, 576), c.cache, c.workspace, c.tables, c.lens, c.max_len, bmm1_scale=c.bmm1,
                     bmm2_scale=c.bmm2, prefix_lens=c.prefix_lens)
    assert torch.equal(out.view_as(c.out), c.out) and math.isfinite(float(out.float().sum()))
