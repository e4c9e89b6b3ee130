"""Selection over vocabularies that are masked by finite values: most of a row is one value, and more
values than a block has room for pass its threshold."""
import math

import pytest
import torch

import paged_mla_decode_03_gb300 as mla
from test_beam import TYPES, reference


def check(logits, scores, k):
    """As tests/test_beam.py's, with the reference over rows less their largest logit: beside the lowest
    fp32, 64 bits (53 of them) do not hold the logarithm of a sum, and without it the score is the same."""
    got = mla.beam_select(logits, scores, k=k)
    torch.cuda.synchronize()
    x = logits.double()
    want, sure = reference(x - x.amax(-1, keepdim=True), scores, k)
    assert sure, "the inputs leave the order open"
    s, t, p = (y.cpu() for y in got)
    for b, rows in enumerate(want):
        assert [(int(w), int(v)) for w, v in zip(p[b], t[b])][:len(rows)] == [(w, v) for _, w, v in rows], b
        for j, (c, _, _) in enumerate(rows):
            assert abs(float(s[b, j]) - c) <= abs(c) * 2.0 ** -24 + 2.0 ** -21
        assert (s[b, len(rows):] == -math.inf).all() and (t[b, len(rows):] == -1).all() and (p[b, len(rows):] == -1).all()


MASKS = {"lowest": None, "-1e4": -1e4}


def masked(kind, B, W, V, live, mask, seed, pad=0):
    """All but `live` tokens of a row masked, others in each row."""
    g = torch.Generator().manual_seed(seed)
    low = torch.finfo(TYPES[kind]).min if MASKS[mask] is None else MASKS[mask]
    x = torch.full((B, W, V + pad), low)
    at = torch.randint(0, V, (B, W, max(live, 1)), generator=g)
    if live:
        x.scatter_(2, at, torch.randn(B, W, live, generator=g) * 2)
    scores = -torch.rand(B, W, generator=g).cumsum(-1) * 2
    return x.to(TYPES[kind]).cuda()[..., :V], scores.cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("B,V,live,k,pad", [(2, 50257, 3, 8, 0), (650, 20001, 5, 8, 1), (1, 131071, 0, 64, 0), (3, 9001, 40, 64, 7),
                                            (4, 2000, 1, 64, 0), (2, 1 << 20, 2, 5, 0)])
def test_fewer_tokens_than_are_wanted(kind, mask, B, V, live, k, pad):
    # (one beam a request: between two, masked scores of -3e38 are equal whatever the beams' own)
    check(*masked(kind, B, 1, V, live, mask, V + live, pad), k)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
def test_some_beams_of_a_request(kind):
    x, c = masked(kind, 4, 3, 30011, 4, "-1e4", 5, pad=2)
    c[1, 1:] = -math.inf
    check(x, c, 20)
    y, d = masked(kind, 4, 5, 30011, 9, "lowest", 6)
    check(y, d, 12)  # the live ones are enough
    y[:, 0, 10007:] = 3.0  # and most of one row the same large value
    check(y, d, 12)


@pytest.mark.gpu
@pytest.mark.parametrize("k", [2, 20])
def test_many_values_in_few_places(k):
    """The largest values all where a few threads read: the threshold lies below thousands of them."""
    B, V = 640, 65536
    g = torch.Generator().manual_seed(k)
    x = torch.rand(B, 1, V, generator=g)
    few = (torch.arange(V) // 4 % 256) < (8 if k <= 16 else 60)
    x[..., few] += 10
    check(x.cuda(), -torch.rand(B, 1, generator=g).cuda(), k)
