"""The order of a selection where scores are equal or nearly so, and how near its normaliser is.

A row's normaliser is its largest logit plus the logarithm of the sum of its terms over the largest
one's own.  Terms of e^-60 and less vanish beside it, so the sum of a row with one logit far above the
others is that logit's term and the quotient 1: such rows' scores are their beams' to the bit.  In
any row a term is off by an exponential's 2^-22, its own argument's rounding (ln 2 times 2^-23 of an
argument of at most some 16 where it counts) and the largest term's 2^-22, and chains of ten sums
by 2^-24 each: 2^-18 bounds them together, were all roundings one way; half of it is asked."""
import math

import numpy as np
import pytest
import torch

import paged_mla_decode_03_gb300 as mla

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def placed(x, offs):
    """The rows of x [W, V] each `offs` values past a 16-byte boundary -> [1, W, V] by a stride that does so."""
    W, V = x.shape
    step = -(-V // 64) * 64 + offs
    flat = torch.zeros(W * step + 64, dtype=x.dtype, device="cuda")
    out = flat.as_strided((1, W, V), (W * step, step, 1))
    out.copy_(x)
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V,W,k,offs", [(50257, 4, 16, 0), (50257, 8, 13, 1), (100003, 8, 64, 3), (20011, 16, 24, 5), (777, 8, 20, 7),
                                        (13, 9, 30, 2), (131071, 8, 5, 1), (4099, 8, 9, 3)])
def test_equal_beams_come_by_index_wherever_their_rows_start(kind, V, W, k, offs):
    g = torch.Generator().manual_seed(V + W)
    row = (torch.randn(V, generator=g) * 3).to(TYPES[kind]).cuda()
    x = placed(row.expand(W, V), offs)
    # the best tokens by logit (of equal ones the lowest), and for each every beam in turn
    order = np.lexsort((np.arange(V), -row.double().cpu().numpy()))
    want = sorted(((-float(row[v]), w, int(v)) for v in order[:k] for w in range(W)))[:k]
    for c in (-1.5, 0.0, -1e-3):
        s, t, p = (y[0].cpu() for y in mla.beam_select(x, torch.full((1, W), c, device="cuda"), k=k))
        assert [(int(w), int(v)) for w, v in zip(p, t)] == [(w, v) for _, w, v in want]
        same = {}
        for j in range(len(want)):  # one score for one logit
            assert same.setdefault(want[j][0], float(s[j])) == float(s[j])
        assert (s[len(want):] == -math.inf).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
def test_contiguous_rows_of_an_odd_vocabulary(kind):
    # (each row starts elsewhere; the beams of a request are the same, of another request others)
    B, W, V, k = 3, 5, 50257, 11
    g = torch.Generator().manual_seed(3)
    row = (torch.randn(B, 1, V, generator=g) * 2).to(TYPES[kind])
    x = row.expand(B, W, V).contiguous().cuda()
    s, t, p = (y.cpu() for y in mla.beam_select(x, torch.full((B, W), -3.0, device="cuda"), k=k))
    for b in range(B):
        r = row[b, 0].double().numpy()
        order = np.lexsort((np.arange(V), -r))[:k]
        want = sorted((-float(r[v]), w, int(v)) for v in order for w in range(W))[:k]
        assert [(int(w), int(v)) for w, v in zip(p[b], t[b])] == [(w, v) for _, w, v in want]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V,offs", [(1, 1), (2, 1), (33, 3), (5003, 1), (50257, 0), (100003, 2)])
def test_rows_with_one_likely_token_have_their_beams_scores(kind, V, offs):
    W = 8
    g = torch.Generator().manual_seed(V)
    top = (torch.rand(W, generator=g) * 20 - 10).to(TYPES[kind])
    at = torch.randint(0, V, (W,), generator=g)
    x = (top.float()[:, None] - 60 - 5 * torch.rand(W, V, generator=g)).to(TYPES[kind])
    x[torch.arange(W), at] = top
    # scores next to one another: half a step of 2^-20 or less between two beams, in mixed order
    c = -0.5 - torch.randperm(W, generator=g).float() * 2.0 ** -24
    s, t, p = (y[0].cpu() for y in mla.beam_select(placed(x.cuda(), offs), c[None].cuda(), k=W))
    order = torch.argsort(-c)
    assert torch.equal(p.long(), order) and torch.equal(t.long(), at[order]) and torch.equal(s, c[order])


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("shape", ["flat", "slope", "two", "near", "usual", "far"])
def test_the_normaliser_is_near(kind, shape):
    """Scores of about 0, so that fp32 shows the normaliser's own error."""
    V, W = 40009, 32
    g = torch.Generator().manual_seed(11)
    if shape == "flat":    # all equal but one
        x = torch.full((W, V), 0.3) + torch.arange(W)[:, None] * 0.37
        x[:, 5] += 1.0
    elif shape == "slope":  # ever larger: every chunk a new maximum
        x = torch.linspace(-1, 0, V) * (1 + torch.arange(W))[:, None] * 0.2 + torch.arange(W)[:, None]
    elif shape == "two":
        x = torch.full((W, V), -50.0)
        x[:, 7], x[:, 30001] = 1.0 + 0.1 * torch.arange(W), 1.3 + 0.05 * torch.arange(W)
    elif shape == "near":  # most of the sum some 8 below the largest
        x = torch.randn(W, V, generator=g) * 0.1 - 8
        x[:, 100] = 0.0
        x += torch.rand(W, 1, generator=g) * 5
    elif shape == "usual":
        x = torch.randn(W, V, generator=g) * 3
    else:                  # 1e6: still by powers of two
        x = (torch.randn(W, V, generator=g) * 2).round() + 1e6 * (kind != "fp16")
    x = x.to(TYPES[kind])
    lse = torch.logsumexp(x.double(), -1)
    top, at = x.double().max(-1)
    c = (lse - top).float()  # the best score is c + top - lse, nearly 0
    x = placed(x.cuda(), 1)
    for w in range(0, W, 4):
        s, t, _ = mla.beam_select(x[:, w:w + 1], c[w:w + 1, None].contiguous().cuda(), k=1)
        want = float(c[w].double() + top[w] - lse[w])
        assert abs(float(s) - want) <= 2.0 ** -19 + 2.0 ** -24 * abs(want), (w, float(s), want)


@pytest.mark.gpu
def test_results_hang_on_no_alignment():
    """The same rows at each offset from 16 bytes, to the bit."""
    for kind in ("fp32", "bf16", "fp16"):
        g = torch.Generator().manual_seed(21)
        x = (torch.randn(4, 30011, generator=g) * 3).to(TYPES[kind]).cuda()
        c = -torch.rand(1, 4, generator=g).cuda()
        base = torch.zeros(4 * 30016 + 64, dtype=x.dtype, device="cuda")
        first = None
        for off in range(8):
            y = base[off:].as_strided((1, 4, 30011), (4 * 30016, 30016, 1), off)
            y.copy_(x)
            got = mla.beam_select(y, c, k=32)
            torch.cuda.synchronize()
            first = first or got
            assert all(torch.equal(a, b) for a, b in zip(first, got)), (kind, off)


def near_logits(kind, step, k, W, n):
    """Rows with n tokens of logits base + step * (0 .. 199), the others far below."""
    g = torch.Generator().manual_seed(k)
    V = 20011
    x = torch.randn(1, W, V, generator=g) * 0.1 - 3
    base = 0 if step < 2.0 ** -20 else 1
    for w in range(W):
        x[0, w, torch.randperm(V, generator=g)[:n]] = base + step * torch.arange(n).remainder(200)
    return x.to(TYPES[kind])


@pytest.mark.gpu
@pytest.mark.parametrize("kind,step,k", [("fp32", 2.0 ** -20, 1), ("fp32", 2.0 ** -20, 7), ("fp32", 2.0 ** -20, 64), ("bf16", 2.0 ** -8, 1),
                                         ("bf16", 2.0 ** -8, 7), ("fp16", 2.0 ** -11, 1), ("fp16", 2.0 ** -11, 7)])
def test_beams_of_one_large_score_come_by_what_they_add(kind, step, k):
    """40 beams of -1e30: 64 bits do not tell their continuations apart, pairs of floats do."""
    W = 40
    x = near_logits(kind, step, k, W, 900)
    got = mla.beam_select(x.cuda(), torch.full((1, W), -1e30, device="cuda"), k=k)
    d = x[0].double()
    d = (d - torch.logsumexp(d, -1, keepdim=True)).numpy()
    rows = [(-d[w, v], w, int(v)) for w in range(W) for v in np.lexsort((np.arange(d.shape[1]), -d[w]))[:k + 1]]
    rows.sort()
    assert all(a[1] == b[1] or b[0] - a[0] > 2.0 ** -19 for a, b in zip(rows[:k], rows[1:k + 1])), "an open order"
    s, t, p = (y[0].cpu() for y in got)
    assert [(int(w), int(v)) for w, v in zip(p, t)] == [(w, v) for _, w, v in rows[:k]]


@pytest.mark.gpu
@pytest.mark.parametrize("kind,step", [("fp32", 2.0 ** -30), ("bf16", 2.0 ** -30), ("fp16", 2.0 ** -24)])
@pytest.mark.parametrize("k", [1, 7, 64])
@pytest.mark.parametrize("many", [False, True])
def test_tokens_of_a_beam_come_by_logit_whatever_its_score(kind, step, k, many):
    """Beside a score of -1e9, logits that differ little make scores that are the same in 48 bits.
    (many: 40 beams that are the same, whose candidates are more than the join has room for.)"""
    W = 40 if many else 3
    x = near_logits(kind, step, k, W, 900 if many else 100)
    c = -1e9 * torch.arange(1, W + 1).float()[None]
    if many:
        x, c = x[:, :1].expand(-1, W, -1).contiguous(), torch.full((1, W), -1e9)
    by_logit = [np.lexsort((np.arange(x.shape[2]), -x[0, w].double().numpy())) for w in range(W)]

    def each_in_order():
        s, t, p = (y[0].cpu() for y in mla.beam_select(x.cuda(), c.cuda(), k=k))
        for w in set(p.tolist()):
            mine = t[p == w].tolist()
            assert mine == [int(v) for v in by_logit[w][:len(mine)]]
        return set(p.tolist())

    # (of beams that are the same, logits whose scores 48 bits tell apart come by turns: 200 steps of
    # 2^-24 are some 25 of a score's)
    assert each_in_order() == {0} or many
    c[0, 1] = c[0, 0]  # two beams of one score
    assert each_in_order() <= {0, 1} or many
