"""A beam search's selection and the reordering of the paged cache, against plain forms.

Selection.  Scores are compared in 64 bits, and the reference's normaliser is in 64 bits.  The
kernel's is off by less than 2^-21 (an exponential's 2^-22 relative, its argument's rounding
2^-25 of at most some 8 in the mean over the distribution, averaged over the terms), so where
the reference's k-th and (k + 1)-th, or any two neighbours, of different beams are nearer than
2^-20 a case says nothing about the order; such a gap in a case is refused as an input.  A
score in fp32 is off by its rounding, 2^-24 of it, and the normaliser's 2^-21."""
import math

import numpy as np
import pytest
import torch

import paged_mla_decode_03_gb300 as mla
from attention_ref import random_cache

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
GAP = 2.0 ** -20


def reference(logits, scores, k, finished=None, end=None):
    """[(score, beam, token)] of each request, and whether its order is beyond doubt."""
    B, W, V = logits.shape
    x, found, sure = logits.double().cpu(), [], True
    for b in range(B):
        rows = []
        for w in range(W):
            c = float(scores[b, w])
            if not math.isfinite(c):
                continue
            if finished is not None and finished[b, w]:
                rows.append((c, w, end))
                continue
            lse = torch.logsumexp(x[b, w], 0)
            if not math.isfinite(float(lse)):
                continue
            # the k + 1 largest logits, of equal ones the lowest tokens
            order = np.lexsort((np.arange(V), -x[b, w].numpy()))[:k + 1]
            rows += [(float(x[b, w, v] - lse) + c, w, int(v)) for v in order if x[b, w, v] > -math.inf]
        rows.sort(key=lambda r: (-r[0], r[1], r[2]))
        for a, c in zip(rows[:k], rows[1:k + 1]):
            if a[1] != c[1] and abs(a[0] - c[0]) < GAP and not _tied(x[b], scores[b], a, c):
                sure = False
        found.append(rows[:k])
    return found, sure


def _tied(x, scores, a, c):
    """Equal by construction: rows with the same logits and scores."""
    return bool(torch.equal(x[a[1]], x[c[1]])) and float(scores[a[1]]) == float(scores[c[1]])


def check(logits, scores, k, finished=None, end=None, **kw):
    got = mla.beam_select(logits, scores, k=k, finished=finished, end_token=end, **kw)
    torch.cuda.synchronize()
    want, sure = reference(logits, scores, k, finished, end)
    assert sure, "the inputs leave the order open"
    s, t, p = (x.cpu() for x in got)
    for b, rows in enumerate(want):
        assert [(int(w), int(v)) for w, v in zip(p[b], t[b])][:len(rows)] == [(w, v) for _, w, v in rows], b
        for j, (c, _, _) in enumerate(rows):
            assert abs(float(s[b, j]) - c) <= abs(c) * 2.0 ** -24 + 2.0 ** -21
        assert (s[b, len(rows):] == -math.inf).all() and (t[b, len(rows):] == -1).all() and (p[b, len(rows):] == -1).all()
    return got


def inputs(kind, B, W, V, seed, spread=3.0, pad=0, off=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, W, V + pad + off, generator=g) * spread
    scores = -torch.rand(B, W, generator=g).cumsum(-1) * 2
    return x.to(TYPES[kind]).cuda()[..., off:off + V], scores.cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("B,W,V,k,pad,off", [
    (1, 1, 1, 1, 0, 0), (1, 1, 1, 3, 0, 0), (2, 3, 2, 5, 0, 0), (1, 4, 33, 4, 1, 0), (3, 2, 100, 64, 0, 3), (1, 4, 8192, 8, 0, 0),
    (2, 4, 16384, 8, 0, 0), (2, 4, 16385, 8, 0, 1), (5, 3, 32768, 6, 7, 0), (1, 8, 100003, 16, 0, 0), (64, 4, 5003, 8, 0, 5),
    (1, 64, 9001, 64, 0, 0), (700, 3, 9, 4, 2, 1), (500, 7, 3, 5, 0, 2), (900, 2, 13, 3, 0, 3), (2, 16, 65537, 32, 3, 2), (300, 5, 1000, 10, 0, 0), (1, 2, 300000, 64, 0, 0)])
def test_select(kind, B, W, V, k, pad, off):
    check(*inputs(kind, B, W, V, 7 * V + k, pad=pad, off=off), k)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("spread", [0.0, 1e-4, 0.3, 30.0])
def test_flat_and_peaked_rows(kind, spread):
    x, c = inputs(kind, 3, 4, 20011, 5, spread=spread)
    check(x, c, 8)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_ties_go_to_the_lowest_beam_and_token(kind):
    x, c = inputs(kind, 2, 4, 40000, 6)
    x = x.clone()
    x[0, 1, 17::100] = 50.0  # 400 equal ones of a row
    x[0, 2, 5:30000] = 40.0  # more than any list holds
    x[1] = x[1, 0]           # beams that are the same
    c[1] = -1.5
    check(x, c, 16)
    check(torch.zeros_like(x), torch.full_like(c, -0.25), 64)
    x[0, :, ::2] = 0.0       # zeros of either sign are equal
    x[0, :, 1::2] = -0.0
    check(x, c, 5)


@pytest.mark.gpu
def test_a_first_step_has_one_beam():
    x, c = inputs("bf16", 4, 8, 30011, 8)
    x = x[:, :1].expand(-1, 8, -1)  # the same row for all beams: stride 0
    c[:, 1:] = -math.inf
    c[:, 0] = 0.0
    _, _, p = check(x, c, 16)
    assert (p == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("flag", [torch.uint8, torch.bool])
def test_ended_beams(flag):
    x, c = inputs("fp32", 5, 6, 12345, 9)
    done = torch.zeros(5, 6, dtype=flag)
    done[0, 0] = done[1, 5] = True
    done[2] = True
    done[3, 1:] = True
    x = x.clone()
    x[0, 0] = math.nan  # not read
    check(x, c, 12, done.cuda(), 77)
    check(x, c, 2, done.cuda(), 0)


@pytest.mark.gpu
def test_masked_and_bad_logits():
    x, c = inputs("fp32", 6, 3, 10007, 10)
    x = x.clone()
    x[0, 0] = -math.inf                # a row that leaves nothing
    x[0, 1, 3:] = -math.inf            # three tokens
    x[1] = -math.inf                   # nothing at all
    x[2, 1, 5000] = math.nan           # no normaliser
    x[2, 2, 9999] = math.inf
    x[3, :, 100:] = torch.finfo(torch.float32).min  # masked by the type's lowest value
    c[4, 0] = math.nan
    c[4, 1] = -math.inf
    c[4, 2] = math.inf
    x[5, 0, :] = -math.inf
    x[5, 0, 777] = -3e38
    check(x, c, 6)


@pytest.mark.gpu
def test_large_scores_and_strides():
    x, c = inputs("bf16", 3, 4, 5001, 11)
    check(x.float() + 1e4, c - 1e4, 8)
    big = torch.randn(4, 3, 2, 5001, device="cuda")  # [W, B, ..]: other strides
    check(big[:, :, 1].transpose(0, 1), c, 8)


@pytest.mark.gpu
def test_given_results_streams_and_graphs():
    x, c = inputs("bf16", 8, 4, 30000, 12)
    out = (torch.full((8, 6), 9.0, device="cuda"), torch.full((8, 6), 9, dtype=torch.int32, device="cuda"),
           torch.full((8, 6), 9, dtype=torch.int32, device="cuda"))
    ws = torch.full((mla.beam_workspace_bytes(8, 4, 6, 30000, torch.bfloat16),), 0xAB, dtype=torch.uint8, device="cuda")
    got = check(x, c, 6, out=out, workspace=ws)
    assert all(a is b for a, b in zip(got, out))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    more = check(x, c, 6, stream=s)
    assert all(torch.equal(a, b) for a, b in zip(more, out))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.beam_select(x, c, k=6, out=out, workspace=ws)
    y, d = inputs("bf16", 8, 4, 30000, 13)
    x.copy_(y)
    c.copy_(d)
    for t in out:
        t.zero_()
    g.replay()
    assert all(torch.equal(a, b) for a, b in zip(mla.beam_select(x, c, k=6), out))
    # two calls at once
    t = torch.cuda.Stream()
    u, e = inputs("fp32", 3, 16, 50021, 14)
    torch.cuda.synchronize()
    for _ in range(4):
        a = mla.beam_select(x, c, k=6, stream=s)
        b = mla.beam_select(u, e, k=20, stream=t)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, mla.beam_select(x, c, k=6)))
    assert all(torch.equal(p, q) for p, q in zip(b, check(u, e, 20)))


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(20))
def test_random_selections(seed):
    rng = np.random.default_rng(seed)
    W = int(rng.choice([1, 2, 3, 5, 8, 13]))
    V = int(np.exp(rng.uniform(0, np.log(150000))))
    B = int(rng.integers(1, max(2, min(40, 600000 // (W * V)))))
    kind = str(rng.choice(["fp32", "bf16", "fp16"]))
    x, c = inputs(kind, B, W, V, 100 + seed, spread=float(rng.uniform(0.2, 5)), pad=int(rng.integers(0, 9)), off=int(rng.integers(0, 9)))
    done = torch.from_numpy(rng.random((B, W)) < rng.choice([0.0, 0.3])).cuda()
    check(x, c, int(rng.integers(1, min(64, 2 * W) + 1)), done, int(rng.integers(V)))


# ------------------------------------------------------------------ reordering

class Beams:
    """Requests with a shared prompt: whole pages of it in common, the page that is still being
    written, pages for rows to come and a spare page of each beam's own."""

    def __init__(self, kind, ps, lens, W, layers, seed=0, ahead=2):
        rng = np.random.default_rng(seed)
        self.kind, self.ps, self.W, self.B = kind, ps, W, len(lens)
        rows, n = [], 0
        spare = []
        for L in lens:
            whole = L // ps
            common = list(range(n, n + whole))
            n += whole
            for _ in range(W):
                rows.append(common + list(range(n, n + 1 + ahead)))
                n += 1 + ahead
                spare.append(n)
                n += 1
        width = max(map(len, rows)) + 1
        order = rng.permutation(n + 3)
        t = np.full((len(rows), width), -7, np.int32)
        for i, r in enumerate(rows):
            t[i, :len(r)] = order[r]
        self.tables = torch.from_numpy(t).cuda()
        self.spare = torch.from_numpy(order[spare].astype(np.int32)).cuda()
        self.lens = torch.tensor([L for L in lens for _ in range(W)], dtype=torch.int32, device="cuda")
        self.caches = [random_cache(kind, n + 3, ps, seed + 10 + i) for i in range(layers)]
        self.parents = torch.from_numpy(rng.integers(0, W, (len(lens), W)).astype(np.int32)).cuda()

    def bytes_of(self, cache, page, rows):
        """The bytes of a page's first rows."""
        raw = cache.view(torch.uint8).view(cache.shape[0], -1)[page]
        if self.kind != "fp4":
            return raw[:rows * (1152 if self.kind == "bf16" else 576)]
        return torch.cat([raw[:rows * 288], raw[self.ps * 288:self.ps * 288 + rows * 36]])

    def check(self, status=0, **kw):
        ps, W = self.ps, self.W
        tables, spare, lens, parents = (x.cpu().numpy().copy() for x in (self.tables, self.spare, self.lens, self.parents))
        before = [c.clone() for c in self.caches]
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        mla.cache_reorder(self.caches, self.tables, self.lens, self.parents, self.spare, status=word, **kw)
        torch.cuda.synchronize()
        assert int(word) == status
        want, kept, written = tables.copy(), spare.copy(), {}
        for b in range(self.B * W):
            p = int(parents[b // W, b % W])
            a = b // W * W + p if 0 <= p < W else b
            whole, rest = divmod(int(lens[b]), ps)
            want[b, :whole] = tables[a, :whole]
            if a != b and rest:
                want[b, whole], kept[b] = spare[b], tables[b, whole]
                written[int(spare[b])] = (int(tables[a, whole]), rest)
        assert (self.tables.cpu().numpy() == want).all() and (self.spare.cpu().numpy() == kept).all()
        for old, new in zip(before, self.caches):
            expect = old.clone()
            for dst, (src, rest) in written.items():
                raw, from_raw = (c.view(torch.uint8).view(c.shape[0], -1) for c in (expect, old))
                if self.kind == "fp4":
                    raw[dst, :rest * 288] = from_raw[src, :rest * 288]
                    at = self.ps * 288
                    raw[dst, at:at + rest * 36] = from_raw[src, at:at + rest * 36]
                else:
                    n = rest * (1152 if self.kind == "bf16" else 576)
                    raw[dst, :n] = from_raw[src, :n]
            assert torch.equal(expect.view(torch.uint8), new.view(torch.uint8))  # nothing else is touched
        return self


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp4"])
@pytest.mark.parametrize("ps,lens,W,layers", [
    (64, [0], 2, 1), (64, [1], 1, 1), (64, [1], 4, 1), (32, [31, 32, 33], 4, 1), (64, [63, 64, 65, 200], 3, 2),
    (32, [1000, 5], 8, 3), (64, [2500], 64, 1), (64, [70] * 40, 5, 2), (32, [40, 41], 2, 70), (32, [3300], 2, 1)])
def test_reorder(kind, ps, lens, W, layers):
    Beams(kind, ps, lens, W, layers, seed=W + layers).check()


@pytest.mark.gpu
def test_swaps_rings_and_parents_that_are_none():
    for parents in ([[1, 0, 3, 2]], [[1, 2, 3, 0]], [[0, 1, 2, 3]], [[3, 3, 3, 3]], [[-1, 0, -1, 2]]):
        b = Beams("bf16", 64, [150], 4, 2, seed=3)
        b.parents.copy_(torch.tensor(parents, dtype=torch.int32))
        b.check().check().check()  # each time on what the last one left


@pytest.mark.gpu
def test_bad_parents_lengths_and_pages_are_flagged():
    b = Beams("e4m3", 32, [70, 50], 3, 1, seed=4)
    b.parents[0, 1] = 3
    b.parents[1, 0] = -2
    b.check(status=2)
    b = Beams("e4m3", 32, [70], 3, 1, seed=4)
    b.parents.copy_(torch.tensor([[1, 2, 0]], dtype=torch.int32))
    saved, tables, spare = b.caches[0].clone(), b.tables.clone(), b.spare.clone()
    for lens in ([70, 71, 70], [-1] * 3, [32 * b.tables.shape[1] + 1] * 3, [2 ** 31 - 1] * 3):
        b.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        mla.cache_reorder(b.caches[0], b.tables, b.lens, b.parents, b.spare, status=word)
        assert int(word) == 1
        assert torch.equal(b.tables, tables) and torch.equal(b.spare, spare)
        assert torch.equal(b.caches[0].view(torch.uint8), saved.view(torch.uint8))
    b.lens.fill_(70)
    for bad in (-1, 2 ** 31 - 1, b.caches[0].shape[0]):
        b.spare.copy_(spare)
        b.tables.copy_(tables)
        b.spare[0] = bad          # no page to copy to
        b.parents.copy_(torch.tensor([[1, 1, 2]], dtype=torch.int32))
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        mla.cache_reorder(b.caches[0], b.tables, b.lens, b.parents, b.spare, status=word)
        assert int(word) == 16 and torch.equal(b.caches[0].view(torch.uint8), saved.view(torch.uint8))


@pytest.mark.gpu
def test_reorder_in_a_graph_and_on_a_stream():
    b = Beams("bf16", 64, [100, 260], 4, 2, seed=5)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    b.check(stream=s)
    c = Beams("bf16", 64, [100, 260], 4, 2, seed=5)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.cache_reorder(c.caches, c.tables, c.lens, c.parents, c.spare)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(b.tables, c.tables) and torch.equal(b.spare, c.spare)
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(b.caches, c.caches))


@pytest.mark.gpu
@pytest.mark.parametrize("B,W,V,ties", [(1, 1, 1, False), (5, 4, 20011, False), (3, 64, 300, False), (4, 8, 9000, True),
                                         (3, 64, 300, True), (2, 64, 9000, True)])
def test_scores_in_place(B, W, V, ties):
    # (rows that are all equal: 64 lists of 64 are more ties than the join has room for)
    x, c = inputs("fp32", B, W, V, 31)
    if ties:
        x.zero_()
        c.zero_()
    want = mla.beam_select(x, c, k=W)
    out = (c, torch.empty_like(want[1]), torch.empty_like(want[2]))
    mla.beam_select(x, c, k=W, out=out)
    assert all(torch.equal(a, b) for a, b in zip(want, out))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp4"])
def test_reorder_past_32_bits_of_the_cache(kind):
    """Pages at the end of a cache of more than 4 GiB."""
    W, ps, rest = 4, 64, 29
    row = {"bf16": 1152, "e4m3": 576, "fp4": 324}[kind]
    dtype, width = {"bf16": (torch.bfloat16, 576), "e4m3": (torch.float8_e4m3fn, 576), "fp4": (torch.uint8, 324)}[kind]
    above = (1 << 32) // (ps * row) + 1
    raw = torch.zeros((above + 2 * W, ps * row), dtype=torch.uint8, device="cuda")
    raw[above:above + W] = torch.randint(0, 256, (W, ps * row), dtype=torch.uint8, device="cuda")
    before = raw[above:above + W].clone()
    ids = torch.arange(above, above + 2 * W, dtype=torch.int32, device="cuda")
    tables, spare = ids[:W].view(W, 1).contiguous(), ids[W:].contiguous()
    lens = torch.full((W,), rest, dtype=torch.int32, device="cuda")
    mla.cache_reorder(raw.view(-1).view(dtype).view(-1, ps, width), tables, lens,
                      torch.tensor([[2, 1, 0, 2]], dtype=torch.int32, device="cuda"), spare)
    assert tables[:, 0].tolist() == [above + W, above + 1, above + W + 2, above + W + 3]
    assert spare.tolist() == [above, above + W + 1, above + 2, above + 3]
    code = 288 if kind == "fp4" else row
    for b, p in enumerate([2, 1, 0, 2]):
        now = raw[int(tables[b, 0])]
        assert torch.equal(now[:rest * code], before[p][:rest * code])
        if kind == "fp4":
            assert torch.equal(now[ps * 288:ps * 288 + rest * 36], before[p][ps * 288:ps * 288 + rest * 36])
    assert torch.equal(raw[above:above + W], before)
