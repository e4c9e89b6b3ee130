"""Decode over a batch whose requests share their first rows, over caches of every format,
against a plain 64-bit form that takes every request by itself (tests/attention_ref.py).
Rows that no query row sees, and the pages that other requests' shared ones replace, are NaN."""
import ctypes

import numpy as np
import pytest
import torch

import paged_mla_decode_03_gb300 as mla
from prefix_case import PrefixCase

P = {"bf16": dict(p_bits=8, p_floor=0.0), "e4m3": {}, "fp4": {}}

CASES = [  # page, group sizes, shared rows, own rows, query lengths, heads, options, whether rows are shared
    (64, [40], [1000], [1, 70, 33], [1], 16, dict(uniform=True), True),
    (32, [40], [1000], [1, 70, 33], [1], 16, {}, True),
    (64, [40], [1024], [0, 1, 64, 200], [1], 16, {}, True),         # requests without a row of their own
    (32, [48], [1600], [0], [1], 16, {}, True),                     # none has one
    (64, [20, 30], [1500, 2100], [5, 400], [1], 32, dict(uniform=False), True),
    (64, [24, 0, 24, 1], [1500, 900, 1291, 700], [9, 130], [1, 2, 3], 16, dict(gap=2, pad=2), True),
    (32, [40], [4000], [50, 3], [1, 2], 32, dict(causal=False), True),
    (64, [30], [9000], [7, 8, 100], [3], 64, {}, True),             # 192 rows a request: they straddle row groups
    (64, [40], [1300], [20, 1], [1], 16, dict(q_fp8=True), True),
    (64, [40], [1300], [20, 1], [1], 16, dict(bmm1=0.0), True),
    (64, [40], [1300], [20, 300], [2], 16, dict(same_pages=False), True),
    (64, [60], [1500], [2, 90], [1], 16, dict(claim=[100000]), True),  # more than a query row sees
    (64, [3], [300], [2, 90], [1], 128, {}, None),                  # little to save
    (64, [1], [300], [0], [1], 16, {}, False),
    (32, [40], [63], [1], [1], 16, {}, False),                      # less than a tile
]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp4"])
@pytest.mark.parametrize("ps,sizes,shared,own,qs,heads,kw,shares", CASES)
def test_shared_prefix(kind, ps, sizes, shared, own, qs, heads, kw, shares):
    if kw.get("claim"):  # only what is the same may be claimed: a request's own rows are none
        own = [0]
    c = PrefixCase(kind, ps, sizes, shared, own, qs, heads, seed=heads + sum(sizes), **kw).run()
    c.check(**P[kind])
    assert shares is None or c.shares() == shares


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp4"])
@pytest.mark.parametrize("seed", range(8))
def test_random_groups(kind, seed):
    rng = np.random.default_rng(600 + seed)
    G = int(rng.integers(1, 5))
    sizes = [int(rng.integers(0, 40)) for _ in range(G)]
    sizes[0] += 1
    top = int(rng.choice([1, 2, 6]))
    qs = [int(x) for x in rng.integers(1, top + 1, 5)]
    shared = [int(x) for x in rng.integers(0, int(rng.choice([100, 1500, 4000])), G)]
    own = [int(x) + top for x in rng.integers(0, int(rng.choice([1, 70, 500])), 6)]
    PrefixCase(kind, int(rng.choice([32, 64])), sizes, shared, own, qs, int(rng.choice([16, 32, 64, 128])),
               causal=bool(rng.integers(2)), q_fp8=bool(rng.integers(3) == 0), gap=int(rng.integers(0, 3)),
               seed=seed).run().check(**P[kind])


WIDE = [  # page, group sizes, shared rows, own rows, query lengths, heads, options: four row groups a group and more
    (64, [16], [3000], [5, 100], [1], 128, dict(uniform=True)),
    (32, [16], [3000], [0], [1], 128, {}),                          # none has a row of its own
    (32, [12, 0, 9, 1], [2500, 500, 4001, 300], [0, 1, 300], [1, 2, 3], 64, dict(gap=2, pad=1)),
    (64, [14], [2000], [64, 3], [2], 64, dict(causal=False, q_fp8=True)),
    (64, [40, 2], [1500, 2000], [64, 3], [1], 32, dict(same_pages=False)),  # one of the groups is not widened
    (64, [5], [30000], [70], [1], 128, {}),                         # few row groups, cut over all workers
]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["e4m3", "fp4"])
@pytest.mark.parametrize("ps,sizes,shared,own,qs,heads,kw", WIDE)
def test_widened_prefix(kind, ps, sizes, shared, own, qs, heads, kw):
    c = PrefixCase(kind, ps, sizes, shared, own, qs, heads, seed=heads + sum(sizes), **kw).run()
    assert mla.mla_decode_kernels_per_run(c.plan.handle) == 5
    c.check(**P[kind])


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["e4m3", "fp4"])
def test_widened_rows_in_a_graph_with_other_lengths(kind):
    c = PrefixCase(kind, 64, [16], [3000], [5, 100], [1], 128, uniform=True, seed=40)
    c.run().check(**P[kind])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for lens in ([700], [0], [2999]):  # fewer widened, none, all again
        c.prefix_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        c.workspace.fill_(0xFF)
        c.out.fill_(3.0)
        g.replay()
        c.check(**P[kind])
    page = int(c.tables[0, 3])
    c.tables[:, 3] = -1
    g.replay()
    c.tables[:, 3] = page
    c.cache[page].zero_()
    c.check(status=16, **P[kind])


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp4"])
def test_one_long_prefix_is_cut_over_every_worker(kind):
    c = PrefixCase(kind, 64, [8], [40000], [1, 30], [1], 16, seed=5).run()
    c.check(**P[kind])
    assert c.shares() and len(c.items()) > 70


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp4"])
def test_through_decode_and_in_a_graph(kind):
    c = PrefixCase(kind, 64, [20, 20], [1500, 1400], [3, 90], [1], 16, seed=2, max_len=1700, uniform=True)
    out, lse = mla.decode(c.query.view(40, 1, 16, 576), c.cache, c.workspace, c.tables, c.lens, 1700, bmm1_scale=c.bmm1,
                          bmm2_scale=c.bmm2, return_lse=True, prefix_lens=c.prefix_lens)
    c.run().check(**P[kind])
    assert torch.equal(out.view_as(c.out), c.out) and torch.equal(lse, c.lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    # other lengths, and a shorter prefix, in the same graph
    c.lens.sub_(1)
    c.ls = [L - 1 for L in c.ls]
    c.prefix_lens.copy_(torch.tensor([900, 0], dtype=torch.int32))
    g.replay()
    c.check(**P[kind])
    # scales read from device memory
    c.out.fill_(3.0)
    c.run(bmm1_scale=torch.tensor([c.bmm1], device="cuda"), bmm2_scale=torch.tensor([c.bmm2], device="cuda"))
    c.check(**P[kind])


@pytest.mark.gpu
def test_repeated_runs_are_equal_on_dirty_workspaces():
    c = PrefixCase("bf16", 64, [33], [2500], [1, 200], [2], 16, seed=9).run()
    torch.cuda.synchronize()
    first = c.out.clone(), c.lse.clone()
    for fill in (0x00, 0xFF, 0x7F):
        c.workspace.fill_(fill)
        c.run()
        torch.cuda.synchronize()
        assert torch.equal(first[0], c.out) and torch.equal(first[1], c.lse)


@pytest.mark.gpu
@pytest.mark.parametrize("indptr", [[0, 30, 20, 40], [-1, 10, 20, 40], [0, 10, 20, 41]])
def test_bad_offsets_are_flagged_and_share_nothing(indptr):
    c = PrefixCase("bf16", 64, [20, 20, 0], [1500, 1400, 0], [3, 90], [1], 16, seed=3)
    c.prefix_indptr.copy_(torch.tensor(indptr, dtype=torch.int32))
    c.run().check(status=256, **P["bf16"])
    assert not c.shares()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp4"])
def test_a_bad_shared_page_is_flagged_and_reads_as_zeros(kind):
    c = PrefixCase(kind, 64, [40], [1500], [10], [1], 16, seed=6)
    page = int(c.tables[0, 3])
    c.tables[:, 3] = c.cache.shape[0]
    c.run()
    c.tables[:, 3] = page
    c.cache[page].zero_()
    c.check(status=16, **P[kind])


@pytest.mark.gpu
def test_two_plans_on_two_streams():
    a = PrefixCase("bf16", 64, [40], [1500], [10, 700], [1], 16, seed=21)
    b = PrefixCase("fp4", 64, [30], [2500], [100, 1], [2], 32, seed=22)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s):
            a.run()
        with torch.cuda.stream(t):
            b.run()
    torch.cuda.synchronize()
    a.check(**P["bf16"])
    b.check(**P["fp4"])


@pytest.mark.gpu
def test_refusals():
    c = PrefixCase("bf16", 64, [4], [100], [10], [1], 16, seed=1)
    q = c.query.view(4, 1, 16, 576)
    call = lambda **kw: mla.decode(q, c.cache, c.workspace, c.tables, c.lens, c.max_len, **kw)  # noqa: E731
    for kw in (dict(prefix_lens=torch.zeros(3, dtype=torch.int32, device="cuda")),   # 3 does not divide 4
               dict(prefix_lens=torch.zeros(2, dtype=torch.int64, device="cuda")),
               dict(prefix_lens=torch.zeros(2, dtype=torch.int32)),
               dict(prefix_lens=torch.zeros(2, 1, dtype=torch.int32, device="cuda")),
               dict(prefix_lens=torch.zeros(0, dtype=torch.int32, device="cuda")),
               dict(prefix_indptr=torch.zeros(2, dtype=torch.int32, device="cuda")),
               dict(prefix_lens=c.prefix_lens, prefix_indptr=torch.zeros(3, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(window=5), dict(sparse_indices=torch.zeros(4, 2, dtype=torch.int32, device="cuda")),
               dict(cp_world=2)):
        with pytest.raises(mla.MlaDecodeError):
            call(prefix_lens=c.prefix_lens, **kw)
    with pytest.raises(mla.MlaDecodeError):  # the other entries refuse the plan
        mla.mla_decode_run(c.plan.handle, c.query, c.cache, c.tables, c.lens, None, 0, 1.0, 1.0, c.out, c.lse, c.workspace)
    with pytest.raises(mla.MlaDecodeError):  # and this one another plan
        p = mla.Plan(batch=4, num_heads=16, max_seq_len_q=1, max_seq_len=200, page_size=64, max_pages_per_req=8,
                     num_pages=64, packed=False, kv_dtype="fp4")
        mla.mla_decode_run_prefix(p.handle, c.query, c.cache, c.tables, c.lens, None, 0, c.prefix_lens, None, 1.0, 1.0,
                                  c.out, c.lse, c.workspace)
    with pytest.raises(mla.MlaDecodeError):
        mla.Plan(batch=4, num_heads=16, max_seq_len_q=1, max_seq_len=200, page_size=64, max_pages_per_req=8,
                 num_pages=64, packed=False, prefix_groups=5)


@pytest.mark.gpu
def test_a_plan_without_groups_refuses_their_lengths():
    c = PrefixCase("bf16", 64, [4], [100], [10], [1], 16, seed=1)
    p = mla.Plan(batch=4, num_heads=16, max_seq_len_q=1, max_seq_len=c.max_len, page_size=64,
                 max_pages_per_req=c.tables.shape[1], num_pages=c.cache.shape[0], packed=False)
    for kw in (dict(prefix_lens=c.prefix_lens), dict(prefix_indptr=c.prefix_lens)):
        with pytest.raises(ValueError):
            p.run(c.query, c.cache, c.tables, c.lens, c.out, workspace=c.workspace, **kw)


@pytest.mark.gpu
def test_the_static_workspace_refuses_a_prefix_plan():
    c = PrefixCase("bf16", 64, [4], [100], [10], [1], 16, seed=1)
    before = c.out.clone()
    rc = mla.load_library().mla_decode_run_static_workspace(
        ctypes.c_void_p(c.plan.handle), c.query.data_ptr(), c.cache.data_ptr(), c.tables.data_ptr(),
        c.lens.data_ptr(), None, ctypes.c_int64(0), ctypes.c_float(1.0), ctypes.c_float(1.0),
        ctypes.c_void_p(c.out.data_ptr()), None, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc != mla.MLA_OK
    torch.cuda.synchronize()
    assert torch.equal(c.out.view(torch.int16), before.view(torch.int16))


@pytest.mark.gpu
def test_repeated_pages_and_no_lse():
    """Every request's table names one page again and again; no LSE is wanted."""
    c = PrefixCase("bf16", 64, [12], [640], [70], [1], 16, seed=3)
    q = c.query.view(12, 1, 16, 576)
    tables = c.tables[:1, :1].repeat(12, c.tables.shape[1]).contiguous()
    lens = torch.full((12,), 640, dtype=torch.int32, device="cuda")
    call = lambda **kw: mla.decode(q, c.cache, c.workspace, tables, lens, 640, bmm1_scale=0.07, **kw)  # noqa: E731
    got = call(prefix_lens=torch.tensor([640], dtype=torch.int32, device="cuda"))
    rows = c.cache.view(-1, 64, 576)[tables[0, 0].item()].double().repeat(10, 1)
    s = q[:, 0].double() @ rows.T * 0.07
    p = torch.softmax(s, -1)
    want, size = p @ rows[:, :512], p @ rows[:, :512].abs()
    # P rounds to bf16 in the sum and in its divisor (2^-8 of `size` each), O once more; a partial
    # to f16, 2^-11 of itself and 2^-39 of its largest, and scores in fp32: 2^-10 of `size`
    assert ((got[:, 0].double() - want).abs() <= 2 ** -8 * (2 * size + want.abs()) + 2 ** -10 * size).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp4"])
def test_pages_past_32_bits_of_the_cache(kind):
    """The same pages at the end of a cache of more than 4 GiB, to the bit."""
    c = PrefixCase(kind, 64, [64], [1500], [20, 300], [1], 16, seed=5)
    q = c.query.view(64, 1, 16, 576)
    page = c.cache[0].numel() * c.cache.element_size()
    above = (1 << 32) // page + 1
    big = torch.zeros((above + c.cache.shape[0], page), dtype=torch.uint8, device="cuda").view(c.cache.dtype)
    big = big.view(-1, *c.cache.shape[1:])
    big.view(torch.uint8)[above:] = c.cache.view(torch.uint8)
    got = [mla.decode(q, cache, c.workspace, tables, c.lens, c.max_len, bmm1_scale=0.07, prefix_lens=c.prefix_lens,
                      prefix_indptr=c.prefix_indptr)
           for cache, tables in ((c.cache, c.tables), (big, c.tables + above))]
    assert torch.equal(got[0].view(torch.int16), got[1].view(torch.int16))


@pytest.mark.gpu
def test_no_request():
    c = PrefixCase("bf16", 64, [4], [100], [10], [1], 16, seed=1)
    out = mla.decode(c.query.view(4, 1, 16, 576)[:0], c.cache, c.workspace, c.tables[:0], c.lens[:0], c.max_len,
                     prefix_lens=c.prefix_lens)
    assert out.shape[0] == 0
