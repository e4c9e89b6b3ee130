"""Decode with a sliding window and sinks, over caches of every format, against
a plain 64-bit form (tests/attention_ref.py).  In every case the rows that no
query row sees are NaN and the pages without a row to see have a page id far
out of range, so an access to one shows."""
import numpy as np
import pytest
import torch

import paged_mla_decode_03_gb300 as mla
from attention_ref import Case

# P as the kernels store it: bf16, or f16 (the default of Case.check)
P = {"bf16": dict(p_bits=8, p_floor=0.0), "e4m3": {}, "fp4": {}}

CASES = [  # page, lengths, query lengths, heads, window, sinks, options
    (64, [1], [1], 16, 1, 0, {}),
    (64, [200, 64, 65], [1, 1, 1], 128, 1, 0, {}),
    (32, [200, 33, 700], [1, 1, 1], 16, 1, 1, {}),
    (64, [1000, 130, 64], [1, 1, 1], 128, 64, 4, {}),
    (32, [1000, 130, 96], [1, 1, 1], 64, 33, 5, {}),
    (64, [900, 70], [4, 4], 128, 100, 0, {}),
    (32, [900, 5, 300], [4, 2, 7], 16, 57, 40, dict(packed=True, pad=2)),
    (64, [2000, 500], [3, 3], 32, 640, 130, {}),
    (64, [2000, 500], [3, 3], 32, 200, 2, dict(causal=False)),
    (32, [400, 90], [40, 70], 16, 20, 3, dict(packed=True)),
    (64, [3000, 10], [1, 1], 128, 2500, 64, dict(max_len=5000)),
    (64, [300, 250], [1, 1], 128, 64, 200, {}),
    (32, [128, 64, 192], [1, 1, 1], 128, 64, 64, {}),
    (64, [700, 333], [2, 2], 128, 130, 7, dict(q_fp8=True)),
    (64, [500, 400], [1, 1], 64, 90, 3, dict(bmm1=0.0)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("kind,widen", [("bf16", False), ("e4m3", False), ("e4m3", True), ("fp4", False)])
@pytest.mark.parametrize("ps,ls,qs,heads,window,sinks,kw", CASES)
def test_window(kind, widen, ps, ls, qs, heads, window, sinks, kw):
    c = Case(kind, ps, ls, qs, heads, window=window, sinks=sinks, seed=heads + window, widen=widen, **kw).run()
    c.check(**P[kind])


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp4"])
@pytest.mark.parametrize("seed", range(8))
def test_random_launches(kind, seed):
    rng = np.random.default_rng(300 + seed)
    packed = bool(rng.integers(2))
    B = int(rng.integers(1, 40))
    top = int(rng.choice([1, 2, 5]))
    qs = [int(rng.integers(1, top + 1)) if packed else top for _ in range(B)]
    ls = [q + int(rng.integers(0, int(rng.choice([3, 70, 700, 2500])))) for q in qs]
    Case(kind, int(rng.choice([32, 64])), ls, qs, int(rng.choice([16, 32, 64, 128])), packed=packed,
         causal=bool(rng.integers(2)), window=int(rng.choice([1, 2, 31, 64, 65, 129, 600])),
         sinks=int(rng.choice([0, 1, 4, 64, 65, 200])), q_fp8=bool(rng.integers(3) == 0),
         seed=seed).run().check(**P[kind])


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp4"])
@pytest.mark.parametrize("window", [300, 301, 2 ** 31 - 1])
def test_a_window_over_everything_hides_nothing(kind, window):
    a = Case(kind, 64, [300, 77], [2, 2], 64, window=window, sinks=5, seed=1).run()
    a.check(**P[kind])
    b = Case(kind, 64, [300, 77], [2, 2], 64, seed=1)
    assert torch.equal(a.tables, b.tables)
    if kind == "fp4":  # the same kernel with and without a window
        b.run()
        assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)
    # one row short of it, the first row of the longer request is out
    Case(kind, 64, [300, 77], [1, 1], 64, window=299, seed=1).run().check(**P[kind])


@pytest.mark.gpu
def test_through_decode_and_in_a_graph():
    c = Case("bf16", 64, [900, 300, 65], [1, 1, 1], 128, window=128, sinks=4, seed=2, max_len=900)
    out, lse = mla.decode(c.query.view(3, 1, 128, 576), c.cache, c.workspace, c.tables, c.lens, 900, bmm1_scale=c.bmm1,
                          bmm2_scale=c.bmm2, return_lse=True, window=128, sinks=4)
    c.run().check(**P["bf16"])
    assert torch.equal(out.view_as(c.out), c.out) and torch.equal(lse, c.lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    # shorter sequences: other pages come into the windows, so all must be there
    d = Case("bf16", 64, [900, 300, 65], [1, 1, 1], 128, seed=2, max_len=900)
    c.cache.copy_(d.cache)
    c.tables.copy_(d.tables)
    c.lens.copy_(torch.tensor([400, 299, 1], dtype=torch.int32))
    c.ls = [400, 299, 1]
    g.replay()
    c.check(**P["bf16"])


@pytest.mark.gpu
def test_host_entry_takes_a_window():
    c = Case("bf16", 64, [500, 90], [1, 1], 16, window=70, sinks=3, seed=4)
    c.run()
    staging = torch.empty(c.plan.staging_bytes(), dtype=torch.uint8, device="cuda")
    h_out = torch.empty(c.out.shape, dtype=torch.bfloat16).pin_memory()
    h_lse = torch.empty(c.lse.shape).pin_memory()
    c.plan.run_host(c.query.cpu().pin_memory(), c.cache, c.tables.cpu().pin_memory(), c.lens.cpu().pin_memory(), h_out,
                    staging=staging, workspace=c.workspace, h_lse=h_lse, bmm1_scale=c.bmm1, bmm2_scale=c.bmm2)
    torch.cuda.synchronize()
    assert torch.equal(h_out, c.out.cpu()) and torch.equal(h_lse, c.lse.cpu())


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp4"])
@pytest.mark.parametrize("ps,bad", [(64, -1), (32, 2 ** 31 - 1), (32, None)])
def test_a_bad_page_in_a_window_is_flagged_and_reads_as_zeros(kind, ps, bad):
    c = Case(kind, ps, [900, 130], [1, 1], 128, window=600, sinks=2, seed=6)
    at = 800 // ps
    page = int(c.bt_host[0, at])
    c.tables[0, at] = c.cache.shape[0] if bad is None else bad  # None: one past the last
    c.run()
    c.tables[0, at] = page  # the reference reads a page of zeros there
    c.cache[page].zero_()
    c.check(status=16, **P[kind])


@pytest.mark.gpu
@pytest.mark.parametrize("kind,window", [("fp4", 0), ("bf16", 20)])
def test_more_row_groups_than_the_small_work_list_takes(kind, window):
    # 1100 row groups: the work list comes from the block form of the partitioner
    rng = np.random.default_rng(8)
    ls = [int(x) for x in rng.integers(1, 65, 1100)]
    Case(kind, 64, ls, [1] * 1100, 128, window=window, seed=8).run().check(**P[kind])


@pytest.mark.gpu
def test_two_plans_on_two_streams():
    """Two windowed decodes in flight at once, each with its own workspace."""
    a = Case("bf16", 64, [900, 700], [1, 1], 128, window=300, seed=21)
    b = Case("fp4", 64, [800, 1500], [2, 2], 64, window=500, sinks=9, seed=22)
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
