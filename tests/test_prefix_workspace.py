"""The workspace of decodes over shared prefixes: the room to widen rows is asked for, never needed."""
import importlib.util
import os
import random
import shutil
import subprocess

import pytest
import torch

import paged_mla_decode_03_gb300 as mla
from prefix_case import PrefixCase
from test_partition_host import CSRC, HERE, ROOT


@pytest.fixture(scope="module")
def totals(tmp_path_factory):
    """(bytes with the room, without, tiles to widen) of plans (B, H, max_q, packed, total_q, max_len, kv, groups)."""
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    out = tmp_path_factory.mktemp("prefix_layout")
    common = open(os.path.join(CSRC, "mla_common.cuh")).read().replace("#include <cuda_runtime.h>\n", "")
    (out / "mla_common_host.h").write_text(common)
    (out / "mla_prefix_host.h").write_text(
        open(os.path.join(CSRC, "mla_prefix.cuh")).read().replace('#include "mla_common.cuh"\n', ""))
    exe = out / "layout"
    r = subprocess.run([cxx, "-std=c++20", "-O1", "-pthread", "-I", str(out), "-I", HERE, "-I", os.path.join(ROOT, "include"),
                        os.path.join(HERE, "prefix_layout.cpp"), "-o", str(exe)], capture_output=True, text=True)
    if r.returncode != 0 and "No such file" in r.stderr:
        pytest.skip("host toolchain lacks C++20 <barrier>: " + r.stderr[-300:])
    assert r.returncode == 0, r.stderr[-3000:]

    def run(plans):
        text = "".join(" ".join(str(int(x)) for x in p) + " 76\n" for p in plans)
        r = subprocess.run([str(exe)], input=text, capture_output=True, text=True)
        assert r.returncode == 0, r.returncode
        return [tuple(int(x) for x in line.split()) for line in r.stdout.splitlines()]
    return run


def test_short_prefixes_under_a_long_bound(totals):
    # seven groups that may be 131072 rows long ask for almost 1 GiB, and do with the rest
    (full, least, tiles), = totals([(7 * 32, 128, 1, 0, 7 * 32, 131072, 2, 7)])
    assert tiles == 7 * 2048 and full > 1 << 30 and least < 40 << 20
    for kv in (0, 1, 2):  # what a run cannot do without hardly hangs on the cache's type
        (a, b, tiles), = totals([(32, 16, 1, 0, 32, 131072, kv, 8)])
        assert a == b < 40 << 20 and tiles == 0


def test_a_workspace_by_the_query_rows_holds_every_plan(totals):
    """64 MiB and a partial's room for each 128 query rows, as a user of the cases of
    perf/more_operators.py keeps: enough for any of them, whatever its prefixes' lengths."""
    spec = importlib.util.spec_from_file_location("more_operators", os.path.join(ROOT, "perf", "more_operators.py"))
    cases = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(cases)
    rng, plans, given = random.Random(7), [], []
    while len(plans) < 6000:
        case = cases.draw(rng)
        if case["op"] != "prefix":
            continue
        sizes, shared, rows, qs = cases._plan(case)
        H, T = case["heads"], sum(qs)
        blocks = -(-T * H // 128) + len(sizes) + sum(-(-q * H // 128) for q in qs) + 256
        given.append((64 << 20) + blocks * (272 << 10))
        plans.append((len(rows), H, max(qs), case["packed"], T, max(rows), ["bf16", "e4m3", "fp4"].index(case["kv"]), len(sizes)))
    got = totals(plans)
    assert all(least <= room for (_, least, _), room in zip(got, given))
    assert any(full > room for (full, _, _), room in zip(got, given))  # (the room to widen is past some of them)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["e4m3", "fp4"])
def test_a_run_without_the_room_widens_nothing(kind):
    c = PrefixCase(kind, 64, [16], [3000], [5, 100], [1], 128, uniform=True, seed=40)
    assert mla.mla_decode_kernels_per_run(c.plan.handle) == 5
    least = c.plan.workspace_least
    assert least == mla.mla_decode_workspace_least(c.plan.handle) < c.plan.workspace_bytes == mla.mla_decode_workspace_size(c.plan.handle)
    c.run().check()
    wide = c.items().shape[0]
    whole = torch.full((least + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    for room in (least, least + 256, least + 4096):
        c.workspace = whole[:room]
        c.workspace.fill_(0xFF)
        c.out.fill_(3.0)
        c.run().check()
        assert (whole[least:] == 0xA5).all() or room > least
        assert (c.items()[:, 3] - c.items()[:, 2]).sum() > 16 * 3000  # the shared rows are in the first list
    out, lse = mla.decode(c.query.view(16, 1, 128, 576), c.cache, whole, c.tables, c.lens, c.max_len, bmm1_scale=c.bmm1,
                          bmm2_scale=c.bmm2, return_lse=True, prefix_lens=c.prefix_lens)
    torch.cuda.synchronize()
    assert torch.equal(out.view_as(c.out), c.out) and torch.equal(lse, c.lse) and wide > 0
    # in a graph too; and less than the least is refused
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    c.out.fill_(3.0)
    g.replay()
    c.check()
    c.workspace = whole[:least - 1]
    with pytest.raises(mla.MlaDecodeError):
        c.run()
    with pytest.raises(ValueError):
        mla.decode(c.query.view(16, 1, 128, 576), c.cache, c.workspace, c.tables, c.lens, c.max_len, prefix_lens=c.prefix_lens)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp4"])
def test_plans_that_cannot_widen_need_what_they_ask_for(kind):
    c = PrefixCase(kind, 64, [4], [700], [5], [1], 16, seed=4)
    assert c.plan.workspace_least == c.plan.workspace_bytes
    p = mla.Plan(batch=4, num_heads=16, max_seq_len_q=1, max_seq_len=c.max_len, page_size=64, kv_dtype=kind,
                 max_pages_per_req=c.tables.shape[1], num_pages=c.cache.shape[0], packed=False)
    assert p.workspace_least == p.workspace_bytes
