"""Decode over a 4-bit cache against a plain 64-bit form (tests/attention_ref.py)."""
import ctypes

import numpy as np
import pytest
import torch

import paged_mla_decode_03_gb300 as mla
from attention_ref import Case, cache_values
from paged_mla_decode_03_gb300 import build as mla_build


@pytest.mark.parametrize("kw,rc", [(dict(sparse_top_k=4), -2), (dict(window=-1), -1), (dict(window=4, sinks=-1), -1),
                                   (dict(sinks=1), -1), (dict(window=4, cp_world=2), -2),
                                   (dict(window=4, sparse_top_k=4, kv_dtype=0), -2)])
def test_refusals(kw, rc):
    mla_build.build()
    p = dict(batch=2, num_heads=16, max_seq_len_q=1, max_seq_len=64, page_size=32, max_pages_per_req=2, num_pages=8,
             kv_dtype=mla.KV_FP4_E2M1)
    p.update(kw)
    with pytest.raises(mla.MlaDecodeError) as e:
        mla.mla_decode_plan(mla.MlaDecodeParams(**p))
    assert e.value.status == rc


CASES = [  # page, lengths, query lengths, heads, options
    (64, [1], [1], 128, {}),
    (64, [64], [1], 128, {}),
    (64, [65, 127, 128], [1, 1, 1], 128, {}),
    (32, [33, 31, 1, 200], [1, 1, 1, 1], 16, {}),
    (32, [70, 97], [4, 4], 32, {}),
    (64, [300, 41], [3, 3], 64, dict(causal=False)),
    (64, [777, 1500], [2, 2], 128, dict(q_fp8=True)),
    (32, [40, 900, 8, 65], [3, 1, 8, 5], 16, dict(packed=True, pad=3)),
    (32, [128, 513], [33, 2], 64, dict(packed=True, causal=False)),
    (64, [20000], [1], 128, {}),
    (64, [9000, 100, 5000], [1, 1, 1], 128, dict(max_len=20000)),
    (64, [400, 210], [1, 1], 128, dict(bmm1=1.5)),
    (32, [400, 210], [1, 1], 16, dict(bmm1=0.0)),
    (64, [400, 65], [1, 1], 32, dict(q_gain=1e-20, bmm1=1e18)),
    (64, [400, 65], [1, 1], 32, dict(q_gain=1e20, bmm1=1e-21)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("ps,ls,qs,heads,kw", CASES)
def test_decode(ps, ls, qs, heads, kw):
    Case("fp4", ps, ls, qs, heads, seed=len(ls) + heads + ps, **kw).run().check()


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(12))
def test_random_launches(seed):
    rng = np.random.default_rng(100 + seed)
    packed = bool(rng.integers(2))
    B = int(rng.integers(1, 12))
    top = int(rng.choice([1, 3, 6]))
    qs = [int(rng.integers(1, top + 1)) if packed else top for _ in range(B)]
    ls = [q + int(rng.integers(0, int(rng.choice([3, 70, 700, 2500])))) for q in qs]
    Case("fp4", int(rng.choice([32, 64])), ls, qs, int(rng.choice([16, 32, 64, 128])), packed=packed,
         causal=bool(rng.integers(2)), q_fp8=bool(rng.integers(3) == 0), seed=seed).run().check()


@pytest.mark.gpu
def test_every_code_and_scale_comes_through():
    """One visible row, so O is V: each code under each finite scale, bit for bit."""
    rows = 64
    c = Case("fp4", 64, [rows] * 4, [1] * 4, 16, seed=3, bmm2=1.0)
    finite = [s for s in range(256) if s & 0x7F != 0x7F]
    scales = torch.tensor(finite + finite[:2], dtype=torch.uint8)  # 256
    for b in range(4):
        page = int(c.bt_host[b, 0])
        flat = c.cache.view(c.cache.shape[0], -1)[page]
        codes = (torch.arange(288) * 2 % 16 + ((torch.arange(288) * 2 + 1) % 16) * 16).to(torch.uint8)
        flat[:rows * 288] = codes.repeat(rows).cuda()
        sc = torch.zeros(rows, 36, dtype=torch.uint8)
        sc[0, :32] = scales[64 * b:64 * b + 32]
        sc[0, 32:] = 0x38
        flat[rows * 288:] = sc.flatten().cuda()
    c.lens.fill_(1)
    c.run()
    assert c.status() == 0
    vals = cache_values(c.cache)
    for b in range(4):
        ref = vals[int(c.bt_host[b, 0]), 0, :512].to(torch.bfloat16)
        assert (c.out[b] == ref).all(), f"request {b}"


@pytest.mark.gpu
def test_more_rows_than_workers_and_items_of_many_tiles():
    rng = np.random.default_rng(5)
    ls = [int(x) for x in rng.integers(1, 1500, 90)]
    Case("fp4", 64, ls, [1] * 90, 128, seed=6).run().check()


@pytest.mark.gpu
def test_repeated_and_back_to_back_calls_agree():
    c = Case("fp4", 64, [3000, 40, 900, 2100], [2] * 4, 128, seed=7).run()
    torch.cuda.synchronize()
    out, lse = c.out.clone(), c.lse.clone()
    for _ in range(20):
        c.run()
    torch.cuda.synchronize()
    assert torch.equal(out, c.out) and torch.equal(lse, c.lse) and c.status() == 0


@pytest.mark.gpu
def test_graph_replay_with_new_lengths_and_device_scales():
    c = Case("fp4", 32, [900, 64, 333], [1] * 3, 64, seed=8, max_len=900)
    b1 = torch.tensor([c.bmm1], device="cuda")
    b2 = torch.tensor([c.bmm2], device="cuda")
    c.run(bmm1_scale=b1, bmm2_scale=b2)
    c.check(what="device scales")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(bmm1_scale=b1, bmm2_scale=b2)
    c.lens -= 60
    c.ls = [L - 60 for L in c.ls]
    b1.mul_(0.5)
    c.bmm1 *= 0.5
    g.replay()
    c.check(what="replay")


@pytest.mark.gpu
def test_bad_pages_are_flagged_and_others_are_right():
    c = Case("fp4", 64, [200, 130], [1, 1], 128, seed=9)
    good = c.tables.clone()
    c.tables[0, 1] = -1
    c.run()
    assert c.status() == 16
    c.tables.copy_(good)
    for t, o, e, _ in c.reference():
        if t == 1:
            assert (c.lse[t].double() - e).abs().max() < 1e-4
    assert torch.isfinite(c.out.float()).all()


@pytest.mark.gpu
def test_context_parallel_ranks_merge_to_the_whole():
    whole = Case("fp4", 32, [500, 77], [2, 2], 16, seed=10, bmm2=1.0).run()
    whole.check()
    W, outs, lses = 2, [], []
    for r in range(W):
        # rank r holds the rows g with g mod W == r
        sub = Case("fp4", 32, [max(1, len(range(r, L, W))) for L in whole.ls], [2, 2], 16, seed=11, bmm2=1.0)
        for b, L in enumerate(whole.ls):
            for k, gpos in enumerate(range(r, L, W)):
                src = whole.cache.view(whole.cache.shape[0], -1)[int(whole.bt_host[b, gpos // 32])]
                dst = sub.cache.view(sub.cache.shape[0], -1)[int(sub.bt_host[b, k // 32])]
                i, j = gpos % 32, k % 32
                dst[j * 288:(j + 1) * 288] = src[i * 288:(i + 1) * 288]
                dst[9216 + j * 36:9216 + (j + 1) * 36] = src[9216 + i * 36:9216 + (i + 1) * 36]
        plan = mla.Plan(batch=2, num_heads=16, max_seq_len_q=2, max_seq_len=sub.max_len, page_size=32,
                        max_pages_per_req=sub.tables.shape[1], num_pages=sub.cache.shape[0], packed=False,
                        kv_dtype="fp4", return_lse=True, cp_world=W, cp_rank=r)
        ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        plan.run(whole.query, sub.cache, sub.tables, sub.lens, sub.out, lse=sub.lse, workspace=ws,
                 bmm1_scale=whole.bmm1, bmm2_scale=1.0, seq_lens_global=whole.lens)
        outs.append(sub.out)
        lses.append(sub.lse)
    out, lse = mla.merge_states(torch.stack(outs), torch.stack(lses))
    for t, o, e, (a, d, v) in whole.reference():
        # the shards' outputs are rounded to bf16 once more
        assert ((out[t].double() - o).abs() <= o.abs() * 2.0 ** -8 + a * 2.0 ** -7 + v * 2.0 ** -32).all()
        assert (lse[t].double() - e).abs().max() < 1e-4


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [16, 128])
def test_written_by_append_then_decoded(heads):
    """The operators as a serving step uses them: append into 4 bits, then decode
    the same tokens over prompt and new rows."""
    ls, qs, ps = [130, 64, 33], [3, 3, 3], 64
    T, B = 9, 3
    g = torch.Generator().manual_seed(12)
    table = mla.rope_table(512)
    cache = torch.zeros(8, ps, 324, dtype=torch.uint8, device="cuda")
    bt = torch.tensor([[5, 0, 3], [2, -1, -1], [7, -1, -1]], dtype=torch.int32, device="cuda")
    w = torch.ones(512, dtype=torch.bfloat16, device="cuda")

    def rows(n):
        return torch.randn(n, 576, generator=g).to(torch.bfloat16).cuda()

    prompt = [L - 3 for L in ls]
    ip = torch.tensor(np.cumsum([0] + prompt), dtype=torch.int32, device="cuda")
    x = rows(sum(prompt))
    mla.cache_append(x[:, :512], x[:, 512:], cache, bt, torch.tensor(prompt, dtype=torch.int32, device="cuda"),
                     rope_table=table, norm_weight=w, qo_indptr=ip)
    sl = torch.tensor(ls, dtype=torch.int32, device="cuda")
    x, qn, qp = rows(T), rows(T * heads).view(T, heads, 576)[..., :512], rows(T * heads).view(T, heads, 576)[..., 512:]
    q = mla.cache_append(x[:, :512], x[:, 512:], cache, bt, sl, rope_table=table, norm_weight=w, q_len=3, q_nope=qn,
                         q_pe=qp)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    out, lse = mla.decode(q.view(B, 3, heads, 576), cache, ws, bt, sl, 130, bmm1_scale=0.07, return_lse=True)
    vals = cache_values(cache)
    for b in range(B):
        j = torch.arange(ls[b], device="cuda")
        k = vals[bt[b].long()[j // ps], j % ps]
        for i in range(3):
            s = q[3 * b + i].double() @ k[:ls[b] - 2 + i].T * float(np.float32(0.07))
            e = torch.logsumexp(s, -1)
            p = torch.exp(s - e[:, None])
            v = k[:ls[b] - 2 + i, :512]
            assert (lse[3 * b + i].double() - e).abs().max() < 1e-4
            o = p @ v
            assert ((out[b, i].double() - o).abs() <= o.abs() * 2.0 ** -8 + (p @ v.abs()) * (2.0 ** -8 + 2.0 ** -11 + 2e-4)).all()
