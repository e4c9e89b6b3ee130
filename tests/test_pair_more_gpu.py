"""More of the decode over 4 bits and with a window: calls that the first tests leave out."""
import ctypes

import pytest
import torch

import paged_mla_decode_03_gb300 as mla
from attention_ref import Case

P = {"bf16": dict(p_bits=8, p_floor=0.0), "e4m3": {}, "fp4": {}}


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp4"])
@pytest.mark.parametrize("ls", [[300, 70, 130], [9000, 200, 4000]])
def test_a_nan_in_a_query_row_is_one_in_its_outputs_and_lse(kind, ls):
    """Whole and split row groups; every other row is right."""
    c = Case(kind, 64, ls, [2] * 3, 16, window=0 if kind == "fp4" else 1 << 20, seed=41)
    hit = [(0, 3, 5), (3, 0, 575), (4, 15, 0), (5, 7, 511)]  # token, head, dim
    clean = c.query.clone()
    for t, h, d in hit:
        c.query[t, h, d] = float("nan")
    c.run()
    for t, h, _ in hit:
        assert c.out[t, h].isnan().all() and c.lse[t, h].isnan()
    dirty = Case(kind, 64, ls, [2] * 3, 16, window=0 if kind == "fp4" else 1 << 20, seed=41)
    dirty.query.copy_(clean)
    dirty.run()
    assert dirty.status() == 0
    for t, h, _ in hit:
        c.out[t, h], c.lse[t, h] = dirty.out[t, h], dirty.lse[t, h]
    assert torch.equal(c.out, dirty.out) and torch.equal(c.lse, dirty.lse)
    dirty.check(**P[kind])


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp4"])
@pytest.mark.parametrize("ls", [[300, 70], [9000, 200]])
def test_a_nan_in_a_visible_row_shows_in_the_lse(kind, ls):
    c = Case(kind, 64, ls, [1, 1], 16, window=0 if kind == "fp4" else 1 << 20, seed=42)
    page, row = int(c.bt_host[0, 2]), 17
    if kind == "fp4":
        c.cache.view(c.cache.shape[0], -1)[page, 64 * 288 + 36 * row + 33] = 0x7F  # a scale of the RoPE dims
    else:
        c.cache.view(torch.uint8 if kind == "e4m3" else torch.int16)[page, row, 530] = 0x7F if kind == "e4m3" else 0x7FFF
    c.run()
    torch.cuda.synchronize()
    assert c.lse[0].isnan().all() and c.out[0].isnan().all()
    for t, o, e, (a, d, v) in c.reference():
        if t == 1:
            assert (c.lse[1].double() - e).abs().max() < 1e-4 and ((c.out[1].double() - o).abs() <= a * 2.0 ** -6).all()


ROW = {"bf16": (576, torch.bfloat16), "e4m3": (576, torch.float8_e4m3fn), "fp4": (324, torch.uint8)}
PAGES = {"bf16": 60000, "e4m3": 120000, "fp4": 210000}  # of 64 rows: past 2^32 bytes


def _far(kind, cache, at):
    """The cache's pages from page ``at`` on of one that is longer than 2^32 bytes."""
    row, dtype = ROW[kind]
    far = torch.empty(PAGES[kind], 64, row, dtype=dtype, device="cuda")
    far[at:at + cache.shape[0]] = cache
    assert at * far[0].numel() * far.element_size() > 1 << 32
    return far


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp4"])
def test_pages_past_four_gigabytes(kind):
    c = Case(kind, 64, [700, 90, 3000], [2] * 3, 64, window=400, sinks=3, seed=43).run()
    c.check(**P[kind])
    out, lse = c.out.clone(), c.lse.clone()
    at = PAGES[kind] - c.cache.shape[0]
    far = _far(kind, c.cache, at)
    got, got_lse = mla.decode(c.query.view(3, 2, 64, 576), far, c.workspace, c.tables + at, c.lens, c.max_len,
                              bmm1_scale=c.bmm1, bmm2_scale=c.bmm2, return_lse=True, window=400, sinks=3)
    torch.cuda.synchronize()
    assert torch.equal(got.view_as(out), out) and torch.equal(got_lse, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp4"])
def test_append_and_gather_past_four_gigabytes(kind):
    T, row, dtype = 9, *ROW[kind]
    g = torch.Generator().manual_seed(44)
    x = torch.randn(T, 576, generator=g).to(torch.bfloat16).cuda()
    tables = torch.randperm(T, generator=g).int().cuda()[:, None]
    lens = torch.arange(1, T + 1, dtype=torch.int32, device="cuda") * 7
    table = mla.rope_table(64)
    near = torch.zeros(T, 64, row, dtype=torch.uint8 if dtype != torch.bfloat16 else torch.bfloat16, device="cuda").view(dtype)
    at = PAGES[kind] - T
    far = _far(kind, near, at)
    for cache, t in ((near, tables), (far, tables + at)):
        mla.cache_append(x[:, :512], x[:, 512:], cache, t, lens, rope_table=table, q_len=1)
    assert torch.equal(far[at:].view(torch.uint8), near.view(torch.uint8)) and near.view(torch.uint8).any()
    assert torch.equal(mla.cache_gather(far, tables + at, lens, q_len=1), mla.cache_gather(near, tables, lens, q_len=1))


def _static(c):
    fn = mla.load_library().mla_decode_run_static_workspace
    vp = ctypes.c_void_p
    fn.argtypes = [vp, vp, vp, vp, vp, vp, ctypes.c_int64, ctypes.c_float, ctypes.c_float, vp, vp, vp]
    fn.restype = ctypes.c_int
    out, lse = torch.full_like(c.out, 3.0), torch.full_like(c.lse, 3.0)
    rc = fn(c.plan.handle, c.query.data_ptr(), c.cache.data_ptr(), c.tables.data_ptr(), c.lens.data_ptr(),
            c.indptr.data_ptr() if c.packed else None, c.query.shape[0] if c.packed else 0, c.bmm1, c.bmm2, out.data_ptr(),
            lse.data_ptr(), torch.cuda.current_stream().cuda_stream)
    return rc, out, lse


@pytest.mark.gpu
@pytest.mark.parametrize("kind,window", [("fp4", 0), ("fp4", 500), ("bf16", 2500), ("e4m3", 500)])
def test_static_workspace(kind, window):
    c = Case(kind, 64, [5000, 70, 900], [3, 1, 2], 128, packed=True, window=window, seed=45, pad=2).run()
    c.check(**P[kind])
    for _ in range(2):
        rc, out, lse = _static(c)
        assert rc == 0
        torch.cuda.synchronize()
        assert torch.equal(out, c.out) and torch.equal(lse, c.lse)


@pytest.mark.gpu
@pytest.mark.parametrize("q_fp8", [False, True])
def test_host_entry_over_4_bits_packed(q_fp8):
    c = Case("fp4", 32, [500, 90, 2000], [1, 4, 2], 16, packed=True, seed=46, q_fp8=q_fp8).run()
    c.check()
    staging = torch.empty(c.plan.staging_bytes(c.T), dtype=torch.uint8, device="cuda")
    h_out, h_lse = torch.empty(c.out.shape, dtype=torch.bfloat16).pin_memory(), torch.empty(c.lse.shape).pin_memory()
    c.plan.run_host(c.query.cpu().pin_memory(), c.cache, c.tables.cpu().pin_memory(), c.lens.cpu().pin_memory(), h_out,
                    staging=staging, workspace=c.workspace, h_qo_indptr=c.indptr.cpu().pin_memory(), total_q=c.T,
                    h_lse=h_lse, bmm1_scale=c.bmm1, bmm2_scale=c.bmm2)
    torch.cuda.synchronize()
    assert torch.equal(h_out, c.out.cpu()) and torch.equal(h_lse, c.lse.cpu())


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
def test_context_parallel_ranks_without_a_row(causal):
    """Five ranks share requests of 3, 130 and 4 rows: some hold none of the short ones."""
    W, ls, qs, H = 5, [3, 130, 4], [2] * 3, 16
    whole = Case("fp4", 32, ls, qs, H, seed=47, bmm2=1.0, causal=causal).run()
    whole.check()
    outs, lses, empty = [], [], 0
    for r in range(W):
        n = [len(range(r, L, W)) for L in ls]
        sub = Case("fp4", 32, [max(1, k) for k in n], qs, H, seed=48, bmm2=1.0, causal=False)
        for b, L in enumerate(ls):
            for k, g in enumerate(range(r, L, W)):
                src = whole.cache.view(whole.cache.shape[0], -1)[int(whole.bt_host[b, g // 32])]
                dst = sub.cache.view(sub.cache.shape[0], -1)[int(sub.bt_host[b, k // 32])]
                i, j = g % 32, k % 32
                dst[j * 288:(j + 1) * 288] = src[i * 288:(i + 1) * 288]
                dst[9216 + j * 36:9216 + (j + 1) * 36] = src[9216 + i * 36:9216 + (i + 1) * 36]
        sub.lens.copy_(torch.tensor(n, dtype=torch.int32))
        plan = mla.Plan(batch=3, num_heads=H, max_seq_len_q=2, max_seq_len=sub.max_len, page_size=32,
                        max_pages_per_req=sub.tables.shape[1], num_pages=sub.cache.shape[0], packed=False, causal=causal,
                        kv_dtype="fp4", return_lse=True, cp_world=W, cp_rank=r)
        ws = torch.full((plan.workspace_bytes,), 0xA5, dtype=torch.uint8, device="cuda")
        plan.run(whole.query, sub.cache, sub.tables, sub.lens, sub.out, lse=sub.lse, workspace=ws,
                 bmm1_scale=whole.bmm1, bmm2_scale=1.0, seq_lens_global=whole.lens if causal else None)
        torch.cuda.synchronize()
        off = mla.mla_decode_status_offset()
        assert int(ws[off:off + 4].view(torch.int32)) == 0
        for b, L in enumerate(ls):
            for i in range(2):
                last = L - 2 + i if causal else L - 1
                if not any(g <= last for g in range(r, L, W)):
                    empty += 1
                    assert (sub.out[2 * b + i] == 0).all() and (sub.lse[2 * b + i] == -float("inf")).all()
        outs.append(sub.out)
        lses.append(sub.lse)
    assert empty >= 6
    out, lse = mla.merge_states(torch.stack(outs), torch.stack(lses))
    for t, o, e, (a, d, v) in whole.reference():
        # the shards' outputs are rounded to bf16 once more
        assert ((out[t].double() - o).abs() <= o.abs() * 2.0 ** -8 + a * (2.0 ** -8 + 2.0 ** -10) + v * 2.0 ** -32).all()
        assert (lse[t].double() - e).abs().max() < 1e-4
