"""More of cache_append and cache_gather: calls that the first tests leave out."""
import pytest
import torch

import paged_mla_decode_03_gb300 as mla
from test_cache_ops import Setup, close_bf16, close_e4m3, new_cache


def _dirty(*shapes):
    """Leaves memory of these shapes full of NaN in the allocator's hands."""
    for s in [torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda") for shape in shapes]:
        del s


@pytest.mark.gpu
def test_rows_without_a_place_are_zeros_in_tensors_that_the_call_makes():
    s = Setup("bf16", 32, [40, 5], [3, 2], 16, packed=True, seed=21, pad=4)
    s.tables[0, 1] = -1  # the page of request 0's tokens
    cache = new_cache("bf16", s.pages, 32)
    _dirty((s.T, 16, 576), (s.T, 576))
    query = mla.cache_append(s.latent, s.k_pe, cache, s.tables, s.lens, rope_table=s.table, norm_weight=s.weight,
                             q_nope=s.q_nope, q_pe=s.q_pe, **s.which)
    _, _, q, tq = s.reference()
    close_bf16(query[3:5], q[3:5], (q.abs() + tq)[3:5], "query")
    assert (query[:3] == 0).all() and (query[5:] == 0).all()
    _dirty((s.T, 16, 576), (s.T, 576))
    rows = mla.cache_gather(cache, s.tables, s.lens, total_q=s.T, **s.which)
    assert (rows[:3] == 0).all() and (rows[5:] == 0).all() and (rows[3:5] != 0).any(-1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("power,eps", [(60, 1e-6), (60, 2.0 ** 100), (60, 2.0 ** 127), (62, 3e38), (70, 3e38), (100, 3e38), (0, 3e38)])
def test_an_eps_beside_a_sum_past_the_range(power, eps):
    """Latents whose squares' sum passes fp32's range, with an eps that counts beside their mean."""
    s = Setup("bf16", 32, [40], [3], 16, packed=False, seed=22)
    g = torch.Generator().manual_seed(23)
    x = torch.randn(3, 576, generator=g)
    x[:, :512] *= 2.0 ** power
    x = x.to(torch.bfloat16).cuda()
    s.latent, s.k_pe = x[:, :512], x[:, 512:]
    cache = new_cache("bf16", s.pages, 32)
    mla.cache_append(s.latent, s.k_pe, cache, s.tables, s.lens, rope_table=s.table, norm_weight=s.weight, eps=eps, q_len=3)
    y, ty, _, _ = s.reference(eps=float(torch.tensor(eps, dtype=torch.float32)))
    s.check(cache, y, ty, 1.0, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("power", [65, 70, 120])
def test_small_latents_beside_huge_ones(power):
    s = Setup("bf16", 32, [40], [2], 16, packed=False, seed=24)
    g = torch.Generator().manual_seed(25)
    x = torch.randn(2, 576, generator=g)
    x[:, :512:2] *= 2.0 ** power
    x[:, 1:512:2] *= 2.0 ** (power - 118)  # normed: about 2^-118
    x = x.to(torch.bfloat16).cuda()
    s.latent, s.k_pe = x[:, :512], x[:, 512:]
    cache = new_cache("bf16", s.pages, 32)
    mla.cache_append(s.latent, s.k_pe, cache, s.tables, s.lens, rope_table=s.table, norm_weight=s.weight, q_len=2)
    y, ty, _, _ = s.reference()
    s.check(cache, y, ty, 1.0, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp4"])
@pytest.mark.parametrize("q_fp8", [False, True])
@pytest.mark.parametrize("heads,packed", [(16, False), (128, True)])
def test_every_cache_with_every_query(kind, q_fp8, heads, packed):
    s = Setup(kind, 64, [70, 64, 3], [3, 3, 3], heads, packed=packed, seed=26, style="half", pad=2 if packed else 0)
    cache = new_cache(kind, s.pages, 64)
    query = torch.full((s.T, heads, 576), 3.0, dtype=torch.bfloat16, device="cuda")
    if q_fp8:
        query = query.to(torch.float8_e4m3fn)
    kvs, qsc = (0.0125 if kind == "e4m3" else 1.0), (0.0110 if q_fp8 else 1.0)
    mla.cache_append(s.latent, s.k_pe, cache, s.tables, s.lens, rope_table=s.table, norm_weight=s.weight,
                     rope_style="half", kv_scale=kvs, q_nope=s.q_nope, q_pe=s.q_pe, query=query, q_scale=qsc, **s.which)
    y, ty, q, tq = s.reference()
    s.check(cache, y, ty, kvs, kind)
    inv = float(torch.tensor(1.0 / qsc, dtype=torch.float32))
    (close_e4m3 if q_fp8 else close_bf16)(query[:s.n], q * inv, (q.abs() + tq) * inv, "query")
    assert (query[s.n:].float() == 3.0).all()
