"""More of the decode over 4 bits and with a window: calls that the first tests leave out."""
import pytest
import torch

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
