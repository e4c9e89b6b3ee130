"""Reordering by tables and spare pages that name no page: flagged, and what the tables name stays whole."""
import pytest
import torch

import paged_mla_decode_03_gb300 as mla
from test_beam import Beams


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp4"])
@pytest.mark.parametrize("where", ["spare", "parent"])
@pytest.mark.parametrize("bad", ["-1", "last", "far"])
def test_a_page_that_is_none_is_not_taken(kind, where, bad):
    b = Beams(kind, 32, [70, 45], 3, 2, seed=4)
    bad = {"-1": -1, "last": b.caches[0].shape[0], "far": 2 ** 31 - 1}[bad]
    b.parents.copy_(torch.tensor([[1, 1, 0], [1, 2, 0]], dtype=torch.int32))
    if where == "spare":
        b.spare[0] = bad      # beam 0 has no page to copy to
    else:
        b.tables[1, 2] = bad  # its parent's page of the last 6 rows is none
    tables, spare = b.tables.cpu().numpy().copy(), b.spare.cpu().numpy().copy()
    before = [c.view(torch.uint8).clone() for c in b.caches]
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.cache_reorder(b.caches, b.tables, b.lens, b.parents, b.spare, status=word)
    torch.cuda.synchronize()
    assert int(word) == 16
    want, kept = tables.copy(), spare.copy()
    want[0, :2] = tables[1, :2]           # whole pages go by reference; the third one's place stays
    want[2, :2], want[2, 2], kept[2] = tables[0, :2], spare[2], tables[2, 2]
    for w, p in ((3, 4), (4, 5), (5, 3)):  # the other request is untouched by it
        want[w, :1], want[w, 1], kept[w] = tables[p, :1], spare[w], tables[w, 1]
    assert (b.tables.cpu().numpy() == want).all() and (b.spare.cpu().numpy() == kept).all()
    for old, new in zip(before, b.caches):  # beam 0's page keeps its rows, and a spare page that is one
        for page in [want[0, 2]] + [kept[0]] * (where == "parent"):
            assert torch.equal(old[page], new.view(torch.uint8)[page])
