"""What ``decode`` refuses over a 4-bit cache or with a window: tensors that the kernels would
read or write past their end, or as another type."""
import pytest
import torch

import paged_mla_decode_03_gb300 as mla

B, SQ, H, PS, PAGES = 3, 2, 16, 32, 8


def _args(device, packed, kind="fp4"):
    cache = (torch.zeros(PAGES, PS, 324, dtype=torch.uint8, device=device) if kind == "fp4" else
             torch.zeros(PAGES, PS, 576, dtype=torch.bfloat16, device=device))
    q = torch.zeros(B * SQ, H, 576, dtype=torch.bfloat16, device=device)
    out = torch.zeros(B * SQ, H, 512, dtype=torch.bfloat16, device=device)
    return dict(query=q if packed else q.view(B, SQ, H, 576), kv_cache=cache,
                workspace=torch.zeros(1 << 20, dtype=torch.uint8, device=device),
                block_tables=torch.arange(B * 2, dtype=torch.int32, device=device).view(B, 2),
                seq_lens=torch.tensor([40, 33, 2], dtype=torch.int32, device=device),
                qo_indptr=torch.tensor([0, 2, 4, 6], dtype=torch.int32, device=device) if packed else None,
                out=out if packed else out.view(B, SQ, H, 512),
                lse=torch.zeros(B * SQ, H, device=device), global_lens=None)


def _twice(t):
    """The same values with a stride of two in the last dim."""
    return torch.stack([t, t], -1)[..., 0]


BAD = [  # argument, what becomes of it, only packed or fixed calls (None: both)
    ("query", _twice, None), ("query", lambda t: t[..., :512].contiguous(), None),
    ("query", lambda t: t.flatten(0, -2), None), ("query", lambda t: t[:-1].contiguous(), False),
    ("kv_cache", lambda t: t[::2], None), ("workspace", lambda t: t[::2], None),
    ("workspace", lambda t: t[:1].expand(1 << 30), None),
    ("seq_lens", lambda t: t.long(), None), ("seq_lens", lambda t: t.float(), None), ("seq_lens", _twice, None),
    ("seq_lens", lambda t: t[0], None), ("seq_lens", lambda t: t[None], None), ("seq_lens", lambda t: t[:2], None),
    ("block_tables", lambda t: t.long(), None), ("block_tables", lambda t: t.t().contiguous().t(), None),
    ("block_tables", lambda t: t[:2], None), ("block_tables", lambda t: t.flatten(), None),
    ("qo_indptr", lambda t: t.long(), True), ("qo_indptr", lambda t: t[:-1], True), ("qo_indptr", _twice, True),
    ("out", lambda t: t.float(), None), ("out", _twice, None), ("out", lambda t: t[:-1], None),
    ("lse", lambda t: t.double(), None), ("lse", lambda t: t.t().contiguous().t(), None), ("lse", lambda t: t[1:], None),
    ("global_lens", lambda t: torch.zeros(B, dtype=torch.int64), None),
    ("global_lens", lambda t: torch.zeros(B + 1, dtype=torch.int32), None),
]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("name,change,when", BAD)
def test_checks(packed, name, change, when):
    """On host tensors: the checks look at types, shapes, strides and devices alone."""
    good = _args("cpu", packed)
    mla._check_decode(**good)
    if when is not None and when != packed:
        return
    with pytest.raises(ValueError):
        mla._check_decode(**{**good, name: change(good[name])})


def test_what_is_left_out_is_not_checked():
    good = _args("cpu", False)
    mla._check_decode(**{**good, "out": None, "lse": None})


@pytest.mark.gpu
@pytest.mark.parametrize("kind,window", [("fp4", 0), ("fp4", 20), ("bf16", 20)])
@pytest.mark.parametrize("packed", [False, True])
def test_through_decode(kind, window, packed):
    good = _args("cuda", packed, kind)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")

    def call(return_lse=True, **kw):
        a = {**good, **kw}
        return mla.decode(a["query"], a["kv_cache"], ws if "workspace" not in kw else a["workspace"], a["block_tables"],
                          a["seq_lens"], 64, qo_indptr=a["qo_indptr"], max_seq_len_q=SQ, out=a["out"], lse=a["lse"],
                          return_lse=return_lse, window=window)

    out, lse = call()
    assert out is good["out"] and lse is good["lse"]
    assert call(out=None, lse=None)[0].shape == good["query"].shape[:-1] + (512,)
    assert call(return_lse=False, lse=good["lse"].double()) is good["out"]  # (an LSE that is not asked for)
    for name, change, when in BAD:
        if name == "global_lens" or (when is not None and when != packed):
            continue
        with pytest.raises(ValueError):
            call(**{name: change(good[name])})
    for name in ("kv_cache", "block_tables", "seq_lens", "out", "lse"):  # on another device
        with pytest.raises(ValueError):
            call(**{name: good[name].cpu()})
    torch.cuda.synchronize()
