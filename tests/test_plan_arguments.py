"""Arguments of a plan that would be taken for others: a window of 2^32 + 5 is not one of 5."""
import pytest
import torch

import paged_mla_decode_03_gb300 as mla
from paged_mla_decode_03_gb300 import build as mla_build


@pytest.mark.parametrize("kw", [dict(window=2 ** 32 + 5), dict(window=2 ** 31), dict(window=-2 ** 32 + 7),
                                dict(window=64, sinks=2 ** 32 + 3), dict(window=64, sinks=2 ** 31)])
def test_windows_and_sinks_past_32_bits(kw):
    mla_build.build()
    with pytest.raises(ValueError):
        mla.Plan(batch=2, num_heads=16, max_seq_len_q=1, max_seq_len=64, page_size=32, max_pages_per_req=2,
                 num_pages=8, packed=False, **kw)


@pytest.mark.parametrize("kv_dtype", ["nvfp4", "int4", "4bit", "FP4", 2, torch.uint8, torch.float16])
def test_a_cache_type_that_is_none(kv_dtype):
    """Taken for bf16, a 4-bit cache's rows would be read three times past their end."""
    mla_build.build()
    with pytest.raises(ValueError):
        mla.Plan(batch=2, num_heads=16, max_seq_len_q=1, max_seq_len=64, page_size=32, max_pages_per_req=2,
                 num_pages=8, packed=False, kv_dtype=kv_dtype)
