"""Scales that the append and the gather refuse (on the host: no address is read)."""
import ctypes

import pytest

import paged_mla_decode_03_gb300 as mla
from test_cache_ops import A, c_append, lib  # noqa: F401


@pytest.mark.parametrize("scale", [1e-39, 2.0 ** -127, 1e-45])
@pytest.mark.parametrize("params,name", [(dict(kv_dtype=1), "kvs"), (dict(kv_dtype=2), "kvs"), (dict(q_dtype=1), "qs")])
def test_a_scale_whose_reciprocal_passes_the_range(lib, params, name, scale):  # noqa: F811
    assert c_append(lib, params, **{name: scale}) == -1


@pytest.mark.parametrize("scale", [1e-39, 1e-45])
def test_gather_refuses_the_same_scales(lib, scale):  # noqa: F811
    p = mla.MlaCacheParams(batch=2, packed=0, q_len=1, page_size=64, max_pages_per_req=4, num_pages=8, kv_dtype=1)
    assert lib.mla_cache_gather(ctypes.byref(p), A, A, A, None, 2, scale, A, None, None) == -1
