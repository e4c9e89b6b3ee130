"""Tensors that the binding makes for a call on a given stream belong to that stream: they
neither take memory that the current stream still uses, nor give theirs back to it."""
import pytest
import torch

import paged_mla_decode_03_gb300 as mla

SLEEP = 40_000_000  # cycles: some 20 ms


def _makers():
    g = torch.Generator().manual_seed(1)
    T, H, ps = 64, 16, 32

    def rows(*shape):
        return torch.randn(*shape, generator=g).to(torch.bfloat16).cuda()

    x, qn, qp = rows(T, 576), rows(T, H, 512), rows(T, H, 64)
    cache = torch.zeros(T, ps, 324, dtype=torch.uint8, device="cuda")
    tables = torch.arange(T, dtype=torch.int32, device="cuda")[:, None]
    lens = torch.full((T,), 7, dtype=torch.int32, device="cuda")
    table = mla.rope_table(32)
    parts = torch.randn(2, 512, 300, generator=g).to(torch.bfloat16).cuda().transpose(1, 2)  # (copied by the call)
    lses = torch.randn(300, 2, generator=g).cuda().t()
    return {
        "merge": lambda s: mla.merge_states(parts, lses, stream=s)[0],
        "append": lambda s: mla.cache_append(x[:, :512], x[:, 512:], cache, tables, lens, rope_table=table, q_len=1,
                                             q_nope=qn, q_pe=qp, stream=s),
        "gather": lambda s: mla.cache_gather(cache, tables, lens, q_len=1, stream=s),
        "table": lambda s: mla.rope_table(4096, stream=s),
    }


@pytest.fixture(scope="module")
def makers():
    m = _makers()
    m["append"](None)
    torch.cuda.synchronize()
    return m


def _as(kind, stream):
    return stream if kind == "object" else stream.cuda_stream


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["object", "handle"])
@pytest.mark.parametrize("name", ["append", "gather", "table", "merge"])
def test_memory_that_the_current_stream_still_uses_is_left_alone(makers, name, kind):
    side = torch.cuda.Stream()
    want = makers[name](None).clone()
    torch.cuda.synchronize()
    used = torch.empty_like(want)
    torch.cuda._sleep(SLEEP)
    used.fill_(7)  # runs after the call below has
    del used
    got = makers[name](_as(kind, side))
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["object", "handle"])
@pytest.mark.parametrize("name", ["append", "gather", "table", "merge"])
def test_memory_that_the_kernel_still_writes_is_not_given_away(makers, name, kind):
    side = torch.cuda.Stream()
    shape = makers[name](None)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
    got = makers[name](_as(kind, side))
    del got
    other = torch.empty_like(shape).fill_(7)
    torch.cuda.synchronize()
    assert (other == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["append", "gather", "table", "merge"])
def test_the_default_stream_by_its_handle(makers, name):
    want = makers[name](None).clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = makers[name](0)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_the_table_is_allocated_on_the_given_stream(monkeypatch):
    """The order of things on the host alone, with the GPU's part taken out."""
    import contextlib
    import types
    on, made = [], []

    @contextlib.contextmanager
    def stream(s):
        on.append(s)
        yield
        on.pop()

    def empty(shape, **kw):
        made.append(list(on))
        return torch.zeros(shape)

    monkeypatch.setattr(mla, "torch", types.SimpleNamespace(
        empty=empty, float32=torch.float32, device=torch.device,
        cuda=types.SimpleNamespace(stream=stream, Stream=torch.cuda.Stream,
                                   ExternalStream=lambda handle, device: ("external", handle, device.index),
                                   default_stream=lambda dev: ("default", dev))))
    monkeypatch.setattr(mla, "load_library", lambda: types.SimpleNamespace(mla_rope_table=lambda *a: 0))
    monkeypatch.setattr(mla, "_call_on", lambda dev, fn, *a: fn(*a))
    monkeypatch.setattr(mla, "_stream_of", lambda s, dev: s)
    for handle in (4096, 0, None):
        mla.rope_table(8, device="cuda:1", stream=handle)
    assert made == [[("external", 4096, 1)], [("default", 1)], []]
