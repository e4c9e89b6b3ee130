"""What the kernels of a decode over shared prefixes rest on, read from the source: a grid sees what the
grids before it wrote once it has itself waited for them, not because a grid between them has."""
import re

from test_pair_ordering import _function, _read


def _first(body, pattern):
    return re.search(pattern, body).start()


def test_the_join_reads_nothing_before_its_wait():
    body = _function(_read("mla_prefix.cu"), "join_prefix_kernel")
    wait = body.index("pdl_wait();")
    assert wait < _first(body, r"kHdrNumCombine") and wait < _first(body, r"=\s*entries\[")


def test_widening_reads_nothing_before_its_wait():
    body = _function(_read("mla_prefix.cu"), "widen_prefix_kernel")
    assert body.index("pdl_wait();") < _first(body, r"of\[groups\]")


def test_every_decode_waits_before_its_work_list():
    src = _read("mla_decode_pair.cu")
    body = src[src.index("decode_pair_kernel(const Problem p"):src.index("cudaLaunchConfig_t pair_launch(")]
    lines = [line.strip() for line in body[:_first(body, r"worker_begin\[worker\]")].split("\n")]
    at = lines.index("pdl_wait();")  # whichever plan it is of
    assert lines[at + 1] == "pdl_launch_dependents();"
