"""What the MMAs across CTA pairs rest on, read from the source: the even CTA issues
MMAs that read what the odd one's threads wrote, so the barriers that both CTAs arrive
at are released and acquired at cluster scope."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_mla_decode_03_gb300", "csrc")


def _read(name):
    return open(os.path.join(CSRC, name)).read()


def _function(text, name):
    """The body of the function of that name (its first definition)."""
    at = re.search(rf"\b{name}\([^;{{]*\{{", text).end()
    depth, end = 1, at
    while depth:
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        end += 1
    return text[at:end]


def test_no_status_is_reported_before_the_partitioner_has_written_the_word():
    """The partitioner releases the decode kernel at its start and stores the whole word later."""
    src = _read("mla_decode_pair.cu")
    body = src[src.index("decode_pair_kernel(const Problem p"):src.index("cudaLaunchConfig_t pair_launch(")]
    first = re.search(r"kHdrStatus[^;]*kStatus\w+", body).start()
    assert "pdl_wait()" in body[:first]


def test_arrivals_at_the_other_cta_release_at_cluster_scope():
    body = _function(_read("sm100_ptx.cuh"), "mbar_arrive_pair")
    arrive = body.index("mbarrier.arrive.")
    assert "relaxed.cluster" in body[arrive:]
    assert re.search(r"fence\.proxy\.async::generic\.release\.\S*\.cluster;", body[:arrive])


def test_waits_on_shared_barriers_acquire_at_cluster_scope():
    """K, V, P, the query and free score buffers: the odd CTA's threads arrive too."""
    src = _read("mla_decode_pair.cu")
    issue = src[src.index("QK issue"):src.index("softmax, correction, epilogue", src.index("QK issue"))]
    waits = re.findall(r"(wait_\w+)\(c, ([A-Z]+_[A-Z]+)", issue)
    assert {b for _, b in waits} == {"S_EMPTY", "Q_FULL", "K_FULL", "V_FULL", "P_FULL"}
    assert all(f == "wait_pair" for f, _ in waits), waits
    body = _function(src, "wait_pair")
    assert "fence_acquire_pair()" in body[body.index("mbar_try_wait_pair"):]
    ptx = _read("sm100_ptx.cuh")
    assert ".relaxed.cluster." in _function(ptx, "mbar_try_wait_pair")
    assert re.search(r"fence\.proxy\.async::generic\.acquire\.\S*\.cluster;", _function(ptx, "fence_acquire_pair"))


def test_what_a_cta_wrote_is_passed_on_with_a_release():
    src = _read("mla_decode_pair.cu")
    assert set(re.findall(r"arrive_leader\(c, ([A-Z]+_[A-Z]+)", src)) == {"Q_FULL", "K_FULL", "V_FULL", "P_FULL"}
    assert "mbar_arrive_pair(" in _function(src, "arrive_leader")
    # the one arrival without a release hands back what was read, not what was written
    assert re.findall(r"mbar_arrive_cluster_relaxed\([^;]*?([A-Z]+_[A-Z]+)", src) == ["S_EMPTY"]
