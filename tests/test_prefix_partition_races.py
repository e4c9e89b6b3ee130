"""The partitioner of plans with shared prefixes under the thread sanitizer: its source on host
threads, one for each CUDA thread, so that shared memory that a warp reads while another
writes it shows, whatever the values come out as."""
import os
import platform
import shutil
import subprocess

import pytest

from test_partition_host import CSRC, HERE, ROOT
from test_prefix_partition import _case


@pytest.fixture(scope="module")
def runner(tmp_path_factory):
    cxx, setarch = shutil.which("g++"), shutil.which("setarch")
    if cxx is None or setarch is None:
        pytest.skip("no g++ or setarch")
    out = tmp_path_factory.mktemp("prefix_races")
    common = open(os.path.join(CSRC, "mla_common.cuh")).read().replace("#include <cuda_runtime.h>\n", "")
    (out / "mla_common_host.h").write_text(
        common.replace("#pragma once", "#pragma once\ninline unsigned char* g_scratch = nullptr;", 1))
    (out / "mla_prefix_host.h").write_text(
        open(os.path.join(CSRC, "mla_prefix.cuh")).read().replace('#include "mla_common.cuh"\n', ""))
    src = open(os.path.join(CSRC, "mla_prefix.cu")).read()
    src = "\n".join(line for line in src[:src.index("// The join:")].split("\n")
                    if not line.startswith("#include") or line.endswith(("<algorithm>", "<climits>")))
    src = src.replace("ptx::pdl_launch_dependents();", "")
    src = src.replace("extern __shared__ __align__(16) unsigned char prefix_smem[];", "unsigned char* prefix_smem = g_scratch;")
    (out / "partition_prefix_host.inc").write_text(src + "}  // namespace mla\n")
    r = subprocess.run([cxx, "-std=c++20", "-O1", "-g", "-fsanitize=thread", "-pthread", "-I", str(out), "-I", HERE, "-I",
                        os.path.join(ROOT, "include"), os.path.join(HERE, "prefix_driver.cpp"), "-o", str(out / "plain")],
                       capture_output=True, text=True)
    if r.returncode != 0 and ("No such file" in r.stderr or "cannot find -l" in r.stderr):
        pytest.skip("host toolchain lacks C++20 <barrier> or the sanitizer: " + r.stderr[-300:])
    assert r.returncode == 0, r.stderr[-3000:]
    # (the sanitizer's shadow wants addresses that are not spread too far)
    exe = out / "run"
    exe.write_text(f'#!/bin/sh\nexec {setarch} {platform.machine()} -R {out}/plain "$@"\n')
    exe.chmod(0o755)
    probe = subprocess.run([str(exe)], capture_output=True, text=True)
    if probe.returncode != 2:  # (no arguments)
        pytest.skip("the thread sanitizer does not start here: " + probe.stderr[-300:])
    return exe, out


@pytest.mark.parametrize("scratch", [False, True])
def test_rows_that_are_widened(runner, scratch):
    assert _case(runner, [32], [20000], lambda i: 100 + 30 * i, [1], 128, False, True, 2, 76, uniform=True, wide=True,
                 global_scratch=scratch) == {0}
    assert _case(runner, [40, 2, 50], [9000, 4000, 7000], lambda i: 3 + i, [3, 1, 2], 64, True, True, 1, 76, gap=2, wide=True,
                 global_scratch=scratch) >= {0, 2}


@pytest.mark.parametrize("scratch", [False, True])
def test_shared_rows_and_requests_on_their_own(runner, scratch):
    assert _case(runner, [96], [6000], lambda i: 64 + 20 * i, [1], 16, False, True, 0, 76, uniform=True,
                 global_scratch=scratch) == {0}
    # nothing is shared: the list is made once more
    assert _case(runner, [8] * 4, [640] * 4, lambda i: 10, [1], 128, False, True, 0, 76, uniform=True,
                 global_scratch=scratch) == set()
    assert _case(runner, [30, 1, 25], [5000, 9000, 3001], lambda i: 5 + i, [1, 3, 2], 16, True, True, 0, 76, gap=3,
                 global_scratch=scratch) >= {0}


@pytest.mark.parametrize("kv", [0, 2])
def test_more_requests_than_threads(runner, kv):
    assert _case(runner, [700, 900], [2000, 1300], lambda i: 1 + i % 90, [1, 2], 16, True, True, kv, 76, gap=5) == {0, 1}
