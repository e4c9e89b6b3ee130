"""Work lists of plans with a sliding window or a 4-bit cache: the partition
kernels' source run on CPU threads, under the sanitizers, against what a work
list has to be (tests/test_partition_host.py holds the other plans to a model)."""
import os
import shutil
import subprocess

import numpy as np
import pytest

from test_partition_host import CSRC, HERE, ROOT, _function_text

TILE, ROWS, OVERHEAD, CUT = 64, 128, 5, 6


@pytest.fixture(scope="module")
def runner(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    out = tmp_path_factory.mktemp("window_partition")
    common = open(os.path.join(CSRC, "mla_common.cuh")).read().replace("#include <cuda_runtime.h>\n", "")
    (out / "mla_common_host.h").write_text(
        common.replace("#pragma once", "#pragma once\ninline unsigned char* g_scratch = nullptr;", 1))
    src = open(os.path.join(CSRC, "mla_partition.cu")).read()
    src = src.replace('#include "mla_common.cuh"\n#include "sm100_ptx.cuh"\n',
                      '#include "shim.h"\n#include "mla_common_host.h"\n')
    src = src.replace("ptx::pdl_launch_dependents();", "")
    src = src.replace("extern __shared__ __align__(16) unsigned char scratch_smem[];",
                      "unsigned char* scratch_smem = g_scratch;")
    (out / "partition_host.inc").write_text(src[:src.index("cudaError_t launch_partition(")] + "}  // namespace mla\n")
    src = open(os.path.join(CSRC, "mla_partition_pair.cu")).read()
    src = src.replace('#include "mla_common.cuh"\n#include "sm100_ptx.cuh"\n', "")
    src = src.replace("ptx::pdl_launch_dependents();", "")
    (out / "partition_pair_host.inc").write_text(src[:src.index("bool partition_pair_picked(")] + "}  // namespace mla\n")
    api = open(os.path.join(CSRC, "mla_api.cu")).read()
    (out / "make_layout.inc").write_text(_function_text(api, "int make_layout(") + "\n")
    exe = out / "window_partition"
    r = subprocess.run([cxx, "-std=c++20", "-O1", "-g", "-fsanitize=address,undefined",
                        "-fno-sanitize-recover=undefined", "-pthread", "-I", str(out), "-I", HERE, "-I",
                        os.path.join(ROOT, "include"), os.path.join(HERE, "window_driver.cpp"), "-o", str(exe)],
                       capture_output=True, text=True)
    if r.returncode != 0 and ("No such file" in r.stderr or "cannot find -l" in r.stderr):
        pytest.skip("host toolchain lacks C++20 <barrier> or the sanitizers: " + r.stderr[-300:])
    assert r.returncode == 0, r.stderr[-3000:]
    return exe, out


def _rows_of(begin, end, skip, sinks):
    """The cache rows that virtual rows [begin, end) stand for."""
    s = -(-sinks // TILE) * TILE
    v = np.arange(begin, end)
    return np.where(v < s, v, v + skip)


def _run(runner, ls, qo, max_q, max_len, H, packed, causal, window, sinks, kv_dtype, n_workers, kernel):
    """The work list (head, items, worker ranges, combine entries), or None where the
    kernel does not take the plan."""
    exe, out = runner
    with open(out / "in.txt", "w") as f:
        f.write(f"{len(ls)} {H} {int(packed)} {max_q} {max_len} {n_workers} {int(causal)} {window} {sinks} "
                f"{kv_dtype} {qo[-1]}\n{' '.join(map(str, ls))}\n{' '.join(map(str, qo))}\n")
    r = subprocess.run([str(exe), str(out / "in.txt"), str(out / "out.txt"), kernel], capture_output=True, text=True,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1"), timeout=300)
    if kernel == "pair" and r.returncode == 4:
        return None
    assert r.returncode == 0, (r.returncode, r.stderr[-3000:])
    return [[int(x) for x in line.split()] for line in open(out / "out.txt").read().split("\n")[:4]]


def _check(runner, ls, qs, H, packed, causal, window, sinks, kv_dtype, n_workers, kernel):
    qo = np.concatenate([[0], np.cumsum(qs)])
    args = (runner, ls, qo, max(qs), max(ls), H, packed, causal, window, sinks, kv_dtype, n_workers)
    got = _run(*args, kernel)
    if got is None:
        return False
    if kernel == "pair":
        assert got == _run(*args, "block")
    head, items, ranges, combine = got
    status, n_items, n_combine, max_partials, max_combine = head
    assert status == 0 and n_combine <= max_combine
    items = [items[10 * i:10 * i + 10] for i in range(n_items)]
    combine = [combine[8 * i:8 * i + 8] for i in range(n_combine)]
    # every item belongs to one worker
    assert ranges[0] == 0 and ranges[-1] == n_items and all(a <= b for a, b in zip(ranges, ranges[1:]))
    by_group, costs, slots = {}, [], []
    for it in items:
        by_group.setdefault((it[0], it[1]), []).append(it)
    for b, (L, q) in enumerate(zip(ls, qs)):
        for g in range(-(-q * H // ROWS)):
            parts = sorted(by_group.pop((b, g)), key=lambda it: it[2])
            # the group's parts follow on one another from the first virtual row to the last
            assert parts[0][2] == 0 and all(a[3] == c[2] for a, c in zip(parts, parts[1:]))
            assert all(it[2] % TILE == 0 and it[2] < it[3] for it in parts)
            end = parts[-1][3]
            skip = L - end
            assert skip >= 0 and skip % TILE == 0
            rows = _rows_of(0, end, skip, sinks if window else 0)
            assert len(set(rows)) == end and rows.max() == L - 1 and rows.min() >= 0
            # every row that a query row of the request sees is among them, and no whole
            # tile more than that needs
            first = (L - q if causal else L - 1) - window + 1 if window else 0
            seen = set(range(max(first, 0), L)) | set(range(min(sinks, L) if window else L))
            assert seen <= set(rows)
            assert len(rows) <= len(seen) + 2 * TILE
            for it in parts:
                assert it[5] == q and it[6] == L and it[7] == qo[b]
                assert (it[4] >= 0) == (len(parts) > 1) and (it[8] >= 0) == (len(parts) > 1)
            if len(parts) > 1:
                e = combine[parts[0][8]]
                assert e[:2] == [b, g] and e[4] == len(parts) and e[5] == q and e[6] == qo[b]
                assert [it[4] for it in parts] == [e[2] + k * e[3] for k in range(len(parts))]
                assert len({it[8] for it in parts}) == 1
                slots += [it[4] for it in parts]
            costs.append((OVERHEAD + -(-end // TILE), len(parts)))
    assert not by_group
    assert n_items == sum(n for _, n in costs) and n_combine == sum(n > 1 for _, n in costs)
    assert len(set(slots)) == len(slots) and all(0 <= s < max_partials for s in slots)
    # uncut where that costs the largest worker no more than kCutTiles tiles
    if len(costs) <= n_workers and max(c for c, _ in costs) <= sum(c for c, _ in costs) // n_workers + CUT:
        assert all(n == 1 for _, n in costs)
        assert max(b - a for a, b in zip(ranges, ranges[1:])) <= 1
    # a worker has at most an even share, a tile, and an overhead for each group it shares in
    share = sum(c for c, _ in costs) / max(1, min(n_workers, sum(c for c, _ in costs) // 4))
    for a, b in zip(ranges, ranges[1:]):
        work = sum(-(-(it[3] - it[2]) // TILE) for it in items[a:b])
        if len(slots):
            assert work <= share + OVERHEAD + 1
    return True


@pytest.mark.parametrize("kernel", ["block", "pair"])
@pytest.mark.parametrize("kv_dtype,window,sinks", [(0, 64, 0), (0, 1000, 4), (1, 130, 70), (2, 0, 0), (2, 33, 1)])
def test_a_batch_of_equal_requests(runner, kernel, kv_dtype, window, sinks):
    assert _check(runner, [2000] * 64, [1] * 64, 128, False, True, window, sinks, kv_dtype, 76, kernel)
    assert _check(runner, [2000] * 3, [4] * 3, 16, False, True, window, sinks, kv_dtype, 76, kernel)
    assert _check(runner, [1], [1], 16, False, True, window, sinks, kv_dtype, 5, kernel)


@pytest.mark.parametrize("kernel", ["block", "pair"])
@pytest.mark.parametrize("seed", range(16))
def test_random_shapes(runner, kernel, seed):
    rng = np.random.default_rng(900 + seed)
    B = int(rng.integers(1, 90))
    packed = bool(rng.integers(2))
    top = int(rng.choice([1, 2, 4, 40]))
    qs = [int(rng.integers(1, top + 1)) if packed else top for _ in range(B)]
    far = int(rng.choice([1, 200, 3001, 40000]))
    ls = [q + int(rng.integers(0, far)) for q in qs]
    window = int(rng.choice([0, 1, 63, 64, 65, 700, 5000]))
    _check(runner, ls, qs, int(rng.choice([16, 32, 64, 128])), packed, bool(rng.integers(2)), window,
           int(rng.choice([0, 1, 64, 65, 500])) if window else 0, 2 if not window else int(rng.integers(3)),
           int(rng.integers(1, 77)), kernel)


@pytest.mark.parametrize("seed", range(8))
def test_bad_lengths_are_flagged_alike(runner, seed):
    """Lengths out of the contract: both forms stay in bounds (the sanitizers look),
    flag the same and leave the same list."""
    rng = np.random.default_rng(70 + seed)
    B = int(rng.integers(1, 40))
    qs = rng.integers(1, 5, B)
    ls = rng.integers(1, 500, B)
    qo = np.concatenate([[0], np.cumsum(qs)])
    qo[int(rng.integers(B + 1))] = int(rng.choice([-7, 0, qo[-1], 2 ** 30]))
    qo[-1] = max(1, qo[-1])
    ls[int(rng.integers(B))] = int(rng.choice([-5, 0, 10 ** 9]))
    args = (runner, ls, qo, 4, 500, 128, True, True, 100, 3, 0, 20)
    got = _run(*args, "pair")
    assert got[0][0] & 3
    assert got == _run(*args, "block")
