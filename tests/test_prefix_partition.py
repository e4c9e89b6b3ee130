"""Work lists of plans with shared prefixes: the partitioner's source run on CPU threads,
under the sanitizers, against what a list has to be: every query row meets every cache row
that it sees exactly once, and the join finds every partial."""
import os
import shutil
import subprocess

import numpy as np
import pytest

from test_partition_host import CSRC, HERE, ROOT

TILE, ROWS = 64, 128


@pytest.fixture(scope="module")
def runner(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    out = tmp_path_factory.mktemp("prefix_partition")
    common = open(os.path.join(CSRC, "mla_common.cuh")).read().replace("#include <cuda_runtime.h>\n", "")
    (out / "mla_common_host.h").write_text(
        common.replace("#pragma once", "#pragma once\ninline unsigned char* g_scratch = nullptr;", 1))
    (out / "mla_prefix_host.h").write_text(
        open(os.path.join(CSRC, "mla_prefix.cuh")).read().replace('#include "mla_common.cuh"\n', ""))
    src = open(os.path.join(CSRC, "mla_prefix.cu")).read()
    for inc in ("<cuda_bf16.h>", "<cuda_fp16.h>", '"mla_common.cuh"', '"mla_prefix.cuh"', '"sm100_ptx.cuh"'):
        src = src.replace(f"#include {inc}\n", "")
    src = src.replace("ptx::pdl_launch_dependents();", "")
    src = src.replace("extern __shared__ __align__(16) unsigned char prefix_smem[];",
                      "unsigned char* prefix_smem = g_scratch;")
    src = src[:src.index("// The join:")] + "}  // namespace mla\n"
    (out / "partition_prefix_host.inc").write_text(src)
    exe = out / "prefix_partition"
    r = subprocess.run([cxx, "-std=c++20", "-O1", "-g", "-fsanitize=address,undefined",
                        "-fno-sanitize-recover=undefined", "-pthread", "-I", str(out), "-I", HERE, "-I",
                        os.path.join(ROOT, "include"), os.path.join(HERE, "prefix_driver.cpp"), "-o", str(exe)],
                       capture_output=True, text=True)
    if r.returncode != 0 and ("No such file" in r.stderr or "cannot find -l" in r.stderr):
        pytest.skip("host toolchain lacks C++20 <barrier> or the sanitizers: " + r.stderr[-300:])
    assert r.returncode == 0, r.stderr[-3000:]
    return exe, out


def _run(runner, ls, qo, max_q, max_len, H, packed, causal, kv, lens, indptr, n_workers, global_scratch=False):
    exe, out = runner
    uniform = indptr is None
    with open(out / "in.txt", "w") as f:
        f.write(f"{len(ls)} {H} {int(packed)} {max_q} {max_len} {n_workers} {int(causal)} {kv} {len(lens)} "
                f"{int(uniform)} {int(global_scratch)} {qo[-1]}\n")
        for v in (ls, qo, lens, [0] * (len(lens) + 1) if uniform else indptr):
            f.write(" ".join(map(str, v)) + "\n")
    r = subprocess.run([str(exe), str(out / "in.txt"), str(out / "out.txt")], capture_output=True, text=True,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1"), timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr[-3000:])
    return [[int(x) for x in line.split()] for line in open(out / "out.txt").read().split("\n")[:4]]


def _check(got, ls, qs, H, causal, lens, indptr, status=0):
    """-> the prefix groups that are shared."""
    head, items, ranges, entries = got
    assert head[0] == status
    n_items, n_entries, max_items, max_entries = head[1:]
    assert n_items <= max_items and n_entries <= max_entries
    assert ranges[0] == 0 and ranges[-1] == n_items and all(a <= b for a, b in zip(ranges, ranges[1:]))
    items = [items[10 * i:10 * i + 10] for i in range(n_items)]
    entries = [entries[9 * i:9 * i + 9] for i in range(n_entries)]
    q0 = np.concatenate([[0], np.cumsum(qs)])
    if indptr is None:
        indptr = [g * (len(ls) // len(lens)) for g in range(len(lens) + 1)]
    group_of = {b: g for g in range(len(lens)) for b in range(indptr[g], indptr[g + 1])}
    # by (first token, number of tokens, row group): a request's, or a prefix group's
    by = {}
    for i, it in enumerate(items):
        assert it[4] in (-1, i) and it[8] == -1 and it[2] % TILE == 0 and it[2] < it[3]
        by.setdefault((it[7], it[5], it[1]), []).append((i, it))
    spans, shared = {}, {}
    for g in range(len(lens)):
        lo, hi = indptr[g], indptr[g + 1]
        if hi - lo < 2:
            continue
        tokens, most = int(q0[hi] - q0[lo]), -(-int(q0[hi] - q0[lo]) * H // ROWS)
        if (int(q0[lo]), tokens, 0) not in by or tokens == qs[lo]:
            continue
        first = next(b for b in range(lo, hi) if ls[b] > 0)
        for k in range(most):
            parts = by.pop((int(q0[lo]), tokens, k))
            P = parts[-1][1][3]
            assert parts[0][1][2] == 0 and all(a[1][3] == c[1][2] for a, c in zip(parts, parts[1:]))
            assert [i for i, _ in parts] == list(range(parts[0][0], parts[0][0] + len(parts)))
            assert 0 < P <= lens[g] and P % TILE == 0 and shared.setdefault(g, P) == P
            for i, it in parts:
                assert it[0] == first and it[4] == i and it[6] == P
                assert it[9] >= P - 1  # the causal bound of the first query row hides nothing
            spans[g, k] = [i for i, _ in parts]
        seen = min(ls[b] - qs[b] + 1 if causal else ls[b] for b in range(lo, hi) if ls[b] > 0)
        assert shared[g] == min(lens[g], seen) // TILE * TILE
    at = 0
    for b, (L, q) in enumerate(zip(ls, qs)):
        if L <= 0:
            continue
        P = shared.get(group_of.get(b), 0)
        for k in range(-(-q * H // ROWS)):
            parts = by.pop((int(q0[b]), q, k), [])
            assert bool(parts) == (L > P)
            if parts:
                assert parts[0][1][2] == P and parts[-1][1][3] == L
                assert all(a[1][3] == c[1][2] for a, c in zip(parts, parts[1:]))
                assert [i for i, _ in parts] == list(range(parts[0][0], parts[0][0] + len(parts)))
            for i, it in parts:
                assert it[0] == b and it[6] == L and it[9] == L - q
                assert (it[4] >= 0) == (P > 0 or len(parts) > 1)
            row0, rows, own, n_own, off, p0, n0, p1, n1 = entries[at]
            at += 1
            assert row0 == q0[b] * H + k * ROWS
            if not P and len(parts) == 1:
                assert rows == 0
                continue
            assert rows == min(ROWS, q * H - k * ROWS)
            assert list(range(own, own + n_own)) == [i for i, _ in parts]
            if not P:
                assert n0 == n1 == 0
                continue
            g = group_of[b]
            row = int(q0[b] - q0[indptr[g]]) * H + k * ROWS
            assert off == row % ROWS and list(range(p0, p0 + n0)) == spans[g, row // ROWS]
            assert list(range(p1, p1 + n1)) == spans.get((g, row // ROWS + 1), [])
            assert off + rows <= ROWS or n1 > 0
    assert at == n_entries and not by
    return set(shared)


def _case(runner, sizes, lens, own, qs, H, packed, causal, kv, n_workers, uniform=False, gap=0, **kw):
    """Groups of `sizes` requests with `lens` shared rows, after and before `gap` requests of
    their own; own(rng-free callable of request) rows past the shared ones."""
    ls, indptr = [own(i) for i in range(gap)], [gap]
    for size, p in zip(sizes, lens):
        ls += [p + own(len(ls) + i) for i in range(size)]
        indptr.append(indptr[-1] + size)
    ls += [own(len(ls) + i) for i in range(gap)]
    qs = [qs[i % len(qs)] for i in range(len(ls))]
    ls = [max(L, q) if L else 0 for L, q in zip(ls, qs)]
    qo = np.concatenate([[0], np.cumsum(qs)])
    got = _run(runner, ls, qo, max(qs), max(ls), H, packed, causal, kv, lens, None if uniform else indptr, n_workers, **kw)
    return _check(got, ls, qs, H, causal, lens, indptr)


def test_a_system_prompt_is_shared(runner):
    assert _case(runner, [96], [6000], lambda i: 64 + 20 * i, [1], 16, False, True, 0, 76, uniform=True) == {0}
    assert _case(runner, [96], [6000], lambda i: 64 + 20 * i, [1], 16, False, True, 0, 76, global_scratch=True) == {0}


def test_beams_are_shared_and_few_are_not(runner):
    assert _case(runner, [8] * 16, [1000 + 400 * g for g in range(16)], lambda i: 1 + 3 * (i // 8), [1], 32, False, True, 1,
                 76, uniform=True) == set(range(16))
    # a call that the card finishes in one item a worker gains nothing
    assert _case(runner, [4], [500], lambda i: 1 + i, [1], 16, False, True, 0, 76, uniform=True) == set()


def test_a_group_without_rows_of_its_own(runner):
    assert _case(runner, [40], [4096], lambda i: 0, [1], 16, False, True, 2, 76, uniform=True) == {0}
    assert _case(runner, [40], [4096], lambda i: i % 2, [2], 16, False, False, 2, 76, uniform=True) == {0}


def test_uneven_groups_and_requests_outside_them(runner):
    assert _case(runner, [30, 1, 25], [5000, 9000, 3001], lambda i: 5 + i, [1, 3, 2], 16, True, True, 0, 76,
                 gap=3) >= {0}


def test_empty_requests_inside_a_group(runner):
    ls = [4100 + i for i in range(40)]
    ls[0] = ls[7] = ls[39] = 0
    qo = list(range(41))
    got = _run(runner, ls, qo, 1, 5000, 16, False, True, 0, [4000], None, 76)
    assert _check(got, ls, [1] * 40, 16, True, [4000], None, status=5) == {0}


@pytest.mark.parametrize("seed", range(24))
def test_random_groups(runner, seed):
    rng = np.random.default_rng(4000 + seed)
    G = int(rng.integers(1, 7))
    sizes = [int(rng.integers(0, 30)) for _ in range(G)]
    if sum(sizes) < G:
        sizes[0] = G
    top = int(rng.choice([1, 2, 5, 37]))
    packed = bool(rng.integers(2))
    qs = [int(x) for x in rng.integers(1, top + 1, 7)] if packed else [top]
    lens = [int(x) for x in rng.integers(0, int(rng.choice([100, 3000, 30000])), G)]
    far = int(rng.choice([1, 100, 5000]))
    more = rng.integers(0, far, 400)
    _case(runner, sizes, lens, lambda i: int(more[i]) + top, qs, int(rng.choice([16, 32, 64, 128])), packed,
          bool(rng.integers(2)), int(rng.integers(3)), int(rng.integers(1, 80)), gap=int(rng.integers(0, 4)),
          global_scratch=bool(rng.integers(2)))


@pytest.mark.parametrize("indptr", [[0, 30, 20, 40], [-1, 10, 20, 40], [0, 10, 20, 41], [0, 2 ** 31 - 1, 5, 40],
                                    [-2 ** 31, 2 ** 31 - 1, -5, 3]])
def test_bad_offsets_share_nothing(runner, indptr):
    ls, qo = [4000 + i for i in range(40)], list(range(41))
    got = _run(runner, ls, qo, 1, 5000, 16, False, True, 0, [4000] * 3, indptr, 76)
    assert _check(got, ls, [1] * 40, 16, True, [0] * 3, [0, 0, 0, 0], status=256) == set()


@pytest.mark.parametrize("seed", range(8))
def test_bad_lengths_stay_in_bounds(runner, seed):
    rng = np.random.default_rng(80 + seed)
    B = 40
    ls, lens = rng.integers(1, 5000, B), rng.integers(0, 5000, 4)
    qo = np.concatenate([[0], np.cumsum(rng.integers(1, 5, B))])
    qo[int(rng.integers(B))] = int(rng.choice([-7, 0, qo[-1], 2 ** 30]))
    ls[int(rng.integers(B))] = int(rng.choice([-5, 0, 10 ** 9]))
    lens[int(rng.integers(4))] = int(rng.choice([-1, -2 ** 31, 2 ** 31 - 1]))
    head = _run(runner, ls, qo, 4, 5000, 64, True, True, 0, lens, None, 76)[0]
    assert head[0] & 3
