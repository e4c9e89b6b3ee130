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
    for inc in ("<cuda_bf16.h>", "<cuda_fp16.h>", '"mla_common.cuh"', '"mla_fp4.cuh"', '"mla_prefix.cuh"', '"sm100_ptx.cuh"'):
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
    return [[int(x) for x in line.split()] for line in open(out / "out.txt").read().split("\n")[:10]]


def _check(got, ls, qs, H, causal, lens, indptr, status=0):
    """-> the prefix groups that are shared."""
    head, items, ranges, entries, segs, wide_items, wide_ranges, wide_segs, wide_groups, (wide_tiles,) = got
    assert head[0] == status
    n_items, n_rg, max_items, max_groups, max_partials = head[1:]
    assert n_items <= max_items and n_rg <= max_groups
    items = [items[10 * i:10 * i + 10] for i in range(n_items)]
    wide_items = [wide_items[i:i + 10] for i in range(0, len(wide_items), 10)]
    entries = [entries[6 * i:6 * i + 6] for i in range(n_rg)]
    segs = [[segs[7 * (9 * r + i):7 * (9 * r + i) + 7] for i in range(9)] for r in range(n_rg)]
    q0 = np.concatenate([[0], np.cumsum(qs)])
    if indptr is None:
        indptr = [g * (len(ls) // len(lens)) for g in range(len(lens) + 1)]
    group_of = {b: g for g in range(len(lens)) for b in range(indptr[g], indptr[g + 1])}
    request_of = np.repeat(np.arange(len(ls)), qs)
    slots, shared, seen, joined = [], {}, {}, {}
    # widened rows: the groups' follow on one another, and fit
    wide = {}
    if wide_tiles:
        at = 0
        for g in range(len(lens)):
            base, tiles, b = wide_groups[3 * g:3 * g + 3]
            assert base == at
            at += tiles
            if tiles:
                wide[g] = base, tiles
                assert b == next(x for x in range(indptr[g], indptr[g + 1]) if ls[x] > 0)
        assert wide_groups[3 * len(lens)] == at <= wide_tiles
    for which, (its, rng) in enumerate([(items, ranges), (wide_items, wide_ranges)]):
        if not rng:
            continue
        assert rng[0] == 0 and rng[-1] == len(its) and all(a <= b for a, b in zip(rng, rng[1:]))
        assert [it[8] for it in its] == sorted(it[8] for it in its)  # a row group's follow on one another
        by = {}
        for i, it in enumerate(its):
            by.setdefault(it[8], []).append((i, it))
        for r, found in by.items():
            parts = [it for _, it in found]
            _, k, _, _, _, tokens, n_seg, start, _, _ = parts[0]
            assert all([it[1], it[5], it[6], it[7]] == [k, tokens, n_seg, start] for it in parts)
            rows = min(ROWS, tokens * H - k * ROWS)
            assert rows > 0 and 1 <= n_seg <= 9
            # the parts follow on one another, and the segments fill them
            assert parts[0][2] == 0 and all(a[3] == c[2] for a, c in zip(parts, parts[1:]))
            assert all(it[2] % TILE == 0 and it[2] < it[3] for it in parts)
            at, is_wide = 0, False
            row_segs = segs[r][:n_seg] if which == 0 else [wide_segs[7 * found[0][0]:7 * found[0][0] + 7]]
            for tile0, b, row0, end, lo, hi, mask in row_segs:
                assert tile0 == at and row0 % TILE == 0 and row0 < end
                at += -(-(end - row0) // TILE)
                assert 0 <= lo < hi <= ROWS
                for q in range(lo, min(hi, rows), H):
                    assert q % H == 0
                    i = (k * ROWS + q) // H  # token of the owner
                    token = start + i
                    own = request_of[token]
                    last, first = mask + i, row0
                    g = group_of.get(own)
                    if which == 1:  # widened rows, in the group's place
                        assert (row0, end) == (wide[g][0] * TILE, sum(wide[g]) * TILE) and mask == 1 << 30
                        last, first = end - row0 - 1, 0
                        assert shared.setdefault(g, last + 1) == last + 1 <= lens[g]
                        assert last + 1 <= (ls[own] - qs[own] + 1 if causal else ls[own]) or ls[own] <= 0
                        seen.setdefault(token, []).append((0, last + 1))
                        continue
                    assert end <= ls[b]
                    if own != b or mask == 1 << 30 and causal:  # shared rows: whole tiles that all see, from the group's first table
                        assert row0 == 0 and end % TILE == 0 and end <= lens[g] and group_of[b] == g and g not in wide
                        assert b == next(x for x in range(indptr[g], indptr[g + 1]) if ls[x] > 0)
                        assert shared.setdefault(g, end) == end
                        assert end <= (ls[own] - qs[own] + 1 if causal else ls[own]) or ls[own] <= 0
                        last = end - 1
                    elif causal:
                        assert last == ls[own] - qs[own] + token - q0[own]
                    seen.setdefault(token, []).append((row0, min(end, last + 1)))
            assert at * TILE == parts[-1][3]
            e = entries[r]
            assert e[0] == start * H + k * ROWS
            needs = len(parts) > 1 or group_of.get(request_of[start + k * ROWS // H]) in wide
            assert e[3 + 2 * which] == (len(parts) if needs else 0)
            if needs:
                joined[r] = rows
                first = e[2 + 2 * which]
                assert [it[4] for it in parts] == list(range(first, first + len(parts)))
                slots += [it[4] for it in parts]
            else:
                assert parts[0][4] == -1
    assert all(e[1] == joined.get(r, 0) for r, e in enumerate(entries))
    assert len(set(slots)) == len(slots) and all(0 <= x < max_partials for x in slots)
    for token, b in enumerate(request_of):  # every row that the token sees, once
        L = ls[b]
        if L <= 0:
            continue
        end = L - qs[b] + token - q0[b] + 1 if causal else L
        spans = sorted(x for x in seen[token] if x[0] < x[1])
        assert spans[0][0] == 0 and spans[-1][1] == end and all(a[1] == c[0] for a, c in zip(spans, spans[1:]))
    return set(shared)


def _case(runner, sizes, lens, own, qs, H, packed, causal, kv, n_workers, uniform=False, gap=0, wide=None, **kw):
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
    assert wide is None or wide == (len(got[5]) > 0)
    return _check(got, ls, qs, H, causal, lens, indptr)


def test_a_system_prompt_is_shared(runner):
    assert _case(runner, [96], [6000], lambda i: 64 + 20 * i, [1], 16, False, True, 0, 76, uniform=True) == {0}
    assert _case(runner, [96], [6000], lambda i: 64 + 20 * i, [1], 16, False, True, 0, 76, global_scratch=True) == {0}


def test_beams_are_shared_and_full_row_groups_are_not(runner):
    assert _case(runner, [8] * 16, [1000 + 400 * g for g in range(16)], lambda i: 1 + 3 * (i // 8), [1], 32, False, True, 1,
                 76, uniform=True) == set(range(16))
    # a row group a request already, and a worker for each
    assert _case(runner, [8] * 4, [640] * 4, lambda i: 10, [1], 128, False, True, 0, 76, uniform=True) == set()


@pytest.mark.parametrize("kv", [1, 2])
def test_rows_that_many_row_groups_walk_are_widened(runner, kv):
    for own in (lambda i: 100 + 30 * i, lambda i: 0, lambda i: i % 2):
        assert _case(runner, [32], [20000], own, [1], 128, False, True, kv, 76, uniform=True, wide=True) == {0}
    assert _case(runner, [40, 2, 50], [9000, 4000, 7000], lambda i: 3 + i, [3, 1, 2], 64, True, True, kv, 76, gap=2, wide=True) >= {0, 2}
    # not over bf16, nor where a prefix group has few row groups
    _case(runner, [32], [20000], lambda i: 9, [1], 128, False, True, 0, 76, uniform=True, wide=False)
    assert _case(runner, [8] * 16, [5000] * 16, lambda i: 9, [1], 32, False, True, kv, 76, uniform=True, wide=False)


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
