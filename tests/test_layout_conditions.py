"""The workspace of plans over a 4-bit cache or with a window: the split partials have the
room that the kernels take, and the plan takes the condition from where they do."""
import os
import re
import shutil
import subprocess

import pytest

from test_partition_host import CSRC, ROOT, _function_text

PROGRAM = r"""
#include <algorithm>
#include <cstdio>
#define __device__
#define __host__
#define __forceinline__ inline
#include "common.h"
#include "mla_decode.h"
namespace {
long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }
constexpr size_t kHeaderBytes = sizeof(int) * mla::kHdrWords;
enum { MLA_OK = 0, MLA_ERR_UNSUPPORTED = -2 };
#include "make_layout.inc"
}
int main() {  // kv type, window, query type, widened -> bytes of a partial row, bytes behind the counters
  for (int kv = 0; kv < 3; ++kv)
    for (int window : {0, 1, 5000})
      for (int q = 0; q < 2; ++q)
        for (int widen = 0; widen < 2; ++widen) {
          mla_decode_params p{};
          p.batch = 40; p.num_heads = 128; p.max_seq_len_q = 3; p.max_seq_len = 4000; p.kv_dtype = kv;
          p.window = window; p.q_dtype = q; p.e4m3_widen = widen;
          mla::Layout lay{};
          if (make_layout(p, 76, 152, 128, &lay)) return 1;
          std::printf("%d %d %d %d %zu %zu\n", kv, window, q, widen,
                      (lay.part_lse - lay.part_o) / ((size_t)128 * lay.max_partials),
                      lay.total - mla::q_split_offset(lay));
        }
}
"""


def _layouts(tmp, change=lambda text: text):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    common = open(os.path.join(CSRC, "mla_common.cuh")).read().replace("#include <cuda_runtime.h>\n", "")
    common = re.sub(r"__device__ __forceinline__ float run_bmm[\s\S]*?\n}\n", "", common)  # (device atomics)
    (tmp / "common.h").write_text(change(common))
    api = open(os.path.join(CSRC, "mla_api.cu")).read()
    (tmp / "make_layout.inc").write_text(_function_text(api, "int make_layout(") + "\n")
    (tmp / "main.cpp").write_text(PROGRAM)
    r = subprocess.run([cxx, "-std=c++20", "-I", str(tmp), "-I", os.path.join(ROOT, "include"), str(tmp / "main.cpp"),
                        "-o", str(tmp / "main")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    out = subprocess.run([str(tmp / "main")], capture_output=True, text=True, check=True).stdout
    return {tuple(int(x) for x in line.split()[:4]): tuple(int(x) for x in line.split()[4:])
            for line in out.strip().split("\n")}


def test_partials_and_query_split_have_their_room(tmp_path):
    for (kv, window, q, widen), (row, behind) in _layouts(tmp_path).items():
        assert row == (2048 if window and kv == 0 else 1024)
        split = kv == 1 and not window and not q and not widen
        assert behind == (2 * 40 * 3 * 128 * 37 * 16 if split else 0)


def test_the_plan_follows_the_kernels_conditions(tmp_path):
    def change(text):
        text, n = re.subn(r"(PartFormat part_format\([^)]*\) \{\s*return )[^;]*;", r"\1kv_dtype == 1 ? kPartF32 : kPartBf16;", text)
        text, m = re.subn(r"(bool fp8_mma\([^)]*\) \{\s*return )[^;]*;", r"\1window == 1;", text)
        assert n == 1 and m == 1
        return text

    for (kv, window, q, _), (row, behind) in _layouts(tmp_path, change).items():
        assert row == (2048 if kv == 1 else 1024)
        assert (behind > 0) == (window == 1 and not q)
