"""Cache append, gather and rotation table against plain 64-bit forms.

Tolerances come from the roundings alone: a rounding to a type is off by at
most half a step, ``torch.finfo(t).eps / 2`` of the value (plus half the
smallest subnormal), and an fp32 step before it by 2^-24 of its terms.  The
rotation of (a, b) has three such steps per output on terms |a c| + |b s|, the
norm five (the sum, the eps, the root, two products): 8 are counted."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

import paged_mla_decode_03_gb300 as mla
from paged_mla_decode_03_gb300 import build as mla_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
F32 = 8 * 2.0 ** -24


def row_bytes(kind):
    return {"bf16": 1152, "e4m3": 576, "fp4": 324}[kind]


def new_cache(kind, pages, ps, fill=0x5A, dev="cuda"):
    raw = torch.full((pages, ps, row_bytes(kind)), fill, dtype=torch.uint8, device=dev)
    return raw if kind == "fp4" else raw.view({"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[kind])


def fp4_parts(cache):
    """(codes [pages, ps, 576] as 64-bit values, scales [pages, ps, 36] in 64 bits)."""
    pages, ps = cache.shape[:2]
    flat = cache.reshape(pages, ps * 324).cpu()
    by = flat[:, :ps * 288].reshape(pages, ps, 288).long()
    code = torch.stack([by & 15, by >> 4], -1).flatten(-2)
    val = E2M1[code & 7] * torch.where(code > 7, -1.0, 1.0)
    sc = flat[:, ps * 288:].reshape(pages, ps, 36).contiguous().view(torch.float8_e4m3fn).double()
    return val, sc


def values(cache, kind):
    if kind != "fp4":
        return cache.double().cpu()
    val, sc = fp4_parts(cache)
    return (val.unflatten(-1, (36, 16)) * sc[..., None]).flatten(-2)


def rotate(x, c, s, style):
    a, b = (x[..., 0::2], x[..., 1::2]) if style == "interleaved" else (x[..., :32], x[..., 32:])
    r, i = a * c - b * s, b * c + a * s
    tr, ti = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    if style == "interleaved":
        return torch.stack([r, i], -1).flatten(-2), torch.stack([tr, ti], -1).flatten(-2)
    return torch.cat([r, i], -1), torch.cat([tr, ti], -1)


def close_bf16(got, ref, terms, what):
    bound = ref.abs() * 2.0 ** -8 + terms * F32 + 2.0 ** -133
    bad = ~((got.double().cpu() - ref).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} values off"


def close_e4m3(got, t, terms, what):
    t2 = t.clamp(-448, 448)
    bad = ~((got.double().cpu() - t2).abs() <= t2.abs() * 2.0 ** -4 + 2.0 ** -10 + terms * F32)
    assert not bad.any(), f"{what}: {int(bad.sum())} values off"


def close_fp4(val, sc, y, terms, what):
    """Each group's scale is e4m3 of amax / 6 and each code the nearest of its value over it."""
    g, tg = y.unflatten(-1, (36, 16)), terms.unflatten(-1, (36, 16))
    want = (g.abs().amax(-1) / 6).clamp(max=448)
    assert ((sc - want).abs() <= want * 2.0 ** -4 + 2.0 ** -10 + tg.amax(-1) * F32).all(), f"{what}: scales"
    s = sc[..., None]
    t = torch.where(s > 0, g / s.clamp(min=2.0 ** -9), torch.zeros_like(g)).clamp(-6, 6)
    half = torch.where(t.abs() < 2, 0.25, torch.where(t.abs() < 4, 0.5, 1.0))
    slop = torch.where(s > 0, tg * F32 / s.clamp(min=2.0 ** -9), torch.zeros_like(g)) + 2.0 ** -21
    bad = ~((val.unflatten(-1, (36, 16)) - t).abs() <= half + slop)
    assert not bad.any(), f"{what}: {int(bad.sum())} codes off"


class Setup:
    """Tokens, tables and lengths of one append; token places worked out on the host."""

    def __init__(self, kind, ps, ls, qs, heads, *, packed, seed=0, pad=0, style="interleaved", table=None):
        rng = np.random.default_rng(seed)
        self.kind, self.ps, self.style, self.heads, self.packed = kind, ps, style, heads, packed
        need = [-(-max(L, 1) // ps) for L in ls]
        pool = sum(need) + 3
        order = rng.permutation(pool).astype(np.int32)
        width = max(need) + 1
        bt = np.full((len(ls), width), -7, np.int32)
        at = 0
        for b, n in enumerate(need):
            bt[b, :n] = order[at:at + n]
            at += n
        self.pages = pool
        self.places = [(int(bt[b, p // ps]), p % ps, p) for b, (L, q) in enumerate(zip(ls, qs))
                       for p in range(L - q, L)]
        self.n = len(self.places)
        self.T = self.n + pad
        g = torch.Generator().manual_seed(seed)
        dev = "cuda"
        kv = torch.randn(self.T, 576 + 24, generator=g).to(torch.bfloat16).to(dev)
        self.latent, self.k_pe = kv[:, 8:520], kv[:, 536:600]
        self.weight = (1 + 0.3 * torch.randn(512, generator=g)).to(torch.bfloat16).to(dev)
        self.q_nope = torch.randn(heads, self.T, 512, generator=g).to(torch.bfloat16).to(dev).transpose(0, 1)
        self.q_pe = torch.randn(self.T, heads, 192, generator=g).to(torch.bfloat16).to(dev)[..., 128:]
        self.tables = torch.from_numpy(bt).to(dev)
        self.lens = torch.tensor(ls, dtype=torch.int32, device=dev)
        self.indptr = torch.tensor(np.cumsum([0] + list(qs)), dtype=torch.int32, device=dev)
        self.which = dict(qo_indptr=self.indptr) if packed else dict(q_len=qs[0])
        self.table = mla.rope_table(max(max(ls), 8)) if table is None else table

    def reference(self, norm=True, eps=1e-6, positions=None):
        """(rows y [n, 576], their fp32 terms, query [n, H, 576], its terms) in 64 bits."""
        n = self.n
        x = self.latent[:n].double().cpu()
        lat = x
        if norm:
            lat = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * self.weight.double().cpu()
        pos = torch.tensor([p for _, _, p in self.places]) if positions is None else positions
        cs = self.table.double().cpu()[pos]
        c, s = cs[:, :32], cs[:, 32:]
        k, tk = rotate(self.k_pe[:n].double().cpu(), c, s, self.style)
        qr, tq = rotate(self.q_pe[:n].double().cpu(), c[:, None], s[:, None], self.style)
        qn = self.q_nope[:n].double().cpu()
        return (torch.cat([lat, k], -1), torch.cat([lat.abs(), tk], -1), torch.cat([qn, qr], -1),
                torch.cat([torch.zeros_like(qn), tq], -1))

    def check(self, cache, y, terms, kv_scale=1.0, what="", skip=()):
        at = torch.tensor([pl[:2] for i, pl in enumerate(self.places) if i not in skip])
        keep = torch.tensor([i for i in range(self.n) if i not in skip])
        inv = float(np.float32(1.0 / kv_scale))
        y, terms = y[keep] * inv, terms[keep] * inv
        if self.kind == "fp4":
            val, sc = fp4_parts(cache)
            close_fp4(val[at[:, 0], at[:, 1]], sc[at[:, 0], at[:, 1]], y, terms, what)
        else:
            (close_bf16 if self.kind == "bf16" else close_e4m3)(cache.cpu().double()[at[:, 0], at[:, 1]], y, terms, what)
        # every other byte of the pool is as it was
        if self.kind == "fp4":
            flat = cache.cpu().reshape(self.pages, -1)
            parts = [flat[:, :self.ps * 288].reshape(self.pages, self.ps, 288),
                     flat[:, self.ps * 288:].reshape(self.pages, self.ps, 36)]
        else:
            parts = [cache.view(torch.uint8).cpu()]
        for part in parts:
            same = (part == 0x5A).all(-1)
            same[at[:, 0], at[:, 1]] = True
            assert same.all(), f"{what}: rows that no token maps to were written"


# ------------------------------------------------------------------ CPU: refusals and layouts

@pytest.fixture(scope="module")
def lib():
    mla_build.build()
    return mla.load_library()


@pytest.mark.parametrize("cls,name", [(mla.MlaCacheParams, "mla_cache_params"), (mla.MlaRopeParams, "mla_rope_params")])
def test_struct_layouts_match_c(cls, name, tmp_path):
    fields = [f[0] for f in cls._fields_]
    prog = ["#include <stdio.h>", "#include <stddef.h>", '#include "mla_decode.h"', "int main(void) {",
            f'printf("%zu\\n", sizeof({name}));'] + [f'printf("%zu\\n", offsetof({name}, {f}));' for f in fields]
    src, exe = tmp_path / "l.c", tmp_path / "l"
    src.write_text("\n".join(prog + ["return 0; }"]))
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    v = [int(x) for x in subprocess.check_output([str(exe)]).split()]
    assert v[0] == ctypes.sizeof(cls) and v[1:] == [getattr(cls, f).offset for f in fields]


A = 1 << 20  # a device address that is never read: every call below is refused on the host


def c_append(lib, params=None, **kw):
    p = dict(batch=2, packed=0, q_len=1, page_size=64, max_pages_per_req=4, kv_dtype=0, num_pages=8, num_heads=16,
             q_dtype=0)
    p.update(params or {})
    a = dict(latent=A, ls=512, k_pe=A, ks=64, w=A, eps=1e-6, table=A, maxp=64, style=0, pos=None, bt=A, sl=A, qo=None,
             T=2, kvs=1.0, cache=A, qn=A, qnt=8192, qnh=512, qp=A, qpt=1024, qph=64, qs=1.0, query=A, status=None)
    a.update(kw)
    return lib.mla_cache_append(
        ctypes.byref(mla.MlaCacheParams(**p)), a["latent"], a["ls"], a["k_pe"], a["ks"], a["w"], a["eps"], a["table"],
        a["maxp"], a["style"], a["pos"], a["bt"], a["sl"], a["qo"], a["T"], a["kvs"], a["cache"], a["qn"], a["qnt"],
        a["qnh"], a["qp"], a["qpt"], a["qph"], a["qs"], a["query"], a["status"], None)


@pytest.mark.parametrize("params,kw,rc", [
    (dict(batch=-1), {}, -1), (dict(kv_dtype=3), {}, -1), (dict(packed=2), {}, -1), (dict(q_len=0), {}, -1),
    (dict(num_pages=0), {}, -1), (dict(max_pages_per_req=0), {}, -1), (dict(page_size=16), {}, -2),
    (dict(num_pages=1 << 26), {}, -2), (dict(num_heads=8), {}, -2), (dict(q_dtype=2), {}, -1),
    (dict(packed=1), {}, -1), ({}, dict(qo=A), -1), ({}, dict(T=3), -1), ({}, dict(T=-1), -1),
    ({}, dict(style=2), -1), ({}, dict(maxp=0), -1), ({}, dict(kvs=0.0), -1), ({}, dict(kvs=2.0), -1),
    (dict(kv_dtype=1), dict(kvs=float("nan")), -1), (dict(kv_dtype=2), dict(kvs=float("inf")), -1),
    ({}, dict(qs=2.0), -1), ({}, dict(eps=-1.0), -1), ({}, dict(eps=float("nan")), -1),
    ({}, dict(qp=None), -1), ({}, dict(query=None), -1), ({}, dict(qp=None, query=None), -1),
    (dict(q_dtype=1), dict(qn=None), -1), ({}, dict(latent=None), -1), ({}, dict(k_pe=None), -1),
    ({}, dict(table=None), -1), ({}, dict(cache=None), -1), ({}, dict(bt=None), -1), ({}, dict(sl=None), -1),
    ({}, dict(latent=A + 2), -4), ({}, dict(ls=516), -4), ({}, dict(k_pe=A + 8), -4), ({}, dict(qpt=1028), -4),
    ({}, dict(qnh=516), -4), ({}, dict(query=A + 8), -4), ({}, dict(cache=A + 8), -4), ({}, dict(w=A + 8), -4),
    ({}, dict(table=A + 4), -4), ({}, dict(pos=A + 2), -4), ({}, dict(status=A + 2), -4), ({}, dict(sl=A + 2), -4),
])
def test_append_refusals(lib, params, kw, rc):
    assert c_append(lib, params, **kw) == rc


@pytest.mark.parametrize("kw,rc", [(dict(kv_scale=0.0), -1), (dict(out=None), -1), (dict(out=A + 8), -4),
                                   (dict(cache=None), -1), (dict(kv_scale=2.0), -1)])
def test_gather_refusals(lib, kw, rc):
    a = dict(cache=A, kv_scale=1.0, out=A)
    a.update(kw)
    p = mla.MlaCacheParams(batch=2, packed=0, q_len=1, page_size=64, max_pages_per_req=4, num_pages=8)
    assert lib.mla_cache_gather(ctypes.byref(p), a["cache"], A, A, None, 2, a["kv_scale"], a["out"], None, None) == rc


@pytest.mark.parametrize("kw", [dict(max_position=0), dict(base=1.0), dict(base=float("nan")), dict(scaling=3),
                                dict(scaling=1, factor=0.0), dict(amplitude=0.0), dict(scaling=2, beta_slow=0.0),
                                dict(scaling=2, beta_fast=0.5), dict(scaling=2, original_max_position=0.0)])
def test_rope_table_refusals(lib, kw):
    p = dict(max_position=8, base=1e4, amplitude=1.0, factor=2.0, original_max_position=4096.0, beta_fast=32.0,
             beta_slow=1.0)
    p.update(kw)
    assert lib.mla_rope_table(ctypes.byref(mla.MlaRopeParams(**p)), A, None) == -1
    assert lib.mla_rope_table(None, A, None) == -1


def test_binding_refusals():
    x = torch.zeros(2, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mla.cache_append(x, x[:, :64], x, x, x, rope_table=x, q_len=1)
    with pytest.raises(ValueError):
        mla.cache_gather(x, x, x)
    with pytest.raises(ValueError):
        mla.rope_table(8, scaling="ntk")


# ------------------------------------------------------------------ GPU

@pytest.mark.gpu
@pytest.mark.parametrize("scaling", [None, "linear", "yarn"])
def test_rope_table(scaling):
    n, factor = 200001, 40.0
    t = mla.rope_table(n, base=10000.0, scaling=scaling, factor=factor, original_max_position=4096, amplitude=1.25).cpu().double()
    i = np.arange(32)
    f = 10000.0 ** (-i / 32.0)
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        edge = [32 * math.log(4096 / (r * 2 * math.pi)) / math.log(10000.0) for r in (32.0, 1.0)]
        low, high = max(0, math.floor(edge[0])), min(63, math.ceil(edge[1]))
        ramp = np.clip((i - low) / (high - low), 0, 1)
        f = f / factor * ramp + f * (1 - ramp)
    for pos in (0, 1, 2, 4095, 131071, 200000):
        a = pos * f
        # fp32 rounding of a value up to 1.25, and 64-bit angles of up to 2e5 turns of 2^-52 each, with slack 4
        tol = 1.25 * 2.0 ** -24 + 4 * pos * 2.0 ** -52
        assert np.abs(t[pos, :32].numpy() - 1.25 * np.cos(a)).max() <= tol
        assert np.abs(t[pos, 32:].numpy() - 1.25 * np.sin(a)).max() <= tol


CASES = [  # kind, page, lengths, query lengths, heads, packed, padding
    ("bf16", 64, [1], [1], 16, False, 0),
    ("bf16", 32, [7, 64, 33], [1, 1, 1], 128, False, 0),
    ("bf16", 32, [40, 5, 1000], [3, 5, 0], 32, True, 5),
    ("e4m3", 64, [129, 64], [2, 2], 64, False, 0),
    ("e4m3", 32, [40, 5, 70, 31], [0, 1, 37, 31], 16, True, 9),
    ("fp4", 64, [65, 64, 1], [1, 1, 1], 16, False, 0),
    ("fp4", 32, [33, 100, 64], [33, 70, 2], 16, True, 1),
    ("fp4", 64, [200, 1, 90], [9, 1, 64], 128, True, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("style", ["interleaved", "half"])
@pytest.mark.parametrize("kind,ps,ls,qs,heads,packed,pad", CASES)
def test_append(kind, ps, ls, qs, heads, packed, pad, style):
    s = Setup(kind, ps, ls, qs, heads, packed=packed, pad=pad, style=style, seed=len(ls) + heads)
    cache = new_cache(kind, s.pages, ps)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_fp8 = kind == "e4m3"
    kvs, qsc = (0.0125, 0.0110) if kind == "e4m3" else (2.5 if kind == "fp4" else 1.0, 1.0)
    query = torch.full((s.T, heads, 576), 3.0, dtype=torch.bfloat16, device="cuda")
    if q_fp8:
        query = query.to(torch.float8_e4m3fn)
    r = mla.cache_append(s.latent, s.k_pe, cache, s.tables, s.lens, rope_table=s.table, norm_weight=s.weight,
                         rope_style=style, kv_scale=kvs, q_nope=s.q_nope, q_pe=s.q_pe, query=query, q_scale=qsc,
                         status=status, **s.which)
    torch.cuda.synchronize()
    assert r is query and int(status) == 0
    y, ty, q, tq = s.reference()
    s.check(cache, y, ty, kvs, kind)
    inv = float(np.float32(1.0 / qsc))
    (close_e4m3 if q_fp8 else close_bf16)(query[:s.n], q * inv, (q.abs() + tq) * inv, "query")
    assert (query[s.n:].float() == 3.0).all(), "padding rows were written"


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp4"])
def test_append_without_norm_or_query_and_with_positions(kind):
    s = Setup(kind, 32, [50, 9], [4, 4], 16, packed=False, seed=5, table=mla.rope_table(9000))
    cache = new_cache(kind, s.pages, 32)
    pos = torch.tensor([8999, 0, 17, 5, 300, 4, 4, 1], dtype=torch.int32)
    assert mla.cache_append(s.latent, s.k_pe, cache, s.tables, s.lens, rope_table=s.table, positions=pos.cuda(),
                            q_len=4) is None
    y, ty, _, _ = s.reference(norm=False, positions=pos.long())
    s.check(cache, y, ty, 1.0, kind)


@pytest.mark.gpu
def test_append_keeps_the_querys_latent_part():
    s = Setup("bf16", 64, [50, 9], [2, 2], 16, packed=False, seed=6)
    cache = new_cache("bf16", s.pages, 64)
    query = torch.full((2, 2, 16, 576), -7.0, dtype=torch.bfloat16, device="cuda")
    mla.cache_append(s.latent, s.k_pe, cache, s.tables, s.lens, rope_table=s.table, norm_weight=s.weight, q_len=2,
                     q_pe=s.q_pe, query=query)
    _, _, q, tq = s.reference()
    assert (query[..., :512] == -7.0).all()
    close_bf16(query.view(4, 16, 576)[..., 512:], q[..., 512:], tq[..., 512:], "query")


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp4"])
def test_append_extreme_values(kind):
    """Zeros (an all-zero group, eps alone under the root), huge and tiny latents."""
    s = Setup(kind, 32, [40], [5], 16, packed=False, seed=7)
    x = torch.zeros(5, 576, dtype=torch.bfloat16, device="cuda")
    x[1] = 1e-30
    x[2] = 3e18
    x[3, :512] = torch.linspace(-1, 1, 512, device="cuda").to(torch.bfloat16)
    x[4, ::17] = 1e4
    s.latent, s.k_pe = x[:, :512], x[:, 512:]
    cache = new_cache(kind, s.pages, 32)
    mla.cache_append(s.latent, s.k_pe, cache, s.tables, s.lens, rope_table=s.table, norm_weight=s.weight, q_len=5)
    y, ty, _, _ = s.reference()
    if kind == "fp4":
        y[2, 512:] = y[2, 512:].clamp(-2688, 2688)  # past the largest 4-bit value: saturates
    s.check(cache, y, ty, 1.0, kind)


@pytest.mark.gpu
def test_bad_places_are_flagged_and_nothing_else_is_lost():
    s = Setup("e4m3", 32, [40, 70, 9, 64], [2, 2, 2, 2], 16, packed=False, seed=8)
    s.tables[1, 2] = s.pages        # page of positions 64..: both tokens of request 1
    s.lens[2] = 1                   # token 0 of request 2 would sit at position -1, token 1 at 0
    pos = torch.tensor([38, 39, 68, 69, 7, 8, 62, 1 << 20], dtype=torch.int32, device="cuda")
    cache = new_cache("e4m3", s.pages, 32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    query = torch.full((8, 16, 576), 3.0, dtype=torch.bfloat16, device="cuda")
    mla.cache_append(s.latent, s.k_pe, cache, s.tables, s.lens, rope_table=s.table, q_len=2, positions=pos,
                     norm_weight=s.weight, q_nope=s.q_nope, q_pe=s.q_pe, query=query, status=status)
    assert int(status) == 16 | 1 | 128
    want = torch.tensor([38, 39, 68, 69, 7, 8, 62, 63])
    y, ty, q, tq = s.reference(positions=want)
    s.places[5] = (int(s.tables[2, 0]), 0, 0)
    bad = (2, 3, 4, 7)
    s.check(cache, y, ty, 1.0, "e4m3", skip=bad)
    keep = [i for i in range(8) if i not in bad]
    close_bf16(query[keep], q[keep], (q.abs() + tq)[keep], "query")
    assert (query[list(bad)] == 3.0).all()
    out = torch.full((8, 576), 2.0, dtype=torch.bfloat16, device="cuda")
    status.zero_()
    mla.cache_gather(cache, s.tables, s.lens, q_len=2, out=out, status=status)
    assert int(status) == 16 | 1 and (out[[2, 3, 4]] == 2.0).all() and not (out[[0, 1, 5, 6]] == 2.0).all(-1).any()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp4"])
@pytest.mark.parametrize("ps", [32, 64])
def test_gather_reads_whole_sequences(kind, ps):
    ls = [1, 31, 64, 65, 300]
    rng = np.random.default_rng(ps)
    need = [-(-L // ps) for L in ls]
    order = rng.permutation(sum(need) + 2).astype(np.int32)
    bt = np.full((5, max(need)), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = order[at:at + n]
        at += n
    raw = torch.from_numpy(rng.integers(0, 256, (sum(need) + 2, ps, row_bytes(kind)), dtype=np.uint8))
    if kind == "bf16":  # finite patterns
        raw = torch.randn(sum(need) + 2, ps, 576).to(torch.bfloat16)
    cache = raw.cuda()
    scale = 1.0 if kind == "bf16" else 0.37
    val = values(cache if kind != "e4m3" else cache.view(torch.float8_e4m3fn), kind)
    ref = torch.cat([val[torch.from_numpy(bt[b]).long()[torch.arange(L) // ps], torch.arange(L) % ps]
                     for b, L in enumerate(ls)])
    ref = (ref.float() * torch.tensor(scale)).to(torch.bfloat16)
    sl = torch.tensor(ls, dtype=torch.int32, device="cuda")
    ip = torch.tensor(np.cumsum([0] + ls), dtype=torch.int32, device="cuda")
    out = mla.cache_gather(cache, torch.from_numpy(bt).cuda(), sl, qo_indptr=ip, total_q=sum(ls), kv_scale=scale).cpu()
    assert torch.equal(out.isnan(), ref.isnan()) and torch.equal(out.nan_to_num(0), ref.nan_to_num(0))


@pytest.mark.gpu
def test_append_many_requests_of_uneven_length():
    """The search for a token's request over more than 32 x 32 of them, empty ones among them."""
    rng = np.random.default_rng(3)
    qs = rng.integers(0, 4, 1500)
    ls = [int(q + rng.integers(0, 50)) for q in qs]
    s = Setup("e4m3", 32, ls, [int(q) for q in qs], 16, packed=True, seed=9, pad=3)
    cache = new_cache("e4m3", s.pages, 32)
    mla.cache_append(s.latent, s.k_pe, cache, s.tables, s.lens, rope_table=s.table, norm_weight=s.weight, **s.which)
    y, ty, _, _ = s.reference()
    s.check(cache, y, ty, 1.0, "e4m3")


@pytest.mark.gpu
def test_append_in_a_graph_and_on_a_side_stream():
    s = Setup("fp4", 32, [33, 64], [1, 1], 16, packed=False, seed=10)
    cache = new_cache("fp4", s.pages, 32)
    out = torch.zeros(2, 576, dtype=torch.bfloat16, device="cuda")
    query = torch.empty(2, 16, 576, dtype=torch.bfloat16, device="cuda")

    def step():
        mla.cache_append(s.latent, s.k_pe, cache, s.tables, s.lens, rope_table=s.table, norm_weight=s.weight, q_len=1,
                         q_nope=s.q_nope, q_pe=s.q_pe, query=query)
        mla.cache_gather(cache, s.tables, s.lens, q_len=1, out=out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    first, q_first = out.clone(), query.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    s.lens -= 20
    g.replay()
    torch.cuda.synchronize()
    got, q_got = out.clone(), query.clone()
    step()
    torch.cuda.synchronize()
    assert torch.equal(out, got) and torch.equal(query, q_got) and not torch.equal(q_got, q_first)
    s.lens += 20
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and torch.equal(query, q_first)


@pytest.mark.gpu
def test_binding_refuses_what_the_kernel_cannot_take():
    s = Setup("bf16", 64, [50, 9], [2, 2], 16, packed=False, seed=11)
    cache = new_cache("bf16", s.pages, 64)
    ok = dict(latent=s.latent, k_pe=s.k_pe, kv_cache=cache, block_tables=s.tables, seq_lens=s.lens, rope_table=s.table,
              norm_weight=s.weight, q_len=2, q_nope=s.q_nope, q_pe=s.q_pe)
    query = mla.cache_append(**ok)
    assert query.shape == (4, 16, 576)
    bad = [dict(latent=s.latent.float()), dict(latent=s.latent[:3]), dict(k_pe=s.k_pe[:, ::2]), dict(k_pe=s.k_pe.cpu()),
           dict(norm_weight=s.weight[:256]), dict(rope_table=s.table.double()), dict(rope_table=s.table[:, :32]),
           dict(seq_lens=s.lens.long()), dict(block_tables=s.tables[:, ::2]), dict(block_tables=s.tables[0]),
           dict(q_len=None), dict(q_len=3), dict(qo_indptr=s.indptr), dict(rope_style="both"), dict(q_pe=s.q_pe[:, :8]),
           dict(q_nope=s.q_nope[..., :256]), dict(query=query[:2]), dict(query=query.half()), dict(q_pe=None),
           dict(positions=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(kv_cache=cache[:, :, :512]),
           dict(kv_cache=cache.half()), dict(status=torch.zeros(2, dtype=torch.int32, device="cuda")),
           dict(q_nope=None)]
    for kw in bad:
        with pytest.raises((ValueError, mla.MlaDecodeError)):
            mla.cache_append(**{**ok, **kw})
    for kw in (dict(kv_scale=0.0), dict(kv_scale=2.0), dict(q_scale=3.0), dict(eps=0.0)):
        with pytest.raises(mla.MlaDecodeError):
            mla.cache_append(**{**ok, **kw})
    for kw in (dict(out=torch.zeros(4, 576, device="cuda")), dict(q_len=None), dict(total_q=5)):
        with pytest.raises(ValueError):
            mla.cache_gather(**{**dict(kv_cache=cache, block_tables=s.tables, seq_lens=s.lens, q_len=2), **kw})
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert mla.cache_gather(cache, s.tables[:0], none, q_len=1).shape == (0, 576)
    e = torch.zeros(0, 576, dtype=torch.bfloat16, device="cuda")
    assert mla.cache_append(e[:, :512], e[:, 512:], cache, s.tables[:0], none, rope_table=s.table, q_len=1) is None
