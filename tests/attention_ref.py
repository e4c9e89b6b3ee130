"""Plain 64-bit form of the paged decode for the tests of its newer variants:
a cache of any format, a sliding window with sinks, rows without a key.  It
also gives, per output, what the tolerance is made of (see ``tolerances``)."""
import math

import numpy as np
import torch

import paged_mla_decode_03_gb300 as mla

E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def cache_values(cache):
    """64-bit values of a cache in any format, [pages, page_size, 576]."""
    if cache.dtype != torch.uint8:
        return cache.double()
    pages, ps = cache.shape[:2]
    flat = cache.reshape(pages, ps * 324)
    by = flat[:, :ps * 288].reshape(pages, ps, 288).long()
    code = torch.stack([by & 15, by >> 4], -1).flatten(-2)
    val = E2M1.to(cache.device)[code & 7] * torch.where(code > 7, -1.0, 1.0)
    sc = flat[:, ps * 288:].reshape(pages, ps, 36).contiguous().view(torch.float8_e4m3fn).double()
    return (val.unflatten(-1, (36, 16)) * sc[..., None]).flatten(-2)


def random_cache(kind, pages, ps, seed, scale=1.0):
    """N(0, 1) rows in the cache's format (4 bits: codes and scales of such rows)."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(pages, ps, 576, generator=g) * scale
    if kind == "bf16":
        return x.to(torch.bfloat16).cuda()
    if kind == "e4m3":
        return x.to(torch.float8_e4m3fn).cuda()
    gr = x.unflatten(-1, (36, 16))
    s = (gr.abs().amax(-1) / 6).to(torch.float8_e4m3fn)
    code = torch.bucketize((gr / s.float().clamp(min=2.0 ** -9)[..., None]).abs(),
                           torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]))
    code = (code + 8 * (gr < 0)).flatten(-2).to(torch.uint8)
    packed = code[..., 0::2] | (code[..., 1::2] << 4)
    flat = torch.cat([packed.reshape(pages, -1), s.view(torch.uint8).reshape(pages, -1)], 1)
    return flat.reshape(pages, ps, 324).contiguous().cuda()


def poison(cache, page, row):
    """Make one cache row NaN (4 bits: its scales)."""
    if cache.dtype != torch.uint8:
        cache.view(torch.uint8)[page, row] = 0x7F if cache.dtype == torch.float8_e4m3fn else 0xFF
        return
    ps = cache.shape[1]
    cache.view(cache.shape[0], -1)[page, ps * 288 + row * 36: ps * 288 + (row + 1) * 36] = 0x7F


class Case:
    """Inputs of one decode.  Rows that nothing may read, and pages that no
    request uses, are NaN; block-table entries of such pages are out of range."""

    def __init__(self, kind, ps, ls, qs, heads, *, packed=False, causal=True, q_fp8=False, window=0, sinks=0,
                 seed=0, bmm1=1 / math.sqrt(192.0), bmm2=0.75, pad=0, max_len=None, q_gain=1.0, widen=False):
        self.__dict__.update(kind=kind, ps=ps, ls=list(ls), qs=list(qs), heads=heads, packed=packed, causal=causal,
                             window=window, sinks=sinks, bmm1=float(np.float32(bmm1)), bmm2=float(np.float32(bmm2)))
        rng = np.random.default_rng(seed)
        need = [-(-L // ps) for L in ls]
        pool = sum(need) + 4
        order = rng.permutation(pool).astype(np.int32)
        bt = np.full((len(ls), -(-(max_len or max(ls)) // ps) + 1), 1 << 28, np.int32)
        self.cache = random_cache(kind, pool, ps, seed)
        raw = torch.zeros(pool, ps, dtype=torch.bool)
        at = 0
        for b, (L, q, n) in enumerate(zip(ls, qs, need)):
            pages = order[at:at + n]
            at += n
            seen = np.zeros(n * ps, bool)
            for i in range(q):
                last = L - q + i if causal else L - 1
                lo = max(0, last - window + 1) if window else 0
                seen[lo:last + 1] = True
                if window:
                    seen[:min(sinks, last + 1)] = True
            for k in range(n):
                if seen[k * ps:(k + 1) * ps].any():
                    bt[b, k] = pages[k]
                    raw[pages[k]] = torch.from_numpy(seen[k * ps:(k + 1) * ps])
        self.bt_host = bt
        self.unseen = (~raw).nonzero()
        for page, row in self.unseen.tolist():
            poison(self.cache, page, row)
        self.tables = torch.from_numpy(bt).cuda()
        self.lens = torch.tensor(ls, dtype=torch.int32, device="cuda")
        self.indptr = torch.tensor(np.cumsum([0] + list(qs)), dtype=torch.int32, device="cuda")
        self.T = sum(qs)
        g = torch.Generator().manual_seed(seed + 1)
        x = (torch.randn(self.T + pad, heads, 576, generator=g) * q_gain).to(torch.bfloat16)
        self.query = (x.float() / q_gain).to(torch.float8_e4m3fn).cuda() if q_fp8 else x.cuda()
        self.split_q = kind == "e4m3" and not widen and not q_fp8 and not 0 < window < (max_len or max(ls))
        self.max_len = max_len or max(ls)
        self.out = torch.full((self.T + pad, heads, 512), 3.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.T + pad, heads), 3.0, dtype=torch.float32, device="cuda")
        self.plan = mla.Plan(batch=len(ls), num_heads=heads, max_seq_len_q=max(qs), max_seq_len=self.max_len,
                             page_size=ps, max_pages_per_req=bt.shape[1], num_pages=pool, packed=packed,
                             max_total_q=self.T + pad, kv_dtype=kind, causal=causal, return_lse=True,
                             q_dtype="e4m3" if q_fp8 else "bf16", window=window, sinks=sinks,
                             e4m3_widen=widen)
        self.workspace = torch.full((self.plan.workspace_bytes,), 0xA5, dtype=torch.uint8, device="cuda")

    def run(self, **kw):
        a = dict(qo_indptr=self.indptr if self.packed else None, total_q=self.query.shape[0] if self.packed else 0,
                 lse=self.lse, workspace=self.workspace, bmm1_scale=self.bmm1, bmm2_scale=self.bmm2)
        a.update(kw)
        self.plan.run(self.query, self.cache, self.tables, self.lens, self.out, **a)
        return self

    def status(self):
        torch.cuda.synchronize()
        off = mla.mla_decode_status_offset()
        return int(self.workspace[off:off + 4].view(torch.int32).item())

    def reference(self):
        """Yields (token, O, lse, terms) in 64 bits; terms: (sum p |v|, bmm1 max sum |q k|,
        sum |v|)."""
        vals = cache_values(self.cache)
        t = 0
        for b, (L, q) in enumerate(zip(self.ls, self.qs)):
            rows = torch.arange(L, device="cuda")
            for i in range(q):
                last = L - q + i if self.causal else L - 1
                ok = rows <= last
                if self.window:
                    ok &= (rows > last - self.window) | (rows < self.sinks)
                j = rows[ok]
                k = vals[self.tables[b].long()[j // self.ps], j % self.ps]
                x = self.query[t].double()
                s = x @ k.T * self.bmm1
                lse = torch.logsumexp(s, -1)
                pr = torch.exp(s - lse[:, None])
                terms = (pr @ k[:, :512].abs()) * abs(self.bmm2), (x.abs() @ k.abs().T).amax(-1) * self.bmm1, \
                    k[:, :512].abs().sum(0) * abs(self.bmm2)
                yield t, pr @ k[:, :512] * self.bmm2, lse, terms
                t += 1

    def qk(self, t):
        """bmm1 max |q| max_j sum |k_j| per head of token t (a bound: every cache row)."""
        if not hasattr(self, "_ksum"):
            self._ksum = float(cache_values(self.cache).abs().sum(-1).nan_to_num(0).max())
        return self.query[t].double().abs().amax(-1) * self._ksum * self.bmm1

    def check(self, p_bits=11, p_floor=2.0 ** -32, what="", status=0):
        """Every row against the reference.  The output's rounding to bf16 is off by
        2^-8 of it; a split request's partials, rounded to bf16 before they are
        joined, by 2^-8 of A = sum p |v|; P, rounded to ``p_bits`` + 1 bits, by
        2^-p_bits of A, and where it underflows by ``p_floor`` of the row's largest P for
        every row of V (f16 and a factor 2^7: the largest P is at least 2^7, half the
        smallest subnormal 2^-25; it shows where the rows of large P hold zeros); an error d of the logits changes O by at most 2 d of A and the
        LSE by d.  d: 576 products in fp32 accumulation, 2^-18 of bmm1 sum |q k|, and
        where a bf16 query enters FP8 MMAs in two parts, 2^-17 of its largest element
        times sum |k|, 2^-17 bmm1 max |q| sum |k| <= 2^-17 bmm1 qk.  All outputs together
        are within 1e-2 in 2-norm (roundings of 2^-8 average out far below)."""
        got, want = [], []
        assert self.status() == status, f"{what}: status {self.status()}"
        out, lse = self.out.double(), self.lse.double()
        for t, o, e, (a, d, v) in self.reference():
            d = d * 2.0 ** -18 + 2e-6 + (self.qk(t) * 2.0 ** -17 if self.split_q else 0.0)
            got.append(out[t])
            want.append(o)
            bound = o.abs() * 2.0 ** -8 + a * (2.0 ** -8 + 2.0 ** -p_bits + 2 * d[:, None]) + v * p_floor + 1e-30
            bad = ~((out[t] - o).abs() <= bound)
            assert not bad.any(), (f"{what} token {t}: {int(bad.sum())} outputs off, worst "
                                   f"{float(((out[t] - o).abs() / bound).nan_to_num(9e9).max()):.3g} x the bound")
            bad = ~((lse[t] - e).abs() <= d + e.abs() * 2.0 ** -22)
            assert not bad.any(), f"{what} token {t}: {int(bad.sum())} LSEs off, {float((lse[t] - e).abs().max()):.3g}"
        err, ref = torch.stack(got) - torch.stack(want), torch.stack(want)
        assert float(err.norm()) <= 1e-2 * float(ref.norm()), f"{what}: 2-norm off by {float(err.norm() / ref.norm()):.3g}"
        assert (self.out[self.T:] == 3.0).all() and (self.lse[self.T:] == 3.0).all(), "rows behind the last request"
