"""Inputs of decodes over shared prefixes for the tests: a Case (tests/attention_ref.py)
whose requests' tables name the same pages for the whole pages of their group's shared rows.
A page that the shared rows end in is each request's own, with the same rows in it."""
import torch

import paged_mla_decode_03_gb300 as mla
from attention_ref import Case


class PrefixCase(Case):
    def __init__(self, kind, ps, sizes, shared, own, qs, heads, *, gap=0, uniform=False, same_pages=True,
                 claim=None, **kw):
        """``sizes`` requests a group with ``shared`` rows each, ``gap`` requests of their own
        before and after; own[i % len(own)] rows past the shared ones, qs likewise."""
        ls, of, indptr = [], [], [gap]
        for size in sizes:
            indptr.append(indptr[-1] + size)
        total = indptr[-1] + gap
        for b in range(total):
            g = next((g for g in range(len(sizes)) if indptr[g] <= b < indptr[g + 1]), -1)
            of.append(g)
            ls.append((shared[g] if g >= 0 else 0) + own[b % len(own)])
        q = [qs[b % len(qs)] for b in range(total)]
        ls = [max(L, n) for L, n in zip(ls, q)]
        self.group_of, self.group_indptr_host = of, indptr
        packed = kw.pop("packed", len(set(q)) > 1)
        super().__init__(kind, ps, ls, q, heads, packed=packed, **kw)
        raw = self.cache.view(torch.uint8).view(self.cache.shape[0], -1)
        for b, g in enumerate(of):
            if g < 0 or b == indptr[g]:
                continue
            whole, rest = divmod(shared[g], ps)
            first = self.tables[indptr[g]]
            seen = ls[b]
            for k in range(min(whole, -(-seen // ps))):
                mine = int(self.tables[b, k])
                if same_pages:
                    self.tables[b, k] = first[k]
                    raw[mine, ps * 288 if kind == "fp4" else 0:] = 0xFF if kind == "bf16" else 0x7F  # NaN
                else:
                    raw[mine] = raw[int(first[k])]
            if rest and whole < -(-seen // ps):
                self._copy_rows(int(first[whole]), int(self.tables[b, whole]), rest)
        self.shared = shared
        claim = shared if claim is None else claim
        self.prefix_lens = torch.tensor(claim, dtype=torch.int32, device="cuda")
        self.prefix_indptr = None if uniform else torch.tensor(indptr, dtype=torch.int32, device="cuda")
        p = self.plan.params
        self.plan = mla.Plan(batch=p.batch, num_heads=heads, max_seq_len_q=p.max_seq_len_q, max_seq_len=p.max_seq_len,
                             page_size=ps, max_pages_per_req=p.max_pages_per_req, num_pages=p.num_pages,
                             packed=packed, max_total_q=p.max_total_q, kv_dtype=kind, causal=self.causal,
                             return_lse=True, q_dtype="e4m3" if p.q_dtype else "bf16", prefix_groups=len(sizes))
        self.split_q = False
        self.workspace = torch.full((self.plan.workspace_bytes,), 0xA5, dtype=torch.uint8, device="cuda")

    def _copy_rows(self, src, dst, n):
        if self.kind == "fp4":
            flat = self.cache.view(self.cache.shape[0], -1)
            flat[dst, :n * 288] = flat[src, :n * 288]
            at = self.ps * 288
            flat[dst, at:at + n * 36] = flat[src, at:at + n * 36]
        else:
            self.cache.view(torch.uint8)[dst, :n] = self.cache.view(torch.uint8)[src, :n]

    def run(self, **kw):
        return super().run(**{**dict(prefix_lens=self.prefix_lens, prefix_indptr=self.prefix_indptr), **kw})

    def items(self):
        """The work list's items, ten numbers each."""
        torch.cuda.synchronize()
        at, _, _ = mla.mla_decode_work_list_layout(self.plan.handle)
        n = int(self.workspace[4:8].view(torch.int32).item())
        return self.workspace[at:at + 40 * n].view(torch.int32).view(n, 10).cpu()

    def shares(self):
        """Whether some row group takes the query rows of several requests."""
        return bool((self.items()[:, 5] > max(self.qs)).any())
