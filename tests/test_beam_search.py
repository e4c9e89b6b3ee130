"""A beam search over the paged cache, as a server would run it: each step appends the chosen
tokens' rows, decodes over the shared prompt, selects the next beams and reorders the cache.
Every beam's hypothesis is kept on the host, and every step its attention is recomputed in 64
bits from a cache of its own that its tokens were appended to in order."""
import math

import pytest
import torch

import paged_mla_decode_03_gb300 as mla
from attention_ref import cache_values
from test_beam import reference

H, V = 16, 96


class Model:
    """Rows, queries and logits by token; enough of a model to search with."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.latent, self.pe = r(V, 512).to(torch.bfloat16).cuda(), r(V, 64).to(torch.bfloat16).cuda()
        self.q_nope = r(V, H, 512).to(torch.bfloat16).cuda()
        self.q_pe = r(V, H, 64).to(torch.bfloat16).cuda()
        self.head = (r(H * 512, V) / math.sqrt(H * 512) * 6).cuda()
        self.weight = torch.ones(512, dtype=torch.bfloat16, device="cuda")
        self.table = mla.rope_table(4096)

    def append(self, tokens, cache, tables, lens, scale, **kw):
        t = torch.as_tensor(tokens, device="cuda").long()
        return mla.cache_append(self.latent[t], self.pe[t], cache, tables, lens, rope_table=self.table,
                                norm_weight=self.weight, kv_scale=scale, q_nope=self.q_nope[t], q_pe=self.q_pe[t], **kw)


def new_cache(kind, pages, ps):
    if kind == "fp4":
        return torch.zeros(pages, ps, 324, dtype=torch.uint8, device="cuda")
    c = torch.zeros(pages, ps, 576, dtype=torch.bfloat16, device="cuda")
    return c if kind == "bf16" else c.to(torch.float8_e4m3fn)


@pytest.mark.gpu
@pytest.mark.parametrize("kind,ps,prompts,W,steps", [
    ("bf16", 32, [70, 33], 3, 70), ("e4m3", 32, [64, 7, 1], 4, 40), ("fp4", 64, [100, 130], 2, 70),
    ("bf16", 64, [1500], 48, 4), ("fp4", 64, [2000, 1800], 40, 3)])
def test_beam_search(kind, ps, prompts, W, steps):
    torch.manual_seed(len(prompts) * W)
    m, B, scale = Model(W), len(prompts), 0.02 if kind == "e4m3" else 1.0
    ahead = -(-steps // ps) + 1
    # beam 0 of each request has the prompt; every beam has pages for new rows and a spare one
    width, n, rows, spare = -(-max(prompts) // ps) + ahead + 1, 0, [], []
    for L in prompts:
        for w in range(W):
            first = L // ps if w == 0 else 0
            own = [-1] * (0 if w == 0 else L // ps) + list(range(n, n + first + ahead + 1))
            n += first + ahead + 1
            rows.append(own + [-1] * (width - len(own)))
            spare.append(n)
            n += 1
    order = torch.randperm(n).int()
    tables = torch.tensor(rows)
    tables = torch.where(tables >= 0, order[tables.clamp(min=0)], -1).int().cuda()
    spare = order[torch.tensor(spare)].cuda()
    layers = [new_cache(kind, n, ps) for _ in range(2)]  # one of them is attended
    cache = layers[1]
    text = [torch.randint(V, (L,)).tolist() for L in prompts]
    for c in layers:
        m.append(sum(text, []), c, tables[::W].contiguous(), torch.tensor(prompts, dtype=torch.int32, device="cuda"),
                 scale, qo_indptr=torch.tensor([0] + torch.tensor(prompts).cumsum(0).tolist(), dtype=torch.int32, device="cuda"))
    lens = torch.tensor([L for L in prompts for _ in range(W)], dtype=torch.int32, device="cuda")
    prefix = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    # all beams continue the prompt, each with another first token
    mla.cache_reorder(layers, tables, lens, torch.zeros(B, W, dtype=torch.int32, device="cuda"), spare, status=status)
    hyps = [text[b] + [(7 * w + b) % V] for b in range(B) for w in range(W)]
    scores = torch.zeros(B, W, device="cuda")
    workspace = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    bmm1 = scale / math.sqrt(192.0)
    for step in range(steps):
        tokens = [h[-1] for h in hyps]
        lens += 1
        for c in layers:
            query = m.append(tokens, c, tables, lens, scale, q_len=1, status=status)
        out, lse = mla.decode(query.view(B * W, 1, H, 576), cache, workspace, tables, lens, int(lens.max()), bmm1_scale=bmm1,
                              bmm2_scale=scale, return_lse=True, prefix_lens=prefix)
        logits = (out.view(B * W, H * 512).float() @ m.head).view(B, W, V)
        if step % 13 == 0 or step >= steps - 3:  # against each hypothesis on its own
            for i, h in enumerate(hyps):
                own = new_cache(kind, -(-len(h) // ps), ps)
                page = torch.arange(own.shape[0], dtype=torch.int32, device="cuda")[None]
                m.append(h, own, page, torch.tensor([len(h)], dtype=torch.int32, device="cuda"), scale, q_len=len(h))
                k = cache_values(own).view(-1, 576)[:len(h)]
                x = query.view(B * W, H, 576)[i].double()
                s = x @ k.T * bmm1
                want = torch.softmax(s, -1) @ k[:, :512] * scale
                # (roundings of 2^-8 of the output, of P and of partials, relative to the sum of p |v|)
                room = (torch.softmax(s, -1) @ k[:, :512].abs()) * scale * 3 * 2.0 ** -8 + 1e-6
                assert ((out[i, 0].double() - want).abs() <= room).all(), (step, i)
                assert ((lse[i].double() - torch.logsumexp(s, -1)).abs() <= 1e-3).all()
        before = scores
        scores, chosen, parents = mla.beam_select(logits, before, k=W)
        found, sure = reference(logits, before, W)
        if sure:
            assert [[(w, v) for _, w, v in r] for r in found] == \
                [list(zip(pr, tr)) for pr, tr in zip(parents.tolist(), chosen.tolist())]
        mla.cache_reorder(layers, tables, lens, parents, spare, status=status)
        p, t = parents.tolist(), chosen.tolist()
        hyps = [hyps[b * W + p[b][w]] + [t[b][w]] for b in range(B) for w in range(W)]
    assert int(status) == 0
    # no page in which a beam still writes, and no spare one, is another's
    left = []
    for i in range(B * W):
        left += [int(x) for x in tables[i, int(lens[i]) // ps:] if x >= 0] + [int(spare[i])]
    assert len(set(left)) == len(left)
