"""Cases for the operators of requests that share rows of the cache.

Three operators, each in a plain form (elementary torch operations) and as the
library's call:

* ``prefix``: decode attention over a batch whose requests share their first
  rows (a system prompt, a document, the prompt of a beam search), which are
  read and multiplied once for all requests of a group.
* ``select``: a step of beam search: the k best continuations of a request's
  beams over the vocabulary.
* ``reorder``: what the step does to the paged cache: each beam's block table
  becomes its parent's, and the page that is still being written is copied.

A 4-bit row is 576 e2m1 codes (two a byte, the even dim in the low nibble) and
36 e4m3 scales, one per 16 dims; a page holds the codes of its rows, then
their scales.
"""
import math
import random

import numpy as np
import torch

own = False

LAT, QK = 512, 576
GROUP, FP4_ROW = 16, 324
BMM1 = 1.0 / math.sqrt(192.0)
KV_SCALE = 5.5 / 448.0  # a calibrated scale of normed latents: their largest magnitude to e4m3's
Q_SCALE = 6.0 / 448.0


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one question, four answers side by side on a small shard: the shortest call there is
        dict(name="prefix_small_bf16", op="prefix", kv="bf16", groups=1, members=4, ragged=False, heads=16, q=1,
             packed=False, page=32, causal=True, q_fp8=False, plo=500, phi=500, lo=1, hi=60, lens=11),
        # a serving batch behind one system prompt, on a tensor-parallel shard
        dict(name="prefix_system_bf16", op="prefix", kv="bf16", groups=1, members=96, ragged=False, heads=16, q=1,
             packed=False, page=64, causal=True, q_fp8=False, plo=6000, phi=6000, lo=64, hi=2048, lens=12),
        # beam search of eight beams in each of sixteen requests
        dict(name="prefix_beams_e4m3", op="prefix", kv="e4m3", groups=16, members=8, ragged=False, heads=32, q=1,
             packed=False, page=64, causal=True, q_fp8=False, plo=1000, phi=8000, lo=1, hi=400, lens=13),
        # many questions about one long document, all heads on one GPU, 4-bit cache
        dict(name="prefix_document_fp4", op="prefix", kv="fp4", groups=1, members=32, ragged=False, heads=128, q=1,
             packed=False, page=64, causal=True, q_fp8=False, plo=65536, phi=65536, lo=100, hi=1500, lens=14),
        # drafted tokens of users of several assistants, groups of uneven size
        dict(name="prefix_drafts_bf16", op="prefix", kv="bf16", groups=6, members=10, ragged=True, heads=64, q=4,
             packed=True, page=64, causal=True, q_fp8=False, plo=2000, phi=20000, lo=4, hi=3000, lens=15),
        # one request, four beams
        dict(name="select_small_fp32", op="select", kind="fp32", batch=1, beams=4, k=4, vocab=32768, row=32768,
             finished=0.0, spread=2.5),
        # a serving batch, a large vocabulary whose rows are padded
        dict(name="select_batch_bf16", op="select", kind="bf16", batch=64, beams=4, k=8, vocab=131071, row=131072,
             finished=0.1, spread=3.0),
        # wide beams that keep twice as many candidates, an odd vocabulary
        dict(name="select_wide_fp32", op="select", kind="fp32", batch=24, beams=16, k=32, vocab=100003, row=100003,
             finished=0.05, spread=2.0),
        # one request's beams, one layer
        dict(name="reorder_small_bf16", op="reorder", kv="bf16", groups=1, beams=4, layers=1, page=64, plo=300, phi=300,
             lo=50, hi=50, lens=21),
        # a batch of beam searches, a stage of a model's layers in one call
        dict(name="reorder_layers_bf16", op="reorder", kv="bf16", groups=48, beams=8, layers=12, page=64, plo=100,
             phi=900, lo=1, hi=120, lens=22),
        # the same over an e4m3 cache with small pages
        dict(name="reorder_layers_e4m3", op="reorder", kv="e4m3", groups=64, beams=4, layers=16, page=32, plo=100,
             phi=900, lo=1, hi=120, lens=23),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "select", "reorder"])
    lens = rng.randrange(1 << 20)
    page = rng.choice([32, 64])
    if op == "select":
        beams = rng.choice([1, 2, 3, 4, 5, 8, 16])
        vocab = _log_int(rng, 40, 150000)
        batch = _log_int(rng, 1, max(1, min(200, 33000000 // (vocab * beams))))
        return dict(op=op, kind=rng.choice(["fp32", "bf16", "fp16"]), batch=batch, beams=beams,
                    k=rng.randint(1, min(64, 2 * beams)), vocab=vocab, row=vocab + rng.choice([0, 0, 1, 8, 61]),
                    finished=rng.choice([0.0, 0.1, 0.5]), spread=rng.uniform(0.5, 4.0))
    if op == "reorder":
        beams = rng.choice([1, 2, 3, 4, 6, 8, 16])
        groups = _log_int(rng, 1, 320 // beams)
        plo, lo = _log_int(rng, 1, 900), rng.randint(0, 60)
        return dict(op=op, kv=rng.choice(["bf16", "e4m3", "fp4"]), groups=groups, beams=beams,
                    layers=rng.choice([1, 2, 5, 12]), page=page, plo=plo, phi=plo + rng.randint(0, 300), lo=lo,
                    hi=lo + rng.randint(0, 120), lens=lens)
    heads = rng.choice([16, 32, 64, 128])
    q = rng.choice([1, 1, 1, 2, 3, 5])
    plo = _log_int(rng, 10, 30000)
    phi = min(60000, int(plo * rng.choice([1.0, 1.5, 3.0])))
    lo = rng.randint(q, 400)
    hi = lo + _log_int(rng, 1, 3000)
    # the products, and the rows of the pool, stay below the largest listed case's
    most = max(2, min(160, 250000000 // ((phi + hi) * heads * q), 250000 // hi))
    members = _log_int(rng, 1, most)
    groups = _log_int(rng, 1, max(1, min(most // members, 200000 // phi)))
    return dict(op=op, kv=rng.choice(["bf16", "e4m3", "fp4"]), groups=groups, members=members,
                ragged=rng.random() < 0.4, heads=heads, q=q, packed=rng.random() < 0.5, page=page,
                causal=rng.random() < 0.75, q_fp8=rng.random() < 0.25, plo=plo, phi=phi, lo=lo, hi=hi, lens=lens)


def _plan(case):
    """(requests of each group, shared rows of each group, rows of each request,
    query tokens of each request): the case alone says them."""
    rng = random.Random(case["lens"])
    G, n = case["groups"], case.get("members", case.get("beams"))
    sizes = [rng.randint(max(1, n // 2), n + n // 2) if case.get("ragged") else n for _ in range(G)]
    shared = [rng.randint(case["plo"], case["phi"]) for _ in range(G)]
    rows, qs = [], []
    for size, p in zip(sizes, shared):
        same = rng.randint(case["lo"], case["hi"])  # (the beams of a search have one length)
        for _ in range(size):
            q = case.get("q", 1)
            q = rng.randint(1, q) if case.get("packed") else q
            more = same if case["op"] == "reorder" else rng.randint(case["lo"], case["hi"])
            rows.append(p + (more if case["op"] == "reorder" else max(more, q)))
            qs.append(q)
    return sizes, shared, rows, qs


def _parents(case):
    """The parent of each beam, by request: the better beams have more children."""
    rng, W = random.Random(case["lens"] + 1), case["beams"]
    return [[min(rng.randrange(W), rng.randrange(W)) for _ in range(W)] for _ in range(case["groups"])]


def work(case):
    if case["op"] == "select":
        rows, k = case["batch"] * case["beams"], case["k"]
        size = 4 if case["kind"] == "fp32" else 2
        return {"bytes": rows * (case["vocab"] * size + 5) + case["batch"] * k * 12, "flops": 4 * rows * case["vocab"]}
    sizes, shared, rows, qs = _plan(case)
    row = {"bf16": 2 * QK, "e4m3": QK, "fp4": FP4_ROW}[case["kv"]]
    ps = case["page"]
    if case["op"] == "reorder":
        # the rows of the page that is being written: read of each beam that others
        # continue, written of each that continues another; the tables, read and written
        W, tail = case["beams"], 0
        for g, kin in enumerate(_parents(case)):
            moved = [p for w, p in enumerate(kin) if p != w]
            tail += (len(moved) + len(set(moved))) * (rows[g * W] % ps) * row * case["layers"]
        return {"bytes": tail + 2 * 4 * sum(-(-L // ps) for L in rows) + 16 * len(rows), "flops": 0}
    H, T = case["heads"], sum(qs)
    qrow = QK * (1 if case["q_fp8"] else 2)
    alone, pairs, at = 0, 0, 0
    for size, p in zip(sizes, shared):
        for L, q in zip(rows[at : at + size], qs[at : at + size]):
            alone += L - p
            pairs += q * L - (q * (q - 1) // 2 if case["causal"] else 0)
        at += size
    meta = 4 * (2 * len(rows) + sum(-(-L // ps) for L in rows))
    return {"bytes": (sum(shared) + alone) * row + T * H * (qrow + 2 * LAT + 4) + meta,
            "flops": 2 * (QK + LAT) * pairs * H}


# ------------------------------------------------------------------ inputs

def _fp4_quantise(y):
    """Rows [..., 576] in fp32 -> (codes uint8 [..., 288], scales e4m3 [..., 36])."""
    g = y.unflatten(-1, (QK // GROUP, GROUP))
    s = (g.abs().amax(-1) * (1.0 / 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    f = s.float()
    t = g * torch.where(f > 0, torch.reciprocal(f), torch.zeros_like(f)).unsqueeze(-1)
    a = t.abs()
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    c = torch.where(torch.signbit(t), c + 8, c).flatten(-2).to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), s


def _make_cache(g, kind, pages, ps):
    if kind == "fp4":
        cache = torch.empty(pages, ps, FP4_ROW, dtype=torch.uint8, device="cuda")
        flat = cache.view(pages, ps * FP4_ROW)
        step = max(1, (1 << 18) // ps)
        for a in range(0, pages, step):
            n = min(step, pages - a)
            c, s = _fp4_quantise(torch.randn(n, ps, QK, generator=g, device="cuda"))
            flat[a : a + n, : ps * 288] = c.flatten(1)
            flat[a : a + n, ps * 288 :] = s.view(torch.uint8).flatten(1)
        return cache
    x = torch.randn(pages, ps, QK, generator=g, device="cuda", dtype=torch.bfloat16)
    return x if kind == "bf16" else (x.float() * (1.0 / KV_SCALE)).clamp_(-448, 448).to(torch.float8_e4m3fn)


def _scale(case):
    return KV_SCALE if case["kv"] == "e4m3" else 1.0


def _device(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _tables(case, g):
    """Block tables and the pool's pages.  The whole pages of a group's shared rows are
    the same pages in all its tables; a page that they end in is each request's own.
    A beam search's tables reach past its rows, and each beam has a spare page."""
    sizes, shared, rows, _ = _plan(case)
    ps, beams = case["page"], case["op"] == "reorder"
    n, at, table, spare, copies = 0, 0, [], [], []
    for size, p in zip(sizes, shared):
        whole = p // ps
        first = list(range(n, n + whole))
        n += whole
        for m in range(size):
            more = (rows[at] // ps + 2 if beams else -(-rows[at] // ps)) - whole
            table.append(first + list(range(n, n + more)))
            if p % ps and m > 0:
                copies.append((table[at - m][whole], n))  # the shared rows in it are the same
            n += more
            if beams:
                spare.append(n)
                n += 1
            at += 1
    pool = n + n // 8 + 1
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    width = max(map(len, table))
    t = torch.tensor(np.array([r + [-1] * (width - len(r)) for r in table]), device="cuda")
    st = dict(tables=torch.where(t >= 0, order[t.clamp(min=0)], torch.full_like(order[:1], -1)).contiguous())
    if beams:
        st["spare"] = order[torch.tensor(spare, device="cuda")].contiguous()
    if copies:
        c = order[torch.tensor(copies, device="cuda")].long()
        st["copies"] = (c[:, 0], c[:, 1])
    return st, pool


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "select":
        B, W, V = case["batch"], case["beams"], case["vocab"]
        kind = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}[case["kind"]]
        # a request's beams say nearly the same; a few tokens stand out
        x = torch.randn(B, W, case["row"], generator=g, device="cuda")
        x += torch.randn(B, 1, case["row"], generator=g, device="cuda") * 1.5
        x *= case["spread"] / 1.8
        scores = -torch.rand(B, W, generator=g, device="cuda").cumsum(-1) * 3.0 - 2.0
        done = torch.rand(B, W, generator=g, device="cuda") < case["finished"]
        return dict(case=case, logits=x.to(kind)[..., :V], scores=scores, finished=done.to(torch.uint8), end=V // 3)
    sizes, shared, rows, qs = _plan(case)
    st, pool = _tables(case, g)
    n = case["layers"] if case["op"] == "reorder" else 1
    caches = [_make_cache(g, case["kv"], pool, case["page"]) for _ in range(n)]
    if "copies" in st:
        a, b = st.pop("copies")
        for c in caches:
            c.view(torch.uint8)[b] = c.view(torch.uint8)[a]
    st.update(case=case, lens=_device(rows), max_len=max(rows))
    if case["op"] == "reorder":
        st.update(caches=caches, parents=_device(_parents(case)))
        return st
    H, T, B = case["heads"], sum(qs), len(rows)
    x = torch.randn(T, H, QK, generator=g, device="cuda", dtype=torch.bfloat16)
    if case["q_fp8"]:
        x = (x.float() * (1.0 / Q_SCALE)).clamp_(-448, 448).to(torch.float8_e4m3fn)
    if not case["packed"]:
        x = x.view(B, case["q"], H, QK)
    blocks = -(-T * H // 128) + len(sizes) + sum(-(-q * H // 128) for q in qs) + 256
    st.update(query=x, cache=caches[0], T=T, bmm1=BMM1 * _scale(case) * (Q_SCALE if case["q_fp8"] else 1.0),
              bmm2=_scale(case), indptr=_device(np.cumsum([0] + qs)),
              group_indptr=_device(np.cumsum([0] + sizes)), prefix=_device(shared), max_prefix=max(shared),
              max_size=max(sizes), max_alone=max(L - p for L, p in zip(rows, np.repeat(shared, sizes))),
              workspace=torch.empty((64 << 20) + blocks * (272 << 10), dtype=torch.uint8, device="cuda"),
              out=torch.empty(*x.shape[:-1], LAT, dtype=torch.bfloat16, device="cuda"),
              lse=torch.empty(T, H, dtype=torch.float32, device="cuda"))
    return st


# ------------------------------------------------------------------ plain forms

def _rows(case, cache, page, row):
    """fp32 values of the cache rows (page, row): index tensors of one shape."""
    if case["kv"] != "fp4":
        return cache[page, row].float()
    pages, ps = cache.shape[0], cache.shape[1]
    flat = cache.view(pages, ps * FP4_ROW)
    codes, scales = flat[:, : ps * 288].unflatten(1, (ps, 288)), flat[:, ps * 288 :].unflatten(1, (ps, 36))
    mag = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda")
    one = torch.cat([mag, -mag])
    pair = torch.stack([one.repeat(16), one.repeat_interleave(16)], -1)  # by byte: low nibble, high nibble
    v = pair[codes[page, row].int()].flatten(-2).unflatten(-1, (QK // GROUP, GROUP))
    return (v * scales[page, row].view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)


def _plain_prefix(st):
    """Both parts padded to their longest: the shared rows once a group, for all its
    query rows, and each request's own rows; one softmax over the two."""
    case = st["case"]
    H, qm, ps = case["heads"], case["q"], case["page"]
    B, G, n = st["tables"].shape[0], st["prefix"].shape[0], st["max_size"]
    L, P = st["lens"].long(), st["prefix"].long()
    first, size = st["group_indptr"][:-1].long(), (st["group_indptr"][1:] - st["group_indptr"][:-1]).long()
    of = torch.searchsorted(st["group_indptr"], torch.arange(B, device="cuda", dtype=torch.int32), right=True) - 1
    ql = (st["indptr"][1:] - st["indptr"][:-1]).long()
    i = torch.arange(qm, device="cuda")
    t = (st["indptr"][:-1].long()[:, None] + i).clamp(max=st["T"] - 1)
    x = st["query"].reshape(st["T"], H, QK)
    x = x.view(torch.uint8)[t].view(torch.float8_e4m3fn).float() if case["q_fp8"] else x[t].float()  # [B, q, H, 576]

    # the group's query rows against the shared rows
    m = torch.arange(n, device="cuda")
    member = (first[:, None] + m).clamp(max=B - 1)
    j = torch.arange(st["max_prefix"], device="cuda")
    jc = torch.minimum(j, P[:, None] - 1)
    keys = _rows(case, st["cache"], st["tables"][first].gather(1, jc // ps).long(), jc % ps)  # [G, P, 576]
    s = torch.matmul(x[member].reshape(G, -1, QK), keys.transpose(1, 2)) * st["bmm1"]
    s.masked_fill_((j >= P[:, None])[:, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(top).exp_()
    mass = p.sum(-1, keepdim=True)
    acc = torch.matmul(p, keys[..., :LAT])
    del s, p, keys
    place = torch.arange(B, device="cuda") - first[of]

    def of_member(v):
        return v.view(G, n, qm, H, -1)[of, place]  # [B, q, H, ..]

    top, mass, acc = of_member(top), of_member(mass), of_member(acc)

    # each request's own rows
    j = P[of][:, None] + torch.arange(st["max_alone"], device="cuda")
    inside = j < L[:, None]
    jc = torch.minimum(j, L[:, None] - 1)
    keys = _rows(case, st["cache"], st["tables"].gather(1, jc // ps).long(), jc % ps)
    last = L[:, None] - ql[:, None] + i if case["causal"] else (L - 1)[:, None].expand(B, qm)
    see = (j[:, None] <= last[..., None]) & inside[:, None]
    s = torch.matmul(x.reshape(B, qm * H, QK), keys.transpose(1, 2)) * st["bmm1"]
    s = s.view(B, qm, H, -1).masked_fill_(~see[:, :, None], -math.inf)
    both = torch.maximum(top, s.amax(-1, keepdim=True))
    p = s.sub_(both).exp_()
    down = (top - both).exp()
    mass = mass * down + p.sum(-1, keepdim=True)
    acc = acc * down + torch.matmul(p.view(B, qm * H, -1), keys[..., :LAT]).view(B, qm, H, LAT)
    tok = torch.arange(st["T"], device="cuda")
    b = torch.searchsorted(st["indptr"], tok.int(), right=True) - 1
    k = tok - st["indptr"][b]
    st["out"].view(st["T"], H, LAT).copy_((acc / mass * st["bmm2"])[b, k])
    st["lse"].copy_((both + mass.log())[b, k, :, 0])
    return {"out": st["out"], "lse": st["lse"]}


def _plain_select(st):
    # in 64 bits: of two candidates that nearly tie, the better one is wanted
    case, V = st["case"], st["case"]["vocab"]
    B, W, k = case["batch"], case["beams"], case["k"]
    x = st["logits"].double()
    top = x.amax(-1, keepdim=True)
    score = x - top
    score = score - score.exp().sum(-1, keepdim=True).log() + st["scores"].double()[..., None]
    done = st["finished"].bool()[..., None]
    only = torch.arange(V, device="cuda") == st["end"]
    score = torch.where(done, torch.where(only, st["scores"].double()[..., None], -math.inf), score)
    best, at = score.view(B, W * V).sort(dim=-1, descending=True, stable=True)  # ties: the lowest index
    best, at = best[:, :k], at[:, :k]
    if W * V < k:
        best = torch.nn.functional.pad(best, (0, k - W * V), value=-math.inf)
        at = torch.nn.functional.pad(at, (0, k - W * V))
    some = best > -math.inf
    none = torch.full_like(at, -1)
    return {"scores": best.float(), "tokens": torch.where(some, at % V, none).int(),
            "parents": torch.where(some, at // V, none).int()}


def _plain_reorder(st):
    case, ps, W = st["case"], st["case"]["page"], st["case"]["beams"]
    n = st["tables"].shape[0]
    b = torch.arange(n, device="cuda")
    parent = b // W * W + st["parents"].long().view(-1)
    moved = parent != b
    L = st["lens"].long()
    old = st["tables"].clone()
    col = torch.arange(old.shape[1], device="cuda")
    whole, rest = L // ps, L % ps
    last = whole.clamp(max=old.shape[1] - 1)[:, None]
    src, mine = old[parent].gather(1, last)[:, 0], old.gather(1, last)[:, 0]
    swap = moved & (rest > 0)
    new = torch.where(col < whole[:, None], old[parent], old)
    new.scatter_(1, last, torch.where(swap, st["spare"], new.gather(1, last)[:, 0])[:, None])
    # the rows of the page that is being written, all reads before any write
    pick = torch.nonzero(swap)[:, 0]
    r = torch.arange(ps, device="cuda")
    from_page, to_page = src[pick].long(), st["spare"][pick].long()
    for c in st["caches"]:
        raw = c.view(torch.uint8).view(c.shape[0], -1)
        if case["kv"] == "fp4":
            parts = (raw[:, : ps * 288].unflatten(1, (ps, 288)), raw[:, ps * 288 :].unflatten(1, (ps, 36)))
        else:
            parts = (raw.unflatten(1, (ps, -1)),)
        for part in parts:
            keep = (r < rest[pick][:, None])[..., None]
            part[to_page] = torch.where(keep, part[from_page], part[to_page])
    st["tables"].copy_(new)
    st["spare"].copy_(torch.where(swap, mine, st["spare"]))
    return {"caches": st["caches"], "tables": st["tables"], "spare": st["spare"]}


# ------------------------------------------------------------------ the library's calls

def _own_prefix(st):
    import paged_mla_decode_03_gb300 as mla
    case = st["case"]
    which = dict(qo_indptr=st["indptr"], max_seq_len_q=case["q"]) if case["packed"] else {}
    if case["ragged"]:
        which["prefix_indptr"] = st["group_indptr"]
    mla.decode(st["query"], st["cache"], st["workspace"], st["tables"], st["lens"], st["max_len"], out=st["out"],
               lse=st["lse"], bmm1_scale=st["bmm1"], bmm2_scale=st["bmm2"],
               mask_type="causal" if case["causal"] else "dense", return_lse=True, prefix_lens=st["prefix"], **which)
    return {"out": st["out"], "lse": st["lse"]}


def _own_select(st):
    import paged_mla_decode_03_gb300 as mla
    scores, tokens, parents = mla.beam_select(st["logits"], st["scores"], k=st["case"]["k"],
                                              finished=st["finished"], end_token=st["end"])
    return {"scores": scores, "tokens": tokens, "parents": parents}


def _own_reorder(st):
    import paged_mla_decode_03_gb300 as mla
    mla.cache_reorder(st["caches"], st["tables"], st["lens"], st["parents"], st["spare"])
    return {"caches": st["caches"], "tables": st["tables"], "spare": st["spare"]}


def run(state):
    op = state["case"]["op"]
    if op == "prefix":
        return _own_prefix(state) if own else _plain_prefix(state)
    if op == "select":
        return _own_select(state) if own else _plain_select(state)
    return _own_reorder(state) if own else _plain_reorder(state)


# ------------------------------------------------------------------ 64 bits

def _exact_keys(case, cache, pages, L):
    ps = case["page"]
    if case["kv"] != "fp4":
        return cache[pages].reshape(-1, QK)[:L].double()
    raw = cache.view(-1, ps * FP4_ROW)[pages]
    by = raw[:, : ps * 288].reshape(-1, 288)[:L].to(torch.int16)
    codes = torch.stack([by & 15, by >> 4], -1).flatten(-2)
    mag = (codes & 7).double()
    e, m = torch.div(mag, 2, rounding_mode="floor"), mag % 2
    val = torch.where(e > 0, (1 + m / 2) * torch.exp2(e - 1), m / 2) * torch.where(codes > 7, -1.0, 1.0)
    sc = raw[:, ps * 288 :].reshape(-1, 36)[:L].contiguous().view(torch.float8_e4m3fn).double()
    return (val.view(L, 36, GROUP) * sc[..., None]).view(L, QK)


def _exact_prefix(st):
    """Every request by itself, over its own table: sharing changes no value."""
    case = st["case"]
    outs, lses, t0 = [], [], 0
    x = st["query"].reshape(st["T"], case["heads"], QK).double()
    _, _, rows, qs = _plan(case)
    for b, (L, q) in enumerate(zip(rows, qs)):
        keys = _exact_keys(case, st["cache"], st["tables"][b, : -(-L // case["page"])].long(), L)
        for i in range(q):
            kk = keys[: L - q + i + 1] if case["causal"] else keys
            s = x[t0 + i] @ kk.T * st["bmm1"]
            lse = torch.logsumexp(s, -1)
            outs.append(torch.exp(s - lse[:, None]) @ kk[:, :LAT] * st["bmm2"])
            lses.append(lse)
        t0 += q
    return {"out": torch.stack(outs).view(st["out"].shape), "lse": torch.stack(lses)}


def _exact_select(st):
    case = st["case"]
    best = []
    for b in range(case["batch"]):
        found = []
        for w in range(case["beams"]):
            s = st["scores"][b, w].double()
            if st["finished"][b, w]:
                found.append(s[None])
            else:
                found.append(s + torch.log_softmax(st["logits"][b, w].double(), 0).topk(min(case["k"], case["vocab"])).values)
        v = torch.cat(found).sort(descending=True).values[: case["k"]]
        best.append(torch.cat([v, v.new_full((case["k"] - v.numel(),), -math.inf)]))
    return {"scores": torch.stack(best), "tokens": None, "parents": None}


def _exact_reorder(st):
    case, ps = st["case"], st["case"]["page"]
    tables, spare = st["tables"].tolist(), st["spare"].tolist()
    new, kept = [list(r) for r in tables], list(spare)
    caches = [c.clone() for c in st["caches"]]
    for g, row in enumerate(st["parents"].tolist()):
        for w, p in enumerate(row):
            b, a = g * case["beams"] + w, g * case["beams"] + p
            whole, rest = divmod(int(st["lens"][b]), ps)
            new[b][:whole] = tables[a][:whole]
            if a == b or rest == 0:
                continue
            new[b][whole], kept[b] = spare[b], tables[b][whole]
            for c, old in zip(caches, st["caches"]):
                d, s = c.view(torch.uint8)[spare[b]].view(-1), old.view(torch.uint8)[tables[a][whole]].view(-1)
                if case["kv"] == "fp4":
                    d[: rest * 288] = s[: rest * 288]
                    d[ps * 288 : ps * 288 + rest * 36] = s[ps * 288 : ps * 288 + rest * 36]
                else:
                    n = rest * QK * (2 if case["kv"] == "bf16" else 1)
                    d[:n] = s[:n]
    return {"caches": [c.double() if case["kv"] != "fp4" else None for c in caches], "tables": _device(new), "spare": _device(kept)}


def exact(case, seed):
    if work(case)["flops"] > 7e11:
        return None
    st = prepare(case, seed)
    return {"prefix": _exact_prefix, "select": _exact_select, "reorder": _exact_reorder}[case["op"]](st)
