"""Cases for the cache and attention operators around the paged MLA decode.

Three operators, each in a plain form (elementary torch operations in fp32) and
as the library's call:

* ``append``: RMS norm of the new tokens' latents, rotation of their RoPE part
  (and of the query's), quantisation to the cache's format (bf16, e4m3 or 4
  bits) and the store into the pages.  e4m3 and 4-bit caches are read back
  with the matching ``cache_gather``, so the rows come back as values.
* ``fp4``: decode attention over a cache held in 4 bits.
* ``window``: decode attention with a sliding window and a few first tokens
  that stay visible (sinks), over a cache of any format.

A 4-bit row is 576 e2m1 codes (two a byte, the even dim in the low nibble) and
36 e4m3 scales, one per 16 dims; a page holds the codes of its rows, then
their scales.
"""
import math
import random

import numpy as np
import torch

own = False

LAT, ROPE, QK = 512, 64, 576
GROUP, FP4_ROW = 16, 324
MAX_POSITION = 163840
BMM1 = 1.0 / math.sqrt(192.0)
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a few chats, one new token each: the shortest call there is
        dict(name="append_small_bf16", op="append", kv="bf16", batch=8, heads=16, q=1, packed=False,
             page=64, style="interleaved", q_fp8=False, lo=1, hi=4096, lens=11),
        # a full decode batch of a model served on one GPU, 4-bit cache
        dict(name="append_batch_fp4", op="append", kv="fp4", batch=128, heads=128, q=1, packed=False,
             page=64, style="interleaved", q_fp8=False, lo=1024, hi=8192, lens=12),
        # drafted tokens being verified, everything quantised to e4m3
        dict(name="append_mtp_e4m3", op="append", kv="e4m3", batch=32, heads=128, q=4, packed=False,
             page=64, style="half", q_fp8=True, lo=2048, hi=16384, lens=13),
        # prompt chunks of uneven length written through the same call
        dict(name="append_prompt_fp4", op="append", kv="fp4", batch=24, heads=128, q=331, packed=True,
             page=32, style="interleaved", q_fp8=False, lo=400, hi=120000, lens=14),
        # two or three short chats on a tensor-parallel shard
        dict(name="fp4_small", op="fp4", kv="fp4", batch=3, heads=16, q=1, packed=False, page=32,
             causal=True, q_fp8=False, lo=1, hi=200, lens=21, spread="uniform"),
        # the serving batch the library's benchmark is about, cache in 4 bits
        dict(name="fp4_batch", op="fp4", kv="fp4", batch=64, heads=128, q=1, packed=False, page=64,
             causal=True, q_fp8=False, lo=1024, hi=8192, lens=22, spread="uniform"),
        # ragged requests with drafted tokens on a tensor-parallel shard
        dict(name="fp4_ragged", op="fp4", kv="fp4", batch=128, heads=16, q=8, packed=True, page=32,
             causal=True, q_fp8=False, lo=8, hi=32768, lens=23, spread="lognormal"),
        # long documents: what a 4-bit cache is bought for
        dict(name="fp4_long", op="fp4", kv="fp4", batch=8, heads=128, q=2, packed=False, page=64,
             causal=True, q_fp8=False, lo=65536, hi=131072, lens=24, spread="uniform"),
        # a few streaming chats with a short window
        dict(name="window_small_bf16", op="window", kv="bf16", batch=4, heads=16, q=1, packed=False,
             page=64, causal=True, q_fp8=False, lo=1, hi=2000, lens=31, spread="uniform", window=128,
             sinks=4),
        # a serving batch whose layers see the last thousand tokens
        dict(name="window_batch_bf16", op="window", kv="bf16", batch=64, heads=128, q=1, packed=False,
             page=64, causal=True, q_fp8=False, lo=1024, hi=32768, lens=32, spread="uniform",
             window=1024, sinks=4),
        # drafted tokens over an e4m3 cache with a wide window
        dict(name="window_mtp_e4m3", op="window", kv="e4m3", batch=32, heads=128, q=4, packed=False,
             page=64, causal=True, q_fp8=False, lo=2048, hi=16384, lens=33, spread="uniform",
             window=4096, sinks=64),
        # ragged requests over a 4-bit cache, an odd window that ends inside pages
        dict(name="window_ragged_fp4", op="window", kv="fp4", batch=128, heads=64, q=3, packed=True,
             page=32, causal=True, q_fp8=False, lo=3, hi=16384, lens=34, spread="lognormal",
             window=777, sinks=9),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "fp4", "window"])
    heads = rng.choice([16, 32, 64, 128])
    page = rng.choice([32, 64])
    packed = rng.random() < 0.5
    q_fp8 = rng.random() < 0.25
    lens = rng.randrange(1 << 20)
    if op == "append":
        q = rng.choice([1, 1, 2, 3, 5, _log_int(rng, 6, 300)])
        batch = _log_int(rng, 1, max(1, min(256, 4000 // q)))
        lo = max(q, _log_int(rng, 1, 2000))
        more = _log_int(rng, 1, max(1, min(16000, 600000 // batch)))
        return dict(op=op, kv=rng.choice(["bf16", "e4m3", "fp4"]), batch=batch, heads=heads, q=q, packed=packed,
                    page=page, style=rng.choice(["interleaved", "half"]), q_fp8=q_fp8, lo=lo,
                    hi=lo + more, lens=lens)
    q = rng.choice([1, 1, 1, 2, 3, 4, 7])
    top = _log_int(rng, 16, 100000)
    # the rows of the pool, and the products, stay below the largest listed case's
    batch = _log_int(rng, 1, max(1, min(200, 600000 // top, (20000000 // top) // (q * heads))))
    lo = max(q, int(top * rng.random()))
    case = dict(op=op, kv="fp4", batch=batch, heads=heads, q=q, packed=packed, page=page,
                causal=rng.random() < 0.75, q_fp8=q_fp8, lo=lo, hi=max(top, lo), lens=lens,
                spread=rng.choice(["uniform", "lognormal"]))
    if op == "window":
        case.update(kv=rng.choice(["bf16", "e4m3", "fp4"]), window=_log_int(rng, 1, 6000),
                    sinks=rng.choice([0, 1, 4, 13, 64, 130]))
    return case


def _lengths(case):
    """(cache lengths, query lengths) of the case's requests: the case alone says them."""
    rng = random.Random(case["lens"])
    B, q = case["batch"], case["q"]
    qs = [rng.randint(max(1, q // 2), q) if case["packed"] else q for _ in range(B)]
    if case.get("spread") == "lognormal":
        mid = math.log(max(1.0, case["hi"] / 8))
        ls = [int(min(max(rng.lognormvariate(mid, 1.0), case["lo"]), case["hi"])) for _ in range(B)]
    else:
        ls = [rng.randint(case["lo"], case["hi"]) for _ in range(B)]
    return [max(a, b) for a, b in zip(ls, qs)], qs


def _visible(case):
    """Per request: (cache rows that some query row sees, query row and cache row pairs)."""
    rows = pairs = 0
    W, S = case.get("window", 0), case.get("sinks", 0)
    for L, q in zip(*_lengths(case)):
        seen = 0
        for i in range(q):
            last = L - q + i if case["causal"] else L - 1
            lo = max(0, last - W + 1) if W else 0
            seen += last + 1 - lo + min(S, lo)
        pairs += seen
        first = L - q if case["causal"] else L - 1
        lo = max(0, first - W + 1) if W else 0
        rows += L - lo + min(S, lo)
    return rows, pairs


def work(case):
    ls, qs = _lengths(case)
    T, H = sum(qs), case["heads"]
    row = {"bf16": 2 * QK, "e4m3": QK, "fp4": FP4_ROW}[case["kv"]]
    qrow = QK * (1 if case["q_fp8"] else 2)
    meta = 4 * (len(ls) + sum(-(-L // case["page"]) for L in ls))
    if case["op"] == "append":
        back = 0 if case["kv"] == "bf16" else T * (row + 2 * QK)
        return {"bytes": T * (2 * QK + 4 * ROPE + row) + T * H * (2 * QK + qrow) + 2 * LAT + back
                + 4 * (2 * len(ls) + T),
                "flops": T * (4 * LAT + 3 * ROPE) + T * H * 3 * ROPE}
    rows, pairs = _visible(case)
    return {"bytes": rows * row + T * H * (qrow + 2 * LAT + 4) + meta, "flops": 2 * (QK + LAT) * pairs * H}


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


def _fp4_parts(cache):
    """Views of a 4-bit cache's codes [pages, page, 288] and scales [pages, page, 36]."""
    pages, ps = cache.shape[0], cache.shape[1]
    flat = cache.view(pages, ps * FP4_ROW)
    return flat[:, : ps * 288].unflatten(1, (ps, 288)), flat[:, ps * 288 :].unflatten(1, (ps, 36))


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _make_cache(g, kind, pages, ps):
    if kind == "fp4":
        cache = torch.empty(pages, ps, FP4_ROW, dtype=torch.uint8, device="cuda")
        codes, scales = _fp4_parts(cache)
        step = max(1, (1 << 18) // ps)
        for a in range(0, pages, step):
            n = min(step, pages - a)
            c, s = _fp4_quantise(torch.randn(n, ps, QK, generator=g, device="cuda"))
            codes[a : a + n] = c
            scales[a : a + n] = s.view(torch.uint8)
        return cache
    x = torch.randn(pages, ps, QK, generator=g, device="cuda", dtype=torch.bfloat16)
    return x if kind == "bf16" else (x.float() * (1.0 / KV_SCALE)).clamp_(-448, 448).to(torch.float8_e4m3fn)


KV_SCALE = 5.5 / 448.0  # a calibrated scale of normed latents: their largest magnitude to e4m3's
Q_SCALE = 6.0 / 448.0


def _scale(case):
    return KV_SCALE if case["kv"] == "e4m3" else 1.0


def prepare(case, seed):
    g = _gen(seed)
    ls, qs = _lengths(case)
    B, ps, H, T = case["batch"], case["page"], case["heads"], sum(qs)
    need = [-(-L // ps) for L in ls]
    width = max(need)
    pool = sum(need) + sum(need) // 8 + 1
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    start = torch.tensor(np.cumsum([0] + need[:-1]), device="cuda")
    at = start[:, None] + torch.arange(width, device="cuda")
    used = torch.arange(width, device="cuda") < torch.tensor(need, device="cuda")[:, None]
    st = dict(case=case, T=T, max_len=max(ls), q_scale=Q_SCALE if case["q_fp8"] else 1.0,
              tables=torch.where(used, order[at.clamp(max=pool - 1)], torch.full_like(order[:1], -1)).contiguous(),
              seq_lens=torch.tensor(ls, dtype=torch.int32, device="cuda"),
              indptr=torch.tensor(np.cumsum([0] + qs), dtype=torch.int32, device="cuda"),
              cache=_make_cache(g, case["kv"], pool, ps))
    if case["op"] == "append":
        # what the layer's projections leave: one tensor for latent and key part, the
        # query's latent part by head (a batched product's output), its RoPE part by token
        kv = torch.randn(T, QK, generator=g, device="cuda") * 1.7
        st.update(kv=kv.to(torch.bfloat16),
                  weight=(1 + 0.2 * torch.randn(LAT, generator=g, device="cuda")).to(torch.bfloat16),
                  q_nope=torch.randn(H, T, LAT, generator=g, device="cuda", dtype=torch.bfloat16).transpose(0, 1),
                  q_pe=torch.randn(T, H, 128 + ROPE, generator=g, device="cuda", dtype=torch.bfloat16)[..., 128:],
                  query=torch.empty(T, H, QK, device="cuda", dtype=torch.float8_e4m3fn if case["q_fp8"] else torch.bfloat16),
                  rows=torch.empty(T, QK, device="cuda", dtype=torch.bfloat16), table=_rope_table())
        return st
    x = torch.randn(T, H, QK, generator=g, device="cuda", dtype=torch.bfloat16)
    if case["q_fp8"]:
        x = (x.float() * (1.0 / Q_SCALE)).clamp_(-448, 448).to(torch.float8_e4m3fn)
    if not case["packed"]:
        x = x.view(B, case["q"], H, QK)
    st.update(query=x, bmm1=BMM1 * _scale(case) * st["q_scale"], bmm2=_scale(case),
              workspace=torch.empty((64 << 20) + 1280 * T * H, dtype=torch.uint8, device="cuda"),
              out=torch.empty(*x.shape[:-1], LAT, dtype=torch.bfloat16, device="cuda"),
              lse=torch.empty(T, H, dtype=torch.float32, device="cuda"))
    return st


def _rope_table():
    """fp32 [positions, 64]: cosines, then sines, of a base-10000 rotation stretched
    for long contexts (low frequencies divided by 40, high ones kept, a ramp between)."""
    i = torch.arange(32, dtype=torch.float64, device="cuda")
    freq = 10000.0 ** (-i / 32)
    low, high = (32 * math.log(4096 / (r * 2 * math.pi)) / math.log(10000.0) for r in (32.0, 1.0))
    ramp = ((i - math.floor(low)) / (math.ceil(high) - math.floor(low))).clamp(0, 1)
    freq = freq / 40 * ramp + freq * (1 - ramp)
    a = torch.arange(MAX_POSITION, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1).float()


# ------------------------------------------------------------------ plain forms

def _tokens(st):
    """(request, index in the request, query length) of every token."""
    t = torch.arange(st["T"], device="cuda")
    b = torch.searchsorted(st["indptr"], t.int(), right=True) - 1
    return b, t - st["indptr"][b], (st["indptr"][1:] - st["indptr"][:-1])[b]


def _rotate(x, cos, sin, style):
    if style == "interleaved":
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    a, b = x[..., :32], x[..., 32:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _rows(case, cache, page, row):
    """fp32 values of the cache rows (page, row): index tensors of one shape."""
    if case["kv"] != "fp4":
        return cache[page, row].float()
    codes, scales = _fp4_parts(cache)
    mag = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda")
    one = torch.cat([mag, -mag])
    pair = torch.stack([one.repeat(16), one.repeat_interleave(16)], -1)  # by byte: low nibble, high nibble
    v = pair[codes[page, row].int()].flatten(-2).unflatten(-1, (QK // GROUP, GROUP))
    return (v * scales[page, row].view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)


def _plain_append(st):
    case, cache = st["case"], st["cache"]
    b, i, q = _tokens(st)
    pos = (st["seq_lens"][b] - q + i).long()
    page, row = st["tables"][b, pos // case["page"]].long(), pos % case["page"]
    x = st["kv"][:, :LAT].float()
    # the sum in 64 bits: a value next to a rounding border of 4 bits shows its last bit
    mean = (x.double().square().sum(-1, keepdim=True)).float() * (1.0 / LAT)
    rstd = (mean + EPS).double().rsqrt().float()
    lat = x * rstd * st["weight"].float()
    cos, sin = st["table"][pos, :32], st["table"][pos, 32:]
    y = torch.cat([lat, _rotate(st["kv"][:, LAT:].float(), cos, sin, case["style"])], -1)
    if case["kv"] == "fp4":
        codes, scales = _fp4_parts(cache)
        c, s = _fp4_quantise(y)
        codes[page, row] = c
        scales[page, row] = s.view(torch.uint8)
    elif case["kv"] == "e4m3":
        cache.view(torch.uint8)[page, row] = (y * (1.0 / KV_SCALE)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        cache[page, row] = y.to(torch.bfloat16)
    qr = _rotate(st["q_pe"].float(), cos[:, None], sin[:, None], case["style"])
    qq = torch.cat([st["q_nope"].float(), qr], -1)
    if case["q_fp8"]:
        st["query"].copy_((qq * (1.0 / Q_SCALE)).clamp(-448, 448))
    else:
        st["query"].copy_(qq)
    if case["kv"] == "bf16":
        return {"cache": cache, "query": st["query"]}
    st["rows"].copy_(_rows(case, cache, page, row) * _scale(case))
    return {"rows": st["rows"], "query": st["query"]}


def _plain_attention(st):
    case = st["case"]
    B, H, qm, ps = case["batch"], case["heads"], case["q"], case["page"]
    W, S = case.get("window", 0), case.get("sinks", 0)
    L = st["seq_lens"].long()[:, None]
    ql = (st["indptr"][1:] - st["indptr"][:-1]).long()[:, None]
    i = torch.arange(qm, device="cuda")
    last = L - ql + i if case["causal"] else (L - 1).expand(B, qm)  # [B, q]
    # the positions that some row may see: the first ones, then the window's
    if W and S + W + qm - 1 < st["max_len"]:
        lo = (last[:, :1] - W + 1).clamp(min=S)
        j = torch.cat([torch.arange(S, device="cuda").expand(B, S), lo + torch.arange(W + qm - 1, device="cuda")], 1)
    else:
        j = torch.arange(st["max_len"], device="cuda").expand(B, -1)
    inside = j < L
    jc = torch.where(inside, j, torch.zeros_like(j))
    page = st["tables"].gather(1, jc // ps).long()
    keys = _rows(case, st["cache"], page, jc % ps)  # [B, N, 576]
    see = (j[:, None] <= last[..., None]) & inside[:, None]
    if W:
        see = see & ((j[:, None] > last[..., None] - W) | (j[:, None] < S))
    t = (st["indptr"][:-1].long()[:, None] + i).clamp(max=st["T"] - 1)
    x = st["query"].reshape(st["T"], H, QK)
    x = x.view(torch.uint8)[t].view(torch.float8_e4m3fn).float() if case["q_fp8"] else x[t].float()
    s = torch.matmul(x.reshape(B, qm * H, QK), keys.transpose(1, 2)) * st["bmm1"]
    s = s.view(B, qm, H, -1).masked_fill_(~see[:, :, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-3e38)
    p = (s - m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, qm * H, -1), keys[..., :LAT]).view(B, qm, H, LAT) / l * st["bmm2"]
    b, k, _ = _tokens(st)
    st["out"].view(st["T"], H, LAT).copy_(o[b, k])
    st["lse"].copy_((m + l.log())[b, k, :, 0])
    return {"out": st["out"], "lse": st["lse"]}


# ------------------------------------------------------------------ the library's calls

def _own_append(st):
    import paged_mla_decode_03_gb300 as mla
    case = st["case"]
    which = dict(qo_indptr=st["indptr"]) if case["packed"] else dict(q_len=case["q"])
    mla.cache_append(st["kv"][:, :LAT], st["kv"][:, LAT:], st["cache"], st["tables"], st["seq_lens"],
                     rope_table=st["table"], norm_weight=st["weight"], eps=EPS, rope_style=case["style"],
                     kv_scale=_scale(case), q_nope=st["q_nope"], q_pe=st["q_pe"], query=st["query"],
                     q_scale=st["q_scale"], **which)
    if case["kv"] == "bf16":
        return {"cache": st["cache"], "query": st["query"]}
    mla.cache_gather(st["cache"], st["tables"], st["seq_lens"], total_q=st["T"], kv_scale=_scale(case),
                     out=st["rows"], **which)
    return {"rows": st["rows"], "query": st["query"]}


def _own_attention(st):
    import paged_mla_decode_03_gb300 as mla
    case = st["case"]
    which = dict(qo_indptr=st["indptr"], max_seq_len_q=case["q"]) if case["packed"] else {}
    if case["op"] == "window":
        which.update(window=case["window"], sinks=case["sinks"])
    mla.decode(st["query"], st["cache"], st["workspace"], st["tables"], st["seq_lens"], st["max_len"],
               out=st["out"], lse=st["lse"], bmm1_scale=st["bmm1"], bmm2_scale=st["bmm2"],
               mask_type="causal" if case["causal"] else "dense", return_lse=True, **which)
    return {"out": st["out"], "lse": st["lse"]}


def run(state):
    if state["case"]["op"] == "append":
        return _own_append(state) if own else _plain_append(state)
    return _own_attention(state) if own else _plain_attention(state)


# ------------------------------------------------------------------ 64 bits

def _e2m1_nearest(t):
    """Nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 by magnitude, a tie to the even code."""
    v = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=t.device)
    a = t.abs().clamp(max=6.0)
    hi = torch.searchsorted(v, a).clamp(min=1)
    below, above = a - v[hi - 1], v[hi] - a
    k = torch.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, hi - 1)
    return v[k] * torch.sign(t)


def _exact_append(st):
    case = st["case"]
    x = st["kv"].double()
    rows, cos, sin, where = [], [], [], []
    ls, qs = _lengths(case)
    for b, (L, q) in enumerate(zip(ls, qs)):
        for i in range(q):
            where.append((b, L - q + i))
    pos = torch.tensor([p for _, p in where], device="cuda")
    req = torch.tensor([b for b, _ in where], device="cuda")
    c, s = st["table"].double()[pos].split(32, -1)
    lat = x[:, :LAT] / torch.sqrt((x[:, :LAT] ** 2).mean(-1, keepdim=True) + EPS) * st["weight"].double()

    def turn(v, c, s):  # as products of complex numbers
        a, b = (v[..., 0::2], v[..., 1::2]) if case["style"] == "interleaved" else v.split(32, -1)
        z = torch.complex(a, b) * torch.complex(c, s)
        return torch.view_as_real(z).flatten(-2) if case["style"] == "interleaved" else torch.cat([z.real, z.imag], -1)

    y = torch.cat([lat, turn(x[:, LAT:], c, s)], -1)
    qq = torch.cat([st["q_nope"].double(), turn(st["q_pe"].double(), c[:, None].expand(-1, case["heads"], -1),
                                                s[:, None].expand(-1, case["heads"], -1))], -1)
    if case["q_fp8"]:
        qq = (qq / Q_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).double()
    if case["kv"] == "bf16":
        cache = st["cache"].double()
        cache[st["tables"].long()[req, pos // case["page"]], pos % case["page"]] = y
        return {"cache": cache, "query": qq}
    if case["kv"] == "e4m3":
        return {"rows": (y / KV_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).double() * KV_SCALE, "query": qq}
    g = y.view(-1, QK // GROUP, GROUP)
    sc = (g.abs().amax(-1, keepdim=True) / 6).to(torch.float8_e4m3fn).double()
    v = torch.where(sc > 0, _e2m1_nearest(g / sc.clamp(min=2.0 ** -10)), torch.zeros_like(g)) * sc
    return {"rows": v.flatten(-2), "query": qq}


def _exact_attention(st):
    case, ps = st["case"], st["case"]["page"]
    W, S, H = case.get("window", 0), case.get("sinks", 0), case["heads"]
    outs, lses, t0 = [], [], 0
    x = st["query"].reshape(st["T"], H, QK).double()
    for b, (L, q) in enumerate(zip(*_lengths(case))):
        pages = st["tables"][b, : -(-L // ps)].long()
        if case["kv"] == "fp4":
            raw = st["cache"].view(-1, ps * FP4_ROW)[pages]
            by = raw[:, : ps * 288].reshape(-1, 288)[:L].to(torch.int16)
            codes = torch.stack([by & 15, by >> 4], -1).flatten(-2)
            mag = (codes & 7).double()
            e, m = torch.div(mag, 2, rounding_mode="floor"), mag % 2
            val = torch.where(e > 0, (1 + m / 2) * torch.exp2(e - 1), m / 2) * torch.where(codes > 7, -1.0, 1.0)
            sc = raw[:, ps * 288 :].reshape(-1, 36)[:L].contiguous().view(torch.float8_e4m3fn).double()
            keys = (val.view(L, 36, GROUP) * sc[..., None]).view(L, QK)
        else:
            keys = st["cache"][pages].reshape(-1, QK)[:L].double()
        j = torch.arange(L, device="cuda")
        for i in range(q):
            last = L - q + i if case["causal"] else L - 1
            ok = j <= last
            if W:
                ok &= (last - j < W) | (j < S)
            kk = keys[ok]
            s = x[t0 + i] @ kk.T * st["bmm1"]
            lse = torch.logsumexp(s, -1)
            outs.append(torch.exp(s - lse[:, None]) @ kk[:, :LAT] * st["bmm2"])
            lses.append(lse)
        t0 += q
    return {"out": torch.stack(outs).view(st["out"].shape), "lse": torch.stack(lses)}


def exact(case, seed):
    if work(case)["flops"] > 6e11:
        return None
    st = prepare(case, seed)
    return _exact_append(st) if case["op"] == "append" else _exact_attention(st)
