"""How near decodes over a 4-bit cache and with a window come to 64 bits, where rows are
split and where they are not (tests/attention_ref.py).

Rounding the exact output to bf16 leaves an error of r (2-norm).  Over V of zero mean the
rounding of P adds its own relative error of P: f16, at most 2^-11 / sqrt(3) in the mean
square = 0.00028 against r / |O| of about 0.0016, together 1.02 r; bf16, like the output's
own rounding, together sqrt(2) r.  Partials rounded to bf16 would add r once more: sqrt(2) r and
sqrt(3) r.  The bounds lie between: 1.1 r and 1.5 r."""
import pytest
import torch

from attention_ref import Case

SPLIT = [(64, [20000], [1], 128), (32, [9000, 7000], [2, 2], 64), (64, [5000, 100, 3000], [3, 1, 2], 128)]
WHOLE = [(64, [500] * 70, [1] * 70, 128), (32, [100, 64], [2, 2], 64)]
BOUND = {"fp4": 1.1, "e4m3": 1.1, "bf16": 1.5}
ALL = 1 << 20  # a window over everything: e4m3 and bf16 caches on the MMAs across CTA pairs


def _case(kind, ps, ls, qs, heads, **kw):
    return Case(kind, ps, ls, qs, heads, packed=len(set(qs)) > 1, window=0 if kind == "fp4" else ALL, **kw)


def _splits(c):
    torch.cuda.synchronize()
    return int(c.workspace[12:16].view(torch.int32).item())  # header word: combine entries


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp4", "e4m3", "bf16"])
@pytest.mark.parametrize("split,shape", [(True, s) for s in SPLIT] + [(False, s) for s in WHOLE])
def test_error_of_all_outputs(kind, split, shape):
    c = _case(kind, *shape, seed=31).run()
    assert (_splits(c) > 0) == split
    want = torch.stack([o for _, o, _, _ in c.reference()])
    rounding = (want.to(torch.bfloat16).double() - want).norm()
    err = (c.out[:c.T].double() - want).norm()
    assert float(err / rounding) <= BOUND[kind], f"{float(err / want.norm()):.5f} of the norm, {float(err / rounding):.3f} r"


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp4", "e4m3", "bf16"])
@pytest.mark.parametrize("shape", SPLIT + WHOLE)
def test_equal_rows_of_v_come_back_exactly(kind, shape):
    """Every V row is the same row v, so O is v whatever P is: the sum that divides is that
    of P as it entered (off by 2^-11 of it in f16, below the 2^-9 of half an output step)."""
    c = _case(kind, *shape, seed=32, bmm1=0.5, bmm2=1.0)
    g = torch.Generator().manual_seed(33)
    code = torch.randint(0, 16, (512,), generator=g, dtype=torch.uint8)
    v = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6])[(code & 7).long()] * torch.where(code > 7, -1.0, 1.0)
    if kind == "fp4":
        flat = c.cache.view(c.cache.shape[0], -1)
        ps = c.cache.shape[1]
        codes, scales = flat[:, :ps * 288].view(-1, ps, 288), flat[:, ps * 288:].view(-1, ps, 36)
        codes[..., :256] = (code[0::2] | (code[1::2] << 4)).cuda()
        scales[..., :32] = 0x38  # 1
    else:
        c.cache[..., :512] = v.to(c.cache.dtype).cuda()
    c.run()
    assert c.status() == 0
    assert (c.out == v.to(torch.bfloat16).cuda()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp4", "e4m3", "bf16"])
@pytest.mark.parametrize("largest", [True, False])
@pytest.mark.parametrize("shape", SPLIT[:2])
def test_split_rows_at_the_ends_of_the_range(kind, largest, shape):
    """The largest and the smallest values that a cache holds pass through the partials.  (bf16:
    the sum of P V is divided at its end, and P is at most 2^8, so 20000 rows of 2^105
    would pass fp32's range.)"""
    c = _case(kind, *shape, seed=34, bmm1=0.5, bmm2=1.0)
    c.query[..., :512] = 0  # scores from the RoPE dims alone
    sign = torch.where(torch.arange(512) % 3 == 0, -1.0, 1.0)
    if kind == "fp4":
        v = sign * (6 * 448.0 if largest else 0.5 * 2.0 ** -9)
        flat = c.cache.view(c.cache.shape[0], -1)
        ps = c.cache.shape[1]
        code = ((7 if largest else 1) + 8 * (sign < 0)).to(torch.uint8)
        flat[:, :ps * 288].view(-1, ps, 288)[..., :256] = (code[0::2] | (code[1::2] << 4)).cuda()
        flat[:, ps * 288:].view(-1, ps, 36)[..., :32] = 0x7E if largest else 0x01
    else:
        v = sign * ({"e4m3": 448.0, "bf16": 2.0 ** 100}[kind] if largest else {"e4m3": 2.0 ** -9, "bf16": 2.0 ** -120}[kind])
        c.cache[..., :512] = v.to(c.cache.dtype).cuda()
    c.run()
    assert c.status() == 0 and _splits(c) > 0
    assert (c.out == v.to(torch.bfloat16).cuda()).all()
