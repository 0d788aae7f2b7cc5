"""Rotated K is stored at the exponent and the codes that are nearest to the exactly rotated values, every one of them:
where terms cancel, where E4M3 is subnormal, and where a row's largest value lies beside 448 times a power of two.

The reference rotates in 64 bits, the angle from the table's 64-bit fractions, and rounds to E4M3's grid in 64 bits. Its
own error, 2^-52 of a pair's values and angle, decides nothing: some 1e-13 of a step of the grid.
"""
import math

import pytest
import torch

import precision_attention_nvfp4_b200 as fp

pytestmark = pytest.mark.gpu


def turned(k, pos, table):
    """k [T, H, d] rotated in 64 bits."""
    turns = pos[:, None] * table.turns                        # wrapping: whole turns are gone
    a = turns.double() * (2 * math.pi / 2.0 ** 64)
    c, s = table.magnitude * a.cos()[:, None], table.magnitude * a.sin()[:, None]
    y, n = k.double(), table.dim // 2
    if table.layout == "half":
        i, j = slice(0, n), slice(n, 2 * n)
    else:
        i, j = slice(0, 2 * n, 2), slice(1, 2 * n, 2)
    p, q = y[..., i].clone(), y[..., j].clone()
    y[..., i], y[..., j] = p * c - q * s, p * s + q * c
    return y


def nearest(y):
    """(values of the codes, exponents) of rows y."""
    a = y.abs().amax(-1)
    m, e = torch.frexp(a)                                     # a = m 2^e, m in [0.5, 1): a <= 448 2^(e - 9) from m <= 0.875
    e = torch.where(a == 0, torch.full_like(e, -63), (e - 9 + (m > 0.875)).clamp(min=-63))
    v = torch.ldexp(y, -e[..., None])
    step = torch.ldexp(torch.ones_like(v), (torch.frexp(v)[1] - 1).clamp(min=-6) - 3)      # (exp2 is not exact)
    return torch.round(v / step) * step, e


def stored(cache, T):
    codes = cache.k_codes.transpose(1, 2).reshape(T, cache.num_heads, cache.head_dim)
    exps = cache.exps[:, :, 0].transpose(1, 2).reshape(T, cache.num_heads)
    return codes.view(torch.float8_e4m3fn).double(), exps.int() - 127


def check(k, pos, table):
    T, H, d = k.shape
    cache = fp.kv_cache(T // 16, H, 16, d)
    fp.cache_write(cache, k, k, torch.arange(T, device="cuda"), rotary=table, positions=pos)
    got, e = stored(cache, T)
    want, we = nearest(turned(k, pos, table))
    assert torch.equal(e, we.int())
    assert int((got != want).sum()) == 0


@pytest.mark.parametrize("d,dim,layout", [(128, 128, "half"), (128, 64, "interleaved"), (64, 64, "interleaved"), (64, 48, "half")])
@pytest.mark.parametrize("large", [0, 14])
@pytest.mark.parametrize("scaling", ["none", "yarn"])
def test_codes_are_the_nearest(d, dim, layout, large, scaling):
    """`large`: a channel 2^large of the others, whose codes are then few bits or subnormal."""
    T, H = 32768, 128 // d
    table = fp.rotary_table(dim, layout=layout, scaling=scaling, factor=8.0)
    for seed in range(6):
        g = torch.Generator(device="cuda").manual_seed(seed)
        k = torch.randn(T, H, d, device="cuda", generator=g)
        k[..., 7 + seed] *= 2.0 ** large
        pos = torch.randint(0, 1 << 20, (T,), device="cuda", generator=g)
        check(k.to(torch.bfloat16), pos, table)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_exponents_beside_a_border(layout):
    """Rows of one pair, picked for a largest value within 2^-22 of 448 times a power of two, on either side."""
    d = 64
    table = fp.rotary_table(d, layout=layout)
    g = torch.Generator(device="cuda").manual_seed(5)
    n = 1 << 25
    pick = []
    for pair in range(0, 32, 2):
        i, j = (pair, pair + d // 2) if layout == "half" else (2 * pair, 2 * pair + 1)
        xy = torch.randn(n, 2, device="cuda", generator=g).to(torch.bfloat16)
        pos = torch.randint(0, 1 << 20, (n,), device="cuda", generator=g)
        a = (pos * table.turns[pair]).double() * (2 * math.pi / 2.0 ** 64)
        x, y = xy[:, 0].double(), xy[:, 1].double()
        m = torch.frexp(torch.maximum((x * a.cos() - y * a.sin()).abs(), (x * a.sin() + y * a.cos()).abs()))[0]
        at = ((m / 0.875 - 1).abs() < 2.0 ** -22).nonzero().flatten()
        k = torch.zeros(len(at), 1, d, dtype=torch.bfloat16, device="cuda")
        k[:, 0, i], k[:, 0, j] = xy[at, 0], xy[at, 1]
        pick.append((k, pos[at]))
    k, pos = (torch.cat(t) for t in zip(*pick))
    T = len(pos) // 16 * 16
    assert T >= 64
    check(k[:T].contiguous(), pos[:T].contiguous(), table)
