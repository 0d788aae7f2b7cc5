"""Scores far from zero (still within fp32) weigh as any others: the softmax knows differences alone. Where a step of fp32
is as large as the range of P (2^27 and more) nothing overflows; below -1e30 a score is still a score.

All keys of a sequence are one row k = -a (1, ..., 1), or a, and all queries a (1, ..., 1) with a a power of two, so that
every score is -d a^2 scale exactly, P is 1 for every key seen, and the result their mean of V: bf16's 2^-8, and the 2^-9
and 2^-11 of P and 2^-22 of exp2 and the sums, below 2^-8, of mean |v|. lse: fp32, 2^-23 for the score and its log2 each.

With more than 32 query rows a KV head the exponent of V's scale is added to the score t (in log2) before the reference:
one rounding of 2^-24 |t| a key, one more for the reference of each half of the keys and of each block that are joined,
below u = 2^-22 |t| in all. So every weight is within 2^-u .. 2^u of the others' common factor, a normalised one within
2^-2u .. 2^2u: (2^2u - 1) mean |v| more; and the result is a mean of V rows with weights above zero whatever u, so never
further from the plain mean than the furthest V row.
"""
import math

import pytest
import torch

import precision_attention_nvfp4_b200 as fp
from test_cache_attention_gpu import held, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("log_a", [8, 10, 11, 12, 13, 14, 20, 40, 50, 60])
@pytest.mark.parametrize("T,group", [(1, 4), (4, 8), (40, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_far_scores(sign, log_a, T, group, d):
    lens = [max(T, 40), 700, 20000]                     # within half a tile; a few tiles; split over many blocks
    cache, table, lengths = make(lens, 1, d, 64, 3, spread=0.3)
    slots = torch.cat([(table[b, :(n + 63) // 64].long()[:, None] * 64 + torch.arange(64, device="cuda")).flatten()[:n]
                       for b, n in enumerate(lens)])
    k = torch.full((len(slots), 1, d), sign * 2.0 ** log_a, dtype=torch.bfloat16, device="cuda")
    v = torch.randn(len(slots), 1, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    fp.cache_write(cache, k, v.to(torch.bfloat16), slots)
    q = torch.full((3, T, group, d), 2.0 ** log_a, dtype=torch.bfloat16, device="cuda")
    out, lse = fp.cache_attention(q, cache, table, lengths, causal=False)
    assert fp.device_error() == 0
    score = sign * d * 2.0 ** (2 * log_a) / math.sqrt(d)
    for b, n in enumerate(lens):
        _, vh = held(cache, table, b, n)
        want, size = torch.from_numpy(vh[0].mean(0)), torch.from_numpy(abs(vh[0]).mean(0))
        err = (out[b].double().cpu() - want).abs()
        tol = 2.0 ** -8 * want.abs() + 2.0 ** -8 * size
        if T * group > 32:
            u = 2.0 ** -22 * abs(score) / math.log(2)
            far = torch.from_numpy(abs(vh[0] - vh[0].mean(0)).max(0))
            tol = tol + torch.minimum((2.0 ** min(2 * u, 100.0) - 1) * size, far * (1 + 2.0 ** -8))
        assert (err <= tol).all()
        assert ((lse[b].double().cpu() - (score + math.log(n))).abs() <= 2.0 ** -21 * abs(score)).all()
