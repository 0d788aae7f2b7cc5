"""How exactly the cache attention weighs V: against the 64-bit oracle, channel by channel.

P is multiplied by the power of two of the key's V row before it is rounded. With c the E4M3 values of V's codes and E
their powers of two, |v| = |c| E,
  P's rounding     more than 32 query rows a KV head: fp16, half a step of 2^-11 of the value; where fp16 is subnormal
                   2^-25, beside 2^10 or more for the row's largest p E: 2^-35 max(p E).
                   Up to 32: fp16, 2^-11, then three E5M2 terms, of which the second and third hold 2^3 and 2^7 of
                   what is left: 2^-3 each, 2^-9, while the first is normal (p E above 2^-14, 2^-24 max(p E)); below,
                   it leaves 2^-17 at most, the second 2^-20, the third 2^-23: 2^-33 max(p E)
  scores           eps, as in test_cache_attention_gpu: twice (numerator and sum)
  accumulation     fp32, 16 keys a step: 2^-23 of the magnitudes a step, L / 16 steps and some of joining
  the result       bf16, 2^-8
so |out - ref| <= 2^-8 |ref| + (P + 2 eps + 2^-23 (L / 16 + 64)) sum p|v| / l + F max(p E) sum |c| / l,
P 2^-11 and F 2^-35, or P 2^-9 + 2^-11 and F 2^-33.
"""
import numpy as np
import pytest
import torch

import precision_attention_nvfp4_b200 as fp
from oracle import codec, serving
from test_cache_attention_gpu import _q, make

pytestmark = pytest.mark.gpu

KERNELS = [(1, 1), (1, 8), (4, 8), (40, 2)]        # queries and group: tiles of 16, 16, 32 and 128 query rows


def held(cache, table, b, n):
    """K [H, n, d], the values of V's codes [H, n, d] and their powers of two [H, n], of the first n tokens."""
    i = torch.arange(n, device="cuda")
    p, o = table[b, i // cache.page_size].long(), i % cache.page_size
    e = cache.exps[p, :, :, o].cpu().numpy()
    k = serving.dequantize_rows(cache.k_codes[p, :, o].cpu().numpy(), e[:, :, 0])
    c = codec.e4m3_decode(cache.v_codes[p, :, o].cpu().numpy())
    return k.swapaxes(0, 1), c.swapaxes(0, 1), np.exp2(e[:, :, 1].astype(np.float64) - 127).T


def check(out, q, cache, table, lens, mode, heads=None):
    """Returns the largest error in units of the bound."""
    worst = 0.0
    for b, n in enumerate(lens):
        k, c, E = held(cache, table, b, n)
        qd = q[b].double().cpu().numpy()
        got = out[b].double().cpu().numpy()
        t, hq, d = qd.shape
        sc, group = d ** -0.5, hq // cache.num_heads
        see = serving.visible(n, t, mode)
        for h in heads or range(hq):
            g = h // group
            s = sc * qd[:, h] @ k[g].T
            s[~see] = -np.inf
            p = np.exp(s - s.max(1, keepdims=True))
            l = p.sum(1)[:, None]
            v = c[g] * E[g][:, None]
            ref, spread = p @ v / l, p @ np.abs(v) / l
            size = (sc * (np.abs(qd[:, h]) @ np.abs(k[g]).T) * see).max(1)
            eps = (sc * 2.0 ** -18 * np.abs(qd[:, h]).max(1) * np.abs(k[g]).sum(1).max() + 2.0 ** -17 * size +
                   2.0 ** -21 + 2.0 ** -23 * np.abs(np.where(see, s, 0)).max(1))[:, None]
            wide = t * group > 32
            floor = 2.0 ** (-35 if wide else -33) * (p * E[g]).max(1)[:, None] * (see.astype(float) @ np.abs(c[g])) / l
            tol = 2.0 ** -8 * np.abs(ref) + ((0 if wide else 2.0 ** -9) + 2.0 ** -11 + 2 * eps + 2.0 ** -23 * (n / 16 + 64)) * spread + floor
            worst = max(worst, float((np.abs(got[:, h] - ref) / np.maximum(tol, 1e-300)).max()))
    return worst


def write(cache, table, b, n, k, v):
    i = torch.arange(n, device="cuda")
    slots = table[b, i // cache.page_size].long() * cache.page_size + i % cache.page_size
    fp.cache_write(cache, k.to(torch.bfloat16).contiguous(), v.to(torch.bfloat16).contiguous(), slots)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,group", KERNELS)
@pytest.mark.parametrize("gap", [8, 12, 14, 17, 20])
def test_small_value_rows_beside_one_strong_channel(d, T, group, gap):
    """Like scores, one row of V with a single large channel, the others 2^-gap of it: in every other channel the
    result is made of small rows alone."""
    B, n = 24, 7
    cache, table, _ = make([n] * B, 1, d, 16, gap + T)
    g = torch.Generator(device="cuda").manual_seed(gap)
    for b in range(B):
        k = torch.randn(n, 1, d, device="cuda", generator=g)
        v = torch.randn(n, 1, d, device="cuda", generator=g) * 2.0 ** -gap
        v[b % n] = 0
        v[b % n, 0, b % d] = 3.0
        write(cache, table, b, n, k, v)
    lengths = torch.full((B,), n, dtype=torch.int32, device="cuda")
    q = _q(gap, B, T, group, d)
    out, _ = fp.cache_attention(q, cache, table, lengths, causal=False)
    assert fp.device_error() == 0
    assert check(out, q, cache, table, [n] * B, "full") <= 1


@pytest.mark.parametrize("d,n", [(64, 40000), (128, 9000)])
@pytest.mark.parametrize("T,group", KERNELS)
@pytest.mark.parametrize("far", [11.0, 15.3, 20.0])
def test_long_flat_tail_behind_a_dominant_key(d, n, T, group, far):
    """One key e^far above all others, whose V is zero in half of the channels: there the tail is all there is."""
    cache, table, lengths = make([n], 1, d, 64, 5)
    g = torch.Generator(device="cuda").manual_seed(6)
    base = torch.randn(d, device="cuda", generator=g).to(torch.bfloat16).float()
    k = torch.zeros(n, 1, d, device="cuda")
    k[777, 0] = base * (far * d ** 0.5 / base.square().sum())
    v = 1 + 0.25 * torch.randn(n, 1, d, device="cuda", generator=g)
    v[777, 0, d // 2:] = 0
    write(cache, table, 0, n, k, v)
    q = (base * (1 + 0.02 * torch.randn(1, T, group, 1, device="cuda", generator=g))).to(torch.bfloat16)
    out, _ = fp.cache_attention(q, cache, table, lengths, causal=False)
    assert fp.device_error() == 0
    assert check(out, q, cache, table, [n], "full") <= 1


@pytest.mark.parametrize("d,page", [(64, 32), (128, 16)])
@pytest.mark.parametrize("T,group", KERNELS)
def test_ordinary_rows(d, page, T, group):
    lens = [max(T, 3), 129, 1500]
    cache, table, lengths = make(lens, 2, d, page, 3 * T + d)
    q = _q(T, len(lens), T, 2 * group, d)
    out, _ = fp.cache_attention(q, cache, table, lengths)
    assert fp.device_error() == 0
    assert check(out, q, cache, table, lens, "causal") <= 1
