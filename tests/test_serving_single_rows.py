"""The stride of an axis of one element is never taken: it may be anything (one token out of a wider, odd buffer)."""
import ctypes

import pytest
import torch

import precision_attention_nvfp4_b200 as fp
from precision_attention_nvfp4_b200 import _lib

PTR = 1 << 20


def test_checks_skip_strides_that_are_not_taken():
    from precision_attention_nvfp4_b200 import build
    build.build()

    def run(**kw):
        f = dict(B=1, T=4, H=2, d=64, sb=0, st=128, sh=64)
        f.update(kw)
        r = _lib.Rows(PTR, *f.values())
        t = _lib.RotaryTable(PTR, 64, 0, 1.0)
        # (without positions: refused in any case, after the rows)
        return fp.library().fpattn_rotary(ctypes.byref(r), ctypes.byref(t), None, 0, 0, ctypes.byref(r), None)

    ok, ali = _lib.ERR_INVALID_ARG, _lib.ERR_ALIGNMENT
    assert run() == run(sb=3) == run(T=1, st=131) == run(H=1, sh=65) == run(T=1, H=1, st=1, sh=1) == ok
    assert run(st=131) == run(sh=65) == run(B=2, sb=3) == run(T=1, st=131, sh=65) == run(H=1, st=131, sh=65) == ali


@pytest.mark.gpu
def test_one_token_of_an_odd_buffer():
    d, T = 64, 1
    buf = torch.randn(1, 8 * d + 3, device="cuda").to(torch.bfloat16)
    x = buf.as_strided((T, 8, d), (8 * d + 3, d, 1))
    assert x.stride(0) % 8
    rot, pos, slot = fp.rotary_table(d), torch.tensor([77], device="cuda"), torch.tensor([5], device="cuda")
    c = x.clone(memory_format=torch.contiguous_format)
    assert torch.equal(fp.rotary(x, pos, rot), fp.rotary(c, pos, rot))
    caches = [fp.kv_cache(1, 2, 16, d) for _ in range(2)]
    for cache, t in zip(caches, (x, c)):
        q = fp.cache_write(cache, t[:, 4:6], t[:, 6:], slot, rotary=rot, positions=pos, q=t[:, :4])
    assert torch.equal(q, fp.rotary(c[:, :4], pos, rot)) and torch.equal(caches[0].k_codes, caches[1].k_codes)
    table, lengths = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.tensor([6], dtype=torch.int32, device="cuda")
    got = fp.cache_attention(x[:, :4].unsqueeze(0), caches[0], table, lengths)
    want = fp.cache_attention(c[:, :4].unsqueeze(0), caches[0], table, lengths)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out = torch.empty(4 * d, dtype=torch.bfloat16, device="cuda").as_strided((1, 4, d), (4 * d + 5, d, 1))
    fp.cache_read(caches[0], slot, out=(out[:, :2], out[:, 2:]))
    k, v = fp.cache_read(caches[0], slot)
    assert torch.equal(out, torch.cat([k, v], 1))
