"""Outputs that share memory with what a call reads or writes elsewhere are refused; heads that lie between one another's
in one projection are not."""
import pytest
import torch

import precision_attention_nvfp4_b200 as fp
from test_cache_attention_gpu import _q, make

pytestmark = pytest.mark.gpu


def test_cache_write_refuses_queries_over_its_keys():
    T, d = 20, 64
    cache, rot = fp.kv_cache(2, 2, 16, d), fp.rotary_table(d)
    slots, pos = torch.arange(T, device="cuda"), torch.arange(T, device="cuda")
    x = _q(0, T, 14, d)
    q, k, v = x[:, :10], x[:, 10:12], x[:, 12:14]
    for kv in ((x[:, 8:10], v), (k, x[:, :2]), (x[:, 9:11], v), (k, x[:, 4:6])):
        with pytest.raises(ValueError):
            fp.cache_write(cache, *kv, slots, rotary=rot, positions=pos, q=q, q_out=q)
    with pytest.raises(ValueError):
        fp.cache_write(cache, k, v, slots, rotary=rot, positions=pos, q=q, q_out=x[:, 1:11])
    with pytest.raises(ValueError):
        fp.cache_write(cache, k, v, slots, rotary=rot, positions=pos, q=q[:, :4], q_out=x[:, 8:12])
    assert torch.equal(x, _q(0, T, 14, d))
    want = fp.cache_write(cache, k, v, slots, rotary=rot, positions=pos, q=q)
    codes = cache.k_codes.clone()
    got = fp.cache_write(cache, k, v, slots, rotary=rot, positions=pos, q=q, q_out=q)     # in place, k and v beside it
    assert got is q and torch.equal(q, want) and torch.equal(cache.k_codes, codes)
    y = _q(1, T, 4, d)
    other = fp.cache_write(cache, k, v, slots, rotary=rot, positions=pos, q=y[:, 0::2], q_out=y[:, 1::2])
    assert torch.equal(other, fp.rotary(_q(1, T, 4, d)[:, 0::2], pos, rot)) and torch.equal(y[:, 0::2], _q(1, T, 4, d)[:, 0::2])


def test_cache_read_refuses_outputs_over_one_another():
    cache, slots = fp.kv_cache(2, 2, 16, 64), torch.arange(20, device="cuda")
    x = torch.full((21, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    for out in ((x[:20, :2], x[:20, :2]), (x[:20, :2], x[:20, 1:3]), (x[:20, :2], x[1:, :2]), (x[:20, :2], x.view(-1)[:2560].view(20, 2, 64))):
        with pytest.raises(ValueError):
            fp.cache_read(cache, slots, out=out)
    assert (x == 7).all()
    fp.cache_read(cache, slots, out=(x[:20, :2], x[:20, 2:]))
    assert not x[:20].any() and (x[20] == 7).all()


def test_cache_attention_refuses_its_two_outputs_over_one_another():
    cache, table, lengths = make([20, 20], 2, 64, 16, 1)
    q = _q(2, 2, 3, 4, 64)
    buf = torch.zeros(q.numel() + 256, dtype=torch.bfloat16, device="cuda")
    out = buf[:q.numel()].view(q.shape)
    for at in (0, q.numel() - 8):
        lse = buf[at:at + 48].view(torch.float32).view(2, 3, 4)
        with pytest.raises(ValueError):
            fp.cache_attention(q, cache, table, lengths, out=out, lse=lse)
    over_q = q.view(-1)[:48].view(torch.float32).view(2, 3, 4)
    with pytest.raises(ValueError):
        fp.cache_attention(q, cache, table, lengths, lse=over_q)
    lse = buf[q.numel():q.numel() + 48].view(torch.float32).view(2, 3, 4)
    fp.cache_attention(q, cache, table, lengths, out=out, lse=lse)
    want = fp.cache_attention(q, cache, table, lengths)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
