"""The serving calls record no graph: they refuse what one would be lost for, and say which caller's tensors they wrote."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import precision_attention_nvfp4_b200 as fp
from test_cache_attention_gpu import _q, make

pytestmark = pytest.mark.gpu

D = 64


def calls():
    """(name, tensor, the call with that tensor) of every tensor that a graph could hang on."""
    cache, table, lengths = make([20, 20], 2, D, 16, 1)
    rot = fp.rotary_table(D)
    x, k, v = _q(1, 20, 4, D), _q(2, 20, 2, D), _q(3, 20, 2, D)
    q = _q(4, 2, 3, 4, D)
    slots, pos = torch.arange(20, device="cuda"), torch.arange(20, device="cuda")
    new = torch.empty_like

    def write(**kw):
        return fp.cache_write(cache, kw.pop("k", k), kw.pop("v", v), slots, rotary=rot, positions=pos, q=kw.pop("q", x), **kw)

    return [("x", x, lambda t: fp.rotary(t, pos, rot)), ("out", new(x), lambda t: fp.rotary(x, pos, rot, out=t)),
            ("k", k, lambda t: write(k=t)), ("v", v, lambda t: write(v=t)), ("q", x, lambda t: write(q=t)),
            ("q_out", new(x), lambda t: write(q_out=t)),
            ("out[0]", new(k), lambda t: fp.cache_read(cache, slots, out=(t, new(k)))),
            ("out[1]", new(k), lambda t: fp.cache_read(cache, slots, out=(new(k), t))),
            ("q", q, lambda t: fp.cache_attention(t, cache, table, lengths)),
            ("out", new(q), lambda t: fp.cache_attention(q, cache, table, lengths, out=t)),
            ("lse", torch.empty(2, 3, 4, device="cuda"), lambda t: fp.cache_attention(q, cache, table, lengths, lse=t))]


def test_what_requires_a_gradient_is_refused():
    for name, t, call in calls():
        call(t)
        with pytest.raises(ValueError, match="gradient"):
            call(t.clone().requires_grad_())
        with torch.no_grad():
            call(t.clone().requires_grad_())


def test_a_forward_mode_tangent_is_refused():
    for name, t, call in calls():
        with fwd.dual_level():
            call(t)
            with pytest.raises(ValueError, match="tangent"):
                call(fwd.make_dual(t, torch.ones_like(t)))


def test_outputs_of_the_caller_count_as_written():
    for name, t, call in calls():
        before = t._version
        call(t)
        assert t._version == before + (1 if name in ("out", "out[0]", "out[1]", "q_out", "lse") else 0), name
    cache, table, lengths = make([20], 2, D, 16, 1)
    q = _q(5, 1, 3, 4, D)
    out = torch.ones_like(q)
    w = torch.ones(D, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    y = (out * w).sum()                                           # saves out
    fp.cache_attention(q, cache, table, lengths, out=out)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
