"""Which pairs of views share an element, against the sets of their elements."""
import itertools
import random

import torch

from precision_attention_nvfp4_b200.serving import _meet


def elements(t):
    at = t.storage_offset()
    return {at + sum(i * s for i, s in zip(ix, t.stride())) for ix in itertools.product(*map(range, t.shape))}


def test_views_of_one_layout_meet_exactly_where_they_share_an_element():
    rng = random.Random(0)
    buf = torch.zeros(4000, dtype=torch.bfloat16)
    met = apart = 0
    for _ in range(3000):
        d = rng.choice([4, 8])

        def view(strides=None):
            shape = (rng.randint(1, 4), rng.randint(1, 4), d)
            strides = strides or (rng.choice([0, d, 2 * d, 3 * d, 8 * d, 20 * d, 24 * d]), rng.choice([d, 2 * d, 3 * d, 16 * d]), 1)
            return buf.as_strided(shape, strides, rng.randrange(160)), strides

        x, strides = view()
        y, _ = view(strides)
        share = bool(elements(x) & elements(y))
        assert _meet(x, y) == share == _meet(y, x)
        met, apart = met + share, apart + (not share)
        z, _ = view()
        assert _meet(x, z) or not elements(x) & elements(z)       # other strides: never missed
    assert met > 300 and apart > 300


def test_heads_of_a_projection():
    x = torch.zeros(50, 16, 64, dtype=torch.bfloat16)
    assert not _meet(x[:, :10], x[:, 10:13]) and not _meet(x[:, 3:10], x[:, :3])
    assert _meet(x[:, :10], x[:, 8:10]) and _meet(x[:, :10], x[:, 9:12]) and _meet(x, x)
    t = x.view(50, 4, 4, 64)                                      # q, q, k, v of every KV head side by side
    assert not _meet(t[:, :, 0], t[:, :, 2]) and _meet(t[:, :, 2], x[:, 2::4])
    assert not _meet(x[:0], x[:0]) and not _meet(x[:25], x[25:])
