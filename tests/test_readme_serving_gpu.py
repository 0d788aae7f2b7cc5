"""The serving lines of the README run as they are written."""
import os

import pytest
import torch

import precision_attention_nvfp4_b200 as fp

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(__file__), os.pardir, "README.md")


def test_serving_lines():
    with open(README) as f:
        code = f.read().split("### Serving", 1)[1].split("```python", 1)[1].split("```", 1)[0]
    B, Hq, d, n = 3, 32, 128, 5
    x = torch.randn(B, Hq + 16, d, device="cuda").to(torch.bfloat16)
    names = dict(fp=fp, B=B, Hq=Hq, d=d, num_pages=12, q=x[:, :Hq], k=x[:, Hq:Hq + 8], v=x[:, Hq + 8:],
                 slots=torch.tensor([200, 300, 520], device="cuda"), pos=torch.tensor([71, 40, 9], device="cuda"),
                 page_table=torch.arange(12, dtype=torch.int32, device="cuda").view(B, 4),
                 lengths=torch.tensor([72, 41, 10], dtype=torch.int32, device="cuda"),
                 starts=torch.arange(B + 1, dtype=torch.int32, device="cuda"), parents=[-1, 0, 0, 1, 3],
                 q_tree=torch.randn(B, n, Hq, d, device="cuda").to(torch.bfloat16))
    exec(code, names)
    assert fp.device_error() == 0
    assert names["out"].shape == (B, n, Hq, d) and torch.isfinite(names["out"].float()).all()
    assert names["k16"].shape == (B, 8, d)
