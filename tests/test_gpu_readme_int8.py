"""README.md's program from the logits to the expert outputs in 8-bit integers, and the example's block, run as they stand
there, in debug mode and with masked tokens, whatever fresh memory holds."""
import os
import re

import pytest
import torch

import moe_routing_fp8_amd as moe
from test_gpu_example import example  # noqa: F401

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _program():
    with open(os.path.join(ROOT, "README.md")) as f:
        text = f.read()
    return re.search(r"From the logits to the expert outputs in 8-bit integers:\s*```python\n(.*?)```", text, re.S)[1]


@pytest.fixture(params=["0", "1"])
def poisoned(request, monkeypatch):
    """Debug mode off and on; fresh floating-point memory holds NaN."""
    fresh = torch.empty

    def empty(*args, **kw):
        t = fresh(*args, **kw)
        return t.fill_(float("nan")) if t.is_floating_point() else t

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setenv("MOE_FP8_DEBUG", request.param)


def test_program_of_the_readme(poisoned):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    T, E, H, I = 50, 256, 128, 64
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    names = {"torch": torch, "moe": moe, "logits": normal(T, E), "bias": 0.01 * normal(E), "dw": normal(T, 8),
             "mask": torch.arange(T, device="cuda") % 3 != 0, "x": normal(T, H).to(torch.bfloat16)}
    for name, N, K in (("up", 2 * I, H), ("down", H, I)):
        codes, sf = moe.moe_cast_int8(normal(E * N, K))
        names["w_" + name], names["sf_" + name] = codes.view(E, N, K), sf.view(E, N)
    exec(compile(_program(), "README.md", "exec"), names)
    out = names["out"]
    assert out.shape == (T, H) and torch.isfinite(out).all()
    assert (out[~names["mask"]] == 0).all() and (out[names["mask"]] != 0).any(1).all()


def test_the_example_with_masked_tokens(example, poisoned):  # noqa: F811
    block = example.Block(256, 128, 16, 2, seed=1)
    residual = torch.randn(40, 256, device="cuda").to(torch.bfloat16)
    mask = torch.arange(40, device="cuda") % 4 != 0
    out, normed, ids, _ = block.serve_int8(residual, token_mask=mask)
    assert torch.isfinite(out).all() and torch.isfinite(normed).all()
    assert torch.equal(out[~mask], residual[~mask]) and (ids[~mask] == -1).all()
