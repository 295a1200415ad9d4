"""examples/moe_block.py: the block norm, the expert products and the balance loss together with the dispatch path."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    spec = importlib.util.spec_from_file_location("moe_block_example", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("tokens,hidden,inter,experts,topk", [(1, 256, 128, 16, 2), (8, 512, 256, 8, 4),
                                                              (40, 256, 128, 4, 2)])
def test_serving_block(example, tokens, hidden, inter, experts, topk):
    """The block against its fp32 form: each of two e4m3 casts is at most 2^-4 off a value (rms below 2^-5), the
    expert output reaches the residual through a gate of about a half next to a residual of the same size."""
    block = example.Block(hidden, inter, experts, topk, seed=tokens)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    residual = torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16)
    for got, want in zip(block.serve(residual), block.serve_plain(residual)):
        assert got.dtype == torch.bfloat16
        assert (got.float() - want).norm() <= 2 ** -4 * want.norm()


def test_training_steps(example):
    first, last = example.train_router()
    assert 1 < first and last < first and last < 1.1 + 0.5 * (first - 1)
    first, last = example.train_norm()
    assert last < 0.2 * first
