"""examples/moe_block.py: the block in 8-bit integers, and the router's weights under automatic differentiation."""
import pytest
import torch

from test_gpu_example import example  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,hidden,inter,experts,topk,groups", [(1, 256, 128, 16, 2, 2), (40, 512, 256, 8, 4, 2),
                                                                     (300, 256, 96, 8, 2, 4)])
def test_serving_in_8_bit_integers(example, tokens, hidden, inter, experts, topk, groups):  # noqa: F811
    """The casts of x, of the activation (a row's largest value is 4 to 8 times its rms, half a step of 1/127 of it
    below 2^-5 of the rms) and the products' bf16 outputs: below 2^-4 of the expert output, which a gate of about a
    half adds to a residual of the same size."""
    block = example.Block(hidden, inter, experts, topk, seed=tokens)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    residual = torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16)
    mask = torch.rand(tokens, generator=g, device="cuda") >= 0.2
    mask[0] = True
    out, normed, ids, weights = block.serve_int8(residual, groups=groups, topk_groups=(groups + 1) // 2,
                                                 token_mask=mask)
    assert (ids[~mask] == -1).all() and (ids[mask] >= 0).all()
    # the experts of a token lie in the groups taken
    kept = (ids[mask] // (experts // groups)).sort(1).values
    assert ((kept[:, 1:] != kept[:, :-1]).sum(1) < (groups + 1) // 2).all()
    for got, want in zip((out, normed), block.int8_plain(residual, ids, weights)):
        assert got.dtype == torch.bfloat16
        assert (got.float() - want)[mask].norm() <= 2 ** -4 * want[mask].norm()
    assert torch.equal(out[~mask], residual[~mask])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_router_gradient(example, score):  # noqa: F811
    """The router's weights' gradient against 64-bit automatic differentiation: fp32 products of 64 terms around
    derivatives of 128 roundings."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x, router = torch.randn(100, 64, generator=g, device="cuda"), torch.randn(64, 32, generator=g, device="cuda") / 8
    values = torch.randn(100, 32, generator=g, device="cuda")
    grad, ids = example.router_gradient(x, router, values, 4, score)
    wide = router.double().cpu().requires_grad_()
    z = (x.double().cpu() @ wide).gather(1, ids.cpu())
    p = torch.softmax(z if score == "softmax" else torch.nn.functional.logsigmoid(z), 1)
    (p * values.double().cpu().gather(1, ids.cpu())).sum().backward()
    size = x.abs().double().cpu().T @ torch.ones(100, 32, dtype=torch.float64)
    assert ((grad.double().cpu() - wide.grad).abs() <= 1024 * 2.0 ** -24 * size * values.abs().max().item()).all()
