"""moe_router's weights and moe_router_backward's gradients within the bounds of the operations that each takes, counted
one by one, in units of 2^-24 (half a step of fp32).

The exponential of the weights (exp_nonpos_exact) is off by 1.5 steps, 3 units, and |x| / 16 units for an exact x.  x, the
distance from the largest chosen logit, is exact for bf16 logits of these ranges (8 significant bits, exponents less than
16 apart); for fp32 logits its rounding adds |x| units.  The plain exponential, behind softmax weights that are not
renormalised, is off by 1 step and the rounding of x log2(e), |x| units, and of log2(e) itself, 0.23 |x|."""
import pytest
import torch

from test_gpu_router import BF16, EPS32, F32, HALF, _need_gpu, _weights  # noqa: F401

import moe_routing_fp8_amd as moe

pytestmark = pytest.mark.gpu

LEVELS = 6          # steps of a sum over up to 64 lanes
MEAN_X = 7.0        # sum of p |x| over a softmax's terms: at most the logarithm of their number, 1024


def _within(err, bound):
    worst = float((err.abs() / bound).max())
    assert worst <= 1, worst


def _run(T, E, K, dtype, spread, score, renorm, scale):
    g = torch.Generator().manual_seed(E * 100 + K)
    z = (spread * torch.randn(T, E, generator=g)).to(dtype)
    gw = torch.randn(T, K, generator=g)
    idx, w = moe.moe_router(z.cuda(), K, score=score, renormalize=renorm, scale=scale)
    grad = moe.moe_router_backward(gw.cuda(), z.cuda(), idx, score=score, renormalize=renorm, scale=scale)
    ids = idx.cpu()
    zd = z.double().requires_grad_()
    want = _weights(zd, ids, score, renorm, scale)
    if score == "sigmoid" and not renorm:
        # by the formula: automatic differentiation takes 1 - s from a rounded s, 1e-4 off where that is 1e-12
        zk = z.double().gather(1, ids)
        want_grad = torch.zeros(T, E, dtype=torch.float64).scatter_(
            1, ids, scale * gw.double() * torch.sigmoid(zk) * torch.sigmoid(-zk))
    else:
        (want_grad,) = torch.autograd.grad((want * gw.double()).sum(), zd)
    return z.double(), ids, gw.double() * scale, w.double().cpu(), want.detach(), grad.double().cpu(), want_grad


SHAPES = [(400, 16, 16), (400, 64, 8), (200, 256, 8), (200, 512, 16), (100, 1024, 12)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,K", SHAPES)
@pytest.mark.parametrize("spread", [1.5, 12.0])
def test_renormalised(T, E, K, score, dtype, spread):
    z, ids, g, w, want, grad, want_grad = _run(T, E, K, dtype, spread, score, True, 2.5)
    zk = z.gather(1, ids)
    high = zk.amax(1, keepdim=True)
    sigmoid = score == "sigmoid"
    x = (zk - (high.clamp(max=0) if sigmoid else high)).clamp(max=0).abs()
    per_x = 1 / 16 + (1 if dtype == F32 else 0)
    # a term: its exponential; a sigmoid's denominator (half of 3, and 1 for the sum) and division
    term = 3 + per_x * x + (4 if sigmoid else 0)
    # the terms' sum: their mean error and the steps over the lanes; the division
    total = 3 + per_x * MEAN_X + (4 if sigmoid else 0) + LEVELS
    share = term + total + 1
    _within(w - want, (share + 1) * EPS32 * want + 1e-37)      # and the scale
    # p (g - sum p g), for sigmoids times 1 - s: g's rounding, those of the sum, the difference and the products
    p = want / 2.5
    rest = torch.sigmoid(-zk) if sigmoid else torch.ones_like(zk)
    # 1 - s: an exponential of |z| exactly, 1 + x, a division, a product
    rest_units = 3 + zk.abs() / 16 + 2.5 + 1 + 1 if sigmoid else torch.zeros_like(zk)
    dot = (p * g).sum(1, keepdim=True)
    dot_err = ((share + 2 + LEVELS) * (p * g).abs()).sum(1, keepdim=True)
    err = p * rest * ((share + 2 + rest_units) * (g - dot).abs() + g.abs() + dot_err) * EPS32
    _within(grad - want_grad, torch.zeros_like(z).scatter_(1, ids, err) + HALF[dtype] * want_grad.abs() * 1.01 + 1e-37)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,E,K", SHAPES)
@pytest.mark.parametrize("spread", [1.5, 12.0])
def test_sigmoids_as_they_are(T, E, K, dtype, spread):
    z, ids, g, w, want, grad, want_grad = _run(T, E, K, dtype, spread, "sigmoid", False, 2.5)
    x = z.gather(1, ids).abs()
    # the exponential (in numerator and denominator: half of 3 there), 1 + x, a division, the scale
    _within(w - want, (3 + x / 16 + 2.5 + 2) * EPS32 * want + 1e-37)
    # g x / (1 + x) / (1 + x): two denominators, two divisions, two products
    err = (3 + x / 16 + 2 * 2.5 + 4) * EPS32 * want_grad.gather(1, ids).abs()
    _within(grad - want_grad, torch.zeros_like(z).scatter_(1, ids, err) + HALF[dtype] * want_grad.abs() * 1.01 + 1e-37)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,E,K", SHAPES)
@pytest.mark.parametrize("spread", [1.5, 12.0])
def test_softmax_as_it_is(T, E, K, dtype, spread):
    z, ids, g, w, want, grad, want_grad = _run(T, E, K, dtype, spread, "softmax", False, 2.5)
    x = (z - z.amax(1, keepdim=True)).abs()
    per_x = 1.23 + (1 if dtype == F32 else 0)
    term = 2 + per_x * x
    total = 2 + per_x * MEAN_X + 15 + LEVELS        # 16 terms a lane, one after another
    s_units = term + total + 2                      # a division, or a reciprocal and a product
    _within(w - want, (s_units.gather(1, ids) + 1) * EPS32 * want + 1e-37)
    # s_e (g_e - sum s g): the sum's terms, g's rounding, the difference and the product
    s = torch.softmax(z, 1)
    sk = s.gather(1, ids)
    dot = (sk * g).sum(1, keepdim=True)
    dot_err = ((s_units.gather(1, ids) + 2 + LEVELS) * (sk * g).abs()).sum(1, keepdim=True)
    ge = torch.zeros_like(z).scatter_(1, ids, g)
    err = s * ((s_units + 2) * (ge - dot).abs() + ge.abs() + dot_err) * EPS32
    _within(grad - want_grad, err + HALF[dtype] * want_grad.abs() * 1.01 + 1e-37)
