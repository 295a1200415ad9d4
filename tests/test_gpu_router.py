"""moe_router and its backward pass against the definition in 64 bits (host): ids equal, weights and gradients within
bounds from the fp32 operations they take, gradients also against 64-bit automatic differentiation and differences."""
import sys

import pytest
import torch

import moe_routing_fp8_amd as moe

pytestmark = pytest.mark.gpu

EPS32 = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32
# half a step of the output type, relative to the value: 8 significant bits leave steps of up to 2^-7 of it
HALF = {t: torch.finfo(t).eps / 2 for t in (BF16, F32)}
FMAX = float(torch.finfo(F32).max)


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def _log(msg):
    sys.__stderr__.write(f"[gpu-router] {msg}\n")
    sys.__stderr__.flush()


def _logits(T, E, dtype=F32, seed=0, spread=1.5):
    g = torch.Generator().manual_seed(seed * 7919 + T * 31 + E)
    return (spread * torch.randn(T, E, generator=g)).to(dtype)


def _clean(z):
    z = torch.where(torch.isnan(z), torch.full_like(z, -float("inf")), z)
    return z.clamp(max=FMAX)


def _scores64(z, score):
    """Scores of cleaned 64-bit logits; rows of nothing but -inf give 0."""
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    return e / e.sum(1, keepdim=True).clamp_min(1e-300)


def _ids(logits, K, score, bias=None, num_groups=1, topk_groups=1, group_score="max", token_mask=None):
    """The chosen experts, from the definition: stable sorts of 64-bit values."""
    T, E = logits.shape
    z = _clean(logits.double())
    s = _scores64(z, score)
    low = -float("inf")
    c = s
    open_ = z > low
    if bias is not None:
        b = bias.double()
        open_ = open_ & (b > low)[None]
        c = s + torch.nan_to_num(b, nan=0.0, posinf=FMAX, neginf=0.0)
    c = torch.where(open_, c, low)
    order = torch.where(open_, z, low) if bias is None else c
    if num_groups > 1:
        by = order if bias is None and group_score == "max" else c
        m = by.view(T, num_groups, -1).sort(dim=2, descending=True).values
        worth = m[:, :, 0] if group_score == "max" else m[:, :, 0] + m[:, :, 1]
        keep = worth.sort(dim=1, descending=True, stable=True).indices[:, :topk_groups]
        allowed = torch.zeros(T, num_groups, dtype=torch.bool).scatter_(1, keep, True)
        order = torch.where(allowed.repeat_interleave(E // num_groups, 1), order, low)
    top = order.sort(dim=1, descending=True, stable=True)
    ids = torch.where(top.values[:, :K] > low, top.indices[:, :K], -1)
    if token_mask is not None:
        ids = torch.where(token_mask[:, None], ids, -1)
    return ids


def _weights(logits, ids, score, renormalize, scale):
    """Weights of given ids in 64 bits; differentiable in the logits."""
    z = logits
    live = ids >= 0
    at = ids.clamp_min(0)
    if renormalize:
        zs = z.gather(1, at)
        r = zs if score == "softmax" else torch.nn.functional.logsigmoid(zs)
        r = torch.where(live, r, -float("inf"))
        r = torch.where(live.any(1, keepdim=True), r, torch.zeros_like(r))
        return scale * torch.where(live, torch.softmax(r, 1), torch.zeros_like(r))
    s = torch.softmax(z, 1) if score == "softmax" else torch.sigmoid(z)
    return scale * torch.where(live, s.gather(1, at), torch.zeros_like(at, dtype=s.dtype))


def _unit(logits):
    """Relative error of a weight: the exponents' arguments (differences of logits, up to `reach`, rounded once, times a
    rounded constant: two roundings each), the exponential's 2 ulp, sums of at most 16 terms a lane and 6 steps over
    the lanes, a division and two products, in numerator and denominator: 96 roundings and 4 for each unit of reach."""
    z = logits.double()
    z = torch.where(torch.isfinite(z), z, torch.zeros_like(z))
    reach = float((z.amax(1) - z.amin(1)).max().clamp_min(z.abs().max())) if z.numel() else 0.0
    return (96 + 4 * min(reach, 104.0)) * EPS32


def _gpu(t):
    return None if t is None else t.cuda()


def _check(logits, K, score="softmax", renormalize=False, scale=1.0, seed=1, **kw):
    T, E = logits.shape
    kg = {k: _gpu(v) if isinstance(v, torch.Tensor) else v for k, v in kw.items()}
    d = logits.cuda()
    idx, w = moe.moe_router(d, K, score=score, renormalize=renormalize, scale=scale, **kg)
    ids = _ids(logits, K, score, **kw)
    assert torch.equal(idx.cpu(), ids), (idx.cpu() - ids).nonzero()[:4]
    z = _clean(logits.double()).clamp_min(-FMAX)  # -inf as a number: e^(it) is 0
    if kw.get("token_mask") is not None:
        z = torch.where(kw["token_mask"][:, None], z, torch.zeros_like(z))
    z.requires_grad_()
    want = _weights(z, ids, score, renormalize, scale)
    unit = _unit(logits if kw.get("token_mask") is None else z.detach())
    err = (w.double().cpu() - want.detach()).abs()
    assert (err <= unit * want.detach().abs() + 1e-37).all(), float((err / want.detach().abs().clamp_min(1e-37)).max())
    g = torch.randn(T, K, generator=torch.Generator().manual_seed(seed))
    got = moe.moe_router_backward(g.cuda(), d, idx, score=score, renormalize=renormalize, scale=scale)
    assert got.dtype == logits.dtype
    (exact,) = torch.autograd.grad((want * g.double()).sum(), z)
    # each derivative is s (g - sum s g): its terms' magnitudes times the weights' error
    s = (want.detach() / scale).abs() if scale else want.detach().abs()
    gs = (abs(scale) * g.double()).abs() * (ids >= 0)
    spread = (s * gs).sum(1, keepdim=True)
    size = torch.zeros(T, E, dtype=torch.float64).scatter_add_(1, ids.clamp_min(0), s * (gs + spread))
    if score == "softmax" and not renormalize:
        size = size + _scores64(z.detach(), "softmax") * spread
    bound = 3 * unit * size + HALF[logits.dtype] * exact.abs() * 1.01 + 1e-37
    assert ((got.double().cpu() - exact).abs() <= bound).all(), \
        float(((got.double().cpu() - exact).abs() / bound).max())
    return idx, w


SHAPES = [(1, 1, 1), (3, 2, 1), (5, 5, 3), (64, 16, 2), (7, 17, 16), (33, 61, 4), (130, 64, 6), (9, 100, 8),
          (65, 128, 8), (257, 256, 8), (6, 257, 8), (11, 384, 6), (5, 512, 16), (4, 1000, 8), (3, 1024, 16)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,K", SHAPES)
def test_shapes(T, E, K, score, dtype):
    z = _logits(T, E, dtype)
    bias = 0.05 * torch.randn(E, generator=torch.Generator().manual_seed(E))
    for renorm in (False, True):
        _log(f"T={T} E={E} K={K} {score} {dtype} renorm={renorm}")
        _check(z, K, score, renorm, 1.0)
        _check(z, K, score, renorm, 2.5, bias=bias)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("T,E,K,G,kept", [(50, 256, 8, 8, 4), (33, 160, 6, 8, 3), (7, 64, 2, 32, 1), (9, 128, 8, 64, 9),
                                          (20, 384, 8, 8, 4), (5, 1024, 16, 64, 5), (6, 66, 4, 3, 2), (4, 12, 3, 4, 2),
                                          (17, 256, 8, 8, 8)])
def test_groups(T, E, K, G, kept, group_score, score, dtype):
    z = _logits(T, E, dtype, seed=2)
    bias = 0.02 * torch.randn(E, generator=torch.Generator().manual_seed(E))
    kw = dict(num_groups=G, topk_groups=kept, group_score=group_score)
    _log(f"T={T} E={E} K={K} G={G}/{kept} {group_score} {score} {dtype}")
    _check(z, K, score, True, 2.5, **kw)
    _check(z, K, score, False, 1.0, bias=bias, **kw)


@pytest.mark.parametrize("E,G", [(61, 1), (256, 8), (600, 4)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_equal_values_go_to_the_lowest_expert(E, G, score):
    """bf16 logits on few values, a bias of few steps, or none at all: most places are ties."""
    g = torch.Generator().manual_seed(E)
    z = (torch.randint(-3, 4, (40, E), generator=g) * 0.5).to(BF16)
    bias = torch.randint(0, 2, (E,), generator=g).float() * 1e-3
    kw = dict(num_groups=G, topk_groups=(G + 1) // 2)
    for gs in ("max", "top2"):
        for b in (None, torch.zeros(E), bias):
            _check(z, 8, score, True, bias=b, group_score=gs, **kw)
            _check(z.float(), 8, score, True, bias=b, group_score=gs, **kw)
    same = torch.full((5, E), 0.25)
    idx, _ = _check(same, 4, score, True)
    assert torch.equal(idx.cpu(), torch.arange(4).expand(5, 4))


@pytest.mark.parametrize("E,G", [(16, 1), (61, 1), (256, 1), (256, 8), (520, 4)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_values_next_to_each_other(E, G, score):
    """A bias that cancels one row's scores leaves values that differ by less than an fp32 step; logits that differ
    by single steps; both need the order of 64 bits."""
    z = _logits(6, E, seed=5)
    bias = (0.75 - _scores64(z[:1].double(), score)[0]).float()
    kw = dict(num_groups=G, topk_groups=(G + 1) // 2, group_score="top2")
    _check(z, 8, score, True, bias=bias, **kw)
    _check(z, 8, score, False, bias=bias, num_groups=G, topk_groups=(G + 1) // 2)
    steps = torch.arange(E, dtype=torch.int32).flip(0) * 3 % 17
    one = (torch.full((4, E), 1.25).view(torch.int32) + steps).view(F32)
    one[1] = -one[1]
    one[2, ::2] = -one[2, ::2]
    one[3] *= 1e-30
    _check(one, 8, score, True, **kw)
    _check(one, 8, score, True, bias=torch.zeros(E), **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [16, 61, 256, 300])
def test_masks_and_missing_experts(score, E):
    z = _logits(20, E, seed=3)
    mask = torch.ones(20, dtype=torch.bool)
    mask[[0, 7, 19]] = False
    z[0], z[7] = float("nan"), float("inf")
    z[1] = -float("inf")              # nothing left
    z[2, 3:] = -float("inf")          # three experts left for eight rounds
    z[3, ::2] = float("nan")          # NaN takes an expert out
    z[4, 5] = float("inf")            # counts as the largest number
    z[5] = torch.finfo(F32).min       # the lowest value is a value
    z[6, 0] = torch.finfo(F32).min
    for renorm in (False, True):
        _check(z, 8, score, renorm, token_mask=mask)
        bias = torch.zeros(E)
        bias[1], bias[2], bias[4] = -float("inf"), float("nan"), 3.0
        _check(z, 8, score, renorm, token_mask=mask, bias=bias)
    if E % 4 == 0:
        z[8, : E // 2] = -float("inf")
        _check(z, 8, score, True, token_mask=mask, num_groups=4, topk_groups=2, group_score="top2")
        _check(z, 8, score, True, token_mask=mask, num_groups=4, topk_groups=3, group_score="max")
    none = torch.zeros(20, dtype=torch.bool)
    idx, w = _check(z, 8, score, True, token_mask=none)
    assert (idx == -1).all() and (w == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shift", [-200.0, -90.0, -30.0, 30.0, 200.0])
def test_far_logits(score, shift):
    """Scores that vanish or saturate in fp32 (and, at +-200, in 64 bits): the weights of a renormalised row hold.
    A sigmoid of +30 or more is 1 to fp32, so there is no bias here that would order such values."""
    z = _logits(16, 64, seed=9) + shift
    _check(z, 4, score, True)


def test_a_large_batch_and_one_token():
    z = _logits(5000, 256, seed=11)
    bias = 0.01 * torch.randn(256, generator=torch.Generator().manual_seed(3))
    kw = dict(num_groups=8, topk_groups=4, group_score="top2", bias=bias)
    idx, w = _check(z, 8, "sigmoid", True, 2.5, **kw)
    one = moe.moe_router(z[17:18].cuda(), 8, score="sigmoid", renormalize=True, scale=2.5, num_groups=8, topk_groups=4,
                         group_score="top2", bias=bias.cuda())
    assert torch.equal(one[0], idx[17:18]) and torch.equal(one[1], w[17:18])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strides_and_alignment(dtype):
    wide = _logits(30, 301, dtype, seed=4)
    for lo, hi in ((0, 256), (1, 257), (3, 64), (2, 301)):
        part = wide[:, lo:hi]
        for score, renorm in (("softmax", False), ("sigmoid", True)):
            d = wide.cuda()[:, lo:hi]
            a = moe.moe_router(d, 4, score=score, renormalize=renorm)
            b = moe.moe_router(part.contiguous().cuda(), 4, score=score, renormalize=renorm)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
            g = torch.randn(30, 4, device="cuda")
            ga = moe.moe_router_backward(g, d, a[0], score=score, renormalize=renorm)
            gb = moe.moe_router_backward(g, part.contiguous().cuda(), a[0], score=score, renormalize=renorm)
            assert torch.equal(ga, gb)


def test_gradient_against_differences():
    """The fp32 weights' difference quotient: with steps of 2^-6 its curvature term is below h^2 times the third
    derivative, which for these functions is at most 2 times the gradient's terms."""
    z = _logits(8, 24, seed=6)
    g = torch.randn(8, 3, generator=torch.Generator().manual_seed(1))
    h = 2.0 ** -6
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            idx, _ = moe.moe_router(z.cuda(), 3, score=score, renormalize=renorm)
            got = moe.moe_router_backward(g.cuda(), z.cuda(), idx, score=score, renormalize=renorm).double().cpu()
            ids = idx.cpu()
            for e in range(0, 24, 5):
                up, down = z.double().clone(), z.double().clone()
                up[:, e] += h
                down[:, e] -= h
                f = [(_weights(v, ids, score, renorm, 1.0) * g.double()).sum(1) for v in (up, down)]
                slope = (f[0] - f[1]) / (2 * h)
                assert ((got[:, e] - slope).abs() <= 4 * h * h * g.double().abs().sum(1)).all()


def test_streams_graphs_and_outputs():
    z = _logits(300, 64, seed=8).cuda()
    bias = torch.zeros(64, device="cuda")
    g = torch.randn(300, 4, device="cuda")
    kw = dict(score="sigmoid", renormalize=True)
    want = moe.moe_router(z, 4, bias=bias, **kw)
    grad = moe.moe_router_backward(g, z, want[0], **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.moe_router(z, 4, bias=bias, stream=side, **kw)
    got_grad = moe.moe_router_backward(g, z, got[0], stream=side, **kw)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got_grad, grad)
    out = (torch.empty_like(want[0]), torch.empty_like(want[1]))
    out_grad = torch.empty_like(grad)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_router(z, 4, bias=bias, out=out, **kw)
        moe.moe_router_backward(g, z, out[0], out=out_grad, **kw)
    for seed in range(3):
        z.copy_(_logits(300, 64, seed=20 + seed))
        graph.replay()
        eager = moe.moe_router(z, 4, bias=bias, **kw)
        assert torch.equal(out[0], eager[0]) and torch.equal(out[1], eager[1])
        assert torch.equal(out_grad, moe.moe_router_backward(g, z, eager[0], **kw))
        torch.cuda.synchronize()


def test_no_tokens():
    z = torch.empty(0, 64, device="cuda")
    idx, w = moe.moe_router(z, 4)
    assert idx.shape == (0, 4) and w.shape == (0, 4)
    assert moe.moe_router_backward(w, z, idx).shape == (0, 64)


def test_ids_that_take_no_part():
    """Ids outside [0, E) in the backward pass: their gradients are not used, whatever they hold."""
    z = _logits(6, 32, seed=7)
    ids = torch.tensor([[0, -1, 5], [-1, -1, -1], [31, 32, 2], [7, 1 << 40, -(1 << 40)], [1, 2, 3], [9, -1, -1]])
    g = torch.randn(6, 3)
    g[0, 1] = float("nan")
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            got = moe.moe_router_backward(g.cuda(), z.cuda(), ids.cuda(), score=score, renormalize=renorm).cpu()
            legal = torch.where((ids >= 0) & (ids < 32), ids, -1)
            zz = z.double().requires_grad_()
            loss = (_weights(zz, legal, score, renorm, 1.0) * torch.where(legal >= 0, g, 0.0).double()).sum()
            (want,) = torch.autograd.grad(loss, zz)
            assert ((got.double() - want).abs() <= 1e-5 * g.nan_to_num().abs().max()).all()
            assert (got[1] == 0).all()


def test_ids_feed_the_token_map():
    """Masked tokens' copies get no slot."""
    z = _logits(100, 32, seed=12).cuda()
    mask = torch.arange(100, device="cuda") % 3 != 0
    idx, _ = moe.moe_router(z, 4, token_mask=mask)
    counts, offsets, pos, row_token = moe.moe_token_map(idx, 32)
    assert int(counts.sum()) == 4 * int(mask.sum()) == int(offsets[-1])
    assert (pos[~mask] == -1).all() and (pos[mask] >= 0).all()
