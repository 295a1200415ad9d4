"""moe_block_norm and its backward pass against the formulas in 64 bits (host), with per-element bounds from the
fp32 operations they take, against torch's 64-bit automatic differentiation, and against differences."""
import sys

import pytest
import torch

import moe_routing_fp8_amd as moe

pytestmark = pytest.mark.gpu

EPS32 = 2.0 ** -24   # unit roundoff of fp32
EPS16 = 2.0 ** -8    # of bf16
# A row's sum of squares: at most 32 additions in a thread and 24 across the workgroup, then the square root's and a
# few products' roundings: 64 roundings on a factor, twice that where two norms follow one another.
ROUNDINGS = 64
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def _log(msg):
    sys.__stderr__.write(f"[gpu-block-norm] {msg}\n")
    sys.__stderr__.flush()


def _inputs(T, H, res, act, block=True, post=True, gate="channel", seed=0):
    g = torch.Generator().manual_seed(seed * 1000003 + T * 131 + H)

    def normal(*shape):
        return torch.randn(*shape, generator=g)

    s = {"residual": (3 * normal(T, H)).to(res), "y": normal(T, H).to(act) if block else None,
         "post_weight": 1 + 0.2 * normal(H) if post and block else None,
         "gate": {"none": None, "channel": 0.4 * normal(H), "token": torch.sigmoid(normal(T, 1))}[
             gate if block else "none"],
         "pre_weight": 1 + 0.2 * normal(H), "residual_scale": 0.75 if block else 1.0}
    s["grad_res_out"], s["grad_normed"] = normal(T, H).to(res), normal(T, H).to(act)
    return s


def _wide(t):
    return None if t is None else t.double()


def _forward64(s, eps):
    """r', n and the rstds in 64 bits, and the sum of magnitudes behind each element of r'."""
    r, y = _wide(s["residual"]), _wide(s["y"])
    post = None
    mag = r.abs()
    if y is not None:
        u = y
        if s["post_weight"] is not None:
            post = 1 / torch.sqrt((y * y).mean(1) + eps)
            u = y * post[:, None] * _wide(s["post_weight"])
        if s["gate"] is not None:
            u = u * _wide(s["gate"])
        mag = (s["residual_scale"] * r).abs() + u.abs()
        r = s["residual_scale"] * r + u
    pre = 1 / torch.sqrt((r * r).mean(1) + eps)
    return r, r * pre[:, None] * _wide(s["pre_weight"]), post, pre, mag


def _close(got, want, bound, name):
    """|got - want| <= bound (+ one rounding to bf16 of a value within the bound)."""
    assert got.shape == want.shape, name
    if got.dtype == BF16:
        bound = bound + EPS16 * (want.abs() + bound) + 2.0 ** -134
    bad = (got.double().cpu() - want).abs() > bound
    assert torch.isfinite(got.float()).all(), name
    assert not bad.any(), (name, int(bad.sum()), float(((got.double().cpu() - want).abs() / bound.clamp_min(1e-300)).max()))


def _gpu(s):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}


def _forward(d, eps=1e-6, **kw):
    return moe.moe_block_norm(d["residual"], d["y"], post_weight=d["post_weight"], gate=d["gate"],
                              residual_scale=d["residual_scale"], pre_weight=d["pre_weight"], eps=eps, with_rstd=True,
                              **kw)


SHAPES = [(1, 1), (3, 7), (2, 8), (5, 64), (4, 65), (1, 512), (33, 520), (7, 1001), (2, 2048), (3, 2049), (1, 4097),
          (2, 7168), (3, 8192), (2, 8200), (2, 9001), (1, 16384), (700, 256), (1500, 40)]
TYPES = [(BF16, BF16), (F32, BF16), (F32, F32), (BF16, F32)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("res,act", TYPES)
def test_forward(T, H, res, act):
    for block, post, gate in ((True, True, "channel"), (True, True, "token"), (True, False, "none"),
                              (True, True, "none"), (True, False, "token"), (False, False, "none")):
        _log(f"forward T={T} H={H} {res} {act} {block} {post} {gate}")
        s = _inputs(T, H, res, act, block, post, gate)
        kw = {} if block else {"act_dtype": act}
        r, n, post_rstd, pre_rstd = _forward(_gpu(s), **kw)
        er, en, epost, epre, mag = _forward64(s, 1e-6)
        if block:
            assert r.dtype == res
            _close(r, er, ROUNDINGS * EPS32 * mag, "res_out")
        else:
            assert r is None
        assert n.dtype == act
        w = (s["pre_weight"].double().abs() * epre[:, None])
        _close(n, en, 2 * ROUNDINGS * EPS32 * (mag * w + en.abs()), "normed")
        # the second factor also carries the errors of r' (mag), by at most their share of the row's norm
        amp = 1 + mag.square().mean(1).sqrt() * epre
        _close(pre_rstd, epre, ROUNDINGS * EPS32 * epre * amp, "pre_rstd")
        if post and block:
            _close(post_rstd, epost, ROUNDINGS * EPS32 * epost, "post_rstd")
        else:
            assert post_rstd is None


def _loss64(s, eps):
    """The scalar whose gradients the backward pass computes, on leaves that torch differentiates in 64 bits."""
    leaf = {k: _wide(s[k]).requires_grad_() for k in ("residual", "y", "post_weight", "gate", "pre_weight")
            if s[k] is not None}
    q = {**s, **leaf}
    r, n = _forward64(q, eps)[:2]
    return ((r * _wide(s["grad_res_out"])).sum() if s["grad_res_out"] is not None else 0) + (
        (n * _wide(s["grad_normed"])).sum()), leaf, r


def _backward(d, r, post_rstd, pre_rstd, **kw):
    return moe.moe_block_norm_backward(d["grad_res_out"], d["grad_normed"], r if r is not None else d["residual"],
                                       d["y"], post_weight=d["post_weight"], gate=d["gate"],
                                       residual_scale=d["residual_scale"], pre_weight=d["pre_weight"],
                                       post_rstd=post_rstd, pre_rstd=pre_rstd, **kw)


def _check_backward(s, o, eps=1e-6, saved_rounding=0.0):
    """Every gradient against 64-bit automatic differentiation.  Bounds: the magnitudes behind each value times the
    roundings of fp32; `saved_rounding`: the relative error of the stored r' (its type's roundoff)."""
    loss, leaf, _ = _loss64(s, eps)
    grads = dict(zip(leaf, torch.autograd.grad(loss, list(leaf.values()))))
    er, en, post, pre, mag = _forward64(s, eps)
    T, H = er.shape
    dn, dr = _wide(s["grad_normed"]), _wide(s["grad_res_out"]) if s["grad_res_out"] is not None else 0 * er
    w = _wide(s["pre_weight"])
    amp = 1 + mag.square().mean(1, keepdim=True).sqrt() * pre[:, None]  # cancellation in r' = s r + g u
    xh = mag * pre[:, None]
    g = (dn * w).abs()
    md = dr.abs() + pre[:, None] * (g + xh * (g * xh).mean(1, keepdim=True))
    unit = (2 * ROUNDINGS * EPS32 + 2 * saved_rounding) * amp
    row = 3 * unit  # xh enters the sum and its factor
    _close(o["grad_residual"], grads["residual"], row * s["residual_scale"] * md, "grad_residual")
    tail = (T + ROUNDINGS) * EPS32
    if s["pre_weight"] is not None:
        _close(o["grad_pre_weight"], grads["pre_weight"], ((row + tail) * dn.abs() * xh).sum(0), "grad_pre_weight")
    if s["y"] is None:
        return
    y = _wide(s["y"]).abs()
    yh = y * post[:, None] if post is not None else y
    pw = _wide(s["post_weight"]).abs() if post is not None else 1.0
    gate = _wide(s["gate"]).abs() if s["gate"] is not None else 1.0
    du = md * gate
    if s["gate"] is not None:
        along = (row + tail) * md * yh * pw
        want = grads["gate"]
        _close(o["grad_gate"], want, along.sum(0) if want.dim() == 1 else (
            (row + ROUNDINGS * EPS32) * md * yh * pw).sum(1, keepdim=True), "grad_gate")
    my = du
    if post is not None:
        _close(o["grad_post_weight"], grads["post_weight"], ((row + tail) * du * yh).sum(0), "grad_post_weight")
        h = du * pw
        my = post[:, None] * (h + yh * (h * yh).mean(1, keepdim=True))
    _close(o["grad_y"], grads["y"], 2 * row.amax() * my if T else my, "grad_y")


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("res,act", TYPES)
def test_backward(T, H, res, act):
    for block, post, gate in ((True, True, "channel"), (True, True, "token"), (True, False, "none"),
                              (False, False, "none")):
        _log(f"backward T={T} H={H} {res} {act} {block} {post} {gate}")
        s = _inputs(T, H, res, act, block, post, gate, seed=1)
        d = _gpu(s)
        r, n, post_rstd, pre_rstd = _forward(d, **({} if block else {"act_dtype": act}))
        o = _backward(d, r, post_rstd, pre_rstd)
        assert o["grad_residual"].dtype == res
        assert (o["grad_y"] is None) == (not block) and (o["grad_gate"] is None) == (gate == "none")
        _check_backward(s, o, saved_rounding=EPS16 if block and res == BF16 else 0.0)


def test_backward_without_one_of_the_gradients():
    s = _inputs(9, 264, F32, F32, seed=2)
    s["grad_res_out"] = None
    d = _gpu(s)
    r, n, post_rstd, pre_rstd = _forward(d)
    _check_backward(s, _backward(d, r, post_rstd, pre_rstd))
    # no norm before the next block: D is the residual path's gradient alone
    s = _inputs(9, 264, F32, F32, seed=3)
    d = _gpu(s)
    r, n, post_rstd, pre_rstd = moe.moe_block_norm(d["residual"], d["y"], post_weight=d["post_weight"], gate=d["gate"],
                                                   residual_scale=0.75, with_rstd=True)
    assert n is None and pre_rstd is None
    assert torch.equal(r, _forward(d)[0])
    o = moe.moe_block_norm_backward(d["grad_res_out"], None, r, d["y"], post_weight=d["post_weight"], gate=d["gate"],
                                    residual_scale=0.75, post_rstd=post_rstd)
    assert o["grad_pre_weight"] is None
    assert torch.equal(o["grad_residual"], 0.75 * d["grad_res_out"])
    z = {**s, "grad_normed": torch.zeros_like(s["grad_normed"])}
    loss, leaf, _ = _loss64(z, 1e-6)
    want = dict(zip(leaf, torch.autograd.grad(loss, list(leaf.values()))))
    for k in ("y", "gate", "post_weight"):
        got = o["grad_" + k].double().cpu()
        assert (got - want[k]).norm() <= 1e-5 * want[k].norm(), k  # 64 roundings of 6e-8, once more for the sums


@pytest.mark.parametrize("gate", ["channel", "token"])
def test_backward_against_differences(gate):
    """Along random directions, (L(p + h v) - L(p - h v)) / 2h of the 64-bit forward equals <gradient, v>."""
    s = _inputs(6, 96, F32, F32, gate=gate, seed=4)
    d = _gpu(s)
    r, n, post_rstd, pre_rstd = _forward(d)
    o = _backward(d, r, post_rstd, pre_rstd)
    gen = torch.Generator().manual_seed(5)
    for key in ("residual", "y", "post_weight", "gate", "pre_weight"):
        v = torch.randn(s[key].shape, generator=gen).double()
        h = 1e-5

        def at(step):
            q = {**s, key: _wide(s[key]) + step * v}
            return float(_loss64(q, 1e-6)[0].detach())

        slope = (at(h) - at(-h)) / (2 * h)
        got = o["grad_" + key].double().cpu()
        # the differences' own error is h^2 (1e-10) and 1e-16 / h of the loss; the gradient's 64 roundings
        scale = float((got * v).abs().sum()) + 1.0
        assert abs(slope - float((got * v).sum())) <= 2e-5 * scale, key


def test_strided_and_unaligned_rows():
    """Rows inside wider tensors, at any offset and stride, give what contiguous copies give."""
    T, H = 37, 264
    s = _inputs(T, H, BF16, BF16, seed=6)
    d = _gpu(s)
    want = _forward(d)
    for offset, stride in ((0, H + 8), (8, 2 * H), (1, H + 3), (3, H + 8)):
        wide = torch.full((T, 2 * H + 16), float("nan"), dtype=BF16, device="cuda")
        buf = wide.as_strided((T, H), (stride, 1), offset)
        buf.copy_(d["residual"])
        wy = torch.full((T, 2 * H + 16), float("nan"), dtype=BF16, device="cuda")
        by = wy.as_strided((T, H), (stride, 1), offset)
        by.copy_(d["y"])
        got = _forward({**d, "residual": buf, "y": by})
        for a, b in zip(got, want):
            # another split of the row over threads: the sums' order may differ
            assert (a.float() - b.float()).abs().max() <= 2 * EPS16 * b.float().abs().max()
        o = moe.moe_block_norm_backward(d["grad_res_out"], d["grad_normed"], buf, by, post_weight=d["post_weight"],
                                        gate=d["gate"], residual_scale=0.75, pre_weight=d["pre_weight"],
                                        post_rstd=want[2], pre_rstd=want[3])
        ref = moe.moe_block_norm_backward(d["grad_res_out"], d["grad_normed"], d["residual"], d["y"],
                                          post_weight=d["post_weight"], gate=d["gate"], residual_scale=0.75,
                                          pre_weight=d["pre_weight"], post_rstd=want[2], pre_rstd=want[3])
        for k in o:
            assert (o[k].float() - ref[k].float()).abs().max() <= 2 * EPS16 * ref[k].float().abs().max(), k


def test_in_place():
    """r' over the residual and n over y: the residual stream of a serving loop."""
    for res, act, H in ((BF16, BF16, 7168), (F32, BF16, 520), (F32, F32, 77)):
        d = _gpu(_inputs(5, H, res, act, seed=7))
        want = _forward(d)
        r, y = d["residual"].clone(), d["y"].clone()
        _forward({**d, "residual": r, "y": y}, out=(r, y, None, None))
        assert torch.equal(r, want[0]) and torch.equal(y, want[1])


def test_rows_of_zeros_and_of_large_values():
    T, H = 4, 512
    s = _inputs(T, H, F32, F32, seed=8)
    s["y"][0] = 0
    s["residual"][0] = 0          # n = 0 * rsqrt(eps)
    s["residual"][1] *= 1e15      # squares near 1e30
    s["y"][2] *= 1e-18            # squares below eps: the factor is rsqrt(eps)
    d = _gpu(s)
    r, n, post_rstd, pre_rstd = _forward(d)
    er, en, epost, epre, mag = _forward64(s, 1e-6)
    assert torch.equal(r[0].cpu(), torch.zeros(H)) and torch.equal(n[0].cpu(), torch.zeros(H))
    _close(r, er, ROUNDINGS * EPS32 * mag, "res_out")
    _close(pre_rstd, epre, 4 * ROUNDINGS * EPS32 * epre, "pre_rstd")
    _close(post_rstd, epost, ROUNDINGS * EPS32 * epost, "post_rstd")
    o = _backward(d, r, post_rstd, pre_rstd)
    assert all(torch.isfinite(v).all() for v in o.values())
    # NaN in a row stays in that row
    d["y"][3, 7] = float("nan")
    r2, n2, _, _ = _forward(d)
    assert torch.isnan(r2[3]).all() and torch.equal(r2[:3], r[:3]) and torch.equal(n2[:3], n[:3])


def test_no_tokens():
    d = _gpu(_inputs(0, 256, BF16, BF16))
    r, n, a, b = _forward(d)
    assert r.shape == (0, 256) and n.shape == (0, 256)
    o = _backward(d, r, a, b)
    for k in ("grad_post_weight", "grad_gate", "grad_pre_weight"):
        assert torch.equal(o[k], torch.zeros_like(o[k]))


def test_same_bits_each_time_and_on_another_stream():
    d = _gpu(_inputs(900, 1024, BF16, BF16, seed=9))
    r, n, a, b = _forward(d)
    first = _backward(d, r, a, b)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        r2, n2, a2, b2 = _forward(d, stream=st)
        again = _backward(d, r2, a2, b2, stream=st)
        st.synchronize()
        assert torch.equal(r, r2) and torch.equal(n, n2) and torch.equal(b, b2)
        assert all(torch.equal(first[k], again[k]) for k in first)


def test_writes_nothing_but_its_outputs():
    """Guard regions around every output keep their bytes."""
    for T, H in ((3, 77), (5, 264)):
        d = _gpu(_inputs(T, H, BF16, BF16, seed=10))
        bufs = {}

        def guarded(shape, dtype):
            n = 1
            for v in shape:
                n *= v
            whole = torch.full((n + 256,), 7.0, dtype=dtype, device="cuda")
            bufs[len(bufs)] = (whole, n)
            return whole[128:128 + n].view(shape)

        out = (guarded((T, H), BF16), guarded((T, H), BF16), guarded((T,), F32), guarded((T,), F32))
        _forward(d, out=out)
        o = {"grad_residual": guarded((T, H), BF16), "grad_y": guarded((T, H), BF16),
             "grad_post_weight": guarded((H,), F32), "grad_gate": guarded((H,), F32),
             "grad_pre_weight": guarded((H,), F32)}
        need = moe.moe_block_norm_backward_workspace_bytes(T, H)
        ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
        _backward(d, out[0], out[2], out[3], out=o, workspace=ws[:need])
        assert (ws[need:] == 0x5A).all()
        for whole, n in bufs.values():
            assert (whole[:128] == 7).all() and (whole[128 + n:] == 7).all()


def test_binding_refusals():
    d = _gpu(_inputs(4, 64, BF16, BF16))
    r, y, w = d["residual"], d["y"], d["post_weight"]
    pw = d["pre_weight"]
    bad = [dict(residual=r.half(), y=y, pre_weight=pw), dict(residual=r, y=y[:3], pre_weight=pw),
           dict(residual=r, y=y.t().contiguous().t(), pre_weight=pw), dict(residual=r, y=y, pre_weight=pw[:63]),
           dict(residual=r, y=y, pre_weight=pw.to(BF16)), dict(residual=r, y=y, gate=torch.ones(4, 64, device="cuda")),
           dict(residual=r, y=y, gate=torch.ones(4, device="cuda")), dict(residual=r),
           dict(residual=r, gate=d["gate"], pre_weight=pw), dict(residual=r, residual_scale=0.5, pre_weight=pw),
           dict(residual=r, y=y, pre_weight=pw, act_dtype=F32), dict(residual=r.cpu(), y=y, pre_weight=pw),
           dict(residual=r[:1].expand(4, 64), y=y, pre_weight=pw),
           dict(residual=r, y=y, pre_weight=pw, out=(None, torch.empty_like(y), None, None)),
           dict(residual=r, y=y, pre_weight=pw, out=(torch.empty_like(r), torch.empty_like(y)[:, :32], None, None))]
    for kw in bad:
        with pytest.raises(ValueError):
            moe.moe_block_norm(**kw)
    with pytest.raises(moe.MoeError, match="UNSUPPORTED"):
        wide = torch.zeros(1, 16385, device="cuda")
        moe.moe_block_norm(wide, pre_weight=torch.ones(16385, device="cuda"))
    with pytest.raises(moe.MoeError, match="INVALID"):
        moe.moe_block_norm(r, y, pre_weight=pw, eps=-1.0)
    out, n, a, b = _forward(d)
    for kw in (dict(pre_weight=None), dict(pre_rstd=None), dict(post_rstd=None), dict(grad_normed=None),
               dict(y=None), dict(grad_res_out=d["grad_res_out"][:2]), dict(workspace=torch.empty(8, device="cuda"))):
        args = dict(grad_res_out=d["grad_res_out"], grad_normed=d["grad_normed"], res_out=out, y=y, post_weight=w,
                    gate=d["gate"], residual_scale=0.75, pre_weight=pw, post_rstd=a, pre_rstd=b)
        args.update(kw)
        with pytest.raises(ValueError):
            moe.moe_block_norm_backward(**args)
    with pytest.raises(moe.MoeError, match="WORKSPACE"):
        _backward(d, out, a, b, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


def test_in_a_graph():
    """Captured once and replayed with new inputs, eager work between: every replay equals the eager result."""
    d = _gpu(_inputs(64, 1024, BF16, BF16, seed=11))
    ws = torch.empty(moe.moe_block_norm_backward_workspace_bytes(64, 1024), dtype=torch.uint8, device="cuda")
    out = _forward(d)
    o = _backward(d, out[0], out[2], out[3], workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _forward(d, out=out)
        _backward(d, out[0], out[2], out[3], workspace=ws, out=o)
    for k in range(3):
        new = _gpu(_inputs(64, 1024, BF16, BF16, seed=20 + k))
        for key in ("residual", "y", "grad_res_out", "grad_normed", "gate"):
            d[key].copy_(new[key])
        graph.replay()
        torch.cuda.synchronize()
        want = _forward(d)
        wo = _backward(d, want[0], want[2], want[3])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(torch.equal(o[key], wo[key]) for key in wo)


def test_more_than_2_to_31_elements():
    """The last rows of 270000 x 8192 equal the same rows alone."""
    T, H = 270000, 8192
    _log("2.2e9 elements")
    g = torch.Generator(device="cuda").manual_seed(12)
    r = torch.empty(T, H, dtype=BF16, device="cuda").normal_(generator=g)
    y = torch.empty(T, H, dtype=BF16, device="cuda").normal_(generator=g)
    w = 1 + 0.1 * torch.randn(H, generator=g, device="cuda")
    out, n, _, _ = moe.moe_block_norm(r, y, post_weight=w, pre_weight=w)
    few = moe.moe_block_norm(r[-600:].clone(), y[-600:].clone(), post_weight=w, pre_weight=w)
    assert torch.equal(out[-600:], few[0]) and torch.equal(n[-600:], few[1])
    assert torch.equal(out[:600], moe.moe_block_norm(r[:600], y[:600], post_weight=w, pre_weight=w)[0])


@pytest.mark.parametrize("post", [False, True])
def test_no_tokens_with_a_token_gate(post):
    H = 96
    w = torch.ones(H, device="cuda")
    r, y = torch.empty(0, H, device="cuda"), torch.empty(0, H, dtype=BF16, device="cuda")
    gate, pw = torch.empty(0, 1, device="cuda"), w if post else None
    out, normed, post_rstd, pre_rstd = moe.moe_block_norm(r, y, pw, gate, 1.0, w, with_rstd=True)
    assert out.shape == normed.shape == (0, H) and pre_rstd.shape == (0,)
    g = {k: torch.full((H,), 7.0, device="cuda") for k in (["grad_post_weight"] if post else []) + ["grad_pre_weight"]}
    g.update(grad_residual=torch.empty_like(r), grad_y=torch.empty_like(y), grad_gate=torch.empty_like(gate))
    moe.moe_block_norm_backward(out, normed, out, y, pw, gate, 1.0, w, post_rstd, pre_rstd, out=g)
    assert int(g["grad_pre_weight"].count_nonzero()) == 0
    assert not post or int(g["grad_post_weight"].count_nonzero()) == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H", [64, 2049, 9001])
@pytest.mark.parametrize("size", [1e-18, 1e-19, 3e-20, 1e-20, 1e-21])
def test_tiny_rows_without_eps(dtype, H, size):
    """eps = 0 and mean squares around and below fp32's smallest normal value.  A square, and the mean, are then off
    by up to half a step of 2^-149 each: the mean by 2^-149, the factor by half of that share of it."""
    g = torch.Generator().manual_seed(H)
    v = (size * (1 + torch.rand(3, H, generator=g))).to(dtype)
    one = torch.ones(H)
    _, n, _, pre = moe.moe_block_norm(v.cuda(), pre_weight=one.cuda(), eps=0.0, with_rstd=True)
    r, _, post, _ = moe.moe_block_norm(torch.zeros(3, H, device="cuda"), v.cuda(), post_weight=one.cuda(), eps=0.0,
                                       with_rstd=True)
    mean = v.double().square().mean(1)
    want = mean.rsqrt()
    share = ROUNDINGS * EPS32 + 2.0 ** -149 / mean
    for rstd in (pre, post):
        _close(rstd, want, share * want, "rstd")
    want = v.double() * want[:, None]
    _close(n, want, share[:, None] * want.abs(), "normed")
    _close(r, want, share[:, None] * want.abs(), "res_out")


def test_outputs_under_another_default_type():
    """torch's default type has no say in the rstds' and the parameter gradients' type."""
    d = _gpu(_inputs(40, 520, F32, BF16))
    want = _forward(d)
    gwant = _backward(d, want[0], want[2], want[3])
    torch.set_default_dtype(BF16)
    try:
        got = _forward(d)
        grads = _backward(d, got[0], got[2], got[3])
    finally:
        torch.set_default_dtype(F32)
    for a, b in [*zip(got, want), *((grads[k], gwant[k]) for k in gwant)]:
        assert a.dtype == b.dtype and torch.equal(a, b)


@pytest.mark.parametrize("res,act", TYPES)
def test_the_norm_alone_takes_its_type_from_the_output(res, act):
    """Without y, and without act_dtype, a given n says which type it is to have."""
    d = _gpu(_inputs(6, 200, res, act, block=False))
    want = moe.moe_block_norm(d["residual"], pre_weight=d["pre_weight"], act_dtype=act, with_rstd=True)
    n, rstd = torch.empty(6, 200, dtype=act, device="cuda"), torch.empty(6, device="cuda")
    got = moe.moe_block_norm(d["residual"], pre_weight=d["pre_weight"], out=(None, n, None, rstd))
    assert got[1] is n and torch.equal(n, want[1]) and torch.equal(rstd, want[3])
    other = BF16 if act == F32 else F32
    with pytest.raises(ValueError, match="normed"):
        moe.moe_block_norm(d["residual"], pre_weight=d["pre_weight"], act_dtype=other, out=(None, n, None, rstd))
    with pytest.raises(ValueError, match="act_dtype"):
        moe.moe_block_norm(d["residual"], pre_weight=d["pre_weight"], out=(None, n.half(), None, rstd))
