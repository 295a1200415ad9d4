"""moe_balance_loss and its backward pass against the formulas in 64 bits (host): counts equal, the rest within
bounds from the fp32 operations they take; gradients against 64-bit automatic differentiation and differences."""
import sys

import pytest
import torch

import moe_routing_fp8_amd as moe

pytestmark = pytest.mark.gpu

EPS32 = 2.0 ** -24
EPS16 = 2.0 ** -8
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def _log(msg):
    sys.__stderr__.write(f"[gpu-balance] {msg}\n")
    sys.__stderr__.flush()


def _inputs(T, E, K, dtype=F32, cuts=None, masked=0.0, seed=0, spread=1.5):
    g = torch.Generator().manual_seed(seed * 7919 + T * 31 + E)
    z = (spread * torch.randn(T, E, generator=g)).to(dtype)
    ids = z.float().topk(K, dim=1).indices
    mask = None
    if masked:
        mask = torch.rand(T, generator=g) >= masked
    off = None if cuts is None else torch.tensor(cuts, dtype=torch.int32)
    S = 1 if off is None else len(cuts) - 1
    return {"logits": z, "topk_idx": ids, "token_mask": mask, "seq_offsets": off,
            "grad_loss": torch.randn(S, generator=g) / S}


def _seqs(s):
    T = s["logits"].shape[0]
    ends = [0, T] if s["seq_offsets"] is None else s["seq_offsets"].tolist()
    live = torch.ones(T, dtype=torch.bool) if s["token_mask"] is None else s["token_mask"]
    for q in range(len(ends) - 1):
        rows = torch.arange(ends[q], max(ends[q], ends[q + 1]))
        yield q, rows[live[rows]]


def _probs64(z, score):
    return torch.softmax(z, 1) if score == "softmax" else torch.softmax(torch.nn.functional.logsigmoid(z), 1)


def _want(s, score):
    z = s["logits"].double().requires_grad_()
    T, E = z.shape
    K = s["topk_idx"].shape[1]
    S = s["grad_loss"].shape[0]
    loss, mean = torch.zeros(S, dtype=torch.float64), torch.zeros(S, E, dtype=torch.float64)
    counts, n = torch.zeros(S, E, dtype=torch.int32), torch.zeros(S, dtype=torch.int32)
    total = 0.0
    for q, rows in _seqs(s):
        n[q] = rows.numel()
        if not rows.numel():
            continue
        ids = s["topk_idx"][rows].flatten()
        ids = ids[(ids >= 0) & (ids < E)]
        counts[q] = torch.bincount(ids, minlength=E)
        pm = _probs64(z[rows], score).mean(0)
        one = E / (K * rows.numel()) * (counts[q].double() * pm).sum()
        mean[q], loss[q] = pm.detach(), one.detach()
        total = total + s["grad_loss"][q].double() * one
    grad = torch.zeros(T, E, dtype=torch.float64)
    if isinstance(total, torch.Tensor):
        (grad,) = torch.autograd.grad(total, z)
    return loss, counts, n, mean, grad


def _bounds(s, score, mean, grad_only=False):
    """Relative roundings of one p: the exponent's argument (its magnitude times 2^-24), two ulps of the
    exponential, up to 16 additions in a lane and 6 across the wave, the division: 48 and the argument's range."""
    z = s["logits"].double()
    z = torch.where(torch.isfinite(z), z, torch.zeros_like(z))
    reach = float((z.amax(1) - z.amin(1)).max()) if z.numel() else 0.0
    return (48 + reach) * EPS32


def _run(d, score, **kw):
    o = moe.moe_balance_loss(d["logits"], d["topk_idx"], score=score, token_mask=d["token_mask"],
                             seq_offsets=d["seq_offsets"], **kw)
    g = moe.moe_balance_loss_backward(d["grad_loss"], d["logits"], o["counts"], o["seq_tokens"],
                                      d["topk_idx"].shape[1], score=score, token_mask=d["token_mask"],
                                      seq_offsets=d["seq_offsets"], stream=kw.get("stream"))
    return o, g


def _gpu(s):
    return {k: v.cuda() if v is not None else None for k, v in s.items()}


def _check(s, o, grad, score):
    loss, counts, n, mean, want = _want(s, score)
    assert torch.equal(o["counts"].cpu(), counts)
    assert torch.equal(o["seq_tokens"].cpu(), n)
    p_unit = _bounds(s, score, mean)
    tokens = n.double()[:, None]
    unit = p_unit + (tokens + 8) * EPS32  # a sum of n terms, however ordered
    got = o["prob_mean"].double().cpu()
    assert ((got - mean).abs() <= unit * mean + 1e-44).all(), float(((got - mean).abs() / mean.clamp_min(1e-30)).max())
    E = counts.shape[1]
    lb = ((unit[:, 0]) + (E + 8) * EPS32) * loss.abs()
    assert ((o["loss"].double().cpu() - loss).abs() <= lb + 1e-44).all()
    # |p_j| (|a_j| + sum |a| p), a = |grad| E / (K n^2) c
    K = s["topk_idx"].shape[1]
    bound = torch.zeros_like(want)
    for q, rows in _seqs(s):
        if not rows.numel():
            continue
        a = s["grad_loss"][q].double().abs() * E / (K * rows.numel() ** 2) * counts[q].double()
        p = _probs64(s["logits"][rows].double(), score)
        bound[rows] = p * (a + (a * p).sum(1, keepdim=True))
    bound = (4 * p_unit + 64 * EPS32) * bound + 1e-44
    assert grad.dtype == s["logits"].dtype
    if grad.dtype == BF16:
        bound = bound + EPS16 * (want.abs() + bound)
    err = (grad.double().cpu() - want).abs()
    assert (err <= bound).all(), float((err / bound).max())


SHAPES = [(1, 1, 1), (1, 2, 1), (5, 16, 2), (64, 16, 2), (9, 64, 6), (3, 61, 4), (130, 128, 8), (700, 60, 4),
          (77, 256, 8), (2049, 256, 8), (513, 300, 8), (40, 512, 16), (33, 1000, 1), (21, 1024, 16)]


@pytest.mark.parametrize("T,E,K", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_one_sequence(T, E, K, score, dtype):
    _log(f"T={T} E={E} K={K} {score} {dtype}")
    s = _inputs(T, E, K, dtype)
    o, g = _run(_gpu(s), score)
    _check(s, o, g, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("cuts", [
    [0, 0], [0, 700], [3, 3, 3, 3], [0, 1, 2, 3, 700], [0, 0, 350, 350, 350, 700, 700], [10, 20, 690],
    list(range(0, 701, 7)), sorted([0, 700] + [(37 * i * i) % 700 for i in range(60)]), [0] * 200 + [700],
    [0] + [8 * i for i in range(70)] + [700] * 3])
def test_packed_sequences(cuts, score):
    """Empty sequences, one-token ones, cuts at and beside the chunks' edges, tokens before and after all of them."""
    _log(f"cuts={cuts[:8]}... {score}")
    for masked, E, K in ((0.0, 64, 4), (0.3, 61, 4)):
        s = _inputs(700, E, K, cuts=cuts, masked=masked, seed=1)
        o, g = _run(_gpu(s), score)
        _check(s, o, g, score)


def test_many_tokens_and_sequences():
    T = 40000
    g = torch.Generator().manual_seed(3)
    cuts = sorted(torch.randint(0, T + 1, (2000,), generator=g).tolist())
    for dtype, cut in ((F32, None), (BF16, cuts)):
        _log(f"T={T} {dtype} sequences={1 if cut is None else len(cut) - 1}")
        s = _inputs(T, 32, 2, dtype, cuts=cut, masked=0.1, seed=2)
        o, grad = _run(_gpu(s), "softmax")
        _check(s, o, grad, "softmax")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_tokens_hold_anything(score):
    s = _inputs(300, 61, 4, cuts=[0, 100, 100, 250], masked=0.4, seed=4)
    d = _gpu(s)
    o, g = _run(d, score)
    junk = {**d, "logits": d["logits"].clone(), "topk_idx": d["topk_idx"].clone()}
    off = ~d["token_mask"]
    off[250:] = True  # in no sequence
    for k, v in enumerate((float("nan"), float("inf"), float("-inf"), 3e38)):
        junk["logits"][off.nonzero().flatten()[k::4]] = v
    junk["topk_idx"][off] = -(1 << 62)
    o2, g2 = _run(junk, score)
    for k in o:
        assert torch.equal(o[k], o2[k]), k
    assert torch.equal(g, g2) and torch.equal(g[off], torch.zeros_like(g[off]))
    # every token masked
    none = {**d, "token_mask": torch.zeros(300, dtype=torch.bool, device="cuda")}
    o3, g3 = _run(none, score)
    assert all(int(v.count_nonzero()) == 0 for v in (*o3.values(), g3))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_infinities_extremes_and_strange_ids(score):
    s = _inputs(40, 48, 4, seed=5)
    z = s["logits"]
    z[:, 5] = float("-inf")          # an expert switched off
    z[3] = float("-inf")             # a row of nothing: p = 0, still a token
    z[4] = -3.4028234663852886e38    # the type's lowest value throughout: an even row
    z[6] = -200.0 + z[6]             # sigmoids far below the smallest number
    z[6, 5] = float("-inf")
    z[7] = 90.0
    z[8, 2] = 1e30
    s["topk_idx"][9] = torch.tensor([7, 7, 7, 7])            # repeated ids count each time
    s["topk_idx"][10] = torch.tensor([-1, 48, 1 << 40, -(1 << 40)])
    d = _gpu(s)
    o, g = _run(d, score)
    ref = {**s, "logits": z.clone()}
    ref["logits"][3] = 0
    ref["logits"][4] = 0  # the same p as any even row, in 64 bits too
    loss, counts, n, mean, want = _want({**ref, "logits": ref["logits"]}, score)
    p3 = _probs64(ref["logits"][3:4].double(), score)[0] / 40
    assert torch.equal(o["counts"].cpu(), counts) and int(o["seq_tokens"]) == 40
    got = o["prob_mean"][0].double().cpu()
    assert (got - (mean[0] - p3)).abs().max() <= 1e-6  # 48 + 40 roundings of numbers below 1
    assert torch.isfinite(g).all()
    off = torch.tensor([t for t in range(40) if t not in (4, 7)], device="cuda")  # those two hold numbers there
    assert int(g[3].count_nonzero()) == 0 and int(g[off, 5].count_nonzero()) == 0
    for t in (6, 8):
        assert (g[t].double().cpu() - want[t]).norm() <= 1e-5 * want[t].norm() + 1e-12, t
    # a NaN makes its row's p NaN, and so its sequence's sums
    d["logits"][11, 1] = float("nan")
    d["seq_offsets"] = torch.tensor([0, 11, 12, 40], dtype=torch.int32, device="cuda")
    d["grad_loss"] = torch.ones(3, device="cuda")
    o, g = _run(d, score)
    assert torch.isnan(o["loss"][1]) and torch.isfinite(o["loss"][[0, 2]]).all()
    assert torch.isnan(g[11]).all() and torch.isfinite(g[:11]).all() and torch.isfinite(g[12:]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("E", [64, 100, 256])
def test_strided_rows(dtype, E):
    s = _inputs(70, E, 4, dtype, seed=6)
    d = _gpu(s)
    want, gwant = _run(d, "softmax")
    for offset, stride in ((0, E + 8), (16, 2 * E), (1, E + 3), (5, E)):
        wide = torch.full((70 * 2 * E + 64,), float("nan"), dtype=dtype, device="cuda")
        view = wide.as_strided((70, E), (stride, 1), offset)
        view.copy_(d["logits"])
        o, g = _run({**d, "logits": view}, "softmax")
        assert torch.equal(o["counts"], want["counts"])
        for a, b in ((o["prob_mean"], want["prob_mean"]), (o["loss"], want["loss"]), (g, gwant)):
            lim = (EPS16 if b.dtype == BF16 else 100 * EPS32) * b.float().abs().max()
            assert (a.float() - b.float()).abs().max() <= lim


def test_gradient_against_differences():
    for score in ("softmax", "sigmoid"):
        s = _inputs(50, 20, 3, cuts=[0, 20, 20, 45], masked=0.2, seed=7)
        _, g = _run(_gpu(s), score)
        v = torch.randn(50, 20, generator=torch.Generator().manual_seed(8)).double()

        def at(h):
            return float((_want({**s, "logits": s["logits"].double() + h * v}, score)[0] *
                          s["grad_loss"].double()).sum())

        h = 1e-5
        slope = (at(h) - at(-h)) / (2 * h)
        got = float((g.double().cpu() * v).sum())
        # the differences' own error: h^2 and 1e-16 / h of the loss
        assert abs(slope - got) <= 1e-6 * float((g.double().cpu() * v).abs().sum()) + 1e-9


def test_no_tokens_and_offsets_out_of_range():
    d = _gpu(_inputs(0, 16, 2, cuts=[0, 0, 0]))
    d["grad_loss"] = torch.ones(2, device="cuda")
    for k, v in moe.moe_balance_loss(d["logits"], d["topk_idx"], seq_offsets=d["seq_offsets"]).items():
        assert int(v.count_nonzero()) == 0, k
    o, g = _run(d, "softmax")
    assert g.shape == (0, 16)
    # offsets outside [0, T] are clamped to it
    s = _inputs(90, 16, 2, cuts=[0, 30, 90], seed=9)
    d = _gpu(s)
    o, g = _run(d, "softmax")
    d["seq_offsets"] = torch.tensor([-5, 30, 1 << 30], dtype=torch.int32, device="cuda")
    o2, g2 = _run(d, "softmax")
    assert all(torch.equal(o[k], o2[k]) for k in o) and torch.equal(g, g2)


def test_same_bits_each_time_and_on_another_stream():
    d = _gpu(_inputs(5000, 256, 8, cuts=[0, 100, 100, 3000, 5000], masked=0.1, seed=10))
    o, g = _run(d, "sigmoid")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        o2, g2 = _run(d, "sigmoid", stream=st)
        st.synchronize()
        assert all(torch.equal(o[k], o2[k]) for k in o) and torch.equal(g, g2)


def test_workspace_may_hold_anything_and_outputs_stay_in_bounds():
    s = _inputs(333, 61, 4, cuts=[0, 50, 50, 333], seed=11)
    d = _gpu(s)
    want, gw = _run(d, "softmax")
    need = moe.moe_balance_loss_workspace_bytes(333, 61, 3)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    out = {"loss": torch.full((3 + 8,), 7.0, device="cuda"),
           "counts": torch.full((3 * 61 + 8,), 7, dtype=torch.int32, device="cuda"),
           "seq_tokens": torch.full((3 + 8,), 7, dtype=torch.int32, device="cuda"),
           "prob_mean": torch.full((3 * 61 + 8,), 7.0, device="cuda")}
    views = {"loss": out["loss"][4:7], "counts": out["counts"][4:-4].view(3, 61), "seq_tokens": out["seq_tokens"][4:7],
             "prob_mean": out["prob_mean"][4:-4].view(3, 61)}
    o, g = _run(d, "softmax", workspace=ws[:need], out=views)
    assert all(torch.equal(want[k], o[k]) for k in want)
    assert (ws[need:] == 0xFF).all()
    for v in out.values():
        assert (v[:4] == 7).all() and (v[-4:] == 7).all()


def test_binding_refusals():
    d = _gpu(_inputs(8, 16, 2))
    z, ids = d["logits"], d["topk_idx"]
    for args, kw in (((z.half(), ids), {}), ((z, ids.int()), {}), ((z, ids[:4]), {}), ((z, ids), {"score": "relu"}),
                     ((z.t(), ids), {}), ((z, ids), {"token_mask": torch.ones(8, device="cuda")}),
                     ((z, ids), {"token_mask": torch.ones(7, dtype=torch.bool, device="cuda")}),
                     ((z, ids), {"seq_offsets": torch.zeros(1, dtype=torch.int32, device="cuda")}),
                     ((z, ids), {"seq_offsets": torch.zeros(2, dtype=torch.int64, device="cuda")}),
                     ((z, ids.cpu()), {}), ((z.cpu(), ids), {})):
        with pytest.raises(ValueError):
            moe.moe_balance_loss(*args, **kw)
    with pytest.raises(moe.MoeError, match="WORKSPACE"):
        moe.moe_balance_loss(z, ids, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(moe.MoeError, match="INVALID"):
        moe.moe_balance_loss(torch.zeros(2, 1025, device="cuda"), torch.zeros(2, 1, dtype=torch.int64, device="cuda"))
    o = moe.moe_balance_loss(z, ids)
    for kw in (dict(grad_loss=torch.ones(2, device="cuda")), dict(counts=o["counts"].long()),
               dict(seq_tokens=o["seq_tokens"].cpu()), dict(out=torch.empty(8, 16, dtype=BF16, device="cuda"))):
        args = dict(grad_loss=d["grad_loss"], logits=z, counts=o["counts"], seq_tokens=o["seq_tokens"], num_topk=2)
        args.update(kw)
        with pytest.raises(ValueError):
            moe.moe_balance_loss_backward(**args)


def test_in_a_graph():
    d = _gpu(_inputs(500, 256, 8, cuts=[0, 200, 200, 500], masked=0.1, seed=12))
    ws = torch.empty(moe.moe_balance_loss_workspace_bytes(500, 256, 3), dtype=torch.uint8, device="cuda")
    out, _ = _run(d, "sigmoid", workspace=ws)
    grad = torch.empty_like(d["logits"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_balance_loss(d["logits"], d["topk_idx"], score="sigmoid", token_mask=d["token_mask"],
                             seq_offsets=d["seq_offsets"], workspace=ws, out=out)
        moe.moe_balance_loss_backward(d["grad_loss"], d["logits"], out["counts"], out["seq_tokens"], 8,
                                      score="sigmoid", token_mask=d["token_mask"], seq_offsets=d["seq_offsets"],
                                      out=grad)
    for k in range(3):
        new = _gpu(_inputs(500, 256, 8, cuts=[0, 10 * k, 300, 500], masked=0.2, seed=30 + k))
        for key in d:
            d[key].copy_(new[key])
        graph.replay()
        torch.cuda.synchronize()
        want, gw = _run(d, "sigmoid")
        torch.cuda.synchronize()
        assert all(torch.equal(out[key], want[key]) for key in want) and torch.equal(grad, gw)


def test_more_than_2_to_31_elements():
    """2100000 x 1024 logits in two sequences: the last 50 tokens' gradient and counts are those of these alone."""
    T, E = 2100000, 1024
    _log("2.2e9 logits")
    g = torch.Generator(device="cuda").manual_seed(13)
    z = torch.empty(T, E, dtype=BF16, device="cuda").normal_(generator=g)
    ids = torch.randint(0, E, (T, 2), generator=g, device="cuda")
    off = torch.tensor([0, T - 50, T], dtype=torch.int32, device="cuda")
    one = torch.ones(2, device="cuda")
    o = moe.moe_balance_loss(z, ids, seq_offsets=off)
    grad = moe.moe_balance_loss_backward(one, z, o["counts"], o["seq_tokens"], 2, seq_offsets=off)
    few = moe.moe_balance_loss(z[-50:].clone(), ids[-50:].clone())
    alone = moe.moe_balance_loss_backward(one[:1], z[-50:].clone(), few["counts"], few["seq_tokens"], 2)
    assert o["seq_tokens"].tolist() == [T - 50, 50]
    assert torch.equal(o["counts"][1], few["counts"][0])
    assert torch.equal(o["counts"][0], torch.bincount(ids[:-50].flatten(), minlength=E).int())
    assert abs(float(o["loss"][1] - few["loss"][0])) <= 1e-5 * float(few["loss"][0])  # other order of 50 additions
    assert torch.equal(grad[-50:], alone)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("center", [-59.0, -40.0, -20.0, -4.0, 4.0])
def test_sigmoid_scores_of_low_rows(dtype, center):
    """One token's p.  A score takes an exponential (1 ulp and half of one), 1 + t, its reciprocal (1 ulp) and a
    product: at most 7 roundings of 2^-24, 7 / sqrt(3) in the mean square over the experts.  What all of a row share is
    the sum's error: some 20 additions, whose roundings meet at random (20 ** 0.5 / sqrt(3)), and four factors.  All
    of it stays below 8 roundings in the mean square; the argument's size must not enter."""
    E = 256
    g = torch.Generator().manual_seed(7)
    z = (center + 0.5 * torch.randn(8, E, generator=g)).to(dtype)
    assert float(z.max(1).values.min()) > -60
    off = torch.arange(9, dtype=torch.int32)
    o = moe.moe_balance_loss(z.cuda(), z.float().topk(4, 1).indices.cuda(), score="sigmoid", seq_offsets=off.cuda())
    want = _probs64(z.double(), "sigmoid")
    err = (o["prob_mean"].double().cpu() / want - 1).square().mean(1).sqrt()
    _log(f"sigmoid near {center} {dtype}: {float(err.max()) / EPS32:.2f} roundings")
    assert float(err.max()) <= 8 * EPS32


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("E", [17, 20, 24, 32, 40, 48, 63, 64])
def test_rows_of_few_experts(E, dtype, score):
    """Whole vectors of logits and single values, a row's vectors on some of its lanes."""
    s = _inputs(300, E, 4, dtype, cuts=[0, 130, 131, 290], masked=0.1, seed=E)
    o, g = _run(_gpu(s), score)
    _check(s, o, g, score)


@pytest.mark.parametrize("T,E,short", [(33000, 64, 16), (33000, 64, 60), (9000, 1024, 20), (5000, 256, 300)])
def test_a_long_sequence_beside_short_ones(T, E, short):
    """One sequence with most of the chunks' slots, and short ones before and after it."""
    _log(f"T={T} E={E} short={short}")
    half = short // 2
    cuts = list(range(0, 3 * half + 1, 3)) + list(range(T - 5 * (short - half), T + 1, 5))
    s = _inputs(T, E, 4, F32, cuts=cuts, masked=0.05, seed=short)
    assert s["grad_loss"].numel() == short + 1
    o, g = _run(_gpu(s), "softmax")
    _check(s, o, g, "softmax")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_rows_of_1024_experts(dtype):
    """The most LDS that a workgroup takes."""
    s = _inputs(4200, 1024, 8, dtype, seed=12)
    o, g = _run(_gpu(s), "sigmoid")
    _check(s, o, g, "sigmoid")


def test_outputs_under_another_default_type():
    """torch's default type has no say in the loss's and the means' type."""
    d = _gpu(_inputs(500, 64, 4, cuts=[0, 200, 500]))
    want, gwant = _run(d, "softmax")
    torch.set_default_dtype(BF16)
    try:
        got, grad = _run(d, "softmax")
    finally:
        torch.set_default_dtype(F32)
    assert all(got[k].dtype == want[k].dtype and torch.equal(got[k], want[k]) for k in want)
    assert torch.equal(grad, gwant)


@pytest.mark.parametrize("T,E,S", [(32768, 256, 1), (40000, 61, 3), (64, 16, 1), (3000, 1000, 8), (20000, 32, 200)])
def test_without_the_means(T, E, S):
    """Outputs without prob_mean, in one, two and three launches, and a workspace of exactly the bytes asked for."""
    cuts = [T * i // S for i in range(S + 1)]
    d = _gpu(_inputs(T, E, 4, cuts=cuts, seed=S))
    want = moe.moe_balance_loss(d["logits"], d["topk_idx"], seq_offsets=d["seq_offsets"])
    out = {k: torch.empty_like(v) for k, v in want.items() if k != "prob_mean"}
    need = moe.moe_balance_loss_workspace_bytes(T, E, S)
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    moe.moe_balance_loss(d["logits"], d["topk_idx"], seq_offsets=d["seq_offsets"], out=out, workspace=ws[:need])
    assert all(torch.equal(out[k], want[k]) for k in out)
    assert (ws[need:] == 0xFF).all()
