"""moe_expert_matvec against the products in 64 bits (host), with the bound of an fp32 sum rounded once to bf16."""
import sys

import pytest
import torch

import moe_routing_fp8_amd as moe

pytestmark = pytest.mark.gpu

EPS32 = 2.0 ** -24
EPS16 = 2.0 ** -8
VALUES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                      dtype=torch.float64)


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def _log(msg):
    sys.__stderr__.write(f"[gpu-matvec] {msg}\n")
    sys.__stderr__.flush()


def _inputs(counts, N, K, x="bf16", group=32, sf="ue8m0", tokens=None, seed=0, lead=0, tail=0):
    """`counts` rows for each expert after `lead` rows of none and before `tail` more; `tokens`: rows of x, reached
    through row_token (some -1)."""
    g = torch.Generator().manual_seed(seed * 101 + N * 7 + K)
    E = len(counts)
    off = torch.tensor([lead] + counts, dtype=torch.int64).cumsum(0).to(torch.int32)
    R = int(off[-1]) + tail
    s = {"expert_offsets": off, "row_token": None, "x_sf": None, "rows": R}
    if tokens is not None:
        s["row_token"] = torch.randint(-1, tokens, (R,), generator=g, dtype=torch.int32)
    X = tokens if tokens is not None else R
    v = torch.randn(X, K, generator=g)
    if x == "e4m3":
        b = v.view(X, K // 128, 128)
        s["x_sf"] = b.abs().amax(2).clamp_min(1e-4) / 448
        s["x"] = (b / s["x_sf"].unsqueeze(2)).view(X, K).to(torch.float8_e4m3fn)
    else:
        s["x"] = v.to(torch.bfloat16)
    s["w"] = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8)
    if sf == "ue8m0":
        s["w_sf"] = torch.randint(110, 130, (E, N, K // group), generator=g, dtype=torch.uint8)
    else:
        s["w_sf"] = torch.rand(E, N, K // group, generator=g) + 0.01
    return s


def _x64(s):
    x = s["x"].double()
    if s["x_sf"] is not None:
        x = (x.view(x.shape[0], x.shape[1] // 128, 128) * s["x_sf"].double().unsqueeze(2)).view(x.shape)
    return x


def _want(s):
    """The sums and the sums of magnitudes, rows of no expert NaN."""
    x = _x64(s)
    E, N, K2 = s["w"].shape
    if s["row_token"] is not None:
        t = s["row_token"].long()
        ok = (t >= 0) & (t < x.shape[0])
        x = torch.where(ok[:, None], x[t.clamp(0, max(0, x.shape[0] - 1))], 0.0)
    out = torch.full((s["rows"], N), float("nan"), dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(out)
    off = s["expert_offsets"].tolist()
    for e in range(E):
        if off[e + 1] <= off[e]:
            continue
        w = VALUES.to(x.device)[torch.stack([s["w"][e] & 15, s["w"][e] >> 4], 2).view(N, 2 * K2).long()]
        sf = s["w_sf"][e].double()
        if s["w_sf"].dtype == torch.uint8:
            sf = torch.pow(2.0, sf - 127)
        w = w * sf.repeat_interleave(2 * K2 // sf.shape[1], 1)
        r = slice(off[e], off[e + 1])
        out[r], mag[r] = x[r] @ w.T, x[r].abs() @ w.abs().T
    return out, mag


def _call(s, **kw):
    c = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    return moe.moe_expert_matvec(c["x"], c["w"], c["w_sf"], x_sf=c["x_sf"], expert_offsets=c["expert_offsets"],
                                 row_token=c["row_token"], **kw)


def _check(s, guard=True):
    R, (E, N, K2) = s["rows"], s["w"].shape
    whole = torch.full((R * N + 256,), 7.0, dtype=torch.bfloat16, device="cuda")
    got = _call(s, out=whole[128:128 + R * N].view(R, N))
    want, mag = _want(s)
    got = got.double().cpu()
    none = torch.isnan(want).all(1)
    assert (got[none] == 7).all()  # rows of no expert keep what was there
    assert (whole[:128] == 7).all() and (whole[128 + R * N:] == 7).all()
    got, want, mag = got[~none], want[~none], mag[~none]
    bound = (2 * K2 + 16) * EPS32 * mag  # an fp32 sum of K products and its few factors, however ordered
    bound = bound + EPS16 * (want.abs() + bound)
    bad = (got - want).abs() > bound
    assert not bad.any(), (int(bad.sum()), float((got - want).abs().max()))


FORMATS = [("bf16", 32, "ue8m0"), ("bf16", 128, "ue8m0"), ("bf16", 32, "f32"), ("bf16", 128, "f32"),
           ("e4m3", 32, "ue8m0"), ("e4m3", 128, "ue8m0"), ("e4m3", 32, "f32"), ("e4m3", 128, "f32")]


@pytest.mark.parametrize("x,group,sf", FORMATS)
@pytest.mark.parametrize("N,K", [(1, 128), (16, 128), (17, 256), (33, 384), (64, 2048), (100, 640), (257, 7168),
                                 (7, 1152)])
def test_formats_and_widths(x, group, sf, N, K):
    _log(f"{x} {group} {sf} N={N} K={K}")
    _check(_inputs([3, 0, 1, 18, 5], N, K, x, group, sf))


@pytest.mark.parametrize("sf", ["ue8m0", "f32"])
@pytest.mark.parametrize("K", [32, 64, 96, 160, 224, 992, 1056])
def test_rows_that_end_inside_a_step(sf, K):
    _log(f"K={K} {sf}")
    _check(_inputs([2, 17, 0, 1], 50, K, "bf16", 32, sf))


@pytest.mark.parametrize("rows", [1, 2, 7, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 128, 129, 300])
@pytest.mark.parametrize("x,group,sf", [("bf16", 32, "ue8m0"), ("e4m3", 32, "ue8m0"), ("bf16", 32, "f32"),
                                        ("e4m3", 128, "f32")])
def test_rows_of_one_matrix(rows, x, group, sf):
    """One matrix without offsets, given as [N, K/2]."""
    _log(f"rows={rows} {x} {group} {sf}")
    s = _inputs([rows], 70, 512, x, group, sf, seed=rows)
    want, mag = _want(s)
    s.update(expert_offsets=None, w=s["w"][0], w_sf=s["w_sf"][0])
    got = _call(s).double().cpu()
    bound = (512 + 16) * EPS32 * mag
    assert ((got - want).abs() <= bound + EPS16 * (want.abs() + bound)).all()


@pytest.mark.parametrize("counts", [[2, 3, 1, 2], [4, 12, 0, 4], [17, 1, 0, 2], [5, 33, 9, 16], [70, 4, 8, 1]])
@pytest.mark.parametrize("x,group,sf", FORMATS)
def test_many_columns(counts, x, group, sf):
    """So many tiles that each wave has one of its own: several blocks of k, few rows and many, the last tiles past
    the columns."""
    for K in (1024, 1536):
        _log(f"many columns {counts} {x} {group} {sf} K={K}")
        s = _inputs(counts, 16400, K, x, group, sf, seed=sum(counts), tokens=9 if K == 1536 else None)
        d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
        want, mag = _want(d)
        got = _call(s).double()
        bound = (K + 16) * EPS32 * mag
        assert ((got - want).abs() <= bound + EPS16 * (want.abs() + bound)).all()


@pytest.mark.parametrize("x,group,sf", FORMATS)
@pytest.mark.parametrize("K", [512, 1024, 2048, 4096, 2176])
def test_few_columns(x, group, sf, K):
    """So few tiles that waves split k, in one, two and four shares, even and not."""
    for counts in ([1], [3, 0, 6], [20, 2], [40]):
        for N in (33, 2100):
            _log(f"few columns {counts} {x} {group} {sf} K={K} N={N}")
            s = _inputs(counts, N, K, x, group, sf, seed=K)
            d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
            want, mag = _want(d)
            got = _call(s).double()
            bound = (K + 16) * EPS32 * mag
            assert ((got - want).abs() <= bound + EPS16 * (want.abs() + bound)).all()


@pytest.mark.parametrize("x,group,sf", FORMATS)
@pytest.mark.parametrize("N,K", [(2050, 2048), (8200, 512), (130, 640)])
def test_more_rows_than_one_pass_takes(x, group, sf, N, K):
    """An expert's passes side by side and in turn, beside experts with few rows or none."""
    for counts in ([72], [500], [300, 0, 9]):
        _log(f"passes {counts} {x} {group} {sf} K={K} N={N}")
        s = _inputs(counts, N, K, x, group, sf, seed=N)
        d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
        want, mag = _want(d)
        got = _call(s).double()
        bound = (K + 16) * EPS32 * mag
        assert ((got - want).abs() <= bound + EPS16 * (want.abs() + bound)).all()


@pytest.mark.parametrize("x", ["bf16", "e4m3"])
def test_expert_loads(x):
    """Experts without rows at either end and between, one expert with everything, rows of no expert around."""
    for counts in ([0, 0, 5], [5, 0, 0], [0] * 70 + [2] + [0] * 70 + [40] + [0] * 9, [1] * 130, [0, 200, 0, 1],
                   [0, 0, 0]):
        for lead, tail in ((0, 0), (2, 3)):
            _log(f"{x} counts={counts[:6]}... {lead} {tail}")
            _check(_inputs(counts, 40, 256, x, lead=lead, tail=tail))


def test_1024_experts():
    _check(_inputs([i % 3 if i % 5 == 0 else 0 for i in range(1024)], 16, 128, "bf16"))


@pytest.mark.parametrize("x,group,sf", [("bf16", 32, "ue8m0"), ("e4m3", 32, "ue8m0"), ("bf16", 128, "f32")])
def test_rows_through_row_token(x, group, sf):
    """Rows gathered by token; -1 gives zeros.  Ids past the rows of x count as -1."""
    s = _inputs([4, 0, 20, 1, 7], 48, 512, x, group, sf, tokens=6, seed=3)
    s["row_token"][2] = -1
    s["row_token"][3] = 6
    s["row_token"][5] = -(1 << 31)
    s["row_token"][6] = (1 << 31) - 1
    _check(s)
    got = _call(s)
    assert int(got[[2, 3, 5, 6]].count_nonzero()) == 0
    # no row of x at all
    s = _inputs([2, 1], 16, 128, x, group, sf, tokens=0)
    assert int(_call(s).count_nonzero()) == 0


def test_every_code_and_scale():
    """One-hot rows read single weights back: every code under every scale whose product bf16 holds."""
    K, group = 512, 32
    G = K // group
    for base in range(0, 256, 16):
        sf = torch.arange(base, base + 16, dtype=torch.uint8).view(1, 1, G).expand(1, 2, G).contiguous()
        codes = torch.arange(K, dtype=torch.int64) % 16
        row = (codes[0::2] | (codes[1::2] << 4)).to(torch.uint8)
        s = {"w": row.view(1, 1, K // 2).expand(1, 2, K // 2).contiguous(), "w_sf": sf, "x_sf": None,
             "row_token": None, "expert_offsets": None, "x": torch.eye(K, dtype=torch.bfloat16)}
        got = _call(s)[:, 0].float().cpu()
        want = (VALUES[codes] * torch.pow(2.0, sf[0, 0].double() - 127).repeat_interleave(group)).to(torch.bfloat16)
        nan = sf[0, 0].repeat_interleave(group) == 255
        # 255 is UE8M0's NaN: a row whose group it scales is NaN, whatever its x
        if base == 240:
            assert torch.isnan(got).all()
            continue
        keep = ~nan & (want.float().abs() >= 2.0 ** -126)
        assert torch.equal(got[keep], want.float()[keep]), base


def test_infinite_and_nan_rows_stay_alone():
    s = _inputs([3, 2], 20, 256, "bf16", seed=5)
    clean = _call(s)
    s["x"][1, 7] = float("nan")
    s["x"][3, 9] = float("inf")
    got = _call(s)
    assert torch.isnan(got[1]).all()
    assert not torch.isfinite(got[3].float()).any()  # inf times a nonzero weight, or inf times 0
    for r in (0, 2, 4):
        assert torch.equal(got[r], clean[r])


def test_as_the_dispatch_uses_it():
    """The framework's own quantised rows and weights: expand, gate and up, SwiGLU, down, combine."""
    T, E, K, H, I = 24, 16, 2, 256, 128
    g = torch.Generator(device="cuda").manual_seed(11)
    scores = torch.randn(T, E, generator=g, device="cuda")
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    w1 = (torch.randn(E * 2 * I, H, generator=g, device="cuda") / H ** 0.5).to(torch.bfloat16)
    q1, sf1, _ = moe.moe_expand_cast(w1, dtype="e2m1", group_size=32, round_sf=True, sf_ue8m0=True)
    q1, sf1 = q1.view(E, 2 * I, H // 2), sf1.view(E, 2 * I, H // 32)
    d = moe.moe_dispatch(scores, x, K, renormalize=True)
    up = moe.moe_expert_matvec(d["out"], q1, sf1, x_sf=d["out_sf"], expert_offsets=d["offsets"])
    s = {"x": d["out"].cpu(), "x_sf": d["out_sf"].cpu(), "w": q1.cpu(), "w_sf": sf1.cpu(), "row_token": None,
         "expert_offsets": d["offsets"].cpu(), "rows": T * K}
    want, mag = _want(s)
    bound = (H + 16) * EPS32 * mag
    assert ((up.double().cpu() - want).abs() <= bound + EPS16 * (want.abs() + bound)).all()
    # without the expand, from the token rows themselves: the same rows within the e4m3 cast's error
    direct = moe.moe_expert_matvec(x, q1, sf1, expert_offsets=d["offsets"], row_token=d["row_token"])
    assert (direct.float() - up.float()).norm() <= 0.06 * direct.float().norm()  # e4m3: 2^-4 at most per value


def test_same_bits_each_time_and_on_another_stream():
    s = _inputs([9, 0, 30, 2], 100, 1024, "e4m3", seed=6)
    first = _call(s)
    c = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        again = moe.moe_expert_matvec(c["x"], c["w"], c["w_sf"], x_sf=c["x_sf"], expert_offsets=c["expert_offsets"],
                                      stream=st)
        st.synchronize()
        assert torch.equal(first, again)


def test_offsets_past_32_bits():
    """A weight tensor of more than 2^32 bytes: the last expert's rows."""
    E, N, K = 40, 16384, 16384  # 5.4 GB of codes
    w = torch.zeros(E, N, K // 2, dtype=torch.uint8, device="cuda")
    sf = torch.full((E, N, K // 32), 127, dtype=torch.uint8, device="cuda")
    w[-1, :, 0] = 0x02           # w[-1, n, 0] = 1
    w[-1, -1, -1] = 0x50         # w[-1, N-1, K-1] = 3
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[-1] = 1
    x = torch.ones(1, K, dtype=torch.bfloat16, device="cuda")
    _log("5.4 GB of codes")
    got = moe.moe_expert_matvec(x, w, sf, expert_offsets=off)
    assert (got[0, :-1] == 1).all() and float(got[0, -1]) == 4.0


def test_no_rows():
    s = _inputs([0, 0], 8, 128)
    assert _call(s).shape == (0, 8)


def test_binding_refusals():
    s = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in _inputs([3, 2], 20, 256).items()}
    e = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in _inputs([3, 2], 20, 256, "e4m3").items()}

    def call(base=s, **kw):
        a = {"x": base["x"], "w_codes": base["w"], "w_sf": base["w_sf"], "x_sf": base["x_sf"],
             "expert_offsets": base["expert_offsets"]}
        a.update(kw)
        return moe.moe_expert_matvec(**a)

    for kw in (dict(x=s["x"].float()), dict(x=s["x"].t()), dict(w_codes=s["w"][:, :, :64]), dict(w_sf=s["w_sf"][:1]),
               dict(w_sf=s["w_sf"][:, :, :3]), dict(w_sf=s["w_sf"].int()), dict(expert_offsets=None),
               dict(expert_offsets=s["expert_offsets"].long()), dict(expert_offsets=s["expert_offsets"][:2]),
               dict(x_sf=torch.ones(5, 2, device="cuda")), dict(row_token=torch.zeros(5, device="cuda")),
               dict(out=torch.empty(5, 19, dtype=torch.bfloat16, device="cuda")), dict(x=s["x"].cpu())):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(ValueError):
        call(e, x_sf=None)
    with pytest.raises(ValueError):
        call(e, x_sf=e["x_sf"][:, :1])
    with pytest.raises(moe.MoeError, match="UNSUPPORTED"):
        call(w_sf=torch.full((2, 20, 16), 127, dtype=torch.uint8, device="cuda"))  # groups of 16
    with pytest.raises(moe.MoeError, match="UNSUPPORTED"):
        call(w_sf=torch.full((2, 20, 4), 127, dtype=torch.uint8, device="cuda"))   # groups of 64
    flat = s["w"].flatten()
    with pytest.raises(moe.MoeError, match="INVALID"):  # codes not 16-byte aligned
        call(w_codes=flat[1:1 + 20 * 128].view(1, 20, 128), w_sf=s["w_sf"][:1], expert_offsets=None)


def test_in_a_graph():
    s = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in _inputs([9, 0, 30, 2], 100, 1024, "e4m3").items()}
    out = torch.empty(41, 100, dtype=torch.bfloat16, device="cuda")

    def go(**kw):
        return moe.moe_expert_matvec(s["x"], s["w"], s["w_sf"], x_sf=s["x_sf"], expert_offsets=s["expert_offsets"], **kw)

    go(out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(out=out)
    for k, counts in enumerate(([41, 0, 0, 0], [0, 1, 0, 40], [10, 10, 11, 10])):
        new = _inputs(counts, 100, 1024, "e4m3", seed=40 + k)
        for key in ("x", "x_sf", "w", "w_sf", "expert_offsets"):
            s[key].copy_(new[key])
        graph.replay()
        torch.cuda.synchronize()
        want = go()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("x", ["bf16", "e4m3"])
def test_no_rows_by_token(x):
    """A batch that reads five rows of x by token and has none of its own."""
    s = _inputs([0, 0], 8, 128, x, tokens=5)
    assert s["row_token"].numel() == 0
    assert _call(s).shape == (0, 8)
    s.update(expert_offsets=None, w=s["w"][:1], w_sf=s["w_sf"][:1])
    assert _call(s).shape == (0, 8)


@pytest.mark.parametrize("K", [512, 32])
def test_scale_bytes_at_the_ends(K):
    """Each code under the scale bytes whose products leave bf16's normal range, and under 255, by rows of weights with
    one code that is not zero; K = 32 takes the code for the last steps."""
    bytes_ = [0, 1, 2, 3, 126, 127, 252, 253, 254, 255]
    N = 16 * len(bytes_)
    w = torch.zeros(1, N, K // 2, dtype=torch.uint8)
    at = (torch.arange(N) * 13) % K
    code = torch.arange(N) % 16
    w[0, torch.arange(N), at // 2] = (code << (4 * (at % 2))).to(torch.uint8)
    sf = torch.full((1, N, K // 32), 127, dtype=torch.uint8)
    b = torch.tensor(bytes_, dtype=torch.uint8).repeat_interleave(16)
    sf[0, torch.arange(N), at // 32] = b
    for x in (1.0, -1.0, 2.0 ** -20, 2.0 ** 20):
        s = {"x": torch.full((3, K), x, dtype=torch.bfloat16), "x_sf": None, "row_token": None, "w": w, "w_sf": sf,
             "expert_offsets": None}
        got = _call(s).float().cpu()
        weight = VALUES[code] * torch.pow(2.0, b.double() - 127)
        weight = torch.where(weight.abs() >= 2.0 ** 128, weight.sign() * float("inf"), weight)
        want = (weight * x).float().to(torch.bfloat16).float()
        nan = b == 255
        assert torch.isnan(got[:, nan]).all()
        assert torch.equal(got[:, ~nan], want[~nan].expand(3, -1)), x
