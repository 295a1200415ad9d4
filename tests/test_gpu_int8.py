"""The 8-bit integer feed-forward: moe_cast_int8 bit for bit, swiglu_cast_int8 within the roundings of its arithmetic,
moe_expert_matmul_int8 bit for bit (its sums are whole numbers), and the run of them from the router to the combine."""
import sys

import pytest
import torch

import moe_routing_fp8_amd as moe

pytestmark = pytest.mark.gpu

EPS32 = 2.0 ** -24
BF16, F32, I8, I32 = torch.bfloat16, torch.float32, torch.int8, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def _log(msg):
    sys.__stderr__.write(f"[gpu-int8] {msg}\n")
    sys.__stderr__.flush()


def _gen(*seed):
    n = 17
    for s in seed:
        n = n * 7919 + s
    return torch.Generator().manual_seed(n % (1 << 31))


def _cast32(x):
    """The definition in fp32 on the host: every operation rounds once there too."""
    v = x.float()
    sf = v.abs().amax(1).clamp_min(127 * 2.0 ** -126) / 127
    return torch.round(v * (1 / sf)[:, None]).to(I8), sf


WIDTHS = [1, 7, 8, 63, 64, 200, 511, 512, 513, 1000, 2048, 2049, 4096, 5001, 7168, 8192, 8200, 20001]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H", WIDTHS)
def test_cast(H, dtype):
    g = _gen(H)
    x = torch.randn(9, H, generator=g)
    x[0] = 0.0
    x[1] *= 1e-38
    x[2] *= 1e30
    x[3, H // 2] = 300.0
    x[4] = -x[4].abs()
    x = x.to(dtype)
    q, sf = moe.moe_cast_int8(x.cuda())
    want, want_sf = _cast32(x)
    assert torch.equal(sf.cpu(), want_sf)
    assert torch.equal(q.cpu(), want)
    assert (q[0] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_cast_rows_of_a_wider_tensor(dtype):
    wide = torch.randn(12, 700, generator=_gen(5)).to(dtype).cuda()
    for lo, hi in ((0, 256), (4, 260), (1, 640), (3, 4)):
        q, sf = moe.moe_cast_int8(wide[:, lo:hi])
        want, want_sf = _cast32(wide[:, lo:hi].cpu())
        assert torch.equal(q.cpu(), want) and torch.equal(sf.cpu(), want_sf)


def _swiglu64(gu, w, clamp):
    l, u = gu.double().chunk(2, dim=1)
    if clamp > 0:
        l, u = l.clamp(max=clamp), u.clamp(-clamp, clamp)
    v = l * torch.sigmoid(l) * u
    return v if w is None else v * w.double()[:, None]


@pytest.mark.parametrize("I", [1, 5, 8, 64, 289, 512, 520, 2048, 2050, 4104, 9000])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("clamp", [0.0, 1.75])
def test_swiglu_cast(I, weighted, clamp):
    g = _gen(I, weighted)
    gu = (2 * torch.randn(7, 2 * I, generator=g)).to(BF16)
    gu[2] = 0.0
    w = torch.rand(7, generator=g) if weighted else None
    q, sf = moe.swiglu_cast_int8(gu.cuda(), None if w is None else w.cuda(), clamp_value=clamp)
    v = _swiglu64(gu, w, clamp)
    # the exponential 3 ulp, 1 + e, the reciprocal 1 ulp, three products: 16 roundings of v
    unit = 16 * EPS32
    want_sf = v.abs().amax(1).clamp_min(127 * 2.0 ** -126) / 127
    assert ((sf.double().cpu() - want_sf).abs() <= (unit + EPS32) * want_sf).all()
    # a code is off by half a step, the error of v, and the inverse scale's and the product's roundings
    err = (q.double().cpu() * sf.double().cpu()[:, None] - v).abs()
    assert (err <= sf.double().cpu()[:, None] * (0.5 + 127 * 3 * EPS32) + unit * v.abs()).all()
    assert (q[2] == 0).all()


def _offsets(counts):
    off = torch.zeros(len(counts) + 1, dtype=I32)
    off[1:] = torch.tensor(counts).cumsum(0)
    return off


def _product(x, x_sf, w, w_sf, off, row_token, dtype, R):
    E, N, K = w.shape
    out = torch.zeros(R, N, dtype=dtype)
    at = row_token.long() if row_token is not None else torch.arange(R)
    known = (at >= 0) & (at < x.shape[0])
    for e in range(E):
        rows = torch.arange(int(off[e]), int(off[e + 1]))
        if rows.numel() == 0:
            continue
        src = at[rows].clamp(0, max(x.shape[0] - 1, 0))
        if x.shape[0] == 0:
            continue
        sums = x[src].double() @ w[e].double().T   # whole numbers below 2^53
        y = (sums.float() * x_sf[src][:, None]) * w_sf[e]
        out[rows] = torch.where(known[rows][:, None], y, torch.zeros_like(y)).to(dtype)
    return out


def _case(counts, N, K, by_token=False, seed=0, X=None):
    g = _gen(N, K, sum(counts), seed)
    E, R = len(counts), sum(counts)
    row_token = None
    if by_token:
        X = X or max(1, R // 2)
        row_token = torch.randint(0, X, (R,), generator=g, dtype=I32)
    else:
        X = R
    x = torch.randint(-128, 128, (X, K), generator=g, dtype=I8)
    w = torch.randint(-128, 128, (E, N, K), generator=g, dtype=I8)
    return {"x": x, "x_sf": torch.rand(X, generator=g) + 0.1, "w": w, "w_sf": torch.rand(E, N, generator=g) - 0.5,
            "off": _offsets(counts), "row_token": row_token}


def _run(s, dtype=BF16, **kw):
    c = {k: v.cuda() if v is not None else None for k, v in s.items()}
    return moe.moe_expert_matmul_int8(c["x"], c["x_sf"], c["w"], c["w_sf"], expert_offsets=c["off"],
                                      row_token=c["row_token"], out_dtype=dtype, **kw)


def _check(s, dtype=BF16):
    R = int(s["off"][-1])
    y = _run(s, dtype)
    want = _product(s["x"], s["x_sf"], s["w"], s["w_sf"], s["off"], s["row_token"], dtype, R)
    assert y.dtype == dtype and torch.equal(y.cpu(), want), (y.cpu() != want).nonzero()[:4]


COUNTS = [[1], [0, 1, 0], [3, 0, 5, 1], [16, 17, 15], [33, 1, 64], [70, 0, 130], [200, 257], [600], [5] * 40]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("N,K", [(64, 128), (256, 256), (100, 640), (4, 16), (130, 2064)])
def test_product_in_whole_chunks(counts, N, K, dtype):
    _log(f"{counts} N={N} K={K} {dtype}")
    _check(_case(counts, N, K), dtype)
    _check(_case(counts, N, K, by_token=True, seed=1), dtype)


@pytest.mark.parametrize("counts", [[1], [0, 3, 20], [40, 0, 9], [300]])
@pytest.mark.parametrize("N,K", [(1, 1), (3, 7), (65, 15), (33, 17), (64, 130), (127, 259), (5, 1999)])
def test_product_at_odd_sizes(counts, N, K):
    _log(f"{counts} N={N} K={K}")
    _check(_case(counts, N, K), BF16)
    _check(_case(counts, N, K, by_token=True, seed=1), F32)


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 31, 33, 63, 65, 127, 128, 129, 255, 256, 257, 511, 513, 1024])
def test_product_row_counts(rows):
    """Every number of rows around the tiles' heights, of one matrix (no offsets) and beside another expert."""
    s = _case([rows], 192, 384, seed=rows)
    c = {k: v.cuda() if v is not None else None for k, v in s.items()}
    y = moe.moe_expert_matmul_int8(c["x"], c["x_sf"], c["w"][0], c["w_sf"][0])
    want = _product(s["x"], s["x_sf"], s["w"], s["w_sf"], s["off"], None, BF16, rows)
    assert torch.equal(y.cpu(), want)
    _check(_case([rows, 7], 320, 144, seed=rows), F32)


@pytest.mark.parametrize("channels", [1, 15, 16, 17, 63, 65, 127, 129, 255, 257, 1021])
def test_product_channel_counts(channels):
    _check(_case([9, 30], channels, 272), BF16)
    _check(_case([300, 280], channels, 160), BF16)


def test_uneven_experts():
    """One expert with nearly all rows, and 300 experts of which few have any."""
    _check(_case([0, 1, 900, 0, 2], 64, 128))
    counts = [0] * 300
    counts[0], counts[17], counts[255], counts[299] = 3, 40, 1, 9
    _check(_case(counts, 48, 96))
    _check(_case([1] * 1000 + [30] + [0] * 23, 16, 64))


def _device_check(s, dtype):
    """As _check, the whole-number sums as 64-bit products on the device."""
    c = {k: v.cuda() if v is not None else None for k, v in s.items()}
    R, N = int(s["off"][-1]), s["w"].shape[1]
    out = torch.full((R, N), 7.0, dtype=dtype, device="cuda")
    y = moe.moe_expert_matmul_int8(c["x"], c["x_sf"], c["w"], c["w_sf"], expert_offsets=c["off"],
                                   row_token=c["row_token"], out=out)
    at = c["row_token"].long() if c["row_token"] is not None else torch.arange(R, device="cuda")
    known = (at >= 0) & (at < c["x"].shape[0])
    at = at.clamp(0, c["x"].shape[0] - 1)
    ends = s["off"].tolist()
    for e in range(len(ends) - 1):
        rows = slice(ends[e], ends[e + 1])
        sums = c["x"][at[rows]].double() @ c["w"][e].double().t().contiguous()
        want = (sums.float() * c["x_sf"][at[rows], None]) * c["w_sf"][e]
        assert torch.equal(y[rows], torch.where(known[rows, None], want, 0.0).to(dtype)), e


# experts and channels for which each tile is chosen on 256 compute units: of 256 x 256, 192 x 256, 128 x 256, 64 x 128
# and 32 x 128; k of one step, of steps and a part, and of many steps
FORMS = [([9000, 0, 8500], 4104), ([0, 700, 200, 300, 1, 500, 250, 600], 5000), ([100, 40, 0, 190, 7] * 4, 3500),
         ([300, 310, 20, 500], 1700), ([129, 0, 33], 600), ([700] * 2 + [0] * 70 + [300] * 2, 2304)]


@pytest.mark.parametrize("counts,N", FORMS)
@pytest.mark.parametrize("K", [16, 128, 272, 656])
def test_product_in_every_tile(counts, N, K):
    _log(f"{counts} N={N} K={K}")
    _device_check(_case(counts, N, K), BF16)
    s = _case(counts, N, K, by_token=True, seed=1)
    s["row_token"][::97] = -1
    _device_check(s, F32)


@pytest.mark.parametrize("counts,N,K", [([700, 650], 1030, 33), ([125] * 16, 1000, 301), ([40, 0, 90], 200, 47)])
def test_product_in_every_tile_at_odd_sizes(counts, N, K):
    _device_check(_case(counts, N, K), BF16)
    _device_check(_case(counts, N, K, by_token=True, seed=1), F32)


def test_debug_mode_checks_activations(monkeypatch):
    x = torch.ones(4, 64, dtype=BF16, device="cuda")
    monkeypatch.setenv("MOE_FP8_DEBUG", "1")
    moe.moe_cast_int8(x)
    moe.swiglu_cast_int8(x)
    x[2, 7] = float("nan")
    for call in (moe.moe_cast_int8, moe.swiglu_cast_int8):
        with pytest.raises(ValueError, match="MOE_CHECK_NONFINITE_ACTIVATION"):
            call(x)


def test_two_streams_at_once():
    """Nothing is shared between calls: two sets of inputs in flight on two streams."""
    sets = [_case([300, 20, 500], 1024, 1024, by_token=True, seed=i) for i in range(2)]
    want = [_run(s) for s in sets]
    held = [{k: v.cuda() for k, v in s.items()} for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(5):
        for i, (c, stream) in enumerate(zip(held, streams)):
            got[i].append(moe.moe_expert_matmul_int8(c["x"], c["x_sf"], c["w"], c["w_sf"], expert_offsets=c["off"],
                                                     row_token=c["row_token"], stream=stream))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


def test_largest_codes_do_not_overflow():
    """-128 times -128 over the longest k: 131071 * 2^14 < 2^31."""
    K = 131071
    x = torch.full((2, K), -128, dtype=I8)
    w = torch.full((1, 3, K), -128, dtype=I8)
    w[0, 1] = 127
    s = {"x": x, "x_sf": torch.ones(2), "w": w, "w_sf": torch.ones(1, 3), "off": _offsets([2]), "row_token": None}
    _check(s, F32)


def test_rows_without_a_token_and_rows_of_no_expert():
    s = _case([5, 0, 4], 64, 128, by_token=True, X=6)
    s["row_token"][1], s["row_token"][6], s["row_token"][8] = -1, 6, 1 << 30
    s["w_sf"][0, 3] = float("nan")  # a row of zeros stays one
    y = _run(s).cpu()
    want = _product(s["x"], s["x_sf"], s["w"], s["w_sf"], s["off"], s["row_token"], BF16, 9)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(y), nan) and torch.equal(y[~nan], want[~nan])
    for r in (1, 6, 8):
        assert (y[r] == 0).all()
    # rows before the first and behind the last expert are left as they were
    s["off"] = torch.tensor([2, 5, 5, 7], dtype=I32)
    out = torch.full((9, 64), 7.0, dtype=BF16, device="cuda")
    y = _run(s, out=out).cpu()
    assert (y[:2] == 7).all() and (y[7:] == 7).all() and (y[6] == 0).all()
    # no token rows at all
    empty = {**s, "x": torch.empty(0, 128, dtype=I8), "x_sf": torch.empty(0), "off": _offsets([5, 0, 4])}
    assert (_run(empty) == 0).all()


def test_bad_offsets_stay_inside():
    """Offsets outside [0, R] or decreasing are clamped: nothing outside the output is written."""
    s = _case([5, 5, 5], 64, 128)
    guard = torch.full((15 + 2, 64), 7.0, dtype=BF16, device="cuda")
    s["off"] = torch.tensor([-4, 6, 3, 99], dtype=I32)
    _run(s, out=guard[1:16])
    assert (guard[0] == 7).all() and (guard[16] == 7).all()


def test_unaligned_tensors():
    """Codes at odd addresses take the byte loads; results are the same bits."""
    s = _case([20, 3], 64, 128)
    want = _product(s["x"], s["x_sf"], s["w"], s["w_sf"], s["off"], None, BF16, 23)

    def shifted(t):
        flat = torch.empty(t.numel() + 16, dtype=t.dtype, device="cuda")[1:1 + t.numel()]
        return flat.copy_(t.flatten()).view(t.shape)

    for x, w in ((shifted(s["x"]), s["w"].cuda()), (s["x"].cuda(), shifted(s["w"]))):
        y = moe.moe_expert_matmul_int8(x, s["x_sf"].cuda(), w, s["w_sf"].cuda(), expert_offsets=s["off"].cuda())
        assert torch.equal(y.cpu(), want)
    out = torch.empty(23 * 64 + 1, dtype=BF16, device="cuda")[1:].view(23, 64)
    assert torch.equal(_run(s, out=out).cpu(), want)


def test_many_rows_past_32_bits():
    """Weights of more than 2^31 and outputs of more than 2^32 bytes: the last expert's last rows are right."""
    E, N, K, R = 5, 65536, 8192, 34000
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GiB of device memory")
    w = torch.zeros(E, N, K, dtype=I8, device="cuda")
    w[-1, -1] = 3
    w[-1, -2, ::2] = -5
    off = torch.tensor([0, 0, 0, 0, 33990, R], dtype=I32, device="cuda")
    x = torch.ones(R, K, dtype=I8, device="cuda")
    y = moe.moe_expert_matmul_int8(x, torch.ones(R, device="cuda"), w, torch.ones(E, N, device="cuda"),
                                   expert_offsets=off)
    assert y.numel() * 2 > 1 << 32
    assert (y[33990:, -1] == 3 * K).all() and (y[33990:, -2] == -5 * K // 2).all()
    assert (y[33990:, :-2] == 0).all() and (y[:33990:997] == 0).all()


def test_streams_and_graphs():
    s = _case([30, 2, 100], 128, 256, by_token=True)
    c = {k: v.cuda() if v is not None else None for k, v in s.items()}
    gu = torch.randn(132, 512, device="cuda").to(BF16)

    def run(stream=None, outs=None):
        o = outs or {}
        q = moe.moe_cast_int8(gu, out=o.get("q"), stream=stream)
        a = moe.swiglu_cast_int8(gu, out=o.get("a"), stream=stream)
        y = moe.moe_expert_matmul_int8(c["x"], c["x_sf"], c["w"], c["w_sf"], expert_offsets=c["off"],
                                       row_token=c["row_token"], out=o.get("y"), stream=stream)
        return [*q, *a, y]

    want = [t.clone() for t in run()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    outs = {"q": tuple(torch.empty_like(t) for t in want[:2]), "a": tuple(torch.empty_like(t) for t in want[2:4]),
            "y": torch.empty_like(want[4])}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(outs=outs)
    for _ in range(3):
        gu.copy_(torch.randn(132, 512, device="cuda"))
        c["x"].copy_(torch.randint(-128, 128, c["x"].shape, device="cuda", dtype=I8))
        graph.replay()
        for a, b in zip([*outs["q"], *outs["a"], outs["y"]], run()):
            assert torch.equal(a, b)
        torch.cuda.synchronize()


def test_no_rows():
    e = torch.empty
    q, sf = moe.moe_cast_int8(e(0, 64, dtype=BF16, device="cuda"))
    assert q.shape == (0, 64) and sf.shape == (0,)
    q, sf = moe.swiglu_cast_int8(e(0, 64, dtype=BF16, device="cuda"))
    assert q.shape == (0, 32)
    w, w_sf = torch.zeros(2, 8, 32, dtype=I8, device="cuda"), torch.zeros(2, 8, device="cuda")
    off = torch.zeros(3, dtype=I32, device="cuda")
    assert moe.moe_expert_matmul_int8(q, sf, w, w_sf, expert_offsets=off).shape == (0, 8)
    y = moe.moe_expert_matmul_int8(torch.zeros(4, 32, dtype=I8, device="cuda"), torch.zeros(4, device="cuda"), w, w_sf,
                                   expert_offsets=off, row_token=e(0, dtype=I32, device="cuda"))
    assert y.shape == (0, 8)


@pytest.mark.parametrize("T,E,K,H,I", [(1, 8, 2, 256, 64), (37, 16, 4, 384, 96), (300, 8, 2, 512, 136)])
def test_from_the_router_to_the_combine(T, E, K, H, I):
    """A block's feed-forward as a user runs it, stage by stage against the definition on the stage's own inputs."""
    g = _gen(T, E, H)
    x = torch.randn(T, H, generator=g).to(BF16)
    logits = torch.randn(T, E, generator=g)
    mask = torch.rand(T, generator=g) >= 0.2
    mask[0] = True
    w1 = torch.randint(-127, 128, (E, 2 * I, H), generator=g, dtype=I8)
    w2 = torch.randint(-127, 128, (E, H, I), generator=g, dtype=I8)
    s1 = (0.5 + torch.rand(E, 2 * I, generator=g)) / (73 * H ** 0.5)
    s2 = (0.5 + torch.rand(E, H, generator=g)) / (73 * I ** 0.5)
    idx, weights = moe.moe_router(logits.cuda(), K, score="sigmoid", renormalize=True, token_mask=mask.cuda())
    counts, offsets, pos, row_token = moe.moe_token_map(idx, E)
    q, sf = moe.moe_cast_int8(x.cuda())
    h = moe.moe_expert_matmul_int8(q, sf, w1.cuda(), s1.cuda(), expert_offsets=offsets, row_token=row_token)
    live = int(offsets[-1])
    a, a_sf = moe.swiglu_cast_int8(h[:live])
    y = torch.zeros(T * K, H, dtype=BF16, device="cuda")
    moe.moe_expert_matmul_int8(a, a_sf, w2.cuda(), s2.cuda(), expert_offsets=offsets, out=y[:live])
    out = moe.moe_combine(y, pos, weights)

    off, rt = offsets.cpu(), row_token.cpu()[:live]
    want_h = _product(*_cast32(x), w1, s1, off, rt, BF16, live)
    assert torch.equal(h[:live].cpu(), want_h)
    want_y = _product(a.cpu(), a_sf.cpu(), w2, s2, off, None, BF16, live)
    assert torch.equal(y[:live].cpu(), want_y)
    p, wts = pos.cpu().long(), weights.double().cpu()
    rows = torch.where((p >= 0)[:, :, None], y.double().cpu()[p.clamp_min(0)], torch.zeros(1, dtype=torch.float64))
    want = (rows * wts[:, :, None]).sum(1)
    size = (rows * wts[:, :, None]).abs().sum(1)
    assert ((out.double().cpu() - want).abs() <= 2.0 ** -8 * want.abs() + 2 * K * EPS32 * size).all()
    assert (out[~mask.cuda()] == 0).all()
