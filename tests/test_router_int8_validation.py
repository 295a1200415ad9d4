"""CPU checks of the routing and of the 8-bit integer casts and products: the C entry points refuse invalid arguments
on the host before any HIP call and return MOE_OK for calls with nothing to do; the binding refuses tensors that do not
fit and allocates outputs of the types that are written (on fake tensors, without a GPU and without a call)."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import moe_routing_fp8_amd as moe
from moe_routing_fp8_amd import _native

INVALID, UNSUPPORTED = 1, 2
FAKE = 0x10000  # a non-null, 256-byte aligned address never dereferenced on the host
NAN, INF = float("nan"), float("inf")
F32, BF16, I8, I32, I64 = torch.float32, torch.bfloat16, torch.int8, torch.int32, torch.int64


@pytest.fixture(scope="module")
def lib():
    return _native.lib()


def _caller(fn, names, ok):
    def call(**kw):
        args = dict(zip(names.split(), ok))
        args.update(kw)
        assert len(args) == len(names.split()), set(args) - set(names.split())
        return fn(*args.values())
    return call


def test_router(lib):
    call = _caller(lib.moe_router, "z dt rs T E K score bias G kept gs renorm scale mask idx w stream",
                   [FAKE, 1, 64, 4, 64, 8, 0, FAKE, 8, 4, 1, 1, 2.5, FAKE, FAKE, FAKE, None])
    assert call(T=-1) == INVALID and call(E=0) == INVALID and call(K=0) == INVALID and call(K=17) == INVALID
    assert call(E=1025, rs=1025, G=1, kept=1) == INVALID and call(rs=63) == INVALID
    assert call(T=(1 << 31) // 16 + 1) == INVALID
    assert call(dt=2) == INVALID and call(dt=-1) == INVALID and call(score=2) == INVALID and call(gs=2) == INVALID
    assert call(renorm=2) == INVALID and call(scale=NAN) == INVALID and call(scale=INF) == INVALID
    assert call(G=0) == INVALID and call(G=7) == INVALID and call(kept=0) == INVALID and call(kept=9) == INVALID
    assert call(G=16, kept=1, K=5) == INVALID                     # four experts cannot give five
    assert call(G=64, kept=64) == INVALID                         # the two best of one
    assert call(E=260, rs=260, G=65, kept=30) == UNSUPPORTED
    assert call(T=1 << 26, E=264, rs=264) == UNSUPPORTED          # 2^32 threads
    assert call(z=None) == INVALID and call(idx=None) == INVALID and call(w=None) == INVALID
    assert call(z=FAKE + 2) == INVALID and call(dt=0, z=FAKE + 1) == INVALID
    assert call(bias=FAKE + 2) == INVALID and call(idx=FAKE + 4) == INVALID and call(w=FAKE + 2) == INVALID
    assert call(T=0, z=None, idx=None, w=None, bias=None) == 0


def test_router_backward(lib):
    call = _caller(lib.moe_router_backward, "g z dt rs T E idx K score renorm scale out stream",
                   [FAKE, FAKE, 0, 64, 4, 64, FAKE, 8, 1, 0, 1.0, FAKE, None])
    assert call(T=-1) == INVALID and call(E=0) == INVALID and call(K=65) == INVALID and call(K=17) == INVALID
    assert call(rs=63) == INVALID and call(dt=2) == INVALID and call(score=-1) == INVALID
    assert call(renorm=-1) == INVALID and call(scale=NAN) == INVALID
    assert call(g=None) == INVALID and call(z=None) == INVALID and call(idx=None) == INVALID
    assert call(out=None) == INVALID and call(out=FAKE + 1) == INVALID and call(idx=FAKE + 4) == INVALID
    assert call(g=FAKE + 2) == INVALID
    assert call(T=1 << 26, E=257, rs=257) == UNSUPPORTED
    assert call(T=0, g=None, z=None, idx=None, out=None) == 0


def test_casts(lib):
    call = _caller(lib.moe_cast_int8, "x dt rs R H out sf stream", [FAKE, 0, 64, 4, 64, FAKE, FAKE, None])
    assert call(R=-1) == INVALID and call(H=0) == INVALID and call(rs=63) == INVALID and call(dt=2) == INVALID
    assert call(x=None) == INVALID and call(out=None) == INVALID and call(sf=None) == INVALID
    assert call(x=FAKE + 1) == INVALID and call(dt=1, x=FAKE + 2) == INVALID and call(sf=FAKE + 2) == INVALID
    assert call(R=1 << 24) == UNSUPPORTED and call(H=(1 << 20) + 1, rs=1 << 21) == UNSUPPORTED
    assert call(R=0, x=None, out=None, sf=None) == 0
    call = _caller(lib.swiglu_cast_int8, "gu R I w clamp out sf stream", [FAKE, 4, 64, FAKE, 0.0, FAKE, FAKE, None])
    assert call(R=-1) == INVALID and call(I=0) == INVALID and call(clamp=NAN) == INVALID
    assert call(gu=None) == INVALID and call(out=None) == INVALID and call(sf=None) == INVALID
    assert call(gu=FAKE + 1) == INVALID and call(w=FAKE + 2) == INVALID and call(sf=FAKE + 2) == INVALID
    assert call(R=1 << 24) == UNSUPPORTED and call(I=(1 << 20) + 1) == UNSUPPORTED
    assert call(R=0, gu=None, out=None, sf=None) == 0


def test_expert_matmul_int8(lib):
    call = _caller(lib.moe_expert_matmul_int8, "x sf X rt R K N E off w wsf dt out stream",
                   [FAKE, FAKE, 5, FAKE, 7, 100, 20, 2, FAKE, FAKE, FAKE, 0, FAKE, None])
    assert call(R=-1) == INVALID and call(X=-1) == INVALID and call(R=1 << 31) == INVALID
    assert call(K=0) == INVALID and call(N=0) == INVALID and call(E=0) == INVALID and call(E=1025) == INVALID
    assert call(dt=2) == INVALID and call(off=None) == INVALID
    assert call(rt=None) == INVALID                               # then x has the rows
    assert call(K=131072) == UNSUPPORTED and call(N=(1 << 20) + 1) == UNSUPPORTED
    assert call(R=1 << 26, N=256) == UNSUPPORTED
    for name in ("x", "sf", "w", "wsf", "out"):
        assert call(**{name: None}) == INVALID
    for name in ("sf", "wsf", "rt", "off"):
        assert call(**{name: FAKE + 2}) == INVALID
    assert call(out=FAKE + 1) == INVALID and call(dt=1, out=FAKE + 2) == INVALID
    assert call(R=0, x=None, sf=None, X=0, rt=None, w=None, wsf=None, out=None) == 0


def test_limits_match_the_header():
    with open(_native.HEADER_PATH) as f:
        text = f.read()
    assert f"#define MOE_GROUP_MAX {_native.MOE_GROUP_MAX} " in text
    assert f"#define MOE_GROUP_TOP2 {_native.MOE_GROUP_TOP2} " in text
    assert "#define MOE_MATMUL_INT8_MAX_INNER 131071 " in text and 131071 * 2 ** 14 < 2 ** 31 <= 131072 * 2 ** 14


@pytest.fixture(params=[torch.float32, torch.bfloat16, torch.float64])
def fake(request, monkeypatch):
    monkeypatch.setattr(_native, "_call", lambda *a: None)
    monkeypatch.setattr(_native, "_ptr", lambda t: None)
    before = torch.get_default_dtype()
    torch.set_default_dtype(request.param)
    try:
        with FakeTensorMode():
            yield lambda *shape, dtype=F32: torch.empty(shape, dtype=dtype, device="cuda")
    finally:
        torch.set_default_dtype(before)


def test_outputs(fake):
    z = fake(6, 64, dtype=BF16)
    idx, w = moe.moe_router(z, 4, bias=fake(64))
    assert (idx.dtype, w.dtype, idx.shape, w.shape) == (I64, F32, (6, 4), (6, 4))
    grad = moe.moe_router_backward(w, z, idx)
    assert grad.dtype == BF16 and grad.shape == (6, 64)
    q, sf = moe.moe_cast_int8(fake(6, 32, dtype=BF16))
    assert (q.dtype, sf.dtype, q.shape, sf.shape) == (I8, F32, (6, 32), (6,))
    q, sf = moe.swiglu_cast_int8(fake(6, 64, dtype=BF16), fake(6))
    assert (q.dtype, sf.dtype, q.shape, sf.shape) == (I8, F32, (6, 32), (6,))
    mats, mat_sf, off = fake(3, 8, 32, dtype=I8), fake(3, 8), fake(4, dtype=I32)
    y = moe.moe_expert_matmul_int8(q, sf, mats, mat_sf, expert_offsets=off)
    assert y.dtype == BF16 and y.shape == (6, 8)
    y = moe.moe_expert_matmul_int8(q, sf, mats, mat_sf, expert_offsets=off, row_token=fake(9, dtype=I32), out_dtype=F32)
    assert y.dtype == F32 and y.shape == (9, 8)
    assert moe.moe_expert_matmul_int8(q, sf, mats[0], mat_sf[0], out=y[:6]).dtype == F32


def test_binding_refuses(fake):
    z = fake(6, 64)
    bad = [
        lambda: moe.moe_router(fake(6, 64, dtype=torch.float16), 4),
        lambda: moe.moe_router(z, 4, score="relu"),
        lambda: moe.moe_router(z, 4, group_score="mean"),
        lambda: moe.moe_router(z, 4, bias=fake(63)),
        lambda: moe.moe_router(z, 4, bias=fake(64, dtype=BF16)),
        lambda: moe.moe_router(z, 4, token_mask=fake(5, dtype=torch.bool)),
        lambda: moe.moe_router(z, 4, out=(fake(6, 4, dtype=I32), fake(6, 4))),
        lambda: moe.moe_router(z, 4, out=(fake(6, 4, dtype=I64), fake(6, 5))),
        lambda: moe.moe_router(fake(64, 6).t(), 4),
        lambda: moe.moe_router_backward(fake(6, 4), z, fake(6, 3, dtype=I64)),
        lambda: moe.moe_router_backward(fake(6, 4), z, fake(6, 4, dtype=I32)),
        lambda: moe.moe_router_backward(fake(6, 4), z, fake(6, 4, dtype=I64), out=fake(6, 64, dtype=BF16)),
        lambda: moe.moe_cast_int8(fake(6, 64, dtype=torch.float16)),
        lambda: moe.moe_cast_int8(z, out=(fake(6, 64, dtype=torch.uint8), fake(6))),
        lambda: moe.moe_cast_int8(z, out=(fake(6, 64, dtype=I8), fake(5))),
        lambda: moe.swiglu_cast_int8(fake(6, 63, dtype=BF16)),
        lambda: moe.swiglu_cast_int8(fake(6, 64, dtype=BF16), fake(5)),
        lambda: moe.swiglu_cast_int8(fake(6, 64, dtype=BF16), out=(fake(6, 64, dtype=I8), fake(6))),
    ]
    x, sf, w, w_sf, off = fake(6, 32, dtype=I8), fake(6), fake(3, 8, 32, dtype=I8), fake(3, 8), fake(4, dtype=I32)
    bad += [
        lambda: moe.moe_expert_matmul_int8(fake(6, 32), sf, w, w_sf, expert_offsets=off),
        lambda: moe.moe_expert_matmul_int8(x, fake(5), w, w_sf, expert_offsets=off),
        lambda: moe.moe_expert_matmul_int8(x, sf, fake(3, 8, 31, dtype=I8), w_sf, expert_offsets=off),
        lambda: moe.moe_expert_matmul_int8(x, sf, w, fake(3, 7), expert_offsets=off),
        lambda: moe.moe_expert_matmul_int8(x, sf, w, w_sf),
        lambda: moe.moe_expert_matmul_int8(x, sf, w, w_sf, expert_offsets=fake(3, dtype=I32)),
        lambda: moe.moe_expert_matmul_int8(x, sf, w, w_sf, expert_offsets=off, row_token=fake(6, dtype=I64)),
        lambda: moe.moe_expert_matmul_int8(x, sf, w, w_sf, expert_offsets=off, out_dtype=torch.float16),
        lambda: moe.moe_expert_matmul_int8(x, sf, w, w_sf, expert_offsets=off, out=fake(6, 9, dtype=BF16)),
        lambda: moe.moe_expert_matmul_int8(x, sf, w, w_sf, expert_offsets=off, out_dtype=F32,
                                           out=fake(6, 8, dtype=BF16)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")


def test_host_tensors_are_refused():
    for call in (lambda: moe.moe_router(torch.zeros(2, 8), 2),
                 lambda: moe.moe_cast_int8(torch.zeros(2, 8)),
                 lambda: moe.swiglu_cast_int8(torch.zeros(2, 8, dtype=BF16)),
                 lambda: moe.moe_expert_matmul_int8(torch.zeros(2, 8, dtype=I8), torch.zeros(2),
                                                    torch.zeros(3, 8, dtype=I8), torch.zeros(3))):
        with pytest.raises(ValueError):
            call()
