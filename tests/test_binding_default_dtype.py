"""The outputs that the binding allocates have the types that the kernels write, whatever torch's default type is: a
narrower one would leave them less memory than is written.  On fake tensors, without a GPU and without a call."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import moe_routing_fp8_amd as moe
from moe_routing_fp8_amd import _native

T, H, E, K, S = 6, 64, 16, 2, 3
F32, BF16, I32, U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8


@pytest.fixture(params=[torch.bfloat16, torch.float64])
def fake(request, monkeypatch):
    monkeypatch.setattr(_native, "_call", lambda *a: None)
    monkeypatch.setattr(_native, "_ptr", lambda t: None)
    monkeypatch.setattr(_native, "_workspace", lambda t, dev: t.numel())
    before = torch.get_default_dtype()
    torch.set_default_dtype(request.param)
    try:
        with FakeTensorMode():
            yield lambda *shape, dtype=F32: torch.empty(shape, dtype=dtype, device="cuda")
    finally:
        torch.set_default_dtype(before)


def _types(out):
    values = out.items() if isinstance(out, dict) else enumerate(out)
    return {k: v.dtype for k, v in values if v is not None}


def test_block_norm(fake):
    r, y, w, gate = fake(T, H), fake(T, H, dtype=BF16), fake(H), fake(T, 1)
    out = moe.moe_block_norm(r, y, w, gate, 0.5, w, with_rstd=True)
    assert _types(out) == {0: F32, 1: BF16, 2: F32, 3: F32}
    for g in (gate, w):
        grads = moe.moe_block_norm_backward(out[0], out[1], out[0], y, w, g, 0.5, w, out[2], out[3])
        assert _types(grads) == {"grad_residual": F32, "grad_y": BF16, "grad_post_weight": F32, "grad_gate": F32,
                                 "grad_pre_weight": F32}


def test_balance_loss(fake):
    z, ids, off = fake(T, E, dtype=BF16), fake(T, K, dtype=torch.int64), fake(S + 1, dtype=I32)
    out = moe.moe_balance_loss(z, ids, seq_offsets=off)
    assert _types(out) == {"loss": F32, "counts": I32, "seq_tokens": I32, "prob_mean": F32}
    assert moe.moe_balance_loss_backward(out["loss"], z, out["counts"], out["seq_tokens"], K,
                                         seq_offsets=off).dtype == BF16


def test_expert_matvec(fake):
    out = moe.moe_expert_matvec(fake(T, H, dtype=BF16), fake(E, 8, H // 2, dtype=U8), fake(E, 8, H // 32, dtype=U8),
                                expert_offsets=fake(E + 1, dtype=I32))
    assert out.dtype == BF16


def test_the_dispatch_path(fake):
    x, scores = fake(T, 128, dtype=BF16), fake(T, E)
    assert _types(moe.moe_topk_gate(scores, K, renormalize=True)) == {0: torch.int64, 1: F32}
    assert set(_types(moe.moe_expand_cast_fp8(x)).values()) <= {U8, F32, torch.float8_e4m3fn}
    assert moe.moe_combine(x, fake(T, 1, dtype=I32), fake(T, 1)).dtype == BF16
