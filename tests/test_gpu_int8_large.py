"""moe_expert_matmul_int8 with many rows and many channels at once, and with offsets that give many experts many rows."""
import pytest
import torch

import moe_routing_fp8_amd as moe
from test_gpu_int8 import BF16, I32, I8, _need_gpu  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [48, 47])
def test_many_rows_by_many_channels(K):
    """2^18 rows by 2^16 channels, 2^24 blocks of 16 by 64, in whole chunks and at an odd length: rows all over the
    output, bit for bit."""
    R, N = 1 << 18, 1 << 16
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GiB of device memory")
    g = torch.Generator(device="cuda").manual_seed(K)
    codes = {"generator": g, "dtype": I8, "device": "cuda"}
    x, w = torch.randint(-128, 128, (R, K), **codes), torch.randint(-128, 128, (2, N, K), **codes)
    x_sf, w_sf = torch.rand(R, generator=g, device="cuda") + 0.1, torch.rand(2, N, generator=g, device="cuda") - 0.5
    half = 100003
    off = torch.tensor([0, half, R], dtype=I32, device="cuda")
    y = moe.moe_expert_matmul_int8(x, x_sf, w, w_sf, expert_offsets=off)
    assert y.shape == (R, N)
    for e, rows in ((0, torch.arange(0, half, 809)), (1, torch.arange(half, R, 809)),
                    (0, torch.arange(half - 40, half)), (1, torch.arange(R - 300, R))):
        rows = rows.cuda()
        sums = x[rows].double() @ w[e].double().t().contiguous()
        assert torch.equal(y[rows], ((sums.float() * x_sf[rows, None]) * w_sf[e]).to(BF16)), (e, int(rows[0]))


@pytest.mark.parametrize("K", [16, 1])
def test_offsets_that_give_every_second_expert_all_rows(K):
    """512 experts of nearly 2^26 rows each, which no valid offsets give: nothing is computed, nothing outside is read.
    (With 2 experts the same rows are computed.)"""
    R, E = (1 << 26) - 1, 1024
    x, x_sf = torch.ones(R, K, dtype=I8, device="cuda"), torch.ones(R, device="cuda")
    w, w_sf = torch.ones(E, 1, K, dtype=I8, device="cuda"), torch.ones(E, 1, device="cuda")
    out = torch.full((R + 2, 1), 7.0, dtype=BF16, device="cuda")
    off = torch.tensor([0, R] * (E // 2) + [0], dtype=I32, device="cuda")
    moe.moe_expert_matmul_int8(x, x_sf, w, w_sf, expert_offsets=off, out=out[1:-1])
    assert (out == 7).all()
    moe.moe_expert_matmul_int8(x, x_sf, w[:2], w_sf[:2], expert_offsets=off[:3], out=out[1:-1])
    assert (out[1:-1] == K).all() and out[0] == 7 and out[-1] == 7
