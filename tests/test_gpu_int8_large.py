"""moe_expert_matmul_int8 with many rows and many channels at once."""
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
