"""Ids as moe_router writes them, -1 where a copy has no expert: their check, and the token maps in debug mode."""
import pytest
import torch

import moe_routing_fp8_amd as moe
from moe_routing_fp8_amd import _native

RANGE, DUPLICATE = 0x04, 0x08
FAKE = 0x10000  # a non-null, 256-byte aligned address never dereferenced on the host


def test_validation():
    """On the host, before any HIP call (CPU)."""
    f = _native.lib().moe_check_routed_idx
    assert f(FAKE, 4, 17, 64, FAKE, None) == 1 and f(FAKE, 4, 0, 64, FAKE, None) == 1
    assert f(FAKE, -1, 8, 64, FAKE, None) == 1 and f(FAKE, 4, 8, 1025, FAKE, None) == 1
    assert f(FAKE + 4, 4, 8, 64, FAKE, None) == 1 and f(FAKE, 4, 8, 64, None, None) == 1
    assert f(None, 4, 8, 64, FAKE, None) == 1 and f(None, 0, 8, 64, FAKE, None) == 0


@pytest.mark.gpu
def test_check():
    for ids, routed, plain in (([[3, 1, 2]], 0, 0), ([[-1, -1, -1]], 0, RANGE | DUPLICATE),
                               ([[3, -1, -1]], 0, RANGE | DUPLICATE), ([[3, -1, 3]], DUPLICATE, RANGE | DUPLICATE), ([[-1, 0, 1], [7, 8, -1]], RANGE, RANGE),
                               ([[-2, 0, -2]], RANGE | DUPLICATE, RANGE | DUPLICATE)):
        idx = torch.tensor(ids, dtype=torch.int64, device="cuda")
        assert int(moe.moe_check_routed_idx(idx, 8)) == routed, ids
        assert int(moe.moe_check_topk_idx(idx, 8)) == plain, ids


@pytest.mark.gpu
@pytest.mark.parametrize("debug", ["0", "1"])
def test_masked_tokens_through_the_maps(debug, monkeypatch):
    z = torch.randn(100, 32, generator=torch.Generator().manual_seed(2)).cuda()
    z[5, 3:] = -float("inf")  # three experts for four rounds
    mask = torch.arange(100, device="cuda") % 3 != 0
    idx, _ = moe.moe_router(z, 4, token_mask=mask)
    assert (idx[~mask] == -1).all() and idx[5].tolist().count(-1) == 1
    monkeypatch.setenv("MOE_FP8_DEBUG", debug)
    for token_map in (moe.moe_token_map, moe.moe_token_map_noalloc):
        counts, offsets, pos, _ = token_map(idx, 32)
        assert int(counts.sum()) == 4 * int(mask.sum()) - 1 == int(offsets[-1])
        assert torch.equal(pos == -1, idx == -1)
    idx[7, 0] = idx[7, 1]
    if debug == "1":
        with pytest.raises(ValueError, match="MOE_CHECK_ID_DUPLICATE"):
            moe.moe_token_map(idx, 32)
