"""moe_router's order where values lie next to each other: ids equal to the definition's stable sorts of 64-bit values."""
import pytest
import torch

from test_gpu_router import BF16, F32, _check, _ids, _need_gpu, _gpu, _log  # noqa: F401

import moe_routing_fp8_amd as moe

pytestmark = pytest.mark.gpu


def _same_ids(z, K, score, **kw):
    kg = {k: _gpu(v) if isinstance(v, torch.Tensor) else v for k, v in kw.items()}
    idx, _ = moe.moe_router(z.cuda(), K, score=score, renormalize=True, **kg)
    want = _ids(z, K, score, **kw)
    wrong = (idx.cpu() != want).any(1)
    assert not wrong.any(), (int(wrong.sum()), wrong.nonzero()[0].tolist(), idx.cpu()[wrong][0], want[wrong][0])


# rows over 16 lanes with 2, 4, 8 and 16 experts a lane, over 64 with 8 and 16
WIDTHS = [16, 61, 100, 256, 300, 1000]


@pytest.mark.parametrize("E", WIDTHS)
def test_equal_experts_on_both_sides_of_the_last_place(E):
    """A little lower, at a lower index, than `copies` equal experts, of which the last place takes some: the lower one
    has the better index and the same leading bits, and gives way to a copy left over."""
    low, high = 1.25, 1.25 + 2.0 ** -23
    for copies in (2, 3, 5):
        for K in (2, 3, 4, 8, 16):
            if K > E:
                continue
            rows = []
            for first in (1, E // 2):
                for extra in (None, low + 2.0 ** -22, low - 2.0 ** -22):
                    z = torch.zeros(E)
                    clear = max(0, K - copies)     # clearly better ones, so that the copies reach the last place
                    z[E - 1 - torch.arange(clear)] = 3.0 + torch.arange(clear)
                    z[first] = low
                    z[first + 2:first + 2 + copies] = high
                    if extra is not None:
                        z[first - 1] = extra
                    rows.append(z)
            z = torch.stack(rows)
            _log(f"E={E} K={K} copies={copies}")
            _same_ids(z, K, "softmax")
            for score in ("softmax", "sigmoid"):
                _same_ids(z, K, score, bias=torch.zeros(E))
            if E % 4 == 0:
                kw = dict(num_groups=2, topk_groups=1) if K <= E // 2 else dict(num_groups=2, topk_groups=2)
                _same_ids(z, K, "sigmoid", **kw)
                _same_ids(z, K, "sigmoid", bias=torch.zeros(E), group_score="top2", **kw)


@pytest.mark.parametrize("E", WIDTHS)
@pytest.mark.parametrize("K", [1, 2, 5, 8, 10, 16])
def test_logits_of_a_few_steps(E, K):
    """Logits on up to four neighbouring fp32 values, in some places: equal and nearly equal experts around every place."""
    g = torch.Generator().manual_seed(E * 31 + K)
    T = 600
    step = torch.randint(0, 4, (T, E), generator=g) * torch.randint(0, 2, (T, 1), generator=g) * 2
    step += torch.randint(0, 2, (T, E), generator=g)
    z = (torch.full((T, E), 1.25).view(torch.int32) + step.int()).view(F32)
    share = torch.rand(T, 1, generator=g) ** 3
    z = torch.where(torch.rand(T, E, generator=g) < share.clamp_min(2.5 / E), z, torch.zeros(1))
    z[::2] = -z[::2]
    _same_ids(z, K, "softmax")
    bias = torch.randint(0, 2, (E,), generator=g).float() * 2.0 ** -23
    for score in ("softmax", "sigmoid"):
        for b in (torch.zeros(E), bias):
            _same_ids(z, K, score, bias=b)


@pytest.mark.parametrize("E,G,kept", [(256, 1, 1), (256, 8, 4), (384, 1, 1), (60, 4, 2), (1024, 16, 6)])
@pytest.mark.parametrize("K", [4, 8])
def test_saturated_scores_with_a_bias_of_few_steps(E, G, kept, K):
    """bf16 logits around 10: the sigmoids differ by less than an fp32 key holds, and many are equal."""
    g = torch.Generator().manual_seed(E + K)
    z = (10 + 1.5 * torch.randn(6000, E, generator=g)).to(BF16)
    for steps in (0, 1, 3):
        bias = torch.randint(-steps, steps + 1, (E,), generator=g).float() * 1e-3
        for group_score in ("max", "top2"):
            _same_ids(z, K, "sigmoid", bias=bias, num_groups=G, topk_groups=kept, group_score=group_score)


@pytest.mark.parametrize("E,G,kept", [(64, 8, 4), (256, 8, 4), (256, 64, 7), (66, 3, 1), (168, 8, 3), (512, 8, 2),
                                      (1000, 8, 5)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_whose_two_best_cancel(E, G, kept, score):
    """One expert of each group lifted and the others pushed down by as much: a group's score is about one, what
    rounding leaves of its two values goes with the bias."""
    g = torch.Generator().manual_seed(E)
    z = 1.3 * torch.randn(12000, E, generator=g)
    for size in (1e3, 1e4, 1e6, 1e9):
        bias = torch.full((G, E // G), -size)
        bias[torch.arange(G), torch.randint(0, E // G, (G,), generator=g)] = size
        one = bias.clone()
        one[1:] = 1e-3 * torch.randint(-60, 61, (G - 1, E // G), generator=g)  # in the first group only
        for b in (bias, one):
            _log(f"E={E} G={G}/{kept} {score} {size}")
            _same_ids(z, min(4, kept * (E // G)), score, bias=b.flatten(), num_groups=G, topk_groups=kept,
                      group_score="top2")


@pytest.mark.parametrize("E", [16, 66, 256, 320])
def test_saturated_logits_without_a_bias(E):
    """Sigmoids that are 1 in 64 bits: experts come by their logits, with groups too; groups judged by their two best are
    equal then and go to the lowest, those judged by their best go by its logit."""
    G, size = 2, E // 2
    z = torch.full((2, E), 40.0)
    z[:, size - 1], z[:, 3] = 42.0, 41.0
    z[1, E - 1] = 43.0
    kw = dict(score="sigmoid", num_groups=G, topk_groups=1)
    idx, _ = moe.moe_router(z.cuda(), 3, group_score="top2", **kw)
    assert idx.tolist() == [[size - 1, 3, 0], [size - 1, 3, 0]]
    idx, _ = moe.moe_router(z.cuda(), 3, group_score="max", **kw)
    assert idx.tolist() == [[size - 1, 3, 0], [E - 1, size, size + 1]]
    # with a bias, one of zeros too, equal scores go to the lowest expert
    idx, _ = moe.moe_router(z.cuda(), 3, group_score="top2", bias=torch.zeros(E, device="cuda"), **kw)
    assert idx.tolist() == [[0, 1, 2]] * 2
