"""One MoE block around the dispatch path, as a serving step and as a training step.

    python examples/moe_block.py

Serving: the norm before the block, the router, the dispatch with its e4m3 cast, the experts' gate and up products
with 4-bit weights, SwiGLU with its cast, the down products, the combine, and then in one pass the norm after the
block, its gate, the residual and the norm before the next block.

Training: the router's balance loss over packed sequences with its gradient, and the block norm's gradients.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_routing_fp8_amd as moe  # noqa: E402

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def quantise(w):
    """Weights [E, N, K] -> e2m1 codes [E, N, K/2] and UE8M0 scales [E, N, K/32]: MXFP4, once, when a model loads."""
    E, N, K = w.shape
    codes, sf, _ = moe.moe_expand_cast(w.reshape(E * N, K).to(torch.bfloat16), dtype="e2m1", group_size=32,
                                       round_sf=True, sf_ue8m0=True)
    return codes.view(E, N, K // 2), sf.view(E, N, K // 32)


def dequantise(codes, sf):
    """The fp32 weights that e2m1 codes and UE8M0 scales stand for."""
    value = torch.tensor(E2M1, device=codes.device)
    w = torch.stack([value[(codes & 15).long()], value[(codes >> 4).long()]], -1).flatten(-2)
    return w * torch.exp2(sf.float() - 127).repeat_interleave(32, -1)


class Block:
    """The weights of one block."""

    def __init__(self, hidden, inter, experts, topk, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, generator=g, device="cuda")

        self.topk, self.experts = topk, experts
        self.norm_before, self.norm_after = 1 + 0.1 * normal(hidden), 1 + 0.1 * normal(hidden)
        self.norm_next, self.gate = 1 + 0.1 * normal(hidden), 0.5 + 0.1 * normal(hidden)
        self.router = normal(hidden, experts) / hidden ** 0.5
        self.up = quantise(normal(experts, 2 * inter, hidden) / hidden ** 0.5)
        self.down = quantise(normal(experts, hidden, inter) / inter ** 0.5)

    def serve(self, residual):
        """residual bf16 [T, H] -> (the new residual, the normed input of the next block)."""
        _, x, _, _ = moe.moe_block_norm(residual, pre_weight=self.norm_before)
        scores = torch.sigmoid(x.float() @ self.router)
        d = moe.moe_dispatch(scores, x, self.topk, renormalize=True)
        up = moe.moe_expert_matvec(d["out"], *self.up, x_sf=d["out_sf"], expert_offsets=d["offsets"])
        act, act_sf = moe.swiglu_cast_fp8(up)
        down = moe.moe_expert_matvec(act, *self.down, x_sf=act_sf, expert_offsets=d["offsets"])
        y = moe.moe_combine(down, d["pos"], d["topk_weights"])
        out, normed, _, _ = moe.moe_block_norm(residual, y, post_weight=self.norm_after, gate=self.gate,
                                               pre_weight=self.norm_next)
        return out, normed

    def serve_plain(self, residual):
        """The same block in fp32 on the dequantised weights, without casts."""
        def norm(v, w):
            return v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-6) * w

        r = residual.float()
        x = norm(r, self.norm_before)
        s, ids = torch.sigmoid(x @ self.router).topk(self.topk, 1)
        s = s / s.sum(1, keepdim=True)
        up, down = dequantise(*self.up), dequantise(*self.down)
        y = torch.zeros_like(r)
        for k in range(self.topk):
            h = torch.bmm(up[ids[:, k]], x.unsqueeze(2)).squeeze(2)
            g, u = h.chunk(2, 1)
            v = torch.nn.functional.silu(g) * u
            y += s[:, k:k + 1] * torch.bmm(down[ids[:, k]], v.unsqueeze(2)).squeeze(2)
        out = r + self.gate * norm(y, self.norm_after)
        return out, norm(out, self.norm_next)


def train_router(steps=60, tokens=512, experts=32, topk=4, rate=4000.0, seed=1):
    """Gradient descent of the logits on the balance loss alone, four packed sequences; returns the mean loss of the
    first and the last step.  It falls to about 1, the loss of an even load."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = torch.randn(tokens, experts, generator=g, device="cuda") + 1.5 * torch.randn(experts, generator=g,
                                                                                          device="cuda")
    offsets = torch.tensor([0, 100, 100, 300, tokens], dtype=torch.int32, device="cuda")  # one is empty
    weight = torch.full((4,), 1 / 3, device="cuda")
    seen = []
    for _ in range(steps):
        ids, _ = moe.moe_topk_gate(logits, topk)
        o = moe.moe_balance_loss(logits, ids, seq_offsets=offsets)
        seen.append((o["loss"] * weight).sum())
        logits -= rate * moe.moe_balance_loss_backward(weight, logits, o["counts"], o["seq_tokens"], topk,
                                                       seq_offsets=offsets)
    return float(seen[0]), float(seen[-1])


def train_norm(steps=40, tokens=256, hidden=512, rate=0.02, seed=2):
    """Fits the gate and norm weights of a block norm to a target; returns the first and the last squared error."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    residual, y = normal(tokens, hidden), normal(tokens, hidden).to(torch.bfloat16)
    want = dict(post_weight=1 + 0.3 * normal(hidden), gate=0.5 + 0.3 * normal(hidden),
                pre_weight=1 + 0.3 * normal(hidden))
    target = moe.moe_block_norm(residual, y, **want)[0]
    have = dict(post_weight=torch.ones(hidden, device="cuda"), gate=torch.full((hidden,), 0.1, device="cuda"),
                pre_weight=torch.ones(hidden, device="cuda"))
    seen = []
    for _ in range(steps):
        out, normed, post, pre = moe.moe_block_norm(residual, y, with_rstd=True, **have)
        diff = out - target
        seen.append(diff.square().mean())
        grads = moe.moe_block_norm_backward(diff / tokens, torch.zeros_like(normed), out, y, post_rstd=post,
                                            pre_rstd=pre, **have)
        for key in have:
            have[key] -= 10 * rate * grads["grad_" + key]
    return float(seen[0]), float(seen[-1])


def main():
    block = Block(hidden=256, inter=128, experts=16, topk=2)
    residual = torch.randn(8, 256, device="cuda").to(torch.bfloat16)
    out, normed = block.serve(residual)
    want, want_normed = block.serve_plain(residual)
    for name, a, b in (("residual", out, want), ("next input", normed, want_normed)):
        print(f"serving, {name}: {float((a.float() - b).norm() / b.norm()):.4f} from the fp32 block (e4m3 casts)")
    first, last = train_router()
    print(f"balance loss: {first:.3f} -> {last:.3f}")
    first, last = train_norm()
    print(f"block norm fit: squared error {first:.4f} -> {last:.4f}")


if __name__ == "__main__":
    main()
