"""One MoE block around the dispatch path, as a serving step and as a training step.

    python examples/moe_block.py

Serving: the norm before the block, the router, the dispatch with its e4m3 cast, the experts' gate and up products
with 4-bit weights, SwiGLU with its cast, the down products, the combine, and then in one pass the norm after the
block, its gate, the residual and the norm before the next block.  The same in 8-bit integers: the routing from the
logits with a bias and groups, one cast of each token, products that read it by token, SwiGLU with its cast.

Training: the router's balance loss over packed sequences with its gradient, the gradient of its weights, and the block
norm's gradients.
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


def quantise_int8(w):
    """Weights [E, N, K] -> int8 codes and one scale for each of the E x N channels."""
    codes, sf = moe.moe_cast_int8(w.reshape(-1, w.shape[2]))
    return codes.view(w.shape), sf.view(w.shape[:2])


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
        up = normal(experts, 2 * inter, hidden) / hidden ** 0.5
        down = normal(experts, hidden, inter) / inter ** 0.5
        self.up, self.down = quantise(up), quantise(down)
        self.up_int8, self.down_int8 = quantise_int8(up), quantise_int8(down)
        self.bias = 0.02 * normal(experts)  # for balance: it moves the choice, not the weights

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

    def serve_int8(self, residual, groups=2, topk_groups=1, token_mask=None):
        """The same in 8-bit integers, with the experts chosen from the best groups; masked tokens get no expert."""
        _, x, _, _ = moe.moe_block_norm(residual, pre_weight=self.norm_before)
        ids, weights = moe.moe_router(x.float() @ self.router, self.topk, score="sigmoid", bias=self.bias,
                                      num_groups=groups, topk_groups=topk_groups, group_score="top2",
                                      renormalize=True, token_mask=token_mask)
        _, offsets, pos, row_token = moe.moe_token_map(ids, self.experts)
        codes, sf = moe.moe_cast_int8(x)
        # the rows behind the last expert's, of masked tokens, stay zeros
        up, down = (torch.zeros(row_token.numel(), w[0].shape[1], dtype=torch.bfloat16, device=x.device)
                    for w in (self.up_int8, self.down_int8))
        moe.moe_expert_matmul_int8(codes, sf, *self.up_int8, expert_offsets=offsets, row_token=row_token, out=up)
        act, act_sf = moe.swiglu_cast_int8(up)
        moe.moe_expert_matmul_int8(act, act_sf, *self.down_int8, expert_offsets=offsets, out=down)
        y = moe.moe_combine(down, pos, weights)
        out, normed, _, _ = moe.moe_block_norm(residual, y, post_weight=self.norm_after, gate=self.gate,
                                               pre_weight=self.norm_next)
        return out, normed, ids, weights

    def int8_plain(self, residual, ids, weights):
        """That block in fp32 on the dequantised weights, without casts, for given experts and weights."""
        def norm(v, w):
            return v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-6) * w

        r = residual.float()
        x = norm(r, self.norm_before)
        up, down = (codes.float() * sf.unsqueeze(2) for codes, sf in (self.up_int8, self.down_int8))
        y = torch.zeros_like(r)
        for k in range(self.topk):
            at = ids[:, k].clamp_min(0)  # a masked token's weight is 0
            g, u = torch.bmm(up[at], x.unsqueeze(2)).squeeze(2).chunk(2, 1)
            v = torch.nn.functional.silu(g) * u
            y += weights[:, k:k + 1] * torch.bmm(down[at], v.unsqueeze(2)).squeeze(2)
        out = r + self.gate * norm(y, self.norm_after)
        return out, norm(out, self.norm_next)

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


class Route(torch.autograd.Function):
    """The router's weights as a differentiable function of its logits."""

    @staticmethod
    def forward(ctx, logits, topk, score):
        ids, weights = moe.moe_router(logits, topk, score=score, renormalize=True)
        ctx.save_for_backward(logits, ids)
        ctx.score = score
        ctx.mark_non_differentiable(ids)
        return weights, ids

    @staticmethod
    def backward(ctx, grad_weights, _):
        logits, ids = ctx.saved_tensors
        return moe.moe_router_backward(grad_weights.contiguous(), logits, ids, score=ctx.score,
                                       renormalize=True), None, None


def router_gradient(x, router, values, topk, score="sigmoid"):
    """d/d router of sum over tokens and choices of weights * values[token, expert], through the kernels."""
    router = router.detach().requires_grad_()
    weights, ids = Route.apply(x @ router, topk, score)
    (weights * values.gather(1, ids)).sum().backward()
    return router.grad, ids


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
    out, normed, ids, weights = block.serve_int8(residual)
    for name, a, b in zip(("residual", "next input"), (out, normed), block.int8_plain(residual, ids, weights)):
        print(f"serving in 8-bit integers, {name}: {float((a.float() - b).norm() / b.norm()):.4f} from the fp32 block")
    first, last = train_router()
    print(f"balance loss: {first:.3f} -> {last:.3f}")
    first, last = train_norm()
    print(f"block norm fit: squared error {first:.4f} -> {last:.4f}")


if __name__ == "__main__":
    main()
