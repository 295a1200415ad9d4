"""Cases of the operators around and inside the MoE block: the norms before and after it, the router's balance loss,
and the experts' products with 4-bit weights.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits, rounded once at the end), or
calls the framework's entry point where ``own`` is true.  ``exact`` computes the same outputs in 64 bits from the
definition.  Shapes are those of the repository's workloads (hidden 7168, 256 experts, top-8, expert width 2048; the
64-token workload with 16 experts, top-2, hidden 256) and odd sizes between them.
"""
import torch

own = False

DEV = "cuda"
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZES = {"bf16": 2, "f32": 4}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
# the largest drawn cases stay within the largest listed ones
NORM_MOST = 4096 * 7168
BALANCE_MOST = 32768 * 256
MATVEC_MOST = 32 * 4096 * 7168


def _norm(name, way, tokens, hidden, act, res, post, gate, block=True):
    return {"name": name, "op": "norm", "pass": way, "tokens": tokens, "hidden": hidden, "act": act, "res": res,
            "block": block, "post": post, "gate": gate, "scale": 1.0 if gate == "none" else 0.875}


def _balance(name, way, tokens, experts, topk, dtype, score, seqs, masked):
    return {"name": name, "op": "balance", "pass": way, "tokens": tokens, "experts": experts, "topk": topk,
            "dtype": dtype, "score": score, "seqs": seqs, "masked": masked}


def _matvec(name, experts, tokens, topk, out, inner, x, group, sf, by_token):
    return {"name": name, "op": "matvec", "experts": experts, "tokens": tokens, "topk": topk, "out": out,
            "inner": inner, "x": x, "group": group, "sf": sf, "by_token": by_token}


def listed():
    return [
        # one token through a layer while serving: latency
        _norm("norm, one token", "forward", 1, 7168, "bf16", "bf16", True, "token"),
        # a prompt's batch: post-norm, layer scale, residual and the next block's pre-norm
        _norm("norm, prompt", "forward", 4096, 7168, "bf16", "bf16", True, "channel"),
        # training, a residual stream kept in 32 bits
        _norm("norm, backward", "backward", 4096, 7168, "bf16", "f32", True, "channel"),
        # training at sizes that fill no vector and no wave
        _norm("norm, odd backward", "backward", 1021, 2049, "bf16", "bf16", True, "token"),
        # the 64-token workload: load statistics for a small step
        _balance("balance, small batch", "forward", 64, 16, 2, "f32", "softmax", 1, False),
        # a layer's batch of eight packed sequences, sigmoid scores
        _balance("balance, packed layer", "train", 4096, 256, 8, "bf16", "sigmoid", 8, False),
        # the large workload: one batch-wide loss and its gradient
        _balance("balance, large batch", "train", 32768, 256, 8, "f32", "softmax", 1, False),
        # many short sequences, some empty, padded tokens masked out, an odd number of experts
        _balance("balance, short ragged", "train", 10007, 61, 4, "f32", "softmax", 311, True),
        # a shared expert's down projection for one token
        _matvec("matvec, shared expert", 1, 1, 1, 7168, 2048, "bf16", 32, "ue8m0", False),
        # one token's eight experts, gate and up, read by token without an expand
        _matvec("matvec, one token", 256, 1, 8, 4096, 7168, "bf16", 32, "ue8m0", True),
        # a decode batch on one of eight ranks (32 local experts): e4m3 rows as the dispatch writes them
        _matvec("matvec, gate and up", 32, 128, 1, 4096, 7168, "e4m3", 32, "ue8m0", False),
        # the same batch's down projection, more rows to an expert, scales in fp32 over 128 channels
        _matvec("matvec, down", 32, 512, 1, 7168, 2048, "bf16", 128, "f32", False),
    ]


def _between(rng, lo, hi):
    """A whole number, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("norm", "balance", "matvec"))
    if op == "norm":
        hidden = rng.choice((_between(rng, 64, 8192), 8 * _between(rng, 8, 1024), 7168))
        block = rng.random() < 0.8
        c = _norm("", rng.choice(("forward", "backward")), _between(rng, 1, min(16384, NORM_MOST // hidden)), hidden,
                  rng.choice(("bf16", "bf16", "f32")), rng.choice(("bf16", "f32")), rng.random() < 0.7,
                  rng.choice(("none", "channel", "token")) if block else "none", block)
        if c["act"] == "f32":
            c["res"] = "f32"
        if not block:
            c["post"] = False
    elif op == "balance":
        experts = rng.choice((_between(rng, 2, 1024), 8 * _between(rng, 1, 64), 256))
        tokens = _between(rng, 1, min(65536, BALANCE_MOST // experts))
        seqs = rng.choice((1, 1, _between(rng, 1, min(512, max(1, tokens // 4)))))
        c = _balance("", rng.choice(("forward", "train")), tokens, experts, min(experts, rng.choice((1, 2, 4, 6, 8))),
                     rng.choice(("f32", "bf16")), rng.choice(("softmax", "sigmoid")), seqs, rng.random() < 0.4)
    else:
        experts = rng.choice((1, _between(rng, 2, 64)))
        x = rng.choice(("bf16", "e4m3"))
        group, sf = rng.choice(((32, "ue8m0"), (32, "ue8m0"), (32, "f32"), (128, "ue8m0"), (128, "f32")))
        step = 128 if x == "e4m3" or group == 128 else 32
        inner = step * _between(rng, 1, 7168 // step)
        out = rng.choice((_between(rng, 1, 7168), 256, 64 * _between(rng, 1, 112)))
        out = max(1, min(out, MATVEC_MOST // (experts * inner)))
        topk = rng.choice((1, 2, 8))
        topk = min(topk, experts)
        c = _matvec("", experts, max(1, _between(rng, 1, 256) // topk), topk, out, inner, x, group, sf,
                    rng.random() < 0.4)
    del c["name"]
    return c


def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _prepare_norm(c, seed):
    g = _generator(seed)
    T, H = c["tokens"], c["hidden"]

    def normal(*shape, dtype=torch.float32, outliers=False):
        v = torch.randn(*shape, generator=g, device=DEV)
        if outliers:
            v = torch.where(torch.rand(*shape, generator=g, device=DEV) < 0.01, 50.0 * v, v)
        return v.to(dtype)

    act, res = DTYPES[c["act"]], DTYPES[c["res"]]
    s = {"case": c, "scale": c["scale"], "y": normal(T, H, dtype=act) if c["block"] else None,
         "post_weight": 1 + 0.1 * normal(H) if c["post"] else None, "pre_weight": 1 + 0.1 * normal(H),
         "gate": {"none": None, "channel": 0.3 * normal(H), "token": torch.sigmoid(normal(T, 1))}[c["gate"]]}
    if c["pass"] == "forward":
        s["residual"] = normal(T, H, dtype=res, outliers=True)
        s["out"] = (torch.empty(T, H, dtype=res, device=DEV) if c["block"] else None,
                    torch.empty(T, H, dtype=act, device=DEV),
                    torch.empty(T, device=DEV) if c["post"] else None, torch.empty(T, device=DEV))
        return s
    # what the forward pass left, and the gradients that arrive
    s["res_out"] = normal(T, H, dtype=res, outliers=True)
    s["pre_rstd"] = torch.rsqrt(s["res_out"].float().square().mean(1) + EPS)
    s["post_rstd"] = torch.rsqrt(s["y"].float().square().mean(1) + EPS) if c["post"] else None
    s["grad_res_out"], s["grad_normed"] = normal(T, H, dtype=res), normal(T, H, dtype=act)
    s["out"] = {"grad_residual": torch.empty(T, H, dtype=res, device=DEV),
                "grad_y": torch.empty(T, H, dtype=act, device=DEV) if c["block"] else None,
                "grad_post_weight": torch.empty(H, device=DEV) if c["post"] else None,
                "grad_gate": torch.empty_like(s["gate"]) if s["gate"] is not None else None,
                "grad_pre_weight": torch.empty(H, device=DEV)}
    return s


def _prepare_balance(c, seed):
    g = _generator(seed)
    T, E, S = c["tokens"], c["experts"], c["seqs"]
    # the experts' popularity differs, as in an unbalanced router
    logits = torch.randn(T, E, generator=g, device=DEV) + 0.7 * torch.randn(E, generator=g, device=DEV)
    logits = logits.to(DTYPES[c["dtype"]])
    ids = logits.float().topk(c["topk"], dim=1).indices
    s = {"case": c, "topk_idx": ids, "score": c["score"], "seq_offsets": None, "token_mask": None}
    if S > 1:  # cuts anywhere: some sequences are empty, the last tokens belong to none
        cuts = torch.randint(0, T + 1, (S + 1,), generator=g, device=DEV).sort().values
        cuts[0] = 0
        s["seq_offsets"] = cuts.to(torch.int32)
    if c["masked"]:  # padded tokens hold anything
        s["token_mask"] = torch.rand(T, generator=g, device=DEV) >= 0.15
        junk = torch.rand(T, generator=g, device=DEV) < 0.5
        logits[junk & ~s["token_mask"]] = float("nan")
    s["logits"] = logits
    s["grad_loss"] = (0.5 + torch.rand(S, generator=g, device=DEV)) / S
    s["out"] = {"loss": torch.empty(S, device=DEV), "counts": torch.empty(S, E, dtype=torch.int32, device=DEV),
                "seq_tokens": torch.empty(S, dtype=torch.int32, device=DEV),
                "prob_mean": torch.empty(S, E, device=DEV)}
    s["grad"] = torch.empty(T, E, dtype=logits.dtype, device=DEV) if c["pass"] == "train" else None
    return s


def _prepare_matvec(c, seed):
    g = _generator(seed)
    E, T, N, K = c["experts"], c["tokens"], c["out"], c["inner"]
    R = T * c["topk"]
    s = {"case": c, "row_token": None, "x_sf": None}
    # each token's copies go to different experts; rows are grouped by expert
    ids = torch.rand(T, E, generator=g, device=DEV).topk(c["topk"], dim=1).indices.flatten()
    s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV),
                              torch.bincount(ids, minlength=E).cumsum(0)]).to(torch.int32)
    s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
    s["rows"] = R
    if c["by_token"]:
        s["row_token"] = (ids.argsort(stable=True) // c["topk"]).to(torch.int32)
    x = torch.randn(T if c["by_token"] else R, K, generator=g, device=DEV)
    if c["x"] == "e4m3":
        v = x.view(x.shape[0], K // 128, 128)
        s["x_sf"] = v.abs().amax(2).clamp_min(1e-4) / 448
        s["x"] = (v / s["x_sf"].unsqueeze(2)).view_as(x).to(torch.float8_e4m3fn)
    else:
        s["x"] = x.to(torch.bfloat16)
    # codes over all sixteen values; scales that give outputs of about one
    s["w"] = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8, device=DEV)
    if c["sf"] == "ue8m0":
        s["w_sf"] = torch.randint(117, 122, (E, N, K // c["group"]), generator=g, dtype=torch.uint8, device=DEV)
    else:
        s["w_sf"] = 0.002 + 0.004 * torch.rand(E, N, K // c["group"], generator=g, device=DEV)
    s["y"] = torch.empty(R, N, dtype=torch.bfloat16, device=DEV)
    return s


def prepare(case, seed):
    return {"norm": _prepare_norm, "balance": _prepare_balance, "matvec": _prepare_matvec}[case["op"]](case, seed)


def _plain_norm_forward(s):
    r, y = s["residual"].float(), s["y"]
    post_rstd = None
    if y is not None:
        u = y.float()
        if s["post_weight"] is not None:
            post_rstd = torch.rsqrt((u * u).mean(1) + EPS)
            u = u * post_rstd[:, None] * s["post_weight"]
        r = s["scale"] * r + (u if s["gate"] is None else s["gate"] * u)
    pre_rstd = torch.rsqrt((r * r).mean(1) + EPS)
    normed = (r * pre_rstd[:, None] * s["pre_weight"]).to(DTYPES[s["case"]["act"]])
    return r.to(s["residual"].dtype) if y is not None else None, normed, post_rstd, pre_rstd


def _plain_norm_backward(s):
    y, gate = s["y"], s["gate"]
    dn, rstd = s["grad_normed"].float(), s["pre_rstd"][:, None]
    xh = s["res_out"].float() * rstd
    g = dn * s["pre_weight"]
    d = s["grad_res_out"].float() + rstd * (g - xh * (g * xh).mean(1, keepdim=True))
    o = {"grad_residual": (s["scale"] * d).to(s["res_out"].dtype), "grad_y": None, "grad_post_weight": None,
         "grad_gate": None, "grad_pre_weight": (dn * xh).sum(0)}
    if y is not None:
        yh = y.float() * (s["post_rstd"][:, None] if s["post_weight"] is not None else 1)
        u = yh * s["post_weight"] if s["post_weight"] is not None else yh
        if gate is not None:
            o["grad_gate"] = (d * u).sum(0) if gate.dim() == 1 else (d * u).sum(1, keepdim=True)
            d = gate * d
        if s["post_weight"] is not None:
            o["grad_post_weight"] = (d * yh).sum(0)
            h = d * s["post_weight"]
            d = s["post_rstd"][:, None] * (h - yh * (h * yh).mean(1, keepdim=True))
        o["grad_y"] = d.to(y.dtype)
    return o


def _plain_balance(s):
    c, S = s["case"], s["case"]["seqs"]
    T, E, K = c["tokens"], c["experts"], c["topk"]
    live = s["token_mask"] if s["token_mask"] is not None else torch.ones(T, dtype=torch.bool, device=DEV)
    seq = torch.zeros(T, dtype=torch.int64, device=DEV)
    if s["seq_offsets"] is not None:
        seq = torch.bucketize(torch.arange(T, device=DEV, dtype=torch.int32), s["seq_offsets"], right=True) - 1
        live = live & (seq < S)
        seq = seq.clamp(max=S - 1)
    z = torch.where(live[:, None], s["logits"].float(), 0.0)
    sig = torch.sigmoid(z)
    p = torch.softmax(z, 1) if s["score"] == "softmax" else sig / sig.sum(1, keepdim=True)
    p = p * live[:, None]
    n = torch.zeros(S, dtype=torch.int32, device=DEV).index_add_(0, seq, live.int())
    sums = p.sum(0)[None] if S == 1 else torch.zeros(S, E, device=DEV).index_add_(0, seq, p)
    at = (seq[:, None] * E + s["topk_idx"]).flatten()
    counts = torch.zeros(S * E, dtype=torch.int32, device=DEV)
    counts = counts.index_add_(0, at, live.int().repeat_interleave(K)).view(S, E)
    many = n.float().clamp_min(1)
    mean = sums / many[:, None]
    loss = (counts.float() * mean).sum(1) * (E / K) / many
    o = {"loss": loss, "counts": counts, "seq_tokens": n, "prob_mean": mean}
    if c["pass"] == "train":
        a = counts.float() * (s["grad_loss"] * (E / K) / (many * many))[:, None]
        a = a[seq]
        d = p * (a - (a * p).sum(1, keepdim=True))
        o["grad"] = (d if s["score"] == "softmax" else d * (1 - sig)).to(s["logits"].dtype)
    return o


def _plain_matvec(s):
    c, off, R = s["case"], s["offsets"].long(), s["rows"]
    E, N, K, G = c["experts"], c["out"], c["inner"], c["inner"] // c["group"]
    count = off[1:] - off[:-1]
    # at most R experts have rows: only their weights are taken apart
    busy = torch.argsort(count, descending=True, stable=True)[:min(E, R)]
    w, sf = (s["w"], s["w_sf"]) if E <= R else (s["w"][busy], s["w_sf"][busy])
    if E <= R:
        busy = torch.arange(E, device=DEV)
    A = w.shape[0]
    value = torch.tensor(E2M1, device=DEV)
    byte = torch.arange(256, device=DEV)
    pair = torch.stack([value[byte & 15], value[byte >> 4]], 1)
    if c["sf"] == "ue8m0":
        sf = (sf.int() << 23).view(torch.float32)
    w = (pair[w.int()].view(A, N, G, c["group"]) * sf[..., None]).view(A, N, K)
    x = s["x"].float()
    if s["x_sf"] is not None:
        x = x * s["x_sf"].repeat_interleave(128, dim=1)
    slot = torch.arange(s["most"], device=DEV)
    row = (off[busy][:, None] + slot).clamp(max=R - 1)
    x = x[s["row_token"].long()[row] if s["row_token"] is not None else row]
    y = torch.matmul(x, w.transpose(1, 2))  # [A, most, N]
    r = torch.arange(R, device=DEV)
    e = torch.bucketize(r, off, right=True) - 1
    place = torch.zeros(E, dtype=torch.int64, device=DEV).index_copy_(0, busy, torch.arange(A, device=DEV))
    return y[place[e], r - off[e]].to(torch.bfloat16)


def _own(s):
    import moe_routing_fp8_amd as moe

    c = s["case"]
    if c["op"] == "norm" and c["pass"] == "forward":
        return moe.moe_block_norm(s["residual"], s["y"], post_weight=s["post_weight"], gate=s["gate"],
                                  residual_scale=s["scale"], pre_weight=s["pre_weight"], eps=EPS, out=s["out"])
    if c["op"] == "norm":
        return moe.moe_block_norm_backward(s["grad_res_out"], s["grad_normed"], s["res_out"], s["y"],
                                           post_weight=s["post_weight"], gate=s["gate"], residual_scale=s["scale"],
                                           pre_weight=s["pre_weight"], post_rstd=s["post_rstd"],
                                           pre_rstd=s["pre_rstd"], out=s["out"])
    if c["op"] == "balance":
        o = moe.moe_balance_loss(s["logits"], s["topk_idx"], score=s["score"], token_mask=s["token_mask"],
                                 seq_offsets=s["seq_offsets"], out=s["out"])
        if c["pass"] == "train":
            grad = moe.moe_balance_loss_backward(s["grad_loss"], s["logits"], o["counts"], o["seq_tokens"],
                                                 c["topk"], score=s["score"], token_mask=s["token_mask"],
                                                 seq_offsets=s["seq_offsets"], out=s["grad"])
            o = {**o, "grad": grad}
        return o
    return moe.moe_expert_matvec(s["x"], s["w"], s["w_sf"], x_sf=s["x_sf"], expert_offsets=s["offsets"],
                                 row_token=s["row_token"], out=s["y"])


def run(state):
    if own:
        return _own(state)
    c = state["case"]
    if c["op"] == "norm":
        return _plain_norm_forward(state) if c["pass"] == "forward" else _plain_norm_backward(state)
    return _plain_balance(state) if c["op"] == "balance" else _plain_matvec(state)


def work(case):
    c = case
    if c["op"] == "norm":
        T, H, a, r = c["tokens"], c["hidden"], SIZES[c["act"]], SIZES[c["res"]]
        vectors = 4 * H * (1 + c["post"] + (c["gate"] == "channel")) + 4 * T * (1 + c["post"] + (c["gate"] == "token"))
        if c["pass"] == "forward":
            return {"bytes": T * H * (2 * (a + r) if c["block"] else a + r) + vectors,
                    "flops": T * H * (12 if c["block"] else 4)}
        return {"bytes": T * H * (3 * (a + r) if c["block"] else a + 3 * r) + 2 * vectors,
                "flops": T * H * (28 if c["block"] else 12)}
    if c["op"] == "balance":
        T, E, K, S, z = c["tokens"], c["experts"], c["topk"], c["seqs"], SIZES[c["dtype"]]
        back = c["pass"] == "train"
        # a gradient needs the counts of the whole sequence: the logits are read twice
        return {"bytes": T * E * z * (3 if back else 1) + 8 * T * K + 8 * S * E + 16 * S + (T if c["masked"] else 0),
                "flops": T * E * (20 if back else 8)}
    E, T, k, N, K = c["experts"], c["tokens"], c["topk"], c["out"], c["inner"]
    busy = E * (1 - (1 - k / E) ** T)  # the experts that a batch is expected to reach
    x = (T if c["by_token"] else T * k) * (2 * K if c["x"] == "bf16" else K + 4 * (K // 128))
    return {"bytes": busy * N * (K // 2 + K // c["group"] * (1 if c["sf"] == "ue8m0" else 4)) + x + 2 * T * k * N,
            "flops": 2 * T * k * N * K}


def _exact_norm(s):
    def wide(t):
        return None if t is None else t.double()

    y, wp, wn, gate, scale = wide(s["y"]), wide(s["post_weight"]), wide(s["pre_weight"]), wide(s["gate"]), s["scale"]
    if s["case"]["pass"] == "forward":
        out, post, h = wide(s["residual"]), None, None
        if y is not None:
            h = y
            if wp is not None:
                post = (y.pow(2).sum(1) / y.shape[1] + EPS).pow(-0.5)
                h = torch.einsum("th,t,h->th", y, post, wp)
            out = out * scale + (h if gate is None else h * gate)
        pre = (out.pow(2).sum(1) / out.shape[1] + EPS).pow(-0.5)
        return out if y is not None else None, torch.einsum("th,t,h->th", out, pre, wn), post, pre
    # the Jacobian of a row's norm, applied: J v = rstd * (v - xh <xh, v> / H)
    H = s["case"]["hidden"]
    a, dn = wide(s["pre_rstd"]).unsqueeze(1), wide(s["grad_normed"])
    xh = wide(s["res_out"]) * a
    v = dn * wn
    total = wide(s["grad_res_out"]) + a * v - a * xh * ((xh * v).sum(1, keepdim=True) / H)
    o = {"grad_residual": total * scale, "grad_y": None, "grad_post_weight": None, "grad_gate": None,
         "grad_pre_weight": torch.einsum("th,th->h", dn, xh)}
    if y is None:
        return o
    yh = y if wp is None else y * wide(s["post_rstd"]).unsqueeze(1)
    into = total if gate is None else total * gate
    if gate is not None:
        along = total * yh * (1.0 if wp is None else wp)
        o["grad_gate"] = along.sum(0) if s["case"]["gate"] == "channel" else along.sum(1).unsqueeze(1)
    o["grad_y"] = into
    if wp is not None:
        o["grad_post_weight"] = torch.einsum("th,th->h", into, yh)
        b, v = wide(s["post_rstd"]).unsqueeze(1), into * wp
        o["grad_y"] = b * v - b * yh * ((yh * v).sum(1, keepdim=True) / H)
    return o


def _exact_balance(s):
    c = s["case"]
    T, E, K, S = c["tokens"], c["experts"], c["topk"], c["seqs"]
    ends = [0, T] if s["seq_offsets"] is None else s["seq_offsets"].tolist()
    live = torch.ones(T, dtype=torch.bool, device=DEV) if s["token_mask"] is None else s["token_mask"].clone()
    z = s["logits"].double()
    o = {"loss": torch.zeros(S, dtype=torch.float64, device=DEV), "counts": None, "seq_tokens": None,
         "prob_mean": torch.zeros(S, E, dtype=torch.float64, device=DEV)}
    grad = torch.zeros(T, E, dtype=torch.float64, device=DEV)
    for q in range(S):
        rows = torch.arange(ends[q], ends[q + 1], device=DEV)
        rows = rows[live[rows]]
        n = rows.numel()
        if n == 0:
            continue
        w = torch.exp(z[rows] - z[rows].amax(1, keepdim=True)) if s["score"] == "softmax" else 1 / (1 + torch.exp(-z[rows]))
        p = w / w.sum(1, keepdim=True)
        f = torch.bincount(s["topk_idx"][rows].flatten(), minlength=E).double() * (E / (K * n))
        o["prob_mean"][q] = p.mean(0)
        o["loss"][q] = f @ p.mean(0)
        # d loss / d p = f / n, through the normalisation, then through the score
        up = (f / n)[None] * s["grad_loss"][q].double()
        through = p * (up - (up * p).sum(1, keepdim=True))
        grad[rows] = through if s["score"] == "softmax" else through * (1 - w)
    if c["pass"] == "train":
        o["grad"] = grad
    return o


def _exact_matvec(s):
    c, ends = s["case"], s["offsets"].tolist()
    value = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    x = s["x"].double()
    if s["x_sf"] is not None:
        x = (x.view(x.shape[0], -1, 128) * s["x_sf"].double().unsqueeze(2)).view(x.shape)
    if s["row_token"] is not None:
        x = x[s["row_token"].long()]
    out = torch.zeros(s["rows"], c["out"], dtype=torch.float64, device=DEV)
    for e in range(c["experts"]):
        if ends[e] == ends[e + 1]:
            continue
        codes = torch.stack([s["w"][e] % 16, s["w"][e] // 16], 2).view(c["out"], c["inner"])
        sf = s["w_sf"][e].double()
        sf = torch.pow(2.0, sf - 127) if c["sf"] == "ue8m0" else sf
        w = value[codes.long()] * sf.repeat_interleave(c["group"], 1)
        out[ends[e]:ends[e + 1]] = x[ends[e]:ends[e + 1]] @ w.T
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "balance": _exact_balance, "matvec": _exact_matvec}[case["op"]](s)
