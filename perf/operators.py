"""Measured cases of the operators that train a pre-norm OmniMoE layer beside its routed forward and backward:

  balance    per-expert counts, the balance loss over the implicit N_r x N_c grid, and its gradients to the tokens
             and the router's weights
  norm       layer norm, forward (with or without an 8-bit checkpoint of the normalised rows) and backward (from the
             kept input, or from that checkpoint), with the sums of the weight's and bias's gradients
  ckpt       activations packed to 8 bits (e4m3 with one power-of-two scale per 32 values) and restored, and the
             routed backward that takes its tokens from such a checkpoint

With own = False `run` computes them in elementary torch operations; with own = True it calls this package.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 32          # values that share a scale in an 8-bit checkpoint
EPS = 1e-5


def listed():
    return [
        # a check-sized layer: what a unit test or a first training step runs; launch latency counts
        {"name": "balance-tiny", "kind": "balance", "L": 256, "d": 256, "N_r": 64, "N_c": 64, "K": 16, "zipf": False, "masked": False},
        # the headline layer's training step: 1.7M experts, about 20 tasks in a group
        {"name": "balance-headline", "kind": "balance", "L": 4096, "d": 1024, "N_r": 1304, "N_c": 1304, "K": 64, "zipf": False, "masked": False},
        # the collapse that the loss is there to undo: few rows and columns take most tasks, counts far above 256
        {"name": "balance-skew", "kind": "balance", "L": 16384, "d": 2048, "N_r": 1024, "N_c": 1024, "K": 128, "zipf": True, "masked": False},
        # a padded batch with no size a power of two
        {"name": "balance-ragged", "kind": "balance", "L": 1777, "d": 776, "N_r": 515, "N_c": 389, "K": 33, "zipf": True, "masked": True},
        # the loss and the counts alone, as a validation step logs them
        {"name": "balance-fwd-small", "kind": "balance_fwd", "L": 4096, "d": 768, "N_r": 512, "N_c": 512, "K": 64, "zipf": False, "masked": False},
        # one decoded token before the layer: latency
        {"name": "norm-one-token", "kind": "norm", "L": 1, "d": 2048, "f32": False, "bias": True, "ckpt": False},
        # the headline layer's norm on the fp32 residual stream, keeping its checkpoint
        {"name": "norm-headline-ckpt", "kind": "norm", "L": 4096, "d": 1024, "f32": True, "bias": True, "ckpt": True},
        # its backward from the kept fp32 input
        {"name": "norm-bwd-headline", "kind": "norm_bwd", "L": 4096, "d": 1024, "f32": True, "bias": True, "ckpt": False},
        # the widest layer's backward from the checkpoint
        {"name": "norm-bwd-ckpt-wide", "kind": "norm_bwd", "L": 16384, "d": 2048, "f32": False, "bias": True, "ckpt": True},
        # a long prefill's activations, packed after the forward and restored before the backward
        {"name": "ckpt-long", "kind": "ckpt", "L": 65536, "d": 2048, "f32": False},
        # the check-sized layer's routed backward from a checkpoint
        {"name": "bwd-ckpt-tiny", "kind": "bwd_ckpt", "L": 256, "d": 256, "N_r": 64, "N_c": 64, "K": 16, "affine": True},
        # an ordinary layer's routed backward from a checkpoint
        {"name": "bwd-ckpt-d1024", "kind": "bwd_ckpt", "L": 2048, "d": 1024, "N_r": 256, "N_c": 256, "K": 64, "affine": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["balance", "balance", "balance_fwd", "norm", "norm_bwd", "ckpt", "bwd_ckpt"])
    if kind in ("balance", "balance_fwd"):
        N_r, N_c = _log_int(rng, 16, 1304), _log_int(rng, 16, 1304)
        return {"kind": kind, "L": _log_int(rng, 64, 8192), "d": 8 * _log_int(rng, 8, 256), "N_r": N_r, "N_c": N_c,
                "K": min(_log_int(rng, 1, 128), N_r * N_c // 2), "zipf": rng.random() < 0.5, "masked": rng.random() < 0.5}
    if kind in ("norm", "norm_bwd"):
        ckpt = rng.random() < 0.5
        d = BLOCK * _log_int(rng, 2, 128) if ckpt else 8 * _log_int(rng, 8, 512)
        return {"kind": kind, "L": _log_int(rng, 1, 16384), "d": d, "f32": rng.random() < 0.5, "bias": rng.random() < 0.7, "ckpt": ckpt}
    if kind == "ckpt":
        return {"kind": kind, "L": _log_int(rng, 16, 32768), "d": BLOCK * _log_int(rng, 2, 128), "f32": rng.random() < 0.5}
    return {"kind": kind, "L": _log_int(rng, 16, 2048), "d": 256 * rng.randint(1, 4), "N_r": _log_int(rng, 32, 256), "N_c": _log_int(rng, 32, 256),
            "K": _log_int(rng, 1, 64), "affine": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs


def _normal(gen, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device=DEV) * std).to(dtype)


def _router_inputs(c, gen):
    """Tokens, router weights and the log-probabilities they give, the way the layer's own workloads draw them."""
    L, d = c["L"], c["d"]
    x = _normal(gen, L, d)
    W = [_normal(gen, n, d, std=d**-0.5) for n in (c["N_r"], c["N_c"])]
    if c.get("zipf"):
        x[:, -1] = 1.0
        for w in W:
            rank = torch.randperm(len(w), generator=gen, device=DEV) + 1
            w[:, -1] = (-1.1 * torch.log(rank.double())).to(w.dtype)
    p = [torch.log_softmax(x.float() @ w.float().T, dim=1) for w in W]
    return x, W, p


def _top_cells(p_r, p_c, K):
    """The K best cells of every token's grid: the best lie at (a, b) with (a + 1)(b + 1) <= K in sorted rows and columns."""
    N_c = p_c.shape[1]
    vr, ir = p_r.topk(min(K, p_r.shape[1]), dim=1)
    vc, ic = p_c.topk(min(K, N_c), dim=1)
    a = torch.arange(1, vr.shape[1] + 1, device=DEV)
    b = torch.arange(1, vc.shape[1] + 1, device=DEV)
    a, b = torch.nonzero(a[:, None] * b[None, :] <= K, as_tuple=True)
    score, at = (vr[:, a] + vc[:, b]).topk(K, dim=1)
    idx = ir[:, a].gather(1, at) * N_c + ic[:, b].gather(1, at)
    return idx.to(torch.int32), torch.softmax(score, dim=1)


def _pow2(code):
    """2^(code - 127), the value of a scale byte (2^-127 too, which is below the smallest normal number)."""
    return torch.exp2(code.double() - 127.0).float()


def _pack(x):
    """Blocks of 32 values as e4m3 times the smallest power of two that lets none pass 448."""
    v = x.float().reshape(len(x), -1, BLOCK)
    m, e = torch.frexp(v.abs().amax(dim=2))                      # amax = m 2^e, m in [0.5, 1)
    code = (e - 9 + (m > 448 / 512).to(e.dtype) + 127).clamp(0, 254)
    code = torch.where(m == 0, torch.zeros_like(code), code)
    q = (v.double() * torch.exp2(127.0 - code.double())[..., None]).float().to(torch.float8_e4m3fn)
    return q.reshape(x.shape).view(torch.uint8), code.to(torch.uint8)


def _values(q, scale):
    """What a checkpoint's bytes stand for, in 32 bits."""
    v = q.view(torch.float8_e4m3fn).float().reshape(*scale.shape, BLOCK)
    return (v * _pow2(scale)[..., None]).reshape(q.shape)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    c, s = case, dict(case)
    kind, L, d = c["kind"], c["L"], c["d"]
    if kind in ("balance", "balance_fwd"):
        s["x"], (s["W_r"], s["W_c"]), (s["p_r"], s["p_c"]) = _router_inputs(c, gen)
        s["idx"], _ = _top_cells(s["p_r"], s["p_c"], c["K"])
        # sequences padded at their ends: about a fifth of the rows, the first one kept
        s["mask"] = torch.rand(L, generator=gen, device=DEV) > 0.2 if c["masked"] else None
        if c["masked"]:
            s["mask"][0] = True
        s["dloss"] = 0.01                                         # the loss's weight in the training objective
    elif kind in ("norm", "norm_bwd"):
        # a residual stream: rows of their own mean and width
        x = torch.randn(L, d, generator=gen, device=DEV) * (0.5 + 2 * torch.rand(L, 1, generator=gen, device=DEV)) + torch.randn(L, 1, generator=gen, device=DEV)
        s["x"] = x if c["f32"] else x.to(torch.bfloat16)
        s["w"] = (1 + 0.2 * torch.randn(d, generator=gen, device=DEV)).to(torch.bfloat16)
        s["b"] = _normal(gen, d, std=0.2) if c["bias"] else None
        if kind == "norm_bwd":
            s["dy"] = torch.randn(L, d, generator=gen, device=DEV)
            v = s["x"].double()
            mean = v.mean(dim=1)
            rstd = ((v - mean[:, None]).square().mean(dim=1) + EPS).rsqrt()
            s["mean"], s["rstd"] = mean.float(), rstd.float()
            if c["ckpt"]:
                s["q"], s["scale"] = _pack(((v - mean[:, None]) * rstd[:, None]).float())
                del s["x"], s["mean"]
    elif kind == "ckpt":
        s["x"] = _normal(gen, L, d, dtype=torch.float32 if c["f32"] else torch.bfloat16)
    else:
        N = c["N_r"] * c["N_c"]
        n, (s["W_r"], s["W_c"]), p = _router_inputs(c, gen)
        s["idx"], s["gate"] = _top_cells(*p, c["K"])
        s["q"], s["scale"] = _pack(n)
        s["W"], s["V"] = (_normal(gen, N, d, std=d**-0.5) for _ in range(2))
        s["w"] = (1 + 0.2 * torch.randn(d, generator=gen, device=DEV)).to(torch.bfloat16) if c["affine"] else None
        s["b"] = _normal(gen, d, std=0.2) if c["affine"] else None
        s["dy"] = torch.randn(L, d, generator=gen, device=DEV)
    return s


# ------------------------------------------------------------- plain forms


def _balance_plain(s, backward):
    L, K, N_r, N_c = s["L"], s["K"], s["N_r"], s["N_c"]
    N = N_r * N_c
    keep = torch.ones(L, dtype=torch.int32, device=DEV) if s["mask"] is None else s["mask"].to(torch.int32)
    counts = torch.zeros(N, dtype=torch.int32, device=DEV)
    counts.scatter_add_(0, s["idx"].reshape(-1).long(), keep[:, None].expand(L, K).reshape(-1))
    n = keep.sum()
    on = keep[:, None] != 0
    P_r = torch.where(on, torch.exp(s["p_r"]), 0.0)
    P_c = torch.where(on, torch.exp(s["p_c"]), 0.0)
    F = counts.float().reshape(N_r, N_c)
    U = P_c @ F.T                                                 # [L, N_r]
    each = (P_r.double() * U.double()).sum(dim=1)
    factor = N / (K * n.double() * n.double())
    loss = (factor * each.sum()).float()
    if not backward:
        return {"counts": counts, "loss": loss, "token_loss": each.float()}
    scale = (s["dloss"] * factor).float()
    ds_r = scale * P_r * (U - each.float()[:, None])
    ds_c = scale * P_c * (P_r @ F - each.float()[:, None])
    x = torch.where(on, s["x"].float(), 0.0)
    return {"counts": counts, "loss": loss, "token_loss": each.float(), "dx": ds_r @ s["W_r"].float() + ds_c @ s["W_c"].float(),
            "dW_r": ds_r.T @ x, "dW_c": ds_c.T @ x}


def _norm_plain(s):
    x = s["x"].float()
    mean = x.mean(dim=1, keepdim=True)
    rstd = torch.rsqrt((x - mean).square().mean(dim=1, keepdim=True) + EPS)
    hat = (x - mean) * rstd
    y = hat * s["w"].float()
    if s["b"] is not None:
        y = y + s["b"].float()
    out = {"y": y.to(torch.bfloat16), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if s["ckpt"]:
        out["restored"] = _values(*_pack(hat)).to(torch.bfloat16)
    return out


def _norm_bwd_plain(s):
    rstd = s["rstd"][:, None]
    hat = _values(s["q"], s["scale"]) if s["ckpt"] else (s["x"].float() - s["mean"][:, None]) * rstd
    g = s["dy"] * s["w"].float()
    dx = rstd * (g - g.mean(dim=1, keepdim=True) - hat * (g * hat).mean(dim=1, keepdim=True))
    return {"dx": dx, "dw": (s["dy"] * hat).sum(dim=0), "db": s["dy"].sum(dim=0) if s["b"] is not None else None}


def _bwd_plain(s):
    N_c, d = s["N_c"], s["d"]
    x = _values(s["q"], s["scale"])
    if s["w"] is not None:
        x = x * s["w"].float() + s["b"].float()
    x = x.to(torch.bfloat16).float()                              # the layer's operand type
    e, g, dy = s["idx"].long(), s["gate"], s["dy"]
    w, v = s["W"][e].float(), s["V"][e].float()                   # [L, K, d]
    h = (w * x[:, None]).sum(dim=2)
    c = (v * dy[:, None]).sum(dim=2)
    sig = 1 / (1 + torch.exp(-h))
    a = h * sig
    dh = g * c * sig * (1 + h * (1 - sig))
    dgate = a * c
    dS = g * (dgate - (g * dgate).sum(dim=1, keepdim=True))
    i, j = e // N_c, e % N_c
    dx = (dh[..., None] * w).sum(dim=1)
    dx += (dS[..., None] * (s["W_r"][i].float() + s["W_c"][j].float())).sum(dim=1)
    sums = [torch.zeros(len(s[k]), d, device=DEV) for k in ("W", "V", "W_r", "W_c")]
    sums[0].index_add_(0, e.reshape(-1), (dh[..., None] * x[:, None]).reshape(-1, d))
    sums[1].index_add_(0, e.reshape(-1), ((g * a)[..., None] * dy[:, None]).reshape(-1, d))
    task = (dS[..., None] * x[:, None]).reshape(-1, d)
    sums[2].index_add_(0, i.reshape(-1), task)
    sums[3].index_add_(0, j.reshape(-1), task)
    return {"dx": dx, "dW": sums[0], "dV": sums[1], "dW_r": sums[2], "dW_c": sums[3]}


# ------------------------------------------------------- the package's calls


def _balance_own(s, backward):
    import atomic_expert_layer_b200 as omni

    cnt = omni.expert_counts(s["idx"], s["N_r"] * s["N_c"], mask=s["mask"])
    fwd = omni.balance_fwd(s["p_r"], s["p_c"], cnt["counts"], cnt["n_tokens"], s["K"], mask=s["mask"])
    out = {"counts": cnt["counts"], "loss": fwd["loss"], "token_loss": fwd["token_loss"]}
    if backward:
        out |= omni.balance_bwd(s["x"], s["W_r"], s["W_c"], s["p_r"], s["p_c"], cnt["counts"], cnt["n_tokens"], s["K"], fwd["token_loss"],
                                dloss=s["dloss"], mask=s["mask"])
    return out


def _norm_own(s):
    import atomic_expert_layer_b200 as omni

    got = omni.layer_norm_fwd(s["x"], s["w"], s["b"], eps=EPS, ckpt=s["ckpt"])
    out = {"y": got["y"], "mean": got["mean"], "rstd": got["rstd"]}
    if s["ckpt"]:
        out["restored"] = omni.act_unpack(got["q"], got["scale"])
    return out


def _norm_bwd_own(s):
    import atomic_expert_layer_b200 as omni

    kept = {"q": s["q"], "scale": s["scale"]} if s["ckpt"] else {"x": s["x"], "mean": s["mean"]}
    return omni.layer_norm_bwd(s["dy"], s["w"], s["rstd"], bias=s["b"] is not None, **kept)


def _ckpt_own(s):
    import atomic_expert_layer_b200 as omni

    return {"restored": omni.act_unpack(*omni.act_pack(s["x"]))}


def _bwd_own(s):
    import atomic_expert_layer_b200 as omni

    return omni.routed_bwd_ckpt(s["q"], s["scale"], s["W"], s["V"], s["W_r"], s["W_c"], s["idx"], s["gate"], s["dy"], w=s["w"], b=s["b"])


def run(state):
    kind = state["kind"]
    if kind in ("balance", "balance_fwd"):
        return (_balance_own if own else _balance_plain)(state, kind == "balance")
    if kind == "norm":
        return (_norm_own if own else _norm_plain)(state)
    if kind == "norm_bwd":
        return (_norm_bwd_own if own else _norm_bwd_plain)(state)
    if kind == "ckpt":
        return _ckpt_own(state) if own else {"restored": _values(*_pack(state["x"])).to(torch.bfloat16)}
    return (_bwd_own if own else _bwd_plain)(state)


# -------------------------------------------------------------------- work


def work(case):
    c = case
    kind, L, d = c["kind"], c["L"], c["d"]
    if kind in ("balance", "balance_fwd"):
        n, N, K = c["N_r"] + c["N_c"], c["N_r"] * c["N_c"], c["K"]
        mask = L if c["masked"] else 0
        fwd = 4 * L * n + 4 * L * K + 4 * N + 4 * L + 4 + mask
        if kind == "balance_fwd":
            return {"bytes": fwd, "flops": 2 * L * N}
        return {"bytes": fwd + 2 * L * d + 2 * n * d + 4 * L * d + 4 * n * d, "flops": 4 * L * N + 4 * L * d * n}
    packed = d + d / BLOCK                                         # bytes of a row's checkpoint
    x = 4 if c.get("f32") else 2
    if kind == "norm":
        out = 2 * d + 8 + ((packed + 2 * d) if c["ckpt"] else 0)
        return {"bytes": L * (x * d + out) + 2 * d * (2 if c["bias"] else 1), "flops": 8 * L * d}
    if kind == "norm_bwd":
        kept = packed if c["ckpt"] else x * d + 4
        return {"bytes": L * (kept + 4 + 8 * d) + (2 + 4) * d + (4 * d if c["bias"] else 0), "flops": 12 * L * d}
    if kind == "ckpt":
        return {"bytes": L * (x * d + packed + 2 * d), "flops": 4 * L * d}
    N, M = c["N_r"] * c["N_c"], L * c["K"]
    used = min(M, N)                                               # expert rows that some task can use
    n = c["N_r"] + c["N_c"]
    return {"bytes": L * packed + 8 * M + 8 * L * d + 4 * d * used + 8 * N * d + 6 * d * n, "flops": 14 * M * d}


# ------------------------------------------------------------------- exact


def _e4m3(v):
    """The nearest multiple of e4m3's step at v, ties to the even one, in 64 bits."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0**-6)))
    step = torch.exp2(e - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _through_8_bits(v):
    """64-bit values after a checkpoint's rounding."""
    b = v.reshape(len(v), -1, BLOCK)
    top = b.abs().amax(dim=2, keepdim=True)
    two = torch.exp2(torch.ceil(torch.log2(torch.where(top > 0, top, 1.0) / 448)).clamp(min=-127))
    return (_e4m3(b / two) * two).reshape(v.shape)


def _restored64(q, scale):
    bits = q.long()
    e, m = (bits >> 3) & 15, bits & 7
    v = torch.where(e > 0, (8 + m) * torch.exp2(e.double() - 10), m * 2.0**-9) * torch.where(bits > 127, -1.0, 1.0)
    return v * torch.exp2(scale.double() - 127).repeat_interleave(BLOCK, dim=1)


def _exact_balance(s, backward):
    """The definition as a whole, differentiated: N times the sum over the grid of the experts' shares of the tasks and of the probability."""
    L, K, N_r, N_c = s["L"], s["K"], s["N_r"], s["N_c"]
    rows = torch.arange(L, device=DEV) if s["mask"] is None else torch.nonzero(s["mask"])[:, 0]
    n = len(rows)
    counts = torch.bincount(s["idx"][rows].reshape(-1).long(), minlength=N_r * N_c)
    share = counts.double().reshape(N_r, N_c) / (K * n)
    x, W_r, W_c = (s[k].double().requires_grad_(backward) for k in ("x", "W_r", "W_c"))
    logp = []
    for p, w in ((s["p_r"], W_r), (s["p_c"], W_c)):
        moved = x[rows] @ w.T                                      # zero, with the logits' derivative
        z = p[rows].double() + (moved - moved.detach())
        logp.append(z - torch.logsumexp(z, dim=1, keepdim=True) + torch.logsumexp(p[rows].double(), dim=1, keepdim=True))
    pr, pc = logp[0].exp(), logp[1].exp()
    each = torch.einsum("ti,ij,tj->t", pr, share, pc) if N_r * N_c < 4096 else ((pc @ share.T) * pr).sum(dim=1)
    loss = N_r * N_c * each.sum() / n
    token = torch.zeros(L, dtype=torch.float64, device=DEV)
    token[rows] = each.detach() * (K * n)
    out = {"counts": None, "loss": loss.detach(), "token_loss": token}
    if backward:
        (s["dloss"] * loss).backward()
        out |= {"dx": x.grad, "dW_r": W_r.grad, "dW_c": W_c.grad}
    return out


def exact(case, seed):
    s = prepare(case, seed)
    kind = s["kind"]
    if kind in ("balance", "balance_fwd"):
        return _exact_balance(s, kind == "balance")
    if kind == "ckpt":
        return {"restored": _through_8_bits(s["x"].double())}
    if kind == "norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        hat = (x - mean[:, None]) / torch.sqrt(var + EPS)[:, None]
        y = hat * s["w"].double() + (0 if s["b"] is None else s["b"].double())
        out = {"y": y, "mean": mean, "rstd": 1 / torch.sqrt(var + EPS)}
        return out | ({"restored": _through_8_bits(hat)} if s["ckpt"] else {})
    if kind == "norm_bwd":
        dy, rstd = s["dy"].double(), s["rstd"].double()
        hat = _restored64(s["q"], s["scale"]) if s["ckpt"] else (s["x"].double() - s["mean"].double()[:, None]) * rstd[:, None]
        g = dy * s["w"].double()
        d = s["d"]
        pull = g.sum(dim=1) / d
        turn = torch.einsum("ij,ij->i", g, hat) / d
        dx = (g - pull[:, None] - hat * turn[:, None]) * rstd[:, None]
        return {"dx": dx, "dw": torch.einsum("ij,ij->j", dy, hat), "db": dy.sum(dim=0) if s["b"] is not None else None}
    # the routed branch, differentiated with its selection fixed
    x = _restored64(s["q"], s["scale"])
    if s["w"] is not None:
        x = x * s["w"].double() + s["b"].double()
    x = x.float().to(torch.bfloat16).double().requires_grad_()
    e = s["idx"].long()
    i, j = e // s["N_c"], e % s["N_c"]
    leaf = {k: s[k].double().requires_grad_() for k in ("W", "V", "W_r", "W_c")}
    # selected scores whose softmax is the given gates, moving with the router's logits
    moved = torch.einsum("td,tkd->tk", x, leaf["W_r"][i] + leaf["W_c"][j])
    gates = s["gate"].double()
    gate = gates.sum(dim=1, keepdim=True) * torch.softmax(gates.log() + moved - moved.detach(), dim=1)
    h = torch.einsum("td,tkd->tk", x, leaf["W"][e])
    y = torch.einsum("tk,tkd->td", gate * h * torch.sigmoid(h), leaf["V"][e])
    y.backward(s["dy"].double())
    return {"dx": x.grad, "dW": leaf["W"].grad, "dV": leaf["V"].grad, "dW_r": leaf["W_r"].grad, "dW_c": leaf["W_c"].grad}
