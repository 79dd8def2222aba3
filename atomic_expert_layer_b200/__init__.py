"""B200 (sm_100a) routed-branch forward of an OmniMoE layer.

The computation lives in libomni.so (hand-written CUDA, C ABI in
include/omni.h).  This package only loads it and marshals torch tensors:
  - ``omni_*`` functions mirror the C entry points argument for argument;
  - ``router_topk``, ``schedule``, ``grouped_expert_fwd``, ``routed_fwd``,
    ``routed_bwd``, ``shared_mlp_fwd`` and ``layer_fwd`` allocate the output
    tensors and a workspace, then call them.
  - ``expert_counts``, ``balance_fwd``, ``balance_bwd``, ``layer_norm_fwd``,
    ``layer_norm_bwd``, ``act_pack``, ``act_unpack`` and ``routed_bwd_ckpt`` do
    the same for what a training step needs beside the routed branch.  They
    check types, shapes and devices (ValueError), run on the device of their
    tensors whichever is current, and allocate on the stream they run on.
"""
from __future__ import annotations

import contextlib

import torch

from ._lib import (OMNI_ROUTER_LOGPROBS_IN, OMNI_TOKEN_ORDER, OMNI_TOPK_BLOCKWISE,  # noqa: F401
                   OMNI_Y_ACCUMULATE, OMNI_EXPERT_DENSE, OMNI_EXPERT_SPARSE,
                   OMNI_X_F32, OMNI_DX_ACCUMULATE,
                   omni_act_pack, omni_act_unpack, omni_balance_bwd,
                   omni_balance_bwd_workspace_size, omni_balance_fwd,
                   omni_balance_fwd_workspace_size, omni_expert_counts, omni_layer_norm_bwd,
                   omni_layer_norm_bwd_workspace_size, omni_layer_norm_fwd, omni_routed_bwd_ckpt,
                   omni_routed_bwd_ckpt_workspace_size,
                   omni_workspace_size_flags, omni_expert_workspace_size_flags,
                   OmniError, load,
                   expert_workspace, omni_expert_workspace_size, omni_get_device_status,
                   omni_grouped_expert_fwd, omni_grouped_expert_fwd_noalloc,
                   omni_noalloc_get_device_status, omni_routed_bwd,
                   omni_routed_bwd_workspace_size, omni_routed_fwd,
                   omni_router_topk,
                   omni_router_workspace_size, omni_schedule, omni_schedule_workspace_size,
                   omni_selftest_wait_timeout, omni_shared_mlp_fwd,
                   omni_shared_mlp_workspace_size, shared_mlp_workspace,
                   omni_workspace_size, router_workspace, schedule_workspace, workspace)

__all__ = [
    "load", "OmniError", "OMNI_ROUTER_LOGPROBS_IN", "OMNI_Y_ACCUMULATE", "OMNI_TOKEN_ORDER", "OMNI_TOPK_BLOCKWISE",
    "OMNI_EXPERT_DENSE", "OMNI_EXPERT_SPARSE", "omni_workspace_size_flags",
    "omni_expert_workspace_size_flags",
    "omni_workspace_size", "omni_router_topk", "omni_schedule", "omni_grouped_expert_fwd",
    "omni_routed_fwd", "omni_get_device_status", "workspace", "omni_grouped_expert_fwd_noalloc",
    "omni_noalloc_get_device_status",
    "router_topk", "schedule", "grouped_expert_fwd", "routed_fwd", "omni_routed_bwd", "routed_bwd",
    "omni_routed_bwd_workspace_size",
    "omni_shared_mlp_workspace_size", "omni_shared_mlp_fwd", "shared_mlp_fwd", "layer_fwd",
    "OMNI_X_F32", "OMNI_DX_ACCUMULATE", "omni_expert_counts", "omni_balance_fwd_workspace_size",
    "omni_balance_fwd", "omni_balance_bwd_workspace_size", "omni_balance_bwd",
    "omni_layer_norm_fwd", "omni_layer_norm_bwd_workspace_size", "omni_layer_norm_bwd",
    "omni_act_pack", "omni_act_unpack", "omni_routed_bwd_ckpt_workspace_size",
    "omni_routed_bwd_ckpt", "expert_counts", "balance_fwd", "balance_bwd", "layer_norm_fwd",
    "layer_norm_bwd", "act_pack", "act_unpack", "routed_bwd_ckpt",
]


def router_topk(x, W_r, W_c, K, ws=None, p_r=None, p_c=None, logprobs_in=False,
                blockwise=False, stream=None):
    """Top-K experts per token.  With logprobs_in, p_r / p_c are inputs and
    x may be None (then pass W_r / W_c as None too).  blockwise (with
    logprobs_in) selects with the blockwise grid scan instead of the
    row / column pruning; the result is the same."""
    if logprobs_in:
        L, N_r = p_r.shape
        N_c = p_c.shape[1]
        d = 0
        dev = p_r.device
    else:
        L, d = x.shape
        N_r, N_c = W_r.shape[0], W_c.shape[0]
        dev = x.device
        p_r = torch.empty((L, N_r), dtype=torch.float32, device=dev) if p_r is None else p_r
        p_c = torch.empty((L, N_c), dtype=torch.float32, device=dev) if p_c is None else p_c
    idx = torch.empty((L, K), dtype=torch.int32, device=dev)
    score = torch.empty((L, K), dtype=torch.float32, device=dev)
    gate = torch.empty((L, K), dtype=torch.float32, device=dev)
    ws = router_workspace(L, N_r, N_c, K, dev) if ws is None else ws
    flags = (OMNI_ROUTER_LOGPROBS_IN if logprobs_in else 0) | (OMNI_TOPK_BLOCKWISE if blockwise else 0)
    omni_router_topk(x, W_r, W_c, L, d, N_r, N_c, K, p_r, p_c, idx, score, gate, flags, ws, stream)
    return dict(p_r=p_r, p_c=p_c, idx=idx, score=score, gate=gate)


def schedule(idx, gate, N, B, ws=None, stream=None):
    L, K = idx.shape
    dev = idx.device
    M, G = L * K, (N + B - 1) // B
    out = dict(task_token=torch.empty(M, dtype=torch.int32, device=dev),
               task_expert=torch.empty(M, dtype=torch.int32, device=dev),
               task_gate=torch.empty(M, dtype=torch.float32, device=dev),
               group_offsets=torch.empty(G + 1, dtype=torch.int32, device=dev),
               group_counts=torch.empty(G, dtype=torch.int32, device=dev),
               active_groups=torch.empty(G, dtype=torch.int32, device=dev),
               num_active=torch.empty(1, dtype=torch.int32, device=dev),
               num_distinct=torch.empty(1, dtype=torch.int32, device=dev))
    ws = schedule_workspace(L, K, N, B, dev) if ws is None else ws
    omni_schedule(idx, gate, L, K, N, B, out["task_token"], out["task_expert"], out["task_gate"],
                  out["group_offsets"], out["group_counts"], out["active_groups"],
                  out["num_active"], out["num_distinct"], ws, stream)
    return out


_EXPERT_MODE = {"auto": 0, "dense": OMNI_EXPERT_DENSE, "sparse": OMNI_EXPERT_SPARSE}


def grouped_expert_fwd(x, W, V, sched, K, B, y=None, accumulate=False, ws=None, stream=None,
                       expert_mode="auto"):
    """expert_mode: "auto" (the library's size rule), "dense" (always try the
    tensor-core tiles for dense experts) or "sparse" (task by task only)."""
    L, d = x.shape
    N = W.shape[0]
    mode = _EXPERT_MODE[expert_mode]
    y = torch.empty((L, d), dtype=torch.float32, device=x.device) if y is None else y
    ws = expert_workspace(L, d, K, N, B, x.device, mode) if ws is None else ws
    omni_grouped_expert_fwd(x, W, V, L, d, K, N, B, sched["task_token"], sched["task_expert"],
                            sched["task_gate"], sched["group_offsets"], sched["active_groups"],
                            sched["num_active"], y, (OMNI_Y_ACCUMULATE if accumulate else 0) | mode,
                            ws, stream)
    return y


def routed_fwd(x, W, V, W_r, W_c, K, B, y=None, ws=None, want_routing=False, accumulate=False,
               token_order=False, stream=None, expert_mode="auto"):
    L, d = x.shape
    N_r, N_c = W_r.shape[0], W_c.shape[0]
    mode = _EXPERT_MODE[expert_mode]
    flags = (OMNI_Y_ACCUMULATE if accumulate else 0) | (OMNI_TOKEN_ORDER if token_order else 0) | mode
    y = torch.empty((L, d), dtype=torch.float32, device=x.device) if y is None else y
    ws = workspace(L, d, N_r, N_c, K, B, x.device, flags) if ws is None else ws
    idx = gate = None
    if want_routing:
        idx = torch.empty((L, K), dtype=torch.int32, device=x.device)
        gate = torch.empty((L, K), dtype=torch.float32, device=x.device)
    omni_routed_fwd(x, W, V, W_r, W_c, L, d, N_r, N_c, K, B, y, idx, gate, flags, ws, stream)
    return (y, idx, gate) if want_routing else y


def routed_bwd(x, W, V, W_r, W_c, idx, gate, dy, dW=None, dV=None, dW_r=None, dW_c=None,
               ws=None, stream=None):
    """Backward of the routed branch with the forward's routing (idx, gate)
    fixed.  Returns dx (new) and the weight gradients, accumulated into the
    given fp32 buffers (new zeroed ones if None)."""
    L, d = x.shape
    N_r, N_c = W_r.shape[0], W_c.shape[0]
    K = idx.shape[1]
    dev = x.device
    f32 = dict(dtype=torch.float32, device=dev)
    dx = torch.empty((L, d), **f32)
    dW = torch.zeros(W.shape, **f32) if dW is None else dW
    dV = torch.zeros(V.shape, **f32) if dV is None else dV
    dW_r = torch.zeros(W_r.shape, **f32) if dW_r is None else dW_r
    dW_c = torch.zeros(W_c.shape, **f32) if dW_c is None else dW_c
    if ws is None:
        ws = torch.empty(omni_routed_bwd_workspace_size(L, d, N_r, N_c, K), dtype=torch.uint8,
                         device=dev)
    omni_routed_bwd(x, W, V, W_r, W_c, L, d, N_r, N_c, K, idx, gate, dy, dx, dW, dV, dW_r, dW_c,
                    0, ws, stream)
    return dict(dx=dx, dW=dW, dV=dV, dW_r=dW_r, dW_c=dW_c)


def shared_mlp_fwd(x, W_g, W_u, W_d, y=None, accumulate=False, ws=None, stream=None):
    """MLP(x) = (SiLU(x W_g^T) * (x W_u^T)) W_d^T into y (fp32), or added to
    it with accumulate=True.  W_g, W_u: [F, d]; W_d: [d, F]; all bf16."""
    L, d = x.shape
    F = W_g.shape[0]
    y = torch.empty((L, d), dtype=torch.float32, device=x.device) if y is None else y
    ws = shared_mlp_workspace(L, d, F, x.device) if ws is None else ws
    omni_shared_mlp_fwd(x, W_g, W_u, W_d, L, d, F, y, OMNI_Y_ACCUMULATE if accumulate else 0, ws,
                        stream)
    return y


def layer_fwd(x, W, V, W_r, W_c, W_g, W_u, W_d, K, B, y=None, ws=None, mlp_ws=None,
              stream=None, norm_w=None, norm_b=None, norm_eps=1e-5):
    """The whole layer: y = routed(x) + MLP(x), as omni_routed_fwd followed by
    omni_shared_mlp_fwd with OMNI_Y_ACCUMULATE on the same stream.  With norm_w
    (and norm_b), x is the residual stream (bf16 or fp32) and the layer takes
    its layer norm."""
    if norm_w is not None:
        x = layer_norm_fwd(x, norm_w, norm_b, eps=norm_eps, stats=False, stream=stream)["y"]
    y = routed_fwd(x, W, V, W_r, W_c, K, B, y=y, ws=ws, stream=stream)
    return shared_mlp_fwd(x, W_g, W_u, W_d, y=y, accumulate=True, ws=mlp_ws, stream=stream)


# ------------------------------------------------------- training operators

_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _need(name, t, dtypes, shape, dev=None):
    """ValueError unless t is a contiguous CUDA tensor of one of the types and
    of this shape (on `dev`, if given)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name}: a CUDA tensor is expected")
    if t.dtype not in (dtypes if isinstance(dtypes, tuple) else (dtypes,)):
        raise ValueError(f"{name}: {dtypes} expected, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(shape)} expected, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor is expected")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name}: on {t.device}, the other tensors on {dev}")
    return t


def _shape(name, t, dims):
    if not isinstance(t, torch.Tensor) or t.dim() != dims:
        raise ValueError(f"{name}: a tensor of {dims} dimensions is expected")
    return t.shape


@contextlib.contextmanager
def _switched(dev, stream):
    with torch.cuda.device(dev):
        with torch.cuda.stream(stream):
            yield


def _on(dev, stream):
    """Makes the tensors' device current, and `stream` (default: that device's
    current one), for the allocations and launches of a call."""
    if stream is not None:
        if stream.device != dev:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
        return _switched(dev, stream)
    if torch.cuda.current_device() != dev.index:
        return torch.cuda.device(dev)
    return contextlib.nullcontext()


def _scratch(ws, n, dev):
    if ws is None:
        return torch.empty(n, dtype=_U8, device=dev)
    return _need("ws", ws, _U8, (ws.numel(),), dev)


def _token_mask(mask, L, dev):
    if mask is None:
        return None
    return _need("mask", mask, (torch.bool, _U8), (L,), dev)


def expert_counts(idx, N, mask=None, ws=None, stream=None):
    """Tasks per expert and kept tokens: counts [N] and n_tokens [1], int32.
    idx [L, K] int32; mask [L] bool or uint8, None = every token counts."""
    L, K = _shape("idx", idx, 2)
    dev = _need("idx", idx, _I32, (L, K)).device
    mask = _token_mask(mask, L, dev)
    with _on(dev, stream):
        counts = torch.empty(max(N, 0), dtype=_I32, device=dev)
        n_tokens = torch.empty(1, dtype=_I32, device=dev)
        ws = _scratch(ws, 256, dev)
        omni_expert_counts(idx, mask, L, K, N, counts, n_tokens, ws)
    return dict(counts=counts, n_tokens=n_tokens)


def balance_fwd(p_r, p_c, counts, n_tokens, K, mask=None, ws=None, stream=None):
    """Balance loss of the router: loss (0-dim) and token_loss [L], fp32.
    p_r, p_c: log-probabilities (router_topk's); counts, n_tokens from
    expert_counts."""
    (L, N_r), (_, N_c) = _shape("p_r", p_r, 2), _shape("p_c", p_c, 2)
    dev = _need("p_r", p_r, _F32, (L, N_r)).device
    _need("p_c", p_c, _F32, (L, N_c), dev)
    _need("counts", counts, _I32, (N_r * N_c,), dev)
    _need("n_tokens", n_tokens, _I32, (1,), dev)
    mask = _token_mask(mask, L, dev)
    with _on(dev, stream):
        loss = torch.empty((), dtype=_F32, device=dev)
        token_loss = torch.empty(L, dtype=_F32, device=dev)
        ws = _scratch(ws, omni_balance_fwd_workspace_size(L, N_r, N_c), dev)
        omni_balance_fwd(p_r, p_c, counts, n_tokens, mask, L, N_r, N_c, K, loss, token_loss, ws)
    return dict(loss=loss, token_loss=token_loss)


def balance_bwd(x, W_r, W_c, p_r, p_c, counts, n_tokens, K, token_loss, dloss=1.0, mask=None,
                dx=None, dW_r=None, dW_c=None, ws=None, stream=None):
    """Gradients of dloss * balance loss.  With a given dx the gradient is
    added to it (routed_bwd's dx), else a new one is returned; dW_r, dW_c are
    accumulated into the given fp32 buffers (new zeroed ones if None)."""
    (L, d), (N_r, _), (N_c, _) = _shape("x", x, 2), _shape("W_r", W_r, 2), _shape("W_c", W_c, 2)
    dev = _need("x", x, _BF16, (L, d)).device
    _need("W_r", W_r, _BF16, (N_r, d), dev)
    _need("W_c", W_c, _BF16, (N_c, d), dev)
    _need("p_r", p_r, _F32, (L, N_r), dev)
    _need("p_c", p_c, _F32, (L, N_c), dev)
    _need("counts", counts, _I32, (N_r * N_c,), dev)
    _need("n_tokens", n_tokens, _I32, (1,), dev)
    _need("token_loss", token_loss, _F32, (L,), dev)
    mask = _token_mask(mask, L, dev)
    flags = 0
    with _on(dev, stream):
        if dx is None:
            dx = torch.empty((L, d), dtype=_F32, device=dev)
        else:
            _need("dx", dx, _F32, (L, d), dev)
            flags = OMNI_DX_ACCUMULATE
        dW_r = torch.zeros((N_r, d), dtype=_F32, device=dev) if dW_r is None else \
            _need("dW_r", dW_r, _F32, (N_r, d), dev)
        dW_c = torch.zeros((N_c, d), dtype=_F32, device=dev) if dW_c is None else \
            _need("dW_c", dW_c, _F32, (N_c, d), dev)
        ws = _scratch(ws, omni_balance_bwd_workspace_size(L, d, N_r, N_c), dev)
        omni_balance_bwd(x, W_r, W_c, p_r, p_c, counts, n_tokens, mask, token_loss, L, d, N_r, N_c,
                         K, float(dloss), dx, dW_r, dW_c, flags, ws)
    return dict(dx=dx, dW_r=dW_r, dW_c=dW_c)


def layer_norm_fwd(x, w, b=None, eps=1e-5, ckpt=False, stats=True, stream=None):
    """Layer norm of the rows of x [L, d] (bf16 or fp32) with weight w and
    optional bias b (bf16): y bf16, with stats also mean and rstd [L] fp32,
    with ckpt also the 8-bit checkpoint (q [L, d], scale [L, d / 32], uint8) of
    the rows before w and b."""
    L, d = _shape("x", x, 2)
    dev = _need("x", x, (_BF16, _F32), (L, d)).device
    _need("w", w, _BF16, (d,), dev)
    if b is not None:
        _need("b", b, _BF16, (d,), dev)
    with _on(dev, stream):
        out = dict(y=torch.empty((L, d), dtype=_BF16, device=dev))
        if stats:
            out |= dict(mean=torch.empty(L, dtype=_F32, device=dev),
                        rstd=torch.empty(L, dtype=_F32, device=dev))
        if ckpt:
            out |= dict(q=torch.empty((L, d), dtype=_U8, device=dev),
                        scale=torch.empty((L, d // 32), dtype=_U8, device=dev))
        omni_layer_norm_fwd(x, w, b, L, d, eps, out["y"], out.get("mean"), out.get("rstd"),
                            out.get("q"), out.get("scale"), OMNI_X_F32 if x.dtype == _F32 else 0)
    return out


def layer_norm_bwd(dy, w, rstd, x=None, mean=None, q=None, scale=None, bias=True, dx=None, dw=None,
                   db=None, ws=None, stream=None):
    """Backward of layer_norm_fwd from its kept input (x, mean) or from its
    checkpoint (q, scale).  With a given dx the gradient is added to it (the
    residual's), else a new one is returned; dw and (with bias) db are
    accumulated into the given fp32 buffers (new zeroed ones if None)."""
    L, d = _shape("dy", dy, 2)
    dev = _need("dy", dy, _F32, (L, d)).device
    _need("w", w, _BF16, (d,), dev)
    _need("rstd", rstd, _F32, (L,), dev)
    flags = 0
    if q is not None:
        if x is not None:
            raise ValueError("x and q: one of the two is expected")
        _need("q", q, _U8, (L, d), dev)
        _need("scale", scale, _U8, (L, d // 32), dev)
        mean = None
    else:
        _need("x", x, (_BF16, _F32), (L, d), dev)
        _need("mean", mean, _F32, (L,), dev)
        flags = OMNI_X_F32 if x.dtype == _F32 else 0
    if db is not None and not bias:
        raise ValueError("db without bias")
    with _on(dev, stream):
        if dx is None:
            dx = torch.empty((L, d), dtype=_F32, device=dev)
        else:
            _need("dx", dx, _F32, (L, d), dev)
            flags |= OMNI_DX_ACCUMULATE
        dw = torch.zeros(d, dtype=_F32, device=dev) if dw is None else \
            _need("dw", dw, _F32, (d,), dev)
        if bias:
            db = torch.zeros(d, dtype=_F32, device=dev) if db is None else \
                _need("db", db, _F32, (d,), dev)
        ws = _scratch(ws, omni_layer_norm_bwd_workspace_size(L, d), dev)
        omni_layer_norm_bwd(x, mean, rstd, q, scale, w, dy, L, d, dx, dw, db, flags, ws)
    return dict(dx=dx, dw=dw, db=db)


def act_pack(x, stream=None):
    """8-bit checkpoint of x [L, d] (bf16 or fp32): q [L, d] e4m3 bytes and
    scale [L, d / 32] bytes; the values are q * 2**(scale - 127)."""
    L, d = _shape("x", x, 2)
    dev = _need("x", x, (_BF16, _F32), (L, d)).device
    with _on(dev, stream):
        q = torch.empty((L, d), dtype=_U8, device=dev)
        scale = torch.empty((L, d // 32), dtype=_U8, device=dev)
        omni_act_pack(x, L, d, q, scale, OMNI_X_F32 if x.dtype == _F32 else 0)
    return q, scale


def act_unpack(q, scale, w=None, b=None, stream=None):
    """The values of a checkpoint, times w and plus b where given, as bf16."""
    L, d = _shape("q", q, 2)
    dev = _need("q", q, _U8, (L, d)).device
    _need("scale", scale, _U8, (L, d // 32), dev)
    for name, t in (("w", w), ("b", b)):
        if t is not None:
            _need(name, t, _BF16, (d,), dev)
    with _on(dev, stream):
        y = torch.empty((L, d), dtype=_BF16, device=dev)
        omni_act_unpack(q, scale, w, b, L, d, y)
    return y


def routed_bwd_ckpt(q, scale, W, V, W_r, W_c, idx, gate, dy, w=None, b=None, dW=None, dV=None,
                    dW_r=None, dW_c=None, ws=None, stream=None):
    """routed_bwd with its tokens restored from a checkpoint,
    x = act_unpack(q, scale, w, b)."""
    (L, d), (N_r, _), (N_c, _) = _shape("q", q, 2), _shape("W_r", W_r, 2), _shape("W_c", W_c, 2)
    K = _shape("idx", idx, 2)[1]
    dev = _need("q", q, _U8, (L, d)).device
    _need("scale", scale, _U8, (L, d // 32), dev)
    for name, t in (("w", w), ("b", b)):
        if t is not None:
            _need(name, t, _BF16, (d,), dev)
    weights = dict(W=(W, N_r * N_c), V=(V, N_r * N_c), W_r=(W_r, N_r), W_c=(W_c, N_c))
    for name, (t, rows) in weights.items():
        _need(name, t, _BF16, (rows, d), dev)
    _need("idx", idx, _I32, (L, K), dev)
    _need("gate", gate, _F32, (L, K), dev)
    _need("dy", dy, _F32, (L, d), dev)
    with _on(dev, stream):
        dx = torch.empty((L, d), dtype=_F32, device=dev)
        grads = dict(dW=dW, dV=dV, dW_r=dW_r, dW_c=dW_c)
        for name, g in grads.items():
            shape = weights[name[1:]][0].shape
            grads[name] = torch.zeros(shape, dtype=_F32, device=dev) if g is None else \
                _need(name, g, _F32, shape, dev)
        ws = _scratch(ws, omni_routed_bwd_ckpt_workspace_size(L, d, N_r, N_c, K), dev)
        omni_routed_bwd_ckpt(q, scale, w, b, W, V, W_r, W_c, L, d, N_r, N_c, K, idx, gate, dy, dx,
                             grads["dW"], grads["dV"], grads["dW_r"], grads["dW_c"], 0, ws)
    return dict(dx=dx, **grads)
