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
                   OMNI_X_F32, OMNI_DX_ACCUMULATE, OMNI_DW_OVERWRITE, _check,
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
    "OMNI_X_F32", "OMNI_DX_ACCUMULATE", "OMNI_DW_OVERWRITE", "omni_expert_counts", "omni_balance_fwd_workspace_size",
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
              stream=None, norm_w=None, norm_b=None, norm_eps=None):
    """The whole layer: y = routed(x) + MLP(x), as omni_routed_fwd followed by
    omni_shared_mlp_fwd with OMNI_Y_ACCUMULATE on the same stream.  With norm_w
    (and norm_b, and norm_eps, 1e-5 where it is None), x is the residual stream
    (bf16 or fp32) and the layer takes its layer norm; norm_b or norm_eps without
    norm_w is a ValueError.  What it allocates belongs to the stream it runs on
    (`stream`, or the current one)."""
    if stream is not None:
        # all of its scratch is released when it returns, while the stream still runs
        with torch.cuda.stream(stream):
            return layer_fwd(x, W, V, W_r, W_c, W_g, W_u, W_d, K, B, y, ws, mlp_ws, None, norm_w,
                             norm_b, norm_eps)
    if norm_w is not None:
        eps = 1e-5 if norm_eps is None else norm_eps
        x = layer_norm_fwd(x, norm_w, norm_b, eps=eps, stats=False)["y"]
    elif norm_b is not None or norm_eps is not None:
        raise ValueError("norm_b and norm_eps belong to a norm: norm_w is missing")
    y = routed_fwd(x, W, V, W_r, W_c, K, B, y=y, ws=ws)
    return shared_mlp_fwd(x, W_g, W_u, W_d, y=y, accumulate=True, ws=mlp_ws)


# ------------------------------------------------------- training operators
# These run once or more per layer and step, some of them for a few
# microseconds, so their checks read each attribute once and the C entry point
# gets plain addresses.

_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _refuse(name, t, dtype, shape, di):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name}: a CUDA tensor is expected")
    if t.dtype != dtype:
        raise ValueError(f"{name}: {dtype} expected, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(shape)} expected, got {tuple(t.shape)}")
    if t.get_device() != di:
        raise ValueError(f"{name}: on cuda:{t.get_device()}, the other tensors on cuda:{di}")
    raise ValueError(f"{name}: a contiguous tensor is expected")


def _at(name, t, dtype, shape, di):
    """Address of t; ValueError unless it is a contiguous tensor of this type
    and shape on device di."""
    try:
        if (t.dtype is dtype and t.shape == shape and t.get_device() == di and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:                              # no tensor
        pass
    _refuse(name, t, dtype, shape, di)


def _size(name, n):
    """n as the C entry points take it; they would see a larger one modulo 2^32."""
    if not n < 1 << 31:
        raise ValueError(f"{name}: {n} is not below 2^31")
    return n


def _rows(name, t):
    """Shape [rows, columns] and device index of a CUDA matrix."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name}: a tensor of 2 dimensions is expected")
    if t.numel() >= 1 << 31:
        _size(name, max(t.shape))
    di = t.get_device()
    if di < 0:
        raise ValueError(f"{name}: a CUDA tensor is expected")
    return (*t.shape, di)


def _bf16_or_f32(name, t, shape, di):
    """Address and OMNI_X_F32 flag of a bf16 or fp32 tensor."""
    if isinstance(t, torch.Tensor) and t.dtype is _F32:
        return _at(name, t, _F32, shape, di), OMNI_X_F32
    return _at(name, t, _BF16, shape, di), 0


def _number(name, v):
    """v as a Python number.  A CUDA tensor is read back, which waits for its
    stream and cannot be captured."""
    if isinstance(v, torch.Tensor) and v.is_cuda and torch.cuda.is_current_stream_capturing():
        raise ValueError(f"{name}: a Python number is expected while a graph is captured")
    return float(v)


def _mask_at(mask, L, di):
    if mask is None:
        return None
    bits = isinstance(mask, torch.Tensor) and mask.dtype is torch.bool
    return _at("mask", mask, torch.bool if bits else _U8, (L,), di)


def _elsewhere(di, stream):
    """Whether a call has to change the current device or stream first."""
    if stream is not None:
        if stream.device.index != di:
            raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{di}")
        return True
    return torch.cuda.current_device() != di


@contextlib.contextmanager
def _on(di, stream):
    """Makes the tensors' device current, and `stream` where one is given, for
    the allocations and launches of a call."""
    with torch.cuda.device(di):
        with torch.cuda.stream(stream):
            yield


def _new(n, dtype, di):
    return torch.empty(n, dtype=dtype, device=di)


def _scratch(ws, n, di):
    """Workspace, its address and its size."""
    if ws is None:
        ws = torch.empty(n, dtype=_U8, device=di)
        return ws, ws.data_ptr(), n
    n = ws.numel() if isinstance(ws, torch.Tensor) else 0
    return ws, _at("ws", ws, _U8, (n,), di), n


# the current stream's handle without a Stream object around it, where torch has that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _queue(di):
    return _raw_stream(di) if _raw_stream else torch.cuda.current_stream(di).cuda_stream


def _grad(name, g, like):
    """An fp32 gradient to accumulate into: the given one, or a zeroed one."""
    if g is None:
        return torch.zeros_like(like, dtype=_F32)
    _at(name, g, _F32, like.shape, like.get_device())
    return g


def _grads(names, given, like):
    """The weight gradients to write: the given fp32 buffers, which are
    accumulated into, or new ones.  All new: OMNI_DW_OVERWRITE spares zeroing
    and reading them; some given: the new ones start at zero."""
    if not any(g is not None for g in given):
        return [torch.empty_like(t, dtype=_F32) for t in like], OMNI_DW_OVERWRITE
    return [_grad(*ngl) for ngl in zip(names, given, like)], 0


def expert_counts(idx, N, mask=None, ws=None, stream=None):
    """Tasks per expert and kept tokens: counts [N] and n_tokens [1], int32.
    idx [L, K] int32; mask [L] bool or uint8, None = every token counts.  Ids
    outside [0, N) are not counted; omni_get_device_status of the workspace, which
    is returned as ws, reports them."""
    L, K, di = _rows("idx", idx)
    _size("N", N)
    if _elsewhere(di, stream):
        with _on(di, stream):
            return expert_counts(idx, N, mask, ws)
    counts, n_tokens = _new(max(N, 0), _I32, di), _new(1, _I32, di)
    ws, ws_at, ws_n = _scratch(ws, 256, di)
    _check("omni_expert_counts", load().omni_expert_counts(
        _at("idx", idx, _I32, (L, K), di), _mask_at(mask, L, di), L, K, N, counts.data_ptr(),
        n_tokens.data_ptr(), ws_at, ws_n, _queue(di)))
    return dict(counts=counts, n_tokens=n_tokens, ws=ws)


def balance_fwd(p_r, p_c, counts, n_tokens, K, mask=None, ws=None, stream=None):
    """Balance loss of the router: loss (0-dim) and token_loss [L], fp32.
    p_r, p_c: log-probabilities (router_topk's); counts, n_tokens from
    expert_counts."""
    L, N_r, di = _rows("p_r", p_r)
    N_c = _rows("p_c", p_c)[1]
    _size("K", K)
    if _elsewhere(di, stream):
        with _on(di, stream):
            return balance_fwd(p_r, p_c, counts, n_tokens, K, mask, ws)
    at = (_at("p_r", p_r, _F32, (L, N_r), di), _at("p_c", p_c, _F32, (L, N_c), di),
          _at("counts", counts, _I32, (N_r * N_c,), di), _at("n_tokens", n_tokens, _I32, (1,), di),
          _mask_at(mask, L, di))
    loss, token_loss = _new((), _F32, di), _new(L, _F32, di)
    lib = load()
    ws, ws_at, ws_n = _scratch(ws, lib.omni_balance_fwd_workspace_size(L, N_r, N_c), di)
    _check("omni_balance_fwd", lib.omni_balance_fwd(
        *at, L, N_r, N_c, K, loss.data_ptr(), token_loss.data_ptr(), ws_at, ws_n, _queue(di)))
    return dict(loss=loss, token_loss=token_loss)


def balance_bwd(x, W_r, W_c, p_r, p_c, counts, n_tokens, K, token_loss, dloss=1.0, mask=None,
                dx=None, dW_r=None, dW_c=None, ws=None, stream=None):
    """Gradients of dloss * balance loss.  With a given dx the gradient is
    added to it (routed_bwd's dx), else a new one is returned; dW_r, dW_c are
    accumulated into the given fp32 buffers (new ones if None).  dloss is a
    number of the host: one on the device is read back first, so the call waits
    for it (and refuses it while a graph is captured)."""
    L, d, di = _rows("x", x)
    N_r, N_c = _rows("W_r", W_r)[0], _rows("W_c", W_c)[0]
    _size("K", K)
    if _elsewhere(di, stream):
        with _on(di, stream):
            return balance_bwd(x, W_r, W_c, p_r, p_c, counts, n_tokens, K, token_loss, dloss, mask,
                               dx, dW_r, dW_c, ws)
    dloss = _number("dloss", dloss)
    at = (_at("x", x, _BF16, (L, d), di), _at("W_r", W_r, _BF16, (N_r, d), di),
          _at("W_c", W_c, _BF16, (N_c, d), di), _at("p_r", p_r, _F32, (L, N_r), di),
          _at("p_c", p_c, _F32, (L, N_c), di), _at("counts", counts, _I32, (N_r * N_c,), di),
          _at("n_tokens", n_tokens, _I32, (1,), di), _mask_at(mask, L, di),
          _at("token_loss", token_loss, _F32, (L,), di))
    (dW_r, dW_c), flags = _grads(("dW_r", "dW_c"), (dW_r, dW_c), (W_r, W_c))
    if dx is None:
        dx = torch.empty_like(x, dtype=_F32)
    else:
        _at("dx", dx, _F32, (L, d), di)
        flags |= OMNI_DX_ACCUMULATE
    lib = load()
    ws, ws_at, ws_n = _scratch(ws, lib.omni_balance_bwd_workspace_size(L, d, N_r, N_c), di)
    _check("omni_balance_bwd", lib.omni_balance_bwd(
        *at, L, d, N_r, N_c, K, dloss, dx.data_ptr(), dW_r.data_ptr(), dW_c.data_ptr(), flags,
        ws_at, ws_n, _queue(di)))
    return dict(dx=dx, dW_r=dW_r, dW_c=dW_c)


def layer_norm_fwd(x, w, b=None, eps=1e-5, ckpt=False, stats=True, stream=None):
    """Layer norm of the rows of x [L, d] (bf16 or fp32) with weight w and
    optional bias b (bf16): y bf16, with stats also mean and rstd [L] fp32,
    with ckpt also the 8-bit checkpoint (q [L, d], scale [L, d / 32], uint8) of
    the rows before w and b."""
    L, d, di = _rows("x", x)
    if _elsewhere(di, stream):
        with _on(di, stream):
            return layer_norm_fwd(x, w, b, eps, ckpt, stats)
    x_at, flags = _bf16_or_f32("x", x, (L, d), di)
    y = torch.empty_like(x, dtype=_BF16)
    out = dict(y=y)
    at = [None, None, None, None]
    if stats:
        out["mean"] = mean = _new(L, _F32, di)
        out["rstd"] = rstd = _new(L, _F32, di)
        at[:2] = mean.data_ptr(), rstd.data_ptr()
    if ckpt:
        out["q"] = q = torch.empty_like(x, dtype=_U8)
        out["scale"] = scale = torch.empty(L, d // 32, dtype=_U8, device=di)
        at[2:] = q.data_ptr(), scale.data_ptr()
    _check("omni_layer_norm_fwd", load().omni_layer_norm_fwd(
        x_at, _at("w", w, _BF16, (d,), di), None if b is None else _at("b", b, _BF16, (d,), di), L,
        d, eps, y.data_ptr(), *at, flags, _queue(di)))
    return out


def layer_norm_bwd(dy, w, rstd, x=None, mean=None, q=None, scale=None, bias=True, dx=None, dw=None,
                   db=None, ws=None, stream=None):
    """Backward of layer_norm_fwd from its kept input (x, mean) or from its
    checkpoint (q, scale).  With a given dx the gradient is added to it (the
    residual's; it may be dy), else a new one is returned; dw and (with bias) db are
    accumulated into the given fp32 buffers (new ones if None)."""
    L, d, di = _rows("dy", dy)
    if (q is not None and x is not None) or (db is not None and not bias):
        raise ValueError("one of x and q, and db only with bias")
    if _elsewhere(di, stream):
        with _on(di, stream):
            return layer_norm_bwd(dy, w, rstd, x, mean, q, scale, bias, dx, dw, db, ws)
    w_at = _at("w", w, _BF16, (d,), di)
    dy_at = _at("dy", dy, _F32, (L, d), di)
    if bias:
        (dw, db), flags = _grads(("dw", "db"), (dw, db), (w, w))
    else:
        (dw,), flags = _grads(("dw",), (dw,), (w,))
    x_at = mean_at = q_at = scale_at = None
    if q is not None:
        q_at = _at("q", q, _U8, (L, d), di)
        scale_at = _at("scale", scale, _U8, (L, d // 32), di)
    else:
        x_at, x_flag = _bf16_or_f32("x", x, (L, d), di)
        mean_at = _at("mean", mean, _F32, (L,), di)
        flags |= x_flag
    if dx is None:
        dx = torch.empty_like(dy)
    else:
        _at("dx", dx, _F32, (L, d), di)
        flags |= OMNI_DX_ACCUMULATE
    lib = load()
    ws, ws_at, ws_n = _scratch(ws, lib.omni_layer_norm_bwd_workspace_size(L, d), di)
    _check("omni_layer_norm_bwd", lib.omni_layer_norm_bwd(
        x_at, mean_at, _at("rstd", rstd, _F32, (L,), di), q_at, scale_at, w_at, dy_at, L, d,
        dx.data_ptr(), dw.data_ptr(), db.data_ptr() if bias else None, flags, ws_at, ws_n,
        _queue(di)))
    return dict(dx=dx, dw=dw, db=db)


def act_pack(x, stream=None):
    """8-bit checkpoint of x [L, d] (bf16 or fp32): q [L, d] e4m3 bytes and
    scale [L, d / 32] bytes; the values are q * 2**(scale - 127)."""
    L, d, di = _rows("x", x)
    if _elsewhere(di, stream):
        with _on(di, stream):
            return act_pack(x)
    x_at, flags = _bf16_or_f32("x", x, (L, d), di)
    q = torch.empty_like(x, dtype=_U8)
    scale = torch.empty(L, d // 32, dtype=_U8, device=di)
    _check("omni_act_pack", load().omni_act_pack(x_at, L, d, q.data_ptr(), scale.data_ptr(), flags,
                                                 _queue(di)))
    return q, scale


def act_unpack(q, scale, w=None, b=None, stream=None):
    """The values of a checkpoint, times w and plus b where given, as bf16."""
    L, d, di = _rows("q", q)
    if _elsewhere(di, stream):
        with _on(di, stream):
            return act_unpack(q, scale, w, b)
    q_at = _at("q", q, _U8, (L, d), di)
    y = torch.empty_like(q, dtype=_BF16)
    _check("omni_act_unpack", load().omni_act_unpack(
        q_at, _at("scale", scale, _U8, (L, d // 32), di),
        None if w is None else _at("w", w, _BF16, (d,), di),
        None if b is None else _at("b", b, _BF16, (d,), di), L, d, y.data_ptr(), _queue(di)))
    return y


def routed_bwd_ckpt(q, scale, W, V, W_r, W_c, idx, gate, dy, w=None, b=None, dW=None, dV=None,
                    dW_r=None, dW_c=None, ws=None, stream=None):
    """routed_bwd with its tokens restored from a checkpoint,
    x = act_unpack(q, scale, w, b)."""
    L, d, di = _rows("q", q)
    N_r, N_c, K = _rows("W_r", W_r)[0], _rows("W_c", W_c)[0], _rows("idx", idx)[1]
    if _elsewhere(di, stream):
        with _on(di, stream):
            return routed_bwd_ckpt(q, scale, W, V, W_r, W_c, idx, gate, dy, w, b, dW, dV, dW_r,
                                   dW_c, ws)
    N = N_r * N_c
    at = (_at("q", q, _U8, (L, d), di), _at("scale", scale, _U8, (L, d // 32), di),
          None if w is None else _at("w", w, _BF16, (d,), di),
          None if b is None else _at("b", b, _BF16, (d,), di), _at("W", W, _BF16, (N, d), di),
          _at("V", V, _BF16, (N, d), di), _at("W_r", W_r, _BF16, (N_r, d), di),
          _at("W_c", W_c, _BF16, (N_c, d), di), L, d, N_r, N_c, K,
          _at("idx", idx, _I32, (L, K), di), _at("gate", gate, _F32, (L, K), di),
          _at("dy", dy, _F32, (L, d), di))
    dx = torch.empty_like(dy)
    (dW, dV, dW_r, dW_c), flags = _grads(("dW", "dV", "dW_r", "dW_c"), (dW, dV, dW_r, dW_c),
                                         (W, V, W_r, W_c))
    lib = load()
    ws, ws_at, ws_n = _scratch(ws, lib.omni_routed_bwd_ckpt_workspace_size(L, d, N_r, N_c, K), di)
    _check("omni_routed_bwd_ckpt", lib.omni_routed_bwd_ckpt(
        *at, dx.data_ptr(), dW.data_ptr(), dV.data_ptr(), dW_r.data_ptr(), dW_c.data_ptr(), flags,
        ws_at, ws_n, _queue(di)))
    return dict(dx=dx, dW=dW, dV=dV, dW_r=dW_r, dW_c=dW_c)
