"""Plain 64-bit forms of the training operators, for their tests: the balance
loss from its definition over all N experts, the layer norm, the 8-bit
checkpoints in integer arithmetic.  They run on the CPU or the GPU and share no
code with the library."""
from __future__ import annotations

import torch

BLOCK = 32


# ------------------------------------------------------------------ balance
def counts_ref(idx, N, mask=None):
    keep = torch.ones(len(idx), dtype=torch.bool, device=idx.device) if mask is None else mask.bool()
    return torch.bincount(idx[keep].reshape(-1).long(), minlength=N), int(keep.sum())


def balance_loss_ref(logits_r, logits_c, counts, n, K, mask=None):
    """N sum_e f_e P_e with the [N] probabilities written out, from logits."""
    keep = torch.ones(len(logits_r), dtype=torch.bool, device=logits_r.device) if mask is None else mask.bool()
    pr = torch.softmax(logits_r[keep], dim=1)
    pc = torch.softmax(logits_c[keep], dim=1)
    N = pr.shape[1] * pc.shape[1]
    if n == 0 or len(pr) == 0:
        return torch.zeros((), dtype=torch.float64, device=logits_r.device)
    P = (pr.T @ pc).reshape(N) / len(pr)
    f = counts.double() / (K * n)
    return N * (f * P).sum()


def balance_ref(x, W_r, W_c, p_r, p_c, counts, n, K, dloss, mask=None):
    """The formulas in 64 bits, with the bounds that the tests hold the kernels
    to: every output's sum of absolute terms (sensitivity to relative errors)."""
    L, N_r, N_c = len(x), p_r.shape[1], p_c.shape[1]
    keep = torch.ones(L, dtype=torch.bool, device=x.device) if mask is None else mask.bool()
    on = keep[:, None]
    zero = torch.zeros((), dtype=torch.float64, device=x.device)
    Pr = torch.where(on, p_r.double().exp(), zero)
    Pc = torch.where(on, p_c.double().exp(), zero)
    F = counts.double().reshape(N_r, N_c)
    U, V = Pc @ F.T, Pr @ F
    tl = (Pr * U).sum(1)
    nl = int(keep.sum())
    ok = n > 0 and nl > 0
    fac = N_r * N_c / (K * n * nl) if ok else 0.0
    c = dloss * fac
    xd, wr, wc = torch.where(on, x.double(), zero), W_r.double(), W_c.double()
    dsr, dsc = c * Pr * (U - tl[:, None]), c * Pc * (V - tl[:, None])
    Ar, Ac = abs(c) * Pr * (U + tl[:, None]), abs(c) * Pc * (V + tl[:, None])
    return dict(loss=fac * tl.sum(), token_loss=tl, dx=dsr @ wr + dsc @ wc, dW_r=dsr.T @ xd,
                dW_c=dsc.T @ xd, dx_sum=(Ar.sum(1) + Ac.sum(1))[:, None], dW_r_sum=Ar.sum(0)[:, None],
                dW_c_sum=Ac.sum(0)[:, None], dx_abs=Ar @ wr.abs() + Ac @ wc.abs(), dW_r_abs=Ar.T @ xd.abs(),
                dW_c_abs=Ac.T @ xd.abs())


# --------------------------------------------------------------- layer norm
def norm_ref(x, w, b, eps):
    x = x.double()
    mean = x.mean(1)
    var = (x - mean[:, None]).square().mean(1)
    rstd = 1 / torch.sqrt(var + eps)
    xh = (x - mean[:, None]) * rstd[:, None]
    y = xh * w.double()
    return (y if b is None else y + b.double()), mean, rstd, xh


def norm_bwd_ref(dy, w, rstd, xh):
    dy, rstd = dy.double(), rstd.double()[:, None]
    g = dy * w.double()
    m0, m1 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = rstd * (g - m0 - xh * m1)
    dx_abs = rstd * (g.abs() + g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    return dict(dx=dx, dw=(dy * xh).sum(0), db=dy.sum(0), dx_abs=dx_abs,
                dw_abs=(dy * xh).abs().sum(0), db_abs=dy.abs().sum(0))


# -------------------------------------------------------------- checkpoints
E4M3 = None


def e4m3_table():
    """The value of every e4m3 byte, from the format's definition."""
    global E4M3
    if E4M3 is None:
        v = []
        for b in range(256):
            e, m = (b >> 3) & 15, b & 7
            x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
            if e == 15 and m == 7:
                x = float("nan")
            v.append(-x if b & 128 else x)
        E4M3 = torch.tensor(v, dtype=torch.float64)
    return E4M3


def pack_ref(x):
    """(q, scale) by search: the nearest table entry, ties to the even byte."""
    x = x.double().cpu()
    L, d = x.shape
    v = x.reshape(L, d // BLOCK, BLOCK)
    fin = torch.where(torch.isfinite(v), v.abs(), 0.0)
    amax = fin.amax(2)
    code = torch.zeros_like(amax, dtype=torch.int64)
    for c in range(1, 248):
        code = torch.where(amax > 448.0 * 2.0 ** (c - 1 - 127), torch.tensor(c), code)
    y = v * torch.exp2(127.0 - code.double())[..., None]
    tab = e4m3_table()[:127]                               # 0 .. 448, ascending
    a = y.abs().nan_to_num(0.0, 0.0, 0.0)
    hi = torch.searchsorted(tab, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dh, dl = tab[hi] - a, a - tab[lo]
    pick = torch.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)) | (a == tab[hi]), hi, lo)
    q = pick + torch.where(torch.signbit(y), 128, 0)
    bad = ~torch.isfinite(v)
    return q.reshape(L, d), code, bad.reshape(L, d)


def unpack_ref(q, scale):
    v = e4m3_table()[q.long().cpu()]
    return v * torch.exp2(scale.double().cpu() - 127).repeat_interleave(BLOCK, dim=1)


# ---------------------------------------------------------- routed backward
def routed_bwd_ref(x, W, V, W_r, W_c, idx, gate, dy):
    """Gradients of sum(dy * routed(x)) by autograd in 64 bits, with the
    selection fixed and the gates a softmax over the selected scores."""
    N_c = len(W_c)
    leaf = [t.double().detach().requires_grad_() for t in (x, W, V, W_r, W_c)]
    x, W, V, W_r, W_c = leaf
    e = idx.long()
    moved = torch.einsum("td,tkd->tk", x, W_r[e // N_c] + W_c[e % N_c])
    g = torch.softmax(gate.double().log() + moved - moved.detach(), dim=1)
    h = torch.einsum("td,tkd->tk", x, W[e])
    y = torch.einsum("tk,tkd->td", g * h * torch.sigmoid(h), V[e])
    y.backward(dy.double())
    return dict(zip(("dx", "dW", "dV", "dW_r", "dW_c"), (t.grad for t in leaf)))


def router_row_magnitude(x, W, V, idx, gate, dy):
    """max over the router's weight gradients of the sums of magnitudes behind
    them: |dS_k| <= g_k (|dgate_k| + sum_j g_j |dgate_j|), times |x|, over all of
    a token's cells (they may sit in one row, whose dS then sum to 0 exactly)."""
    x, dy, g = x.double(), dy.double(), gate.double()
    e = idx.long()
    h = torch.einsum("td,tkd->tk", x, W.double()[e])
    c = torch.einsum("td,tkd->tk", dy, V.double()[e])
    dg = (h * torch.sigmoid(h) * c).abs()
    dS = g * (dg + (g * dg).sum(1, keepdim=True))
    return float((dS.sum(1)[:, None] * x.abs()).max())
