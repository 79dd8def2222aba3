"""GPU tests of the training operators (per-expert counts, balance loss, layer
norm, 8-bit checkpoints, the routed backward from a checkpoint) against plain
64-bit forms on the same inputs.

Tolerances, fixed before the first run.  They are elementwise: a bound on the
relative error of every term, times the sum of the terms' magnitudes, which the
reference returns beside the value.
  balance  exp(p) and ds enter their products as two fp16 values, hi + lo: what
           is lost is at most 2^-11 of lo, which is at most 2^-11 of the value.
           2^-16 is asked for each (the halves' bound in bf16).  Each fp32
           addition in the tensor core loses at most 2^-23 of the running sum
           of magnitudes; a product over k terms takes 2 k / 16 (hi, lo) or
           3 k / 16 (F_lo) additions of 16-term sums.  exp and the few other
           fp32 operations: 2^-20.  x and W become fp16 with their largest
           magnitude at 2^14 at least, where fp16's smallest step is 2^-24:
           half of it is 2^-39 of the largest, for each value however small.
  norm     y is rounded to bf16 once (2^-8 of itself); the fp32 arithmetic
           before it is off by at most a few units of 2^-24 per operation: mean
           and variance are sums of d terms in chunks of at most 64 and a tree,
           (64 + 16) 2^-24 < 2^-17 of the mean magnitude.
  dw, db   sums over the rows, each addition 2^-24: at most L + 64 of them.
  routed_bwd_ckpt  the bar of omni_routed_bwd (2e-4 of the largest reference
           gradient, 2e-4 in rel-L2): the same kernels on the restored tokens.
"""
import numpy as np
import pytest
import torch

import atomic_expert_layer_b200 as omni
from atomic_expert_layer_b200 import configs, inputs

import _train_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    omni.load()


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _within(got, want, tol, what):
    got, want = got.double(), want.double()
    bad = ~((got - want).abs() <= tol)
    if bad.any():
        at = tuple(i[0].item() for i in torch.nonzero(bad, as_tuple=True)) if bad.dim() else ()
        t = tol[at].item() if torch.is_tensor(tol) and tol.dim() else float(tol)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {at}: "
                             f"{got[at].item()} for {want[at].item()}, tolerance {t}")


# ---------------------------------------------------------------- counts
@pytest.mark.parametrize("L,K,N,masked", [(1, 1, 1, False), (1, 5, 7, False), (37, 3, 50, True),
                                          (4096, 16, 4096, True), (1000, 33, 3, False),
                                          (2048, 64, 1 << 20, False),
                                          (16384, 64, 1000, True),       # the crowded table
                                          (16400, 65, 1 << 20, False),   # ... with few repeats
                                          (40000, 33, 1, True)])         # ... one expert
def test_expert_counts(L, K, N, masked):
    g = _gen(L + K)
    idx = torch.randint(0, N, (L, K), generator=g, device=DEV, dtype=torch.int32)
    mask = torch.rand(L, generator=g, device=DEV) > 0.4 if masked else None
    if masked:
        idx[~mask] = -7                                 # ids of padding are not read
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    out = omni.expert_counts(idx, N, mask=mask, ws=ws)
    want, n = ref.counts_ref(idx, N, mask)
    assert torch.equal(out["counts"].long(), want)
    assert out["n_tokens"].item() == n
    assert omni.omni_get_device_status(ws) == 0


def test_expert_counts_reports_a_bad_id_and_counts_the_rest():
    idx = torch.tensor([[0, 5], [16, 3], [-1, 3]], dtype=torch.int32, device=DEV)
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    out = omni.expert_counts(idx, 16, ws=ws)
    assert omni.omni_get_device_status(ws) == 1         # OMNI_DEV_BAD_EXPERT
    want = torch.zeros(16, dtype=torch.int32)
    want[0] = want[5] = 1
    want[3] = 2
    assert torch.equal(out["counts"].cpu(), want) and out["n_tokens"].item() == 3
    none = omni.expert_counts(idx, 16, mask=torch.zeros(3, dtype=torch.bool, device=DEV))
    assert none["n_tokens"].item() == 0 and not none["counts"].any()


@pytest.mark.parametrize("bad", [-1, 16, 1 << 30])
def test_expert_counts_keeps_its_status(bad):
    """A bad id is found out without a workspace of the caller's."""
    idx = torch.tensor([[0, 5], [3, 3]], dtype=torch.int32, device=DEV)
    assert omni.omni_get_device_status(omni.expert_counts(idx, 16)["ws"]) == 0
    idx[1, 0] = bad
    out = omni.expert_counts(idx, 16)
    assert omni.omni_get_device_status(out["ws"]) == 1 and int(out["counts"].sum()) == 3
    ws = torch.empty(512, dtype=torch.uint8, device=DEV)
    assert omni.expert_counts(idx, 16, ws=ws)["ws"] is ws and omni.omni_get_device_status(ws) == 1


# --------------------------------------------------------------- balance
def _balance_inputs(L, d, N_r, N_c, K, seed, masked=False, hot=False):
    """Log-probabilities of a router on random tokens; hot: all tokens on a few
    experts (counts up to L), with a row and a column at probability near 1."""
    g = _gen(seed)
    x = torch.randn(L, d, generator=g, device=DEV).to(torch.bfloat16)
    W = [(torch.randn(n, d, generator=g, device=DEV) * d ** -0.5).to(torch.bfloat16) for n in (N_r, N_c)]
    s = [x.float() @ w.float().T for w in W]
    if hot:
        for z in s:
            z[:, 0] += 6
    p = [torch.log_softmax(z, 1) for z in s]
    if hot:
        idx = torch.arange(K, device=DEV, dtype=torch.int32).expand(L, K).contiguous()
    else:
        idx = torch.randint(0, N_r * N_c, (L, K), generator=g, device=DEV, dtype=torch.int32)
    mask = None
    if masked:
        mask = torch.rand(L, generator=g, device=DEV) > 0.3
        mask[0] = True
    return x, W[0], W[1], p[0].contiguous(), p[1].contiguous(), idx, mask


def _delta(N_r, N_c, d, L, big):
    """Relative error of a term of U, V or l (first), and with that of ds and its products."""
    per = 3 if big else 2
    adds = per * max(N_r, N_c) / 16 + 64
    one = 2 * 2.0 ** -16 + 2.0 ** -20 + adds * 2.0 ** -23
    prod = 2.0 ** -16 + 2.0 ** -20 + (2 * max(N_r + N_c + 126, L) / 16 + 64) * 2.0 ** -23
    return one, 2 * one + 2.0 ** -16 + prod


def _check_balance(x, W_r, W_c, p_r, p_c, idx, mask, K, dloss=0.37, ws_fill=0xff):
    L, d = x.shape
    N_r, N_c = len(W_r), len(W_c)
    cnt = omni.expert_counts(idx, N_r * N_c, mask=mask)
    n = cnt["n_tokens"].item()
    big = bool((cnt["counts"] > 256).any())
    one, delta = _delta(N_r, N_c, d, L, big)
    want = ref.balance_ref(x, W_r, W_c, p_r, p_c, cnt["counts"], n, K, dloss, mask)
    ws = torch.full((omni.omni_balance_fwd_workspace_size(L, N_r, N_c),), ws_fill, dtype=torch.uint8, device=DEV)
    fwd = omni.balance_fwd(p_r, p_c, cnt["counts"], cnt["n_tokens"], K, mask=mask, ws=ws)
    assert omni.omni_get_device_status(ws) == 0
    _within(fwd["token_loss"], want["token_loss"], one * want["token_loss"] + 1e-30, "token_loss")
    _within(fwd["loss"], want["loss"], (one + 2.0 ** -23) * want["loss"] + 1e-30, "loss")
    ws = torch.full((omni.omni_balance_bwd_workspace_size(L, d, N_r, N_c),), ws_fill, dtype=torch.uint8, device=DEV)
    got = omni.balance_bwd(x, W_r, W_c, p_r, p_c, cnt["counts"], cnt["n_tokens"], K, fwd["token_loss"],
                           dloss=dloss, mask=mask, ws=ws)
    assert omni.omni_get_device_status(ws) == 0
    top = {"dx": max(float(W_r.abs().max()), float(W_c.abs().max()))}
    top["dW_r"] = top["dW_c"] = float((x if mask is None else x[mask]).abs().max())
    for name in ("dx", "dW_r", "dW_c"):
        tol = delta * want[name + "_abs"] + 2.0 ** -39 * top[name] * want[name + "_sum"] + 1e-30
        _within(got[name], want[name], tol, name)
        # far inside the worst case, the whole is good to 1e-4, but for what fp32
        # itself leaves where U and l cancel: token_loss is an fp32 output, so
        # its rounding alone moves ds by up to c P l 2^-24, and by linearity the
        # outputs by 2^-24 of the sums of magnitudes (32000 times the result for
        # the hot experts beside 96 columns: 1.9e-3 of it; torch in fp32 is
        # 2.1e-4 off there)
        norm = want[name].norm()
        tol = 1e-4 * norm + 2.0 ** -24 * want[name + "_abs"].norm() + 1e-30
        assert (got[name].double() - want[name]).norm() <= tol, name
    return cnt, fwd, got


@pytest.mark.parametrize("L,d,N_r,N_c,K,masked,hot", [
    (256, 256, 64, 64, 16, False, False),       # the tiny layer
    (1, 8, 1, 1, 1, False, False),              # smallest sizes: one expert
    (1, 64, 3, 5, 2, False, False),             # one token
    (130, 72, 65, 63, 5, True, False),          # ragged tiles on every axis
    (300, 200, 300, 17, 9, True, False),        # two column tiles beside a narrow axis
    (1000, 776, 257, 389, 33, True, False),     # odd sizes, d off the tile grid
    (700, 256, 40, 300, 4, False, True),        # counts above 256: the F_lo product
    (4096, 1024, 1304, 1304, 64, False, False),  # the headline grid
    (640, 2048, 1024, 96, 128, True, True),     # widest tokens, hot experts, a mask
    (64, 64, 2100, 8, 2, False, False),         # a long axis against a short one
])
def test_balance(L, d, N_r, N_c, K, masked, hot):
    x, W_r, W_c, p_r, p_c, idx, mask = _balance_inputs(L, d, N_r, N_c, min(K, N_r * N_c), L + d, masked, hot)
    _check_balance(x, W_r, W_c, p_r, p_c, idx, mask, idx.shape[1])


@pytest.mark.parametrize("ex,ew", [(60, -50), (-70, 30), (100, 20), (0, -100)])
def test_balance_scales_of_x_and_w(ex, ew):
    """Operands far from 1 are scaled by powers of two and back: the same bounds."""
    x, W_r, W_c, p_r, p_c, idx, _ = _balance_inputs(150, 64, 40, 70, 5, 3)
    x, W_r, W_c = (t.float() * 2.0 ** e for t, e in ((x, ex), (W_r, ew), (W_c, ew)))
    x, W_r, W_c = (t.to(torch.bfloat16) for t in (x, W_r, W_c))
    _check_balance(x, W_r, W_c, p_r, p_c, idx, None, 5)


def test_balance_ranges_within_x_and_w():
    """Columns of x and W from 1 down to 2^-30 of the largest; zero columns;
    all of x zero; a weight of the loss far from 1."""
    x, W_r, W_c, p_r, p_c, idx, _ = _balance_inputs(150, 64, 40, 70, 5, 3)
    s = torch.exp2(-torch.arange(64, device=DEV) * 30.0 / 63).float()
    x, W_r, W_c = ((t.float() * s).to(torch.bfloat16) for t in (x, W_r, W_c))
    x[:, 5] = 0
    W_r[:, 9] = 0
    _check_balance(x, W_r, W_c, p_r, p_c, idx, None, 5)
    _check_balance(x, W_r, W_c, p_r, p_c, idx, None, 5, dloss=1e-28)
    _check_balance(torch.zeros_like(x), W_r, W_c, p_r, p_c, idx, None, 5)


def test_balance_offsets_past_32_bits():
    """L * (N_r + N_c) past 2^31: the last rows, and a weight gradient that only
    the last rows reach."""
    L, d, N_r, N_c, K, n = 1_070_000, 8, 1024, 1024, 2, 96
    g = _gen(5)
    x = torch.zeros(L, d, dtype=torch.bfloat16, device=DEV)
    x[-n:] = torch.randn(n, d, generator=g, device=DEV).to(torch.bfloat16)
    W_r, W_c = (torch.randn(m, d, generator=g, device=DEV).to(torch.bfloat16) for m in (N_r, N_c))
    p_r, p_c = (torch.full((L, m), -np.log(m), device=DEV) for m in (N_r, N_c))
    for p in (p_r, p_c):
        p[-n:] = torch.log_softmax(torch.randn(n, p.shape[1], generator=g, device=DEV), 1)
    idx = torch.randint(0, N_r * N_c, (L, K), generator=g, device=DEV, dtype=torch.int32)
    assert L * (N_r + N_c) > 2 ** 31
    cnt = omni.expert_counts(idx, N_r * N_c)
    fwd = omni.balance_fwd(p_r, p_c, cnt["counts"], cnt["n_tokens"], K)
    got = omni.balance_bwd(x, W_r, W_c, p_r, p_c, cnt["counts"], cnt["n_tokens"], K, fwd["token_loss"], dloss=1e6)
    tail = ref.balance_ref(x[-n:], W_r, W_c, p_r[-n:], p_c[-n:], cnt["counts"], L, K, 1e6 * n / L)
    one, delta = _delta(N_r, N_c, d, L, False)
    _within(fwd["token_loss"][-n:], tail["token_loss"], one * tail["token_loss"], "token_loss")
    # elsewhere p is even: token_loss is the mean count
    mean = L * K / (N_r * N_c)
    assert abs(fwd["token_loss"][:-n].double().mean().item() - mean) < 1e-4 * mean
    _within(got["dx"][-n:], tail["dx"], delta * tail["dx_abs"] + 1e-30, "dx")
    for k in ("dW_r", "dW_c"):
        _within(got[k], tail[k], delta * tail[k + "_abs"] + 1e-30, k)


def test_balance_against_differences():
    """Directional derivatives of the definition over all N experts (64 bits)."""
    L, d, N_r, N_c, K, dloss = 40, 64, 12, 9, 4, 1.3
    x, W_r, W_c, p_r, p_c, idx, mask = _balance_inputs(L, d, N_r, N_c, K, 9, masked=True)
    z = [x.double() @ w.double().T for w in (W_r, W_c)]
    p_r, p_c = (torch.log_softmax(v, 1).float() for v in z)
    cnt, _, got = _check_balance(x, W_r, W_c, p_r, p_c, idx, mask, K, dloss)
    n = cnt["n_tokens"].item()
    args = [x.double(), W_r.double(), W_c.double()]

    def loss(x, W_r, W_c):
        return dloss * ref.balance_loss_ref(x @ W_r.T, x @ W_c.T, cnt["counts"], n, K, mask)

    g = _gen(1)
    for at, name in enumerate(("dx", "dW_r", "dW_c")):
        v = torch.randn(args[at].shape, generator=g, device=DEV, dtype=torch.float64)
        up, dn = list(args), list(args)
        up[at], dn[at] = args[at] + 1e-5 * v, args[at] - 1e-5 * v
        num = (loss(*up) - loss(*dn)) / 2e-5
        # the kernels' 1e-4 of the gradient's norm, times the direction's share
        tol = 1e-4 * got[name].double().norm() * v.norm() / v.numel() ** 0.5 * 4
        assert abs(num - (got[name].double() * v).sum()) <= tol + 1e-9


def test_balance_accumulates_into_given_gradients():
    L, d, N_r, N_c, K = 200, 136, 70, 90, 6
    x, W_r, W_c, p_r, p_c, idx, _ = _balance_inputs(L, d, N_r, N_c, K, 4)
    cnt = omni.expert_counts(idx, N_r * N_c)
    fwd = omni.balance_fwd(p_r, p_c, cnt["counts"], cnt["n_tokens"], K)
    args = (x, W_r, W_c, p_r, p_c, cnt["counts"], cnt["n_tokens"], K, fwd["token_loss"])
    fresh = omni.balance_bwd(*args)
    again = omni.balance_bwd(*args)
    base = {k: torch.randn_like(v) for k, v in fresh.items()}
    added = omni.balance_bwd(*args, **{k: v.clone() for k, v in base.items()})
    for k in fresh:
        assert torch.equal(fresh[k], again[k])           # the same on every run
        assert torch.equal(added[k], base[k] + fresh[k])  # one fp32 addition


def test_balance_masked_rows_hold_anything():
    """Padding rows of x, p_r, p_c with NaN and infinities, ids out of range:
    results as without those rows; masked rows of dx are zero, and stay as they
    were when added to."""
    L, d, N_r, N_c, K = 150, 64, 33, 40, 3
    x, W_r, W_c, p_r, p_c, idx, _ = _balance_inputs(L, d, N_r, N_c, K, 8)
    mask = torch.ones(L, dtype=torch.bool, device=DEV)
    mask[100:] = False
    mask[::7] = False
    clean = _check_balance(x, W_r, W_c, p_r, p_c, idx, mask, K)
    for t, v in ((x, float("nan")), (p_r, float("inf")), (p_c, float("nan"))):
        t[~mask] = v
    idx[~mask] = 1 << 30
    cnt = omni.expert_counts(idx, N_r * N_c, mask=mask)
    fwd = omni.balance_fwd(p_r, p_c, cnt["counts"], cnt["n_tokens"], K, mask=mask)
    got = omni.balance_bwd(x, W_r, W_c, p_r, p_c, cnt["counts"], cnt["n_tokens"], K, fwd["token_loss"],
                           dloss=0.37, mask=mask)
    assert torch.equal(fwd["loss"], clean[1]["loss"]) and not fwd["token_loss"][~mask].any()
    for k in got:
        assert torch.equal(got[k], clean[2][k]), k
    assert not got["dx"][~mask].any()
    kept = torch.randn(L, d, device=DEV)
    dx = omni.balance_bwd(x, W_r, W_c, p_r, p_c, cnt["counts"], cnt["n_tokens"], K, fwd["token_loss"],
                          dloss=0.37, mask=mask, dx=kept.clone())["dx"]
    assert torch.equal(dx[~mask], kept[~mask])


@pytest.mark.parametrize("L,N_r,N_c", [(1, 1, 2), (2, 3, 4), (3, 5, 66), (40, 7, 71), (37, 2, 1), (33, 40, 262)])
@pytest.mark.parametrize("offset", [0, 1, 2, 3])
def test_balance_axes_at_any_address(L, N_r, N_c, offset):
    """Log-probabilities from any 4-byte boundary on, NaN around them: bit for
    bit the results of arrays of their own."""
    d, K = 64, 2
    x, W_r, W_c, p_r, p_c, idx, mask = _balance_inputs(L, d, N_r, N_c, K, L, masked=True)
    cnt = omni.expert_counts(idx, N_r * N_c, mask=mask)

    def within(p):
        room = torch.full((p.numel() + 16,), float("nan"), device=DEV)
        at = room[4 + offset:4 + offset + p.numel()].view_as(p)
        return at.copy_(p)

    def both(p_r, p_c):
        fwd = omni.balance_fwd(p_r, p_c, cnt["counts"], cnt["n_tokens"], K, mask=mask)
        return {**fwd, **omni.balance_bwd(x, W_r, W_c, p_r, p_c, cnt["counts"], cnt["n_tokens"], K,
                                          fwd["token_loss"], mask=mask)}

    want, got = both(p_r, p_c), both(within(p_r), within(p_c))
    for k in want:
        assert torch.equal(want[k], got[k]) and torch.isfinite(got[k]).all(), k


def test_balance_all_rows_masked():
    L, d, N_r, N_c, K = 20, 64, 8, 8, 2
    x, W_r, W_c, p_r, p_c, idx, _ = _balance_inputs(L, d, N_r, N_c, K, 2)
    mask = torch.zeros(L, dtype=torch.bool, device=DEV)
    cnt = omni.expert_counts(idx, 64, mask=mask)
    fwd = omni.balance_fwd(p_r, p_c, cnt["counts"], cnt["n_tokens"], K, mask=mask)
    got = omni.balance_bwd(x, W_r, W_c, p_r, p_c, cnt["counts"], cnt["n_tokens"], K, fwd["token_loss"], mask=mask)
    assert fwd["loss"].item() == 0 and not fwd["token_loss"].any()
    for k in got:
        assert not got[k].any(), k


def test_balance_impossible_rows_and_columns():
    """Log-probabilities of -inf and of fp32's lowest value are probabilities of 0."""
    L, d, N_r, N_c, K = 90, 64, 30, 50, 4
    x, W_r, W_c, p_r, p_c, idx, _ = _balance_inputs(L, d, N_r, N_c, K, 12)
    p_r[:, 5] = float("-inf")
    p_c[::2, 7] = torch.finfo(torch.float32).min
    p_r[3] = float("-inf")
    p_r[3, 4] = 0.0                                      # one row holds everything
    _check_balance(x, W_r, W_c, p_r, p_c, idx, None, K)


def test_balance_counts_summed_over_replicas():
    """counts and n_tokens may be sums over replicas: large counts, n > L."""
    L, d, N_r, N_c, K = 96, 64, 20, 24, 3
    x, W_r, W_c, p_r, p_c, idx, mask = _balance_inputs(L, d, N_r, N_c, K, 6, masked=True)
    cnt = omni.expert_counts(idx, N_r * N_c, mask=mask)
    counts, n_tokens = cnt["counts"] * 4099 + 70000, cnt["n_tokens"] * 5000
    n = n_tokens.item()
    one, delta = _delta(N_r, N_c, d, L, True)
    want = ref.balance_ref(x, W_r, W_c, p_r, p_c, counts, n, K, 1.0, mask)
    fwd = omni.balance_fwd(p_r, p_c, counts, n_tokens, K, mask=mask)
    _within(fwd["loss"], want["loss"], (one + 2.0 ** -15) * want["loss"], "loss")
    got = omni.balance_bwd(x, W_r, W_c, p_r, p_c, counts, n_tokens, K, fwd["token_loss"], mask=mask)
    for name in ("dx", "dW_r", "dW_c"):
        # counts above 2^16 are themselves taken to 16 bits: 2^-16 more on U and l
        _within(got[name], want[name], (delta + 2.0 ** -15) * want[name + "_abs"] + 1e-30, name)


# Bars that hold the balance gradients to fp32's accuracy, relative to the
# results however small they are.  Rounding errors of single terms average out
# of a norm; what stays is the tensor core's cutting off towards zero, at most
# 2^-23 of the running sum at an instruction and about half of that on average.
# Over the 16 to 32 instructions of an accumulator, whose sum grows as they go,
# that is 3e-7 to 6e-7 of a product of mixed signs, and 2e-6 with four times as
# many: 1.5e-6 is asked for.
# Where U and l cancel, their errors do not shrink with the difference.  U, V and
# l are sums of positive terms, all cut off the same way: by up to 4.5 x 2^-23 in
# accumulators of two K steps (8 instructions of hi halves, sum of 1/8 .. 8/8),
# by up to 8.5 x 2^-23 in those of four, which hold two fifths of a sum at most:
# 6.1 x 2^-23 in all.  l can lose less, by the place of its leading bits, so all
# U - l and V - l of a token move by up to 6.1 x 2^-23 l.  Beside that, the terms'
# own roundings (2^-24 each, of U, l and the difference) are 2^-23 one by one
# (root of the sum of squares).
SHIFT, EACH = 6.1 * 2.0 ** -23, 2.0 ** -23
BAR = 1.5e-6


def _cancelled(x, W_r, W_c, p_r, p_c, counts, n, K, dloss, mask):
    """What the errors of U and l leave in dx, dW_r and dW_c where they cancel:
    norms of the shift by c P l, and of the separate terms c P (U + l)."""
    keep = torch.ones(len(x), dtype=torch.bool, device=DEV) if mask is None else mask.bool()
    Pr, Pc = (p[keep].double().exp() for p in (p_r, p_c))
    F = counts.double().reshape(Pr.shape[1], Pc.shape[1])
    U, V = Pc @ F.T, Pr @ F
    tl = (Pr * U).sum(1, keepdim=True)
    c = abs(dloss) * F.numel() / (K * n * int(keep.sum()))
    xd, wr, wc = x[keep].double(), W_r.double(), W_c.double()
    shift = dict(dx=(c * tl * (Pr @ wr)).norm() + (c * tl * (Pc @ wc)).norm(),
                 dW_r=(c * (Pr * tl).T @ xd).norm(), dW_c=(c * (Pc * tl).T @ xd).norm())
    Ar, Ac = (c * Pr * (U + tl)).square(), (c * Pc * (V + tl)).square()
    each = dict(dx=Ar @ wr.square() + Ac @ wc.square(), dW_r=Ar.T @ xd.square(), dW_c=Ac.T @ xd.square())
    return {k: float(SHIFT * shift[k] + EACH * each[k].sum().sqrt()) for k in shift}


def _check_balance_to_fp32(x, W_r, W_c, p_r, p_c, counts, n_tokens, K, dloss=1.0, mask=None, cancels=True):
    """Gradients within BAR of their norm (with `cancels` also what _cancelled
    gives), every token's loss within 2^-18 of itself.  That is the sum of: 4.5 x
    2^-23 cut off; 2^-20 for the up to 150 additions after that (5 times the root
    of the sum of squares of 2^-24 each, uniformly); 2^-21 for exp and the halves
    of P, and 2^-22 for the other exp: 18.5 x 2^-23 in all, and 2^-18 is 32."""
    n = n_tokens.item()
    want = ref.balance_ref(x, W_r, W_c, p_r, p_c, counts, n, K, dloss, mask)
    fwd = omni.balance_fwd(p_r, p_c, counts, n_tokens, K, mask=mask)
    floor = 2.0 ** -36 * float(counts.max())             # P's 2^-39 of 1, beside the largest count
    _within(fwd["token_loss"], want["token_loss"], 2.0 ** -18 * want["token_loss"] + floor, "token_loss")
    _within(fwd["loss"], want["loss"], 2.0 ** -18 * want["loss"], "loss")
    got = omni.balance_bwd(x, W_r, W_c, p_r, p_c, counts, n_tokens, K, fwd["token_loss"], dloss=dloss, mask=mask)
    more = _cancelled(x, W_r, W_c, p_r, p_c, counts, n, K, dloss, mask) if cancels else {}
    for k in ("dx", "dW_r", "dW_c"):
        err, norm = float((got[k].double() - want[k]).norm()), float(want[k].norm())
        assert norm > 0 and err <= BAR * norm + more.get(k, 0.0), (k, err / norm)
    return fwd, got, want


@pytest.mark.parametrize("ex,ew,dloss", [(0, -101, 1.0), (-101, 0, 1.0), (-118, -118, 2.0 ** 40),
                                         (-128, -129, 2.0 ** 50), (120, -20, 2.0 ** -30), (-60, 122, 2.0 ** -30),
                                         (0, 0, 2.0 ** -100), (100, 100, 2.0 ** -140)])
def test_balance_operands_of_any_magnitude(ex, ew, dloss):
    """x and W from bf16's subnormal numbers to near its largest, weights of the
    loss to match: as near to their gradients as ordinary ones."""
    x, W_r, W_c, p_r, p_c, idx, _ = _balance_inputs(150, 64, 40, 70, 5, 3)
    x, W_r, W_c = (t.float() * 2.0 ** (e // 2) * 2.0 ** (e - e // 2) for t, e in ((x, ex), (W_r, ew), (W_c, ew)))
    x, W_r, W_c = (t.to(torch.bfloat16) for t in (x, W_r, W_c))
    cnt = omni.expert_counts(idx, 40 * 70)
    _check_balance_to_fp32(x, W_r, W_c, p_r, p_c, cnt["counts"], cnt["n_tokens"], 5, dloss=dloss)


def _collapsed(L, N_r, N_c, K, spread, seed, d=64):
    """All tokens on the same K experts, whatever their log-probabilities, whose
    logits have this spread."""
    g = _gen(seed)
    x = torch.randn(L, d, generator=g, device=DEV).to(torch.bfloat16)
    W_r, W_c = ((torch.randn(n, d, generator=g, device=DEV) * d ** -0.5).to(torch.bfloat16) for n in (N_r, N_c))
    p_r, p_c = (torch.log_softmax(spread * torch.randn(L, n, generator=g, device=DEV), 1) for n in (N_r, N_c))
    idx = (torch.arange(K, device=DEV) * (N_c + 1) % (N_r * N_c)).int().expand(L, K).contiguous()
    cnt = omni.expert_counts(idx, N_r * N_c)
    return x, W_r, W_c, p_r.contiguous(), p_c.contiguous(), cnt["counts"], cnt["n_tokens"]


@pytest.mark.parametrize("L,N_r,N_c,K,spread", [(4096, 1304, 1304, 1, 0.01), (4096, 1304, 1304, 1, 1.0),
                                                (2048, 1304, 1304, 64, 1.0), (512, 8192, 8192, 1, 0.01),
                                                (512, 8192, 8192, 1, 1.0), (700, 8192, 40, 3, 3.0),
                                                (3000, 257, 389, 1, 8.0)])
def test_balance_of_a_collapsed_router(L, N_r, N_c, K, spread):
    """Few experts take every task while the probabilities are spread over all:
    the gradients are many powers of two below the largest count, and differ as
    much between tokens.  Each token's dx is held to the bar by itself."""
    x, W_r, W_c, p_r, p_c, counts, n = _collapsed(L, N_r, N_c, K, spread, L + K)
    _, got, want = _check_balance_to_fp32(x, W_r, W_c, p_r, p_c, counts, n, K)
    # a token's P are good to 2^-21 and 2^-39 of 1 each; l is a product of two
    rows = want["dx"].norm(dim=1)
    low = 2.0 ** -39 * (torch.exp(-p_r[:, :K].double().amin(1)) + torch.exp(-p_c.double()[:, (torch.arange(K) * (N_c + 1) % N_c)].amin(1)))
    err = (got["dx"].double() - want["dx"]).norm(dim=1)
    more = 2.0 ** -21 * want["dx_abs"].norm(dim=1)
    assert (err <= (4 * BAR + 4 * low) * rows + more).all(), float((err / rows).max())


@pytest.mark.parametrize("top", [1.0, 2.5, 3.98])
@pytest.mark.parametrize("count", [1, 1023, 1025, 2047])
def test_balance_probabilities_up_to_their_limit(top, count):
    """exp(p) may be anything below 3.99, normalised or not: ds stays in range,
    at counts on both sides of a power of two."""
    L, N_r, N_c = 70, 65, 130
    x, W_r, W_c, p_r, p_c, _, _ = _balance_inputs(L, 64, N_r, N_c, 1, 17)
    for p in (p_r, p_c):
        p[:, 3] = np.log(top)
        p[::3, 5] = np.log(top)
    counts = torch.zeros(N_r, N_c, dtype=torch.int32, device=DEV)
    counts[3, 3] = counts[5, 3] = counts[40, 100] = count
    n = torch.full((1,), 4000, dtype=torch.int32, device=DEV)
    _check_balance_to_fp32(x, W_r, W_c, p_r, p_c, counts.reshape(-1), n, 1)


def test_balance_a_token_without_numbers():
    """NaN in one token's probabilities reaches its own dx and the weights'
    gradients, and nothing else."""
    L, d, N_r, N_c, K = 90, 64, 30, 50, 4
    x, W_r, W_c, p_r, p_c, idx, _ = _balance_inputs(L, d, N_r, N_c, K, 12)
    cnt = omni.expert_counts(idx, N_r * N_c)

    def step():
        f = omni.balance_fwd(p_r, p_c, cnt["counts"], cnt["n_tokens"], K)
        return {**f, **omni.balance_bwd(x, W_r, W_c, p_r, p_c, cnt["counts"], cnt["n_tokens"], K, f["token_loss"])}

    clean = step()
    p_r[17, 4] = float("nan")
    got = step()
    rest = torch.arange(L, device=DEV) != 17
    for k in ("token_loss", "dx"):
        assert torch.equal(got[k][rest], clean[k][rest]) and torch.isnan(got[k][17]).all()
    assert all(torch.isnan(got[k]).all() for k in ("loss", "dW_r", "dW_c"))


def test_balance_headline_grid_to_fp32():
    """What accumulators of two K steps are for: with eight, 2e-6 (the scale that
    BAR is set against)."""
    x, W_r, W_c, p_r, p_c, idx, _ = _balance_inputs(4096, 1024, 1304, 1304, 64, 31)
    cnt = omni.expert_counts(idx, 1304 * 1304)
    _check_balance_to_fp32(x, W_r, W_c, p_r, p_c, cnt["counts"], cnt["n_tokens"], 64, cancels=False)


def _counts_past_2048(kind, N_r, N_c, g):
    """Counts on a grid whose axes take several K steps: what fp16's rounding of
    them leaves (none up to 2048) is a third product."""
    few = torch.randint(0, 9, (N_r, N_c), generator=g, device=DEV, dtype=torch.int32)
    if kind == "border":                                 # one count past 2048, in the last tile of both axes
        few[N_r - 1, N_c - 1] = 2049
    elif kind == "2048":                                 # none
        few[N_r - 1, N_c - 1] = 2048
    elif kind == "some":                                 # odd counts here and there
        for i, j in ((0, 0), (N_r // 2, N_c - 1), (N_r - 1, N_c // 3)):
            few[i, j] = 4097 + 2 * i + j
    elif kind == "all":                                  # every one, up to 2^22
        few = torch.randint(0, 1 << 22, (N_r, N_c), generator=g, device=DEV, dtype=torch.int32)
        few[0, :3] = torch.tensor([(1 << 22) - 1, 1 << 22, 2049], dtype=torch.int32, device=DEV)
    else:                                                # up to 2^31 - 1: to 22 bits
        few = torch.randint(0, 1 << 30, (N_r, N_c), generator=g, device=DEV, dtype=torch.int32)
        few[0, :3] = torch.tensor([(1 << 22) + 1, (1 << 31) - 1, 3], dtype=torch.int32, device=DEV)
    return few.reshape(-1)


@pytest.mark.parametrize("kind", ["border", "2048", "some", "all", "largest"])
@pytest.mark.parametrize("L,N_r,N_c,masked", [(300, 257, 389, True),      # 5 and 7 K steps
                                              (200, 300, 1100, False),    # 5 and 18
                                              (260, 1304, 1000, False)])  # 21 and 16
def test_balance_counts_past_2048(L, N_r, N_c, masked, kind):
    """The product with the counts' remainders over several K steps, odd numbers
    of them (its first step shares an accumulator with the last of the others),
    several tiles, a lead of three and four steps."""
    x, W_r, W_c, p_r, p_c, _, mask = _balance_inputs(L, 64, N_r, N_c, 1, L + N_r, masked)
    counts = _counts_past_2048(kind, N_r, N_c, _gen(N_c))
    n = torch.full((1,), 5000, dtype=torch.int32, device=DEV)
    fwd, got, want = _check_balance_to_fp32(x, W_r, W_c, p_r, p_c, counts, n, 3, mask=mask)
    # each expert by itself: tokens that are certain of one cell have its count as their loss
    at = torch.tensor([[0, 0], [0, 1], [0, 2], [N_r // 2, N_c - 1], [N_r - 1, N_c // 3], [N_r - 1, N_c - 1]], device=DEV)
    p_r, p_c = (torch.full((len(at), m), float("-inf"), device=DEV) for m in (N_r, N_c))
    for k, p in enumerate((p_r, p_c)):
        p[torch.arange(len(at), device=DEV), at[:, k]] = 0.0
    sure = omni.balance_fwd(p_r, p_c, counts, n, 3)["token_loss"].double()
    exact = counts[at[:, 0] * N_c + at[:, 1]].double()
    assert torch.equal(sure[exact <= 1 << 22], exact[exact <= 1 << 22])
    assert ((sure - exact).abs() <= 2.0 ** -22 * exact).all()


# ------------------------------------------------------------------ norm
def _rows(L, d, dtype, seed):
    g = _gen(seed)
    x = torch.randn(L, d, generator=g, device=DEV) * (0.1 + 3 * torch.rand(L, 1, generator=g, device=DEV))
    x += 4 * torch.randn(L, 1, generator=g, device=DEV)
    w = (1 + 0.3 * torch.randn(d, generator=g, device=DEV)).to(torch.bfloat16)
    b = (0.3 * torch.randn(d, generator=g, device=DEV)).to(torch.bfloat16)
    return x.to(dtype), w, b, torch.randn(L, d, generator=g, device=DEV)


NORM_SIZES = [(1, 8), (1, 2048), (2, 32), (3, 40), (5, 256), (7, 264), (33, 776), (64, 1000), (4, 1024),
              (6, 1032), (19, 1536), (600, 2048), (3, 2056), (2, 4096), (2, 5000), (3, 8192), (4097, 320)]


@pytest.mark.parametrize("L,d", NORM_SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("bias", [True, False])
def test_layer_norm(L, d, dtype, bias):
    x, w, b, dy = _rows(L, d, dtype, L + d)
    b = b if bias else None
    eps = 1e-5
    out = omni.layer_norm_fwd(x, w, b, eps=eps)
    y, mean, rstd, xh = ref.norm_ref(x, w, b, eps)
    e = 2.0 ** -17
    big = x.double().abs().amax(1)
    _within(out["mean"], mean, e * big, "mean")
    # the variance moves by e of itself, and by the square of the mean's error
    _within(out["rstd"], rstd, rstd * (e + (e * big * rstd) ** 2), "rstd")
    exh = (e * big * rstd)[:, None] + 2 * e * xh.abs()
    wd = w.double().abs()
    _within(out["y"], y, 2.0 ** -8 * y.abs() + (1 + 2.0 ** -7) * (exh * wd) + 2.0 ** -22 * (y.abs() + 1), "y")

    got = omni.layer_norm_bwd(dy, w, out["rstd"], x=x, mean=out["mean"], bias=bias)
    xk = (x.double() - out["mean"].double()[:, None]) * out["rstd"].double()[:, None]
    want = ref.norm_bwd_ref(dy, w, out["rstd"], xk)
    _within(got["dx"], want["dx"], 2.0 ** -17 * want["dx_abs"] + 1e-30, "dx")
    adds = (L + 64) * 2.0 ** -24 + 2.0 ** -21
    _within(got["dw"], want["dw"], adds * want["dw_abs"] + 1e-30, "dw")
    if bias:
        _within(got["db"], want["db"], adds * want["db_abs"] + 1e-30, "db")
    else:
        assert got["db"] is None


@pytest.mark.parametrize("L,d", [(1, 32), (3, 96), (37, 512), (9, 1024), (5, 1056), (130, 2048), (2, 8192)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_layer_norm_checkpoint(L, d, dtype):
    x, w, b, dy = _rows(L, d, dtype, L * d)
    plain = omni.layer_norm_fwd(x, w, b)
    out = omni.layer_norm_fwd(x, w, b, ckpt=True)
    for k in plain:
        assert torch.equal(plain[k], out[k]), k          # the checkpoint changes nothing else
    _, _, _, xh = ref.norm_ref(x, w, b, 1e-5)
    kept = ref.unpack_ref(out["q"], out["scale"]).to(DEV)
    # half a step of e4m3 (2^-4), or 2^-10 of the scale, beside the fp32 error of
    # xh (which a value at a rounding border can turn into a whole step more)
    s = torch.exp2(out["scale"].double() - 127).repeat_interleave(32, 1)
    _within(kept, xh, 2.0 ** -4 * xh.abs() + 2.0 ** -10 * s + 2.0 ** -15 * (1 + x.double().abs().amax(1, keepdim=True) * plain["rstd"].double()[:, None]), "xh")
    # no block wastes a power of two, none passes 448
    top = out["q"].reshape(L, -1, 32).bitwise_and(127).amax(2)
    assert int(top.max()) <= 126 and (top >= 112).all()
    # the values that the layer sees again
    n = omni.act_unpack(out["q"], out["scale"], w, b)
    exact = kept * w.double() + b.double()
    assert torch.equal(n, exact.float().to(torch.bfloat16))
    got = omni.layer_norm_bwd(dy, w, out["rstd"], q=out["q"], scale=out["scale"])
    want = ref.norm_bwd_ref(dy, w, out["rstd"], kept)
    _within(got["dx"], want["dx"], 2.0 ** -17 * want["dx_abs"] + 1e-30, "dx")
    adds = (L + 64) * 2.0 ** -24 + 2.0 ** -21
    _within(got["dw"], want["dw"], adds * want["dw_abs"] + 1e-30, "dw")
    _within(got["db"], want["db"], adds * want["db_abs"] + 1e-30, "db")


@pytest.mark.parametrize("d", [32, 96, 1024, 8192])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_checkpoint_changes_nothing_where_the_norm_overflows(d, dtype):
    """Rows whose variance is 0 in fp32 beside eps = 0, infinities and NaN: y with
    a checkpoint is y without one, bit for bit (the checkpoint holds NaN)."""
    x, w, b, _ = _rows(5, d, torch.float32, d)
    x[1] *= 1e-30
    x[2, d // 2] = float("inf")
    x[3, 3] = float("nan")
    x[4] = 0
    x = x.to(dtype)
    for bias in (b, None):
        plain, out = (omni.layer_norm_fwd(x, w, bias, eps=0.0, ckpt=c) for c in (False, True))
        assert torch.isinf(plain["y"][1].float()).any()  # (w has no zeros, x - mean hardly any)
        for k in plain:
            assert torch.equal(plain[k].nan_to_num(77.0, 88.0, -88.0), out[k].nan_to_num(77.0, 88.0, -88.0)), k
        assert torch.equal(out["q"][1] & 127 == 127, ~torch.isfinite(plain["y"][1].float()))


def test_layer_norm_against_differences():
    L, d, eps = 6, 64, 1e-5
    x, w, b, dy = _rows(L, d, torch.float32, 77)
    out = omni.layer_norm_fwd(x, w, b, eps=eps)
    got = omni.layer_norm_bwd(dy, w, out["rstd"], x=x, mean=out["mean"])
    args = [x.double(), w.double(), b.double()]
    f = lambda x, w, b: (dy.double() * ref.norm_ref(x, w, b, eps)[0]).sum()  # noqa: E731
    g = _gen(2)
    for at, name in enumerate(("dx", "dw", "db")):
        v = torch.randn(args[at].shape, generator=g, device=DEV, dtype=torch.float64)
        up, dn = list(args), list(args)
        up[at], dn[at] = args[at] + 1e-5 * v, args[at] - 1e-5 * v
        num = (f(*up) - f(*dn)) / 2e-5
        assert abs(num - (got[name].double() * v).sum()) <= 1e-4 * got[name].double().norm() * v.norm()


def test_norm_and_checkpoint_offsets_past_32_bits():
    """L * d past 2^31: rows at both ends, forward, checkpoint and backward."""
    L, d = 1_050_000, 2048
    assert L * d > 2 ** 31
    x = torch.ones(L, d, dtype=torch.bfloat16, device=DEV)
    ends = torch.cat([torch.arange(8), torch.arange(L - 8, L)]).to(DEV)
    sub, w, b, dy = _rows(16, d, torch.bfloat16, 12)
    x[ends] = sub
    f = omni.layer_norm_fwd(x, w, b, ckpt=True)
    want = omni.layer_norm_fwd(sub, w, b, ckpt=True)
    for k in want:
        assert torch.equal(f[k][ends], want[k]), k
    assert torch.equal(f["y"][1000], b)                  # a constant row: xh = 0
    q, scale = omni.act_pack(x)
    assert torch.equal(omni.act_unpack(q, scale)[ends], omni.act_unpack(*omni.act_pack(sub)))
    del x, q, scale
    big = torch.zeros(L, d, device=DEV)
    big[ends] = dy
    g = omni.layer_norm_bwd(big, w, f["rstd"], q=f["q"], scale=f["scale"], dx=big)
    h = omni.layer_norm_bwd(dy, w, want["rstd"], q=want["q"], scale=want["scale"], dx=dy.clone())
    assert torch.equal(g["dx"][ends], h["dx"]) and not g["dx"][8:-8].any()
    _within(g["dw"], h["dw"], 2.0 ** -18 * h["dw"].abs().double() + 2.0 ** -18 * float(dy.abs().max()), "dw")


def test_layer_norm_rows_without_spread():
    """Constant rows (xh = 0), rows of zeros, and rows whose mean is far above
    their spread, where a variance from sums of squares would cancel."""
    d = 512
    x = torch.zeros(4, d, device=DEV)
    x[1] = 3.0
    x[2] = 1e4 + torch.arange(d, device=DEV) * 2.0 ** -4
    x[3, 0] = 1e-20
    w = torch.ones(d, dtype=torch.bfloat16, device=DEV)
    out = omni.layer_norm_fwd(x, w, None, eps=1e-5, ckpt=True)
    y, mean, rstd, xh = ref.norm_ref(x, w, None, 1e-5)
    assert not out["y"][:2].any() and not out["q"][:2].any()
    assert torch.isfinite(out["y"].float()).all()
    # row 2: the mean is off by at most 2^-17 of 1e4 (0.08), against a spread of 9.2
    _within(out["y"][2], y[2], 2.0 ** -8 * y[2].abs() + 0.01, "y")
    _within(out["rstd"], rstd, 1e-4 * rstd, "rstd")


def test_layer_norm_gradients_accumulate_and_repeat():
    L, d = 301, 776
    x, w, b, dy = _rows(L, d, torch.float32, 5)
    f = omni.layer_norm_fwd(x, w, b)
    kept = dict(x=x, mean=f["mean"])
    one = omni.layer_norm_bwd(dy, w, f["rstd"], **kept)
    two = omni.layer_norm_bwd(dy, w, f["rstd"], **kept)
    base = {k: torch.randn_like(v) for k, v in one.items()}
    add = omni.layer_norm_bwd(dy, w, f["rstd"], **kept, **{k: v.clone() for k, v in base.items()})
    for k in one:
        assert torch.equal(one[k], two[k])
        assert torch.equal(add[k], base[k] + one[k])
    # dx in place of dy
    ws = torch.empty(omni.omni_layer_norm_bwd_workspace_size(L, d), dtype=torch.uint8, device=DEV)
    inplace, dw, db = dy.clone(), torch.zeros(d, device=DEV), torch.zeros(d, device=DEV)
    omni.omni_layer_norm_bwd(x, f["mean"], f["rstd"], None, None, w, inplace, L, d, inplace, dw, db,
                             omni.OMNI_X_F32, ws)
    assert torch.equal(inplace, one["dx"]) and torch.equal(dw, one["dw"]) and torch.equal(db, one["db"])
    # dx added to dy itself
    inplace = dy.clone()
    got = omni.layer_norm_bwd(inplace, w, f["rstd"], **kept, dx=inplace)
    assert torch.equal(inplace, dy + one["dx"])
    assert torch.equal(got["dw"], one["dw"]) and torch.equal(got["db"], one["db"])


@pytest.mark.parametrize("fill", [0, 0xff])
def test_every_workspace_reports_its_own_call(fill):
    """The status word that a caller reads afterwards is the call's, whatever the
    workspace held: all of the operators that take one."""
    L, d, N_r, N_c, K = 33, 256, 20, 30, 4
    x, W_r, W_c, p_r, p_c, idx, _ = _balance_inputs(L, d, N_r, N_c, K, 4)
    r, w, b, dy = _rows(L, d, torch.float32, 9)
    W = V = torch.zeros(N_r * N_c, d, dtype=torch.bfloat16, device=DEV)
    q, scale = omni.act_pack(x)
    ws = lambda n: torch.full((n,), fill, dtype=torch.uint8, device=DEV)     # noqa: E731
    used = [ws(256), ws(omni.omni_balance_fwd_workspace_size(L, N_r, N_c)),
            ws(omni.omni_balance_bwd_workspace_size(L, d, N_r, N_c)), ws(omni.omni_layer_norm_bwd_workspace_size(L, d)),
            ws(omni.omni_routed_bwd_ckpt_workspace_size(L, d, N_r, N_c, K))]
    cnt = omni.expert_counts(idx, N_r * N_c, ws=used[0])
    fwd = omni.balance_fwd(p_r, p_c, cnt["counts"], cnt["n_tokens"], K, ws=used[1])
    omni.balance_bwd(x, W_r, W_c, p_r, p_c, cnt["counts"], cnt["n_tokens"], K, fwd["token_loss"], ws=used[2])
    f = omni.layer_norm_fwd(r, w, b)
    omni.layer_norm_bwd(dy, w, f["rstd"], x=r, mean=f["mean"], ws=used[3])
    gate = torch.full((L, K), 1 / K, device=DEV)
    omni.routed_bwd_ckpt(q, scale, W, V, W_r, W_c, idx, gate, dy, ws=used[4])
    assert [omni.omni_get_device_status(t) for t in used] == [0] * 5


def test_bindings_give_what_the_wrappers_give():
    """The omni_* bindings with buffers of the caller's, bit for bit (the routed
    backward's atomics aside), and what their outputs leave alone."""
    L, d, N_r, N_c, K = 33, 256, 20, 30, 4
    x, W_r, W_c, p_r, p_c, idx, mask = _balance_inputs(L, d, N_r, N_c, K, 4, masked=True)
    r, w, b, dy = _rows(L, d, torch.float32, 9)
    new = lambda t: torch.full_like(t, 7)                # noqa: E731
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)

    def same(got, want):
        for g, v in zip(got, want):
            assert torch.equal(g, v)

    c = omni.expert_counts(idx, N_r * N_c, mask=mask)
    out = new(c["counts"]), new(c["n_tokens"])
    omni.omni_expert_counts(idx, mask, L, K, N_r * N_c, *out, ws)
    same(out, (c["counts"], c["n_tokens"]))
    f = omni.balance_fwd(p_r, p_c, c["counts"], c["n_tokens"], K, mask=mask)
    out = new(f["loss"]), new(f["token_loss"])
    omni.omni_balance_fwd(p_r, p_c, c["counts"], c["n_tokens"], mask, L, N_r, N_c, K, *out, ws)
    same(out, (f["loss"], f["token_loss"]))
    n = omni.layer_norm_fwd(r, w, b, ckpt=True)
    out = [new(n[k]) for k in ("y", "mean", "rstd", "q", "scale")]
    omni.omni_layer_norm_fwd(r, w, b, L, d, 1e-5, *out, omni.OMNI_X_F32)
    same(out, [n[k] for k in ("y", "mean", "rstd", "q", "scale")])
    packed = omni.act_pack(x)
    out = [new(t) for t in packed]
    omni.omni_act_pack(x, L, d, *out, 0)
    same(out, packed)
    y = new(x)
    omni.omni_act_unpack(*packed, w, b, L, d, y)
    same([y], [omni.act_unpack(*packed, w, b)])
    W, V = ((torch.randn(N_r * N_c, d, generator=_gen(s), device=DEV) * 0.1).to(torch.bfloat16) for s in (1, 2))
    gate = torch.full((L, K), 1 / K, device=DEV)
    g = omni.routed_bwd_ckpt(*packed, W, V, W_r, W_c, idx, gate, dy, w=w, b=b)
    names = ("dx", "dW", "dV", "dW_r", "dW_c")
    for flags, start in ((0, 1.0), (omni.OMNI_DW_OVERWRITE, float("nan"))):
        out = [torch.full_like(g[k], start) for k in names]
        omni.omni_routed_bwd_ckpt(*packed, w, b, W, V, W_r, W_c, L, d, N_r, N_c, K, idx, gate, dy, *out, flags, ws)
        for k, t in zip(names, out):
            base = start if flags == 0 and k != "dx" else 0.0
            assert (t - base - g[k]).norm() <= 1e-5 * (g[k].norm() + base * g[k].numel() ** 0.5), k


@pytest.mark.parametrize("L,d", [(3, 8), (1000, 8), (700, 776), (5000, 1024), (300, 8192)])
def test_rows_written_in_place(L, d):
    """y over a bf16 x, dx over an fp32 x: bit for bit what separate arrays give."""
    x, w, b, dy = _rows(L, d, torch.bfloat16, L)
    want = omni.layer_norm_fwd(x, w, b)
    omni.omni_layer_norm_fwd(x, w, b, L, d, 1e-5, x, None, None, None, None, 0)
    assert torch.equal(x, want["y"])
    x = _rows(L, d, torch.float32, L + 1)[0]
    f = omni.layer_norm_fwd(x, w, b)
    kept = dict(mean=f["mean"])
    want = omni.layer_norm_bwd(dy, w, f["rstd"], x=x, **kept)
    base = x.clone()
    got = omni.layer_norm_bwd(dy, w, f["rstd"], x=x, **kept, dx=x)
    assert torch.equal(x, base + want["dx"]) and got["dx"] is x
    assert torch.equal(got["dw"], want["dw"]) and torch.equal(got["db"], want["db"])


def test_overwrite_does_not_read_the_gradients():
    """OMNI_DW_OVERWRITE on buffers full of NaN, through the C entry points."""
    L, d, N_r, N_c, K = 70, 256, 20, 30, 4
    nan = lambda *shape: torch.full(shape, float("nan"), device=DEV)     # noqa: E731
    x, W_r, W_c, p_r, p_c, idx, _ = _balance_inputs(L, d, N_r, N_c, K, 4)
    cnt = omni.expert_counts(idx, N_r * N_c)
    fwd = omni.balance_fwd(p_r, p_c, cnt["counts"], cnt["n_tokens"], K)
    want = omni.balance_bwd(x, W_r, W_c, p_r, p_c, cnt["counts"], cnt["n_tokens"], K, fwd["token_loss"],
                            dW_r=torch.zeros(N_r, d, device=DEV))
    dx, dW_r, dW_c = nan(L, d), nan(N_r, d), nan(N_c, d)
    ws = torch.empty(omni.omni_balance_bwd_workspace_size(L, d, N_r, N_c), dtype=torch.uint8, device=DEV)
    omni.omni_balance_bwd(x, W_r, W_c, p_r, p_c, cnt["counts"], cnt["n_tokens"], None, fwd["token_loss"], L, d,
                          N_r, N_c, K, 1.0, dx, dW_r, dW_c, omni.OMNI_DW_OVERWRITE, ws)
    for got, k in ((dx, "dx"), (dW_r, "dW_r"), (dW_c, "dW_c")):
        assert torch.equal(got, want[k]), k
    r, w, b, dy = _rows(L, d, torch.float32, 9)
    n = omni.layer_norm_fwd(r, w, b)
    want = omni.layer_norm_bwd(dy, w, n["rstd"], x=r, mean=n["mean"], dw=torch.zeros(d, device=DEV))
    dx, dw, db = nan(L, d), nan(d), nan(d)
    ws = torch.empty(omni.omni_layer_norm_bwd_workspace_size(L, d), dtype=torch.uint8, device=DEV)
    omni.omni_layer_norm_bwd(r, n["mean"], n["rstd"], None, None, w, dy, L, d, dx, dw, db,
                             omni.OMNI_X_F32 | omni.OMNI_DW_OVERWRITE, ws)
    for got, k in ((dx, "dx"), (dw, "dw"), (db, "db")):
        assert torch.equal(got, want[k]), k


# ----------------------------------------------------------- checkpoints
@pytest.mark.parametrize("L,d", [(1, 32), (1, 64), (3, 96), (50, 224), (17, 2048), (3, 8224)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_pack_and_unpack_are_exact(L, d, dtype):
    g = _gen(L + d)
    x = torch.randn(L, d, generator=g, device=DEV) * torch.exp2(40 * torch.rand(L, d // 32, generator=g, device=DEV) - 20).repeat_interleave(32, 1)
    x = x.to(dtype)
    x[0, :32] = 0
    q, scale = omni.act_pack(x)
    wq, wcode, bad = ref.pack_ref(x)
    assert not bad.any()
    assert torch.equal(scale.cpu().long(), wcode)
    assert torch.equal(q.cpu().long() & 127, wq & 127)
    v = ref.unpack_ref(q, scale)
    assert torch.equal(v, ref.unpack_ref(wq, wcode))
    assert torch.equal(omni.act_unpack(q, scale).cpu(), v.to(torch.bfloat16))


def test_pack_borders_and_special_values():
    """Ties, powers of two, the largest and smallest numbers, infinities, NaN."""
    rows = [
        [448.0, 1.0], [448.0 + 2.0 ** -14, 1.0], [449.0, -449.0], [447.0, 1.0625], [1.0, 1.0625],
        [1.75, 1.0], [2.0 ** -20, 2.0 ** -30], [3.3895313892515355e38, 1.0], [1e-38, 1e-39],
        [1e-44, -1e-44], [float("inf"), 5.0], [float("nan"), -7.0], [float("-inf"), 0.0],
        [256.0, 0.001953125], [256.0, 0.0009765625], [256.0, 0.00146484375],
    ]
    x = torch.zeros(len(rows), 32)
    for i, r in enumerate(rows):
        x[i, :2] = torch.tensor(r)
        x[i, 31] = r[1]
    wq, wcode, bad = ref.pack_ref(x)
    q, scale = omni.act_pack(x.to(DEV))
    q, scale = q.cpu().long(), scale.cpu().long()
    assert torch.equal(scale, wcode)
    assert ((q & 127)[bad] == 127).all()
    assert torch.equal((q & 127)[~bad], (wq & 127)[~bad])
    sign = (x < 0) & ~bad
    assert ((q >> 7)[sign] == 1).all()
    assert torch.isnan(omni.act_unpack(*omni.act_pack(x.to(DEV)))[10, 0])


def test_unpack_reads_every_byte_and_scale():
    """All 256 bytes under all scales: the value times 2^(scale - 127), to bf16."""
    q = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    scale = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 8)
    got = omni.act_unpack(q.to(DEV), scale.to(DEV)).cpu()
    v = ref.unpack_ref(q, scale)[:255]                   # 255 is no scale that pack writes
    want = v.float().to(torch.bfloat16)                  # fp32 holds the value or rounds it to a subnormal
    ok = (got[:255] == want) | (torch.isnan(got[:255]) & torch.isnan(want))
    assert ok.all()


# ------------------------------------------- routed backward from 8 bits
@pytest.mark.parametrize("L,d,N_r,N_c,K,affine", [(256, 256, 64, 64, 16, True), (1, 256, 8, 8, 4, False),
                                                  (33, 768, 40, 30, 7, True), (50, 2048, 64, 48, 32, False)])
def test_routed_bwd_from_a_checkpoint(L, d, N_r, N_c, K, affine):
    cfg = configs.LayerConfig("ckpt", L, d, N_r, N_c, K, 32)
    t = inputs.make_inputs(cfg, DEV, seed=L)
    _, w, b, dy = _rows(L, d, torch.float32, 3)
    w, b = (w, b) if affine else (None, None)
    q, scale = omni.act_pack(t["x"])
    x = omni.act_unpack(q, scale, w, b)
    r = omni.router_topk(x, t["W_r"], t["W_c"], K)
    args = (t["W"], t["V"], t["W_r"], t["W_c"])
    ws = torch.full((omni.omni_routed_bwd_ckpt_workspace_size(L, d, N_r, N_c, K),), 0xff, dtype=torch.uint8, device=DEV)
    got = omni.routed_bwd_ckpt(q, scale, *args, r["idx"], r["gate"], dy, w=w, b=b, ws=ws)
    assert omni.omni_get_device_status(ws) == 0
    same = omni.routed_bwd(x, *args, r["idx"], r["gate"], dy)
    want = ref.routed_bwd_ref(x, *args, r["idx"], r["gate"], dy)
    # dS is fp32: off by up to 2^-22 of the magnitudes it is a difference of,
    # which is all there is where a row's dS cancel (a token whose cells sit in
    # one row: the gradient is 0)
    slack = 2.0 ** -22 * ref.router_row_magnitude(x, t["W"], t["V"], r["idx"], r["gate"], dy)
    for k in want:
        top = want[k].abs().max()
        floor = slack if k in ("dW_r", "dW_c") else 0.0
        assert (got[k].double() - want[k]).abs().max() <= 2e-4 * top + floor, k
        assert (got[k].double() - want[k]).norm() <= 2e-4 * want[k].norm() + floor * want[k].numel() ** 0.5, k
        assert (got[k] - same[k]).abs().max() <= 1e-5 * top + 2 * floor, k


# --------------------------------------------------------------- together
def _train_step(res, p, K, B, eps=1e-5, alpha=0.01):
    """One pre-norm routed layer, forward and backward, as a training step runs
    it: norm with a checkpoint, routed branch added to the residual stream,
    balance loss, then the backward from the checkpoint alone."""
    f = omni.layer_norm_fwd(res, p["w"], p["b"], eps=eps, ckpt=True)
    rt = omni.router_topk(f["y"], p["W_r"], p["W_c"], K)
    N = len(p["W"])
    sched = omni.schedule(rt["idx"], rt["gate"], N, B)
    out = omni.grouped_expert_fwd(f["y"], p["W"], p["V"], sched, K, B, y=res.clone(), accumulate=True)
    cnt = omni.expert_counts(rt["idx"], N)
    bal = omni.balance_fwd(rt["p_r"], rt["p_c"], cnt["counts"], cnt["n_tokens"], K)
    dy = out                                              # gradient of 0.5 |out|^2
    g = omni.routed_bwd_ckpt(f["q"], f["scale"], p["W"], p["V"], p["W_r"], p["W_c"], rt["idx"],
                             rt["gate"], dy, w=p["w"], b=p["b"])
    n = omni.act_unpack(f["q"], f["scale"], p["w"], p["b"])
    omni.balance_bwd(n, p["W_r"], p["W_c"], rt["p_r"], rt["p_c"], cnt["counts"], cnt["n_tokens"], K,
                     bal["token_loss"], dloss=alpha, dx=g["dx"], dW_r=g["dW_r"], dW_c=g["dW_c"])
    norm = omni.layer_norm_bwd(g["dx"], p["w"], f["rstd"], q=f["q"], scale=f["scale"], dx=dy.clone())
    return dict(out=out, loss=bal["loss"], n=n, idx=rt["idx"], gate=rt["gate"], p_r=rt["p_r"], p_c=rt["p_c"],
                counts=cnt["counts"], rstd=f["rstd"], q=f["q"], scale=f["scale"], dx=norm["dx"],
                dw=norm["dw"], db=norm["db"], **{k: g[k] for k in ("dW", "dV", "dW_r", "dW_c")})


def _layer_params(cfg, seed):
    t = inputs.make_inputs(cfg, DEV, seed=seed)
    _, w, b, _ = _rows(1, cfg.d, torch.float32, seed)
    return dict(w=w, b=b, **{k: t[k] for k in ("W", "V", "W_r", "W_c")})


def test_a_training_step_of_the_layer():
    cfg = configs.LayerConfig("step", 200, 512, 40, 48, 12, 32)
    p = _layer_params(cfg, 6)
    res = _rows(cfg.L, cfg.d, torch.float32, 21)[0]
    s = _train_step(res, p, cfg.K, cfg.B)
    # the same chain in 64 bits, from the checkpoint's values and the routing
    kept = ref.unpack_ref(s["q"], s["scale"]).to(DEV)
    r = ref.routed_bwd_ref(s["n"], p["W"], p["V"], p["W_r"], p["W_c"], s["idx"], s["gate"], s["out"])
    b = ref.balance_ref(s["n"], p["W_r"], p["W_c"], s["p_r"], s["p_c"], s["counts"], cfg.L, cfg.K, 0.01)
    assert abs(s["loss"].item() - b["loss"].item()) <= 1e-4 * b["loss"].item()
    dn = r["dx"] + b["dx"]
    norm = ref.norm_bwd_ref(dn, p["w"], s["rstd"], kept)
    want = dict(dW=r["dW"], dV=r["dV"], dW_r=r["dW_r"] + b["dW_r"], dW_c=r["dW_c"] + b["dW_c"],
                dx=s["out"].double() + norm["dx"], dw=norm["dw"], db=norm["db"])
    for k in want:                                        # the routed backward's bar holds for the chain
        assert (s[k].double() - want[k]).norm() <= 2e-4 * want[k].norm(), k


def test_layer_fwd_with_its_norm():
    cfg = configs.TINY
    p = _layer_params(cfg, 3)
    F = configs.mlp_hidden(cfg.d)
    m = inputs.make_mlp_weights(cfg.d, F, DEV, seed=3)
    res = _rows(cfg.L, cfg.d, torch.float32, 4)[0]
    args = (p["W"], p["V"], p["W_r"], p["W_c"], m["W_g"], m["W_u"], m["W_d"], cfg.K, cfg.B)
    n = omni.layer_norm_fwd(res, p["w"], p["b"])["y"]
    want = omni.layer_fwd(n, *args)
    got = omni.layer_fwd(res, *args, norm_w=p["w"], norm_b=p["b"])
    assert (got - want).norm() <= 1e-5 * want.norm()     # the expert sum's order varies between runs


@pytest.mark.parametrize("L,dtype", [(1, torch.float32), (3, torch.bfloat16), (16, torch.float32), (17, torch.float32)])
def test_layer_fwd_with_its_norm_on_few_tokens(L, dtype):
    """Decode steps (the fused step up to 16 tokens) and the first size past them."""
    cfg = configs.TINY
    p = _layer_params(cfg, 3)
    m = inputs.make_mlp_weights(cfg.d, configs.mlp_hidden(cfg.d), DEV, seed=3)
    res = _rows(L, cfg.d, dtype, 4 + L)[0]
    args = (p["W"], p["V"], p["W_r"], p["W_c"], m["W_g"], m["W_u"], m["W_d"], cfg.K, cfg.B)
    for eps in (None, 1e-3):
        n = omni.layer_norm_fwd(res, p["w"], p["b"], **({} if eps is None else dict(eps=eps)))["y"]
        want = omni.layer_fwd(n, *args)
        got = omni.layer_fwd(res, *args, norm_w=p["w"], norm_b=p["b"], norm_eps=eps)
        assert (got - want).norm() <= 1e-5 * want.norm()


# ----------------------------------------------- streams, graphs, workspaces
def _flat(s):
    return {k: v.clone() for k, v in s.items()}


def test_calls_on_two_streams_at_once():
    """Two batches on two streams, each with its own outputs and workspaces
    (allocated by the wrappers on those streams), interleaved many times."""
    sets = []
    for seed in (1, 2):
        x, W_r, W_c, p_r, p_c, idx, mask = _balance_inputs(500, 256, 130, 70, 8, seed, masked=seed == 2)
        r, w, b, dy = _rows(500, 256, torch.float32, seed)
        sets.append((x, W_r, W_c, p_r, p_c, idx, mask, r, w, b, dy))

    def step(a, stream):
        x, W_r, W_c, p_r, p_c, idx, mask, r, w, b, dy = a
        c = omni.expert_counts(idx, 130 * 70, mask=mask, stream=stream)
        f = omni.balance_fwd(p_r, p_c, c["counts"], c["n_tokens"], 8, mask=mask, stream=stream)
        g = omni.balance_bwd(x, W_r, W_c, p_r, p_c, c["counts"], c["n_tokens"], 8, f["token_loss"],
                             mask=mask, stream=stream)
        n = omni.layer_norm_fwd(r, w, b, ckpt=True, stream=stream)
        h = omni.layer_norm_bwd(dy, w, n["rstd"], q=n["q"], scale=n["scale"], stream=stream)
        return dict(loss=f["loss"], gx=g["dx"], gr=g["dW_r"], gc=g["dW_c"], y=n["y"], dx=h["dx"], dw=h["dw"])

    want = [step(a, None) for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(10):
        got = [step(a, s) for a, s in zip(sets, streams)]
        torch.cuda.synchronize()
        for w_, g_ in zip(want, got):
            for k in w_:
                assert torch.equal(w_[k], g_[k]), k


@pytest.mark.parametrize("norm", [False, True])
def test_layer_fwd_on_a_stream_keeps_its_scratch(norm):
    """The call returns while its stream is still busy; what is allocated and
    written on the current stream meanwhile is none of its scratch."""
    cfg = configs.TINY
    p = _layer_params(cfg, 3)
    m = inputs.make_mlp_weights(cfg.d, configs.mlp_hidden(cfg.d), DEV, seed=3)
    res = _rows(cfg.L, cfg.d, torch.bfloat16, 8)[0]
    args = (p["W"], p["V"], p["W_r"], p["W_c"], m["W_g"], m["W_u"], m["W_d"], cfg.K, cfg.B)
    given = dict(norm_w=p["w"], norm_b=p["b"]) if norm else {}
    want = omni.layer_fwd(res, *args, **given)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(20_000_000)
    got = omni.layer_fwd(res, *args, **given, stream=stream)
    over = [torch.zeros(n, dtype=torch.uint8, device=DEV) for n in (1 << k for k in range(9, 25)) for _ in range(4)]
    torch.cuda.synchronize()
    assert (got - want).norm() <= 1e-5 * want.norm() and not any(t.any() for t in over)


def test_captured_and_replayed():
    """The chain in a CUDA graph, replayed on new inputs in the same buffers; a
    second graph that shares the workspaces, replayed in turn with the first."""
    L, d, N_r, N_c, K = 300, 256, 70, 90, 8
    first = _balance_inputs(L, d, N_r, N_c, K, 1, masked=True)
    second = _balance_inputs(L, d, N_r, N_c, K, 2, masked=True)
    r1, w, b, dy = _rows(L, d, torch.float32, 1)
    r2 = _rows(L, d, torch.float32, 2)[0]
    buf = [t.clone() for t in first]
    res = r1.clone()
    ws = dict(c=torch.empty(256, dtype=torch.uint8, device=DEV),
              f=torch.empty(omni.omni_balance_fwd_workspace_size(L, N_r, N_c), dtype=torch.uint8, device=DEV),
              b=torch.empty(omni.omni_balance_bwd_workspace_size(L, d, N_r, N_c), dtype=torch.uint8, device=DEV),
              n=torch.empty(omni.omni_layer_norm_bwd_workspace_size(L, d), dtype=torch.uint8, device=DEV))

    def step():
        x, W_r, W_c, p_r, p_c, idx, mask = buf
        c = omni.expert_counts(idx, N_r * N_c, mask=mask, ws=ws["c"])
        f = omni.balance_fwd(p_r, p_c, c["counts"], c["n_tokens"], K, mask=mask, ws=ws["f"])
        g = omni.balance_bwd(x, W_r, W_c, p_r, p_c, c["counts"], c["n_tokens"], K, f["token_loss"],
                             mask=mask, ws=ws["b"])
        n = omni.layer_norm_fwd(res, w, b, ckpt=True)
        h = omni.layer_norm_bwd(dy, w, n["rstd"], q=n["q"], scale=n["scale"], ws=ws["n"])
        p = omni.act_pack(n["y"])
        return dict(counts=c["counts"], loss=f["loss"], gx=g["dx"], gr=g["dW_r"], gc=g["dW_c"], y=n["y"],
                    dx=h["dx"], dw=h["dw"], db=h["db"], restored=omni.act_unpack(*p))

    def fill(src, r):
        for t, s in zip(buf, src):
            t.copy_(s)
        res.copy_(r)

    want = []
    for src, r in ((first, r1), (second, r2)):
        fill(src, r)
        want.append(_flat(step()))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    for turn in range(4):
        at = turn % 2
        fill(*((first, r1), (second, r2))[at])
        g, out = graphs[turn // 2 % 2]
        g.replay()
        torch.cuda.synchronize()
        for k in want[at]:
            assert torch.equal(out[k], want[at][k]), (turn, k)


@pytest.mark.parametrize("n", [1 << 31, (1 << 32) + 64])
def test_wrappers_refuse_numbers_past_31_bits(n):
    idx = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    p = torch.zeros(4, 8, device=DEV)
    W, x = torch.zeros(8, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV)
    cnt = omni.expert_counts(idx, 64)
    for call in (lambda: omni.expert_counts(idx, n), lambda: omni.balance_fwd(p, p, cnt["counts"], cnt["n_tokens"], n),
                 lambda: omni.balance_bwd(x, W, W, p, p, cnt["counts"], cnt["n_tokens"], n, p[:, 0].contiguous())):
        with pytest.raises(ValueError, match="not below 2\\^31"):
            call()


def test_dloss_on_the_device():
    """Read back outside a capture; refused in one, which goes on without harm."""
    L, d, N_r, N_c, K = 50, 64, 12, 20, 3
    x, W_r, W_c, p_r, p_c, idx, _ = _balance_inputs(L, d, N_r, N_c, K, 5)
    cnt = omni.expert_counts(idx, N_r * N_c)
    fwd = omni.balance_fwd(p_r, p_c, cnt["counts"], cnt["n_tokens"], K)
    args = (x, W_r, W_c, p_r, p_c, cnt["counts"], cnt["n_tokens"], K, fwd["token_loss"])
    want = omni.balance_bwd(*args, dloss=0.25)
    scale = torch.tensor(0.25, device=DEV)
    got = omni.balance_bwd(*args, dloss=scale)
    assert all(torch.equal(got[k], want[k]) for k in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError, match="dloss"):
            omni.balance_bwd(*args, dloss=scale)
        got = omni.balance_bwd(*args, dloss=0.25)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)


def test_wrappers_refuse_what_does_not_fit():
    x, w, b, dy = _rows(4, 64, torch.float32, 1)
    f = omni.layer_norm_fwd(x, w, b)
    idx = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    p = torch.zeros(4, 8, device=DEV)
    counts, n = torch.zeros(64, dtype=torch.int32, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV)
    for call in (
            lambda: omni.layer_norm_fwd(x.half(), w), lambda: omni.layer_norm_fwd(x, w.float()),
            lambda: omni.layer_norm_fwd(x, w[:32]), lambda: omni.layer_norm_fwd(x.t().contiguous().t(), w),
            lambda: omni.layer_norm_fwd(x[0], w), lambda: omni.layer_norm_bwd(dy, w, f["rstd"]),
            lambda: omni.layer_norm_bwd(dy, w, f["rstd"], x=x, mean=f["mean"], q=x.byte()),
            lambda: omni.layer_norm_bwd(dy, w, f["rstd"][:2], x=x, mean=f["mean"]),
            lambda: omni.layer_norm_bwd(dy, w, f["rstd"], x=x, mean=f["mean"], bias=False, db=dy[0]),
            lambda: omni.act_unpack(x.byte(), x.byte()), lambda: omni.expert_counts(idx.long(), 64),
            lambda: omni.expert_counts(idx, 64, mask=torch.ones(3, dtype=torch.bool, device=DEV)),
            lambda: omni.balance_fwd(p, p, counts[:60], n, 2), lambda: omni.balance_fwd(p.double(), p, counts, n, 2),
            lambda: omni.balance_fwd(p, p, counts, n, 2, mask=torch.ones(4, device=DEV))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: omni.layer_norm_fwd(x, w, eps=-1.0), lambda: omni.expert_counts(idx, 0),
                 lambda: omni.balance_fwd(p, p, counts, n, 0),
                 lambda: omni.layer_norm_fwd(x[:, :40].contiguous(), w[:40].contiguous(), ckpt=True),
                 lambda: omni.balance_fwd(p, p, counts, n, 2, ws=torch.empty(256, dtype=torch.uint8, device=DEV))):
        with pytest.raises(omni.OmniError):
            call()
