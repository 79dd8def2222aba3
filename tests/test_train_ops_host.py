"""The training operators on the host: the references that their GPU tests use,
against differences and brute force, workspace sizes, and the refusals of the C
entry points and of the wrappers.  Nothing here reaches a GPU."""
import ctypes

import pytest
import torch

import atomic_expert_layer_b200 as omni
from atomic_expert_layer_b200 import _lib, build

import _train_ref as ref


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def _p(v):
    return ctypes.c_void_p(v)


FAKE = _p(1 << 20)                       # 16-byte aligned, never dereferenced
ODD = _p((1 << 20) + 2)
BIG = 1 << 34
APART = [_p(i << 24) for i in range(2, 7)]       # five gradients that share no memory


# ------------------------------------------------------------- references
def test_balance_reference_against_differences():
    """d(dloss * loss) along random directions of x, W_r, W_c, by central
    differences of the definition over all N experts (64 bits: the step 1e-5
    leaves 1e-10 of truncation and 1e-11 of rounding, relative to O(1) slopes)."""
    g = torch.Generator().manual_seed(3)
    L, d, N_r, N_c, K, dloss = 11, 16, 5, 7, 3, 0.7
    x, W_r, W_c = (torch.randn(n, d, generator=g, dtype=torch.float64) for n in (L, N_r, N_c))
    idx = torch.stack([torch.randperm(N_r * N_c, generator=g)[:K] for _ in range(L)]).int()
    mask = torch.rand(L, generator=g) > 0.3
    counts, n = ref.counts_ref(idx, N_r * N_c, mask)
    assert counts.sum() == n * K

    def loss(x, W_r, W_c):
        return dloss * ref.balance_loss_ref(x @ W_r.T, x @ W_c.T, counts, n, K, mask)

    got = ref.balance_ref(x, W_r, W_c, torch.log_softmax(x @ W_r.T, 1),
                          torch.log_softmax(x @ W_c.T, 1), counts, n, K, dloss, mask)
    assert abs(dloss * got["loss"] - loss(x, W_r, W_c)) < 1e-12
    args = [x, W_r, W_c]
    for at, name in enumerate(("dx", "dW_r", "dW_c")):
        for _ in range(4):
            v = torch.randn(args[at].shape, generator=g, dtype=torch.float64)
            up, dn = list(args), list(args)
            up[at], dn[at] = args[at] + 1e-5 * v, args[at] - 1e-5 * v
            num = (loss(*up) - loss(*dn)) / 2e-5
            assert abs(num - (got[name] * v).sum()) < 1e-7 * max(1.0, abs(num))


def test_balance_reference_is_one_when_even():
    # every expert taken once, uniform probabilities: N * N * (1/N)(1/N) = 1
    N_r, N_c = 4, 6
    idx = torch.arange(24).reshape(12, 2).int()
    counts, n = ref.counts_ref(idx, 24)
    z = torch.zeros(12, N_r, dtype=torch.float64), torch.zeros(12, N_c, dtype=torch.float64)
    assert abs(ref.balance_loss_ref(*z, counts, n, 2) - 1) < 1e-12


def test_norm_reference_against_differences():
    g = torch.Generator().manual_seed(5)
    L, d, eps = 4, 24, 1e-5
    x, dy = (torch.randn(L, d, generator=g, dtype=torch.float64) for _ in range(2))
    w, b = (torch.randn(d, generator=g, dtype=torch.float64) for _ in range(2))
    _, _, rstd, xh = ref.norm_ref(x, w, b, eps)
    got = ref.norm_bwd_ref(dy, w, rstd, xh)
    f = lambda x, w, b: (dy * ref.norm_ref(x, w, b, eps)[0]).sum()  # noqa: E731
    for at, name in enumerate(("dx", "dw", "db")):
        args = [x, w, b]
        v = torch.randn(args[at].shape, generator=g, dtype=torch.float64)
        up, dn = list(args), list(args)
        up[at], dn[at] = args[at] + 1e-5 * v, args[at] - 1e-5 * v
        num = (f(*up) - f(*dn)) / 2e-5
        assert abs(num - (got[name] * v).sum()) < 1e-7 * max(1.0, abs(num))


def test_pack_reference_by_hand():
    x = torch.zeros(1, 64)
    x[0, 0], x[0, 1], x[0, 2], x[0, 3] = 448.0, -1.0, 449.0, 0.0
    q, code, _ = ref.pack_ref(x)
    # 449 > 448: scale 2, so -1 is -0.5 and 449 / 2 = 224.5 rounds to 224
    assert code[0, 0] == 128 and code[0, 1] == 0
    v = ref.unpack_ref(q, code)
    assert v[0, :4].tolist() == [448.0, -1.0, 448.0, 0.0]
    x[0, 2] = 0
    q, code, _ = ref.pack_ref(x)
    assert code[0, 0] == 127 and ref.unpack_ref(q, code)[0, 0] == 448.0


# ------------------------------------------------------- sizes and refusals
def test_workspace_sizes(lib):
    assert omni.omni_balance_fwd_workspace_size(0, 8, 8) == 0
    assert omni.omni_balance_fwd_workspace_size(8, 8193, 8) == 0
    assert omni.omni_balance_bwd_workspace_size(8, 12, 8, 8) == 0           # d % 8
    L, d, N_r, N_c = 100, 64, 70, 60
    pr, pc = 128, 64
    up = lambda v: -(-v // 256) * 256                                       # noqa: E731
    fwd = 256 + 2 * up(2 * L * pc) + 2 * up(2 * N_r * pc) + up(8)     # and two sums a tile and token
    assert omni.omni_balance_fwd_workspace_size(L, N_r, N_c) - fwd in [up(4 * 2 * t * L) for t in (1, 2)]
    bwd = (256 + 4 * up(2 * L * (pr + pc)) + 2 * up(2 * N_r * pc) + 2 * up(2 * N_c * pr) + up(2 * L * d) +
           up(2 * (pr + pc) * d))
    assert omni.omni_balance_bwd_workspace_size(L, d, N_r, N_c) == bwd
    assert omni.omni_layer_norm_bwd_workspace_size(5, 12) == 0
    assert omni.omni_layer_norm_bwd_workspace_size(5, 8200) == 0
    assert omni.omni_layer_norm_bwd_workspace_size(5, 1000) % 256 == 0
    b = omni.omni_routed_bwd_workspace_size(7, 256, 8, 8, 4)
    assert omni.omni_routed_bwd_ckpt_workspace_size(7, 256, 8, 8, 4) == b + up(2 * 7 * 256)
    assert omni.omni_routed_bwd_ckpt_workspace_size(7, 256, 8, 8, 0) == 0


def _try_all_pointers(fn, args, pointers, optional=()):
    """Each required pointer as NULL is refused (OMNI_ERR_INVALID_ARG)."""
    for i in pointers:
        if i in optional:
            continue
        bad = list(args)
        bad[i] = None
        assert fn(*bad) == -1, i


def test_expert_counts_refusals(lib):
    ok = [FAKE, None, 4, 2, 16, FAKE, FAKE, FAKE, 256, None]
    _try_all_pointers(lib.omni_expert_counts, ok, (0, 5, 6, 7))
    for at, v, rc in ((2, 0, -1), (3, 0, -1), (4, 0, -1), (8, 255, -3), (7, ODD, -1), (0, ODD, -1),
                      (2, 1 << 30, -2)):
        bad = list(ok)
        bad[at] = v
        if at == 2 and rc == -2:
            bad[3] = 2
        assert lib.omni_expert_counts(*bad) == rc, (at, v)


def test_balance_refusals(lib):
    ok = [FAKE, FAKE, FAKE, FAKE, None, 4, 8, 8, 2, FAKE, FAKE, FAKE, BIG, None]
    _try_all_pointers(lib.omni_balance_fwd, ok, (0, 1, 2, 3, 9, 10, 11))
    for at, v, rc in ((5, 0, -1), (6, 0, -1), (7, -1, -1), (8, 0, -1), (6, 8193, -2), (7, 8193, -2),
                      (12, 1000, -3), (0, ODD, -1), (11, _p((1 << 20) + 16), -1), (5, (1 << 30) + 1, -2)):
        bad = list(ok)
        bad[at] = v
        assert lib.omni_balance_fwd(*bad) == rc, (at, v)
    ok = [FAKE] * 7 + [None, FAKE, 4, 64, 8, 8, 2, 1.0, *APART[:3], 0, FAKE, BIG, None]
    _try_all_pointers(lib.omni_balance_bwd, ok, (0, 1, 2, 3, 4, 5, 6, 8, 15, 16, 17, 19))
    for at, v, rc in ((9, 0, -1), (10, 0, -1), (10, 12, -2), (11, 9000, -2), (13, 0, -1), (18, 1, -1),
                      (20, 1000, -3), (0, ODD, -1), (15, _p((1 << 20) + 4), -1), (3, ODD, -1), (9, (1 << 30) + 1, -2)):
        bad = list(ok)
        bad[at] = v
        assert lib.omni_balance_bwd(*bad) == rc, (at, v)


def test_layer_norm_refusals(lib):
    ok = [FAKE, FAKE, None, 4, 64, 1e-5, FAKE, None, None, None, None, 0, None]
    _try_all_pointers(lib.omni_layer_norm_fwd, ok, (0, 1, 6))
    for at, v, rc in ((3, 0, -1), (4, 0, -1), (4, 12, -2), (4, 8200, -2), (5, -1.0, -1),
                      (5, float("nan"), -1), (9, FAKE, -1), (10, FAKE, -1), (11, 1, -1),
                      (11, 128, -1), (0, ODD, -1), (2, ODD, -1), (6, ODD, -1), (7, ODD, -1)):
        bad = list(ok)
        bad[at] = v
        assert lib.omni_layer_norm_fwd(*bad) == rc, (at, v)
    # a checkpoint needs whole blocks of 32
    assert lib.omni_layer_norm_fwd(FAKE, FAKE, None, 4, 40, 1e-5, FAKE, None, None, FAKE, FAKE, 0,
                                   None) == -2
    ok = [FAKE, FAKE, FAKE, None, None, FAKE, FAKE, 4, 64, APART[0], APART[1], None, 0, FAKE, BIG, None]
    _try_all_pointers(lib.omni_layer_norm_bwd, ok, (0, 1, 2, 5, 6, 9, 10, 13))
    for at, v, rc in ((7, 0, -1), (8, 12, -2), (3, FAKE, -1), (4, FAKE, -1), (12, 2, -1), (14, 100, -3),
                      (6, ODD, -1), (13, _p((1 << 20) + 8), -1), (11, ODD, -1)):
        bad = list(ok)
        bad[at] = v
        assert lib.omni_layer_norm_bwd(*bad) == rc, (at, v)


def test_checkpoint_refusals(lib):
    ok = [FAKE, 4, 64, FAKE, FAKE, 0, None]
    _try_all_pointers(lib.omni_act_pack, ok, (0, 3, 4))
    for at, v, rc in ((1, 0, -1), (2, 40, -2), (5, 2, -1), (0, ODD, -1), (3, ODD, -1)):
        bad = list(ok)
        bad[at] = v
        assert lib.omni_act_pack(*bad) == rc, (at, v)
    ok = [FAKE, FAKE, None, None, 4, 64, FAKE, None]
    _try_all_pointers(lib.omni_act_unpack, ok, (0, 1, 6))
    for at, v, rc in ((4, 0, -1), (5, 48, -2), (3, FAKE, -1), (6, ODD, -1), (2, ODD, -1)):
        bad = list(ok)
        bad[at] = v
        assert lib.omni_act_unpack(*bad) == rc, (at, v)
    ok = [FAKE, FAKE, None, None, FAKE, FAKE, FAKE, FAKE, 4, 256, 8, 8, 2] + [FAKE] * 3 + APART + [0, FAKE, BIG, None]
    _try_all_pointers(lib.omni_routed_bwd_ckpt, ok, (0, 1, 4, 5, 6, 7, *range(13, 21), 22))
    for at, v, rc in ((8, 0, -1), (9, 264, -2), (12, 65, -1), (21, 1, -1), (23, 256, -3), (3, FAKE, -1),
                      (16, ODD, -1)):
        bad = list(ok)
        bad[at] = v
        assert lib.omni_routed_bwd_ckpt(*bad) == rc, (at, v)


@pytest.mark.parametrize("shift", [0, 1, 2])
def test_gradients_that_share_memory_are_refused(lib, shift):
    """One buffer for two gradients, or one that begins inside another: their
    tiles would update it at the same time."""
    def refused(fn, args, at, n):
        for i, a in enumerate(at):
            for b in at[:i]:
                bad = list(args)
                bad[b] = _p(args[a].value - (0, 16, -4 * (n[i] - 4))[shift])
                assert fn(*bad) == -1, (a, b)

    L, d, N_r, N_c = 4, 256, 12, 8
    tied = [FAKE] * 7 + [None, FAKE, L, d, N_r, N_c, 2, 1.0, *APART[:3], 0, FAKE, BIG, None]
    refused(lib.omni_balance_bwd, tied, (15, 16, 17), (L * d, N_r * d, N_c * d))
    norm = [FAKE, FAKE, FAKE, None, None, FAKE, _p(9 << 24), L, d, *APART[:3], 0, FAKE, BIG, None]
    refused(lib.omni_layer_norm_bwd, norm, (9, 10, 11), (L * d, d, d))
    if shift:
        # dx may be dy, but not begin inside it
        norm[9] = _p(norm[6].value + 16 * (2 * shift - 3))
        assert lib.omni_layer_norm_bwd(*norm) == -1
    routed = [FAKE, FAKE, None, None, FAKE, FAKE, FAKE, FAKE, L, d, N_r, N_c, 2, FAKE, FAKE, FAKE,
              *APART, 0, FAKE, BIG, None]
    refused(lib.omni_routed_bwd_ckpt, routed, (16, 17, 18, 19, 20),
            (L * d, N_r * N_c * d, N_r * N_c * d, N_r * d, N_c * d))
    routed[15] = _p(APART[0].value + 16 * shift)                 # nor dx and dy
    assert lib.omni_routed_bwd_ckpt(*routed) == -1


@pytest.mark.parametrize("at", range(5), ids=["dx", "dW", "dV", "dW_r", "dW_c"])
@pytest.mark.parametrize("shift", [0, 16, -1])
def test_no_gradient_shares_memory_with_dy(lib, at, shift):
    """Clearing or adding to a gradient would change the dy that the backward
    reads: every one of the five at dy, inside it, and reaching into it."""
    L, d, N_r, N_c = 4, 256, 12, 8
    n = (L * d, N_r * N_c * d, N_r * N_c * d, N_r * d, N_c * d)
    args = [FAKE, FAKE, None, None, FAKE, FAKE, FAKE, FAKE, L, d, N_r, N_c, 2, FAKE, FAKE, _p(9 << 24),
            *APART, 0, FAKE, BIG, None]
    args[16 + at] = _p((9 << 24) + (shift if shift >= 0 else 16 - 4 * n[at]))
    for flags in (0, omni.OMNI_DW_OVERWRITE):
        args[21] = flags
        assert lib.omni_routed_bwd_ckpt(*args) == -1


@pytest.mark.parametrize("at", [0, 1], ids=["idx", "gate"])
def test_routed_bwd_refuses_misaligned_routing(lib, at):
    """idx and gate are read 4 bytes at a time: off that grid they are refused
    on the host, as the other arrays are."""
    ckpt = [FAKE, FAKE, None, None, FAKE, FAKE, FAKE, FAKE, 4, 256, 8, 8, 2, FAKE, FAKE, _p(9 << 24),
            *APART, 0, FAKE, BIG, None]
    ckpt[13 + at] = ODD
    assert lib.omni_routed_bwd_ckpt(*ckpt) == -1
    bwd = [FAKE] * 5 + [4, 256, 8, 8, 2, FAKE, FAKE, _p(9 << 24), *APART, 0, FAKE, BIG, None]
    bwd[10 + at] = ODD
    assert lib.omni_routed_bwd(*bwd) == -1


@pytest.mark.parametrize("n", [1 << 31, (1 << 32) + 3])
def test_wrappers_refuse_sizes_past_31_bits(lib, n):
    """The C entry points take sizes of 32 bits: 2^32 + 3 rows would run as 3."""
    def rows(dtype, columns):
        return torch.zeros(1, columns, dtype=dtype).expand(n, columns)

    bf, f, u = rows(torch.bfloat16, 64), rows(torch.float32, 64), rows(torch.uint8, 64)
    w, i = torch.zeros(64, dtype=torch.bfloat16), rows(torch.int32, 1)
    for call in (lambda: omni.layer_norm_fwd(bf, w), lambda: omni.layer_norm_bwd(f, w, f[:, 0], x=f, mean=f[:, 0]),
                 lambda: omni.act_pack(bf), lambda: omni.act_unpack(u, u[:, :2]), lambda: omni.expert_counts(i, 16),
                 lambda: omni.balance_fwd(f, f, i, i, 2)):
        with pytest.raises(ValueError, match="not below 2\\^31"):
            call()


@pytest.mark.parametrize("shift", [0, 16, -16, "end"])
def test_outputs_over_rows_still_to_be_read_are_refused(lib, shift):
    """Other threads would write over rows that a thread has yet to read.  Only a
    row written in place, byte for byte where it was read, is sound."""
    L, d, N = 4, 64, 96
    x = 16 << 24

    def over(args, at, n_in, n_out):
        bad = list(args)
        bad[at] = _p(x + (n_in - 16 if shift == "end" else shift if shift >= 0 else 16 - n_out))
        return bad

    fwd = [_p(x), FAKE, None, L, d, 1e-5, APART[0], None, None, None, None, 0, None]
    if shift != 0:                                       # y over x itself, both bf16, is in place
        assert lib.omni_layer_norm_fwd(*over(fwd, 6, 2 * L * d, 2 * L * d)) == -1
    fwd[11] = omni.OMNI_X_F32
    assert lib.omni_layer_norm_fwd(*over(fwd, 6, 4 * L * d, 2 * L * d)) == -1
    fwd[9], fwd[10] = APART[1], APART[2]
    assert lib.omni_layer_norm_fwd(*over(fwd, 9, 4 * L * d, L * d)) == -1
    bwd = [_p(x), FAKE, FAKE, None, None, FAKE, _p(9 << 24), L, d, *APART[:3], 0, FAKE, BIG, None]
    assert lib.omni_layer_norm_bwd(*over(bwd, 9, 2 * L * d, 4 * L * d)) == -1
    if shift != 0:                                       # dx over x itself, both fp32, is in place
        bwd[12] = omni.OMNI_X_F32
        assert lib.omni_layer_norm_bwd(*over(bwd, 9, 4 * L * d, 4 * L * d)) == -1
    bwd[0], bwd[3], bwd[4], bwd[12] = None, _p(x), FAKE, 0
    assert lib.omni_layer_norm_bwd(*over(bwd, 9, L * d, 4 * L * d)) == -1
    for flags, size in ((0, 2), (omni.OMNI_X_F32, 4)):
        pack = [_p(x), L, d, APART[0], FAKE, flags, None]
        assert lib.omni_act_pack(*over(pack, 3, size * L * d, L * d)) == -1
    unpack = [_p(x), FAKE, None, None, L, d, APART[0], None]
    assert lib.omni_act_unpack(*over(unpack, 6, L * d, 2 * L * d)) == -1
    counts = [_p(x), None, L, 16, N, APART[0], APART[1], FAKE, 256, None]
    assert lib.omni_expert_counts(*over(counts, 5, 4 * L * 16, 4 * N)) == -1


def test_layer_fwd_refuses_half_a_norm(lib):
    x, w = torch.zeros(4, 256, dtype=torch.bfloat16), torch.ones(256, dtype=torch.bfloat16)
    for given in (dict(norm_b=w), dict(norm_eps=1e-6), dict(norm_b=w, norm_eps=0.0)):
        with pytest.raises(ValueError, match="norm_w is missing"):
            omni.layer_fwd(x, x, x, x, x, x, x, x, 2, 32, **given)


def test_wrappers_refuse_cpu_tensors(lib):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(64, dtype=torch.bfloat16)
    p = torch.zeros(4, 8)
    i = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: omni.layer_norm_fwd(x, w), lambda: omni.act_pack(x),
                 lambda: omni.act_unpack(x.view(torch.uint8), w.view(torch.uint8)),
                 lambda: omni.expert_counts(i, 16),
                 lambda: omni.balance_fwd(p, p, torch.zeros(64, dtype=torch.int32), i, 2),
                 lambda: omni.layer_norm_bwd(p, w, p)):
        with pytest.raises(ValueError):
            call()
