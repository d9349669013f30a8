"""The delta rule's plans: which kernel takes a call goes by how many 16-column
slices of (b, h) there are, so every count and width has its own instance.  Each
is held to test_delta_gpu's bars, on a few sequences of the batch (the oracle runs
token by token).  With s = ceil(Dv / 16) slices: up to 148 of them all together take
four warps a slice, up to 148 pairs two slices a block, more a warp a slice and as
many slices a block (1, 2, 4, 8) as end soonest."""
import numpy as np
import pytest
import torch

import oracle
from test_delta_gpu import BAR16, BAR32, BAR_STATE, built, dev, la, make, slice_err  # noqa: F401

pytestmark = pytest.mark.gpu

# B, H, Hk, Dv: BH s
PLANS = [
    (30, 1, 1, 128),  # 240: two slices a block
    (30, 1, 1, 112),  # 210, the last block with one
    (20, 2, 1, 128),  # 320: four a block, one round
    (38, 2, 2, 64),   # 304: four a block
    (38, 2, 1, 128),  # 608: eight a block
    (38, 2, 2, 112),  # 532: eight a block, the last one idle
    (75, 2, 1, 16),   # 150: one a block
    (75, 2, 2, 32),   # 300: two a block
]


def f64(t):
    return np.asarray(t.detach().cpu().double().numpy()) if hasattr(t, "detach") else np.asarray(t, np.float64)


def at(t, rows):
    return None if t is None else t[rows]


def gradients_near(got, args, dy, kind, dS, scale, rows, dtype, twice=1.0):
    """test_delta_gpu.check_backward's bars, for some sequences of the batch."""
    q, k, v, beta, lg, S0 = args
    picked = [at(t, rows) for t in (q, k, v, beta)]
    want = oracle.delta_backward(*picked, at(dy, rows), kind, at(lg, rows) if kind == 2 else lg, at(S0, rows), at(dS, rows), scale)
    mine = [at(t, rows) if i != 4 or kind == 2 else None for i, t in enumerate(got)]
    low = twice * 2 * (BAR_STATE if dtype == torch.bfloat16 else BAR32)
    own = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    for name, x, r in zip(("dq", "dk", "dv"), mine, want):
        assert slice_err(x, r) <= own + low, name
    assert slice_err(mine[5], want[5]) <= low, "d_init_state"
    rep = v.shape[1] // q.shape[1]
    norm = lambda t: np.linalg.norm(f64(t), axis=-1)  # noqa: E731
    terms = np.abs(np.repeat((f64(picked[0]) * want[0]).sum(-1), rep, 1)) + np.repeat(norm(picked[1]) * norm(want[1]), rep, 1) \
        + norm(picked[2]) * norm(want[2])
    size = np.linalg.norm(terms, axis=-1) + 1e-30
    assert (np.linalg.norm(f64(mine[3]) - want[3], axis=-1) <= low * (size + np.linalg.norm(want[3], axis=-1))).all(), "dbeta"
    if kind == 2:
        assert (np.linalg.norm(f64(mine[4]) - want[4], axis=-1) <= low * (size + np.linalg.norm(want[4], axis=-1))).all(), "d_log_g"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Dk", [32, 64, 128])
@pytest.mark.parametrize("B,H,Hk,Dv", PLANS)
def test_every_plan(B, H, Hk, Dv, Dk, dtype):
    T, scale, rows = 270, 0.25, [0, B // 2, B - 1]  # five chunks: every stage is used again
    if dtype == torch.float32 and Dv % 16 == 0:
        Dv -= 3  # values that end inside a slice
    args = make(B, H, Hk, T, Dk, Dv, dtype, seed=Dk + Dv)
    g = torch.Generator().manual_seed(1)
    dy, dS = torch.randn(args[2].shape, generator=g).to(dtype), 0.3 * torch.randn(B, H, Dk, Dv, generator=g)
    q, k, v, beta, lg, S0 = dev(*args)
    y, S = la().delta_forward(q, k, v, beta, 2, lg, S0, q_scale=scale)
    ry, rS = oracle.delta_forward(*(t[rows] for t in args[:4]), 2, args[4][rows], args[5][rows], scale)
    assert slice_err(y[rows], ry) <= (BAR16 if dtype == torch.bfloat16 else BAR32)
    assert slice_err(S[rows], rS) <= (BAR_STATE if dtype == torch.bfloat16 else BAR32)
    got = la().delta_backward(q, k, v, beta, dy.cuda(), 2, lg, S0, dS.cuda(), q_scale=scale)
    gradients_near(got, args, dy, 2, dS, scale, rows, dtype)
    again = la().delta_backward(q, k, v, beta, dy.cuda(), 2, lg, S0, dS.cuda(), q_scale=scale)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    if dtype == torch.bfloat16:  # a decay per head: three planes an operand
        lg1 = make(1, H, Hk, 1, 16, 16, kind=1)[4]
        got = la().delta_backward(q, k, v, beta, dy.cuda(), 1, lg1.cuda(), S0, dS.cuda(), q_scale=scale)
        gradients_near(got, (*args[:4], lg1, args[5]), dy, 1, dS, scale, rows, dtype)


def test_offsets_beyond_32_bits():
    # 64 heads: y has more than 2^31 elements, the records 6.8 GB; each head is what it is alone
    H, T, D = 64, 262144 + 65, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    q, k, v = rn(1, H, T, D), rn(1, H, T, D), rn(1, H, T, D)
    q.mul_(D ** -0.5)
    k.mul_(D ** -0.5)
    beta, lg = torch.rand(1, H, T, generator=g, device="cuda"), -0.1 * torch.rand(1, H, T, generator=g, device="cuda")
    y, S = la().delta_forward(q, k, v, beta, 2, lg)
    assert y.numel() > 2 ** 31
    for h in (0, 40, 63):
        one = [t[:, h:h + 1] for t in (q, k, v, beta, lg)]
        ya, Sa = la().delta_forward(*one[:4], 2, one[4])
        assert slice_err(y[:, h:h + 1, -4096:], f64(ya[:, :, -4096:])) <= BAR16
        assert slice_err(S[:, h:h + 1], f64(Sa)) <= 2 * BAR_STATE


def test_gradients_offsets_beyond_32_bits():
    # the states' planes pass 2^31 elements (64 heads x 1025 chunks x 2 x 128 x 128), the workspace 16 GB
    H, T, D = 64, 65536 + 33, 128
    g = torch.Generator(device="cuda").manual_seed(4)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    q, k, v, dy = rn(1, H, T, D), rn(1, H, T, D), rn(1, H, T, D), rn(1, H, T, D)
    q.mul_(D ** -0.5)
    k.mul_(D ** -0.5)
    beta, lg = torch.rand(1, H, T, generator=g, device="cuda"), -0.1 * torch.rand(1, H, T, generator=g, device="cuda")
    assert la().delta_backward_workspace_size(1, H, T, D, D, decay_kind=2) > 2 ** 33
    got = la().delta_backward(q, k, v, beta, dy, 2, lg)
    for h in (0, 40, 63):
        alone = la().delta_backward(*(t[:, h:h + 1].contiguous() for t in (q, k, v, beta, dy)), 2, lg[:, h:h + 1].contiguous())
        for i, (a, b) in enumerate(zip(got, alone)):
            ends = [slice(0, 512), slice(T - 512, T)] if i < 5 else [slice(None)]
            for e in ends:
                x, r = (a[:, h:h + 1][:, :, e], b[:, :, e]) if i < 5 else (a[:, h:h + 1], b)
                assert slice_err(x, f64(r)) <= (2.0 ** -7 if i < 3 else 0) + 8 * BAR_STATE, i


@pytest.mark.parametrize("beta_value,sign,inverse", [(1.0, 1, 2.0), (1.9, 1, 20.0), (1.9, -1, 20.0)])
@pytest.mark.parametrize("dtype,unit", [(torch.bfloat16, BAR_STATE), (torch.float32, BAR32)])
def test_one_key_repeated(dtype, unit, beta_value, sign, inverse):
    # I + A diag(beta) far from the identity: its inverse's columns sum to `inverse` (beta (1 - beta)^n), and that
    # many times the operands' rounding reaches the state.  One plane less (2^-16 instead of 2^-24, 2^-8 instead of
    # 2^-16) would be 5e-4 and above 0.1.
    q, k, v, beta, _, S0 = make(1, 2, 2, 300, 64, 64, dtype, kind=0, seed=12)
    k = k[:, :, :1].expand_as(k).contiguous()
    k[:, :, ::2] *= sign
    beta[:] = beta_value
    y, S = la().delta_forward(*dev(q, k, v, beta), 0, None, *dev(S0))
    ry, rS = oracle.delta_forward(q, k, v, beta, 0, None, S0)
    assert slice_err(S, rS) <= inverse * unit
    assert slice_err(y, ry) <= inverse * unit + (BAR16 if dtype == torch.bfloat16 else 0)


@pytest.mark.parametrize("Dk", [64, 128])
def test_gradients_of_a_loss_on_the_last_tokens(Dk):
    # many tokens (two planes an operand) of which four have a gradient of y: dbeta and d log g keep the bar
    # against their own terms
    B, H, T, Dv = 4, 4, 600, 64
    args = make(B, H, 2, T, Dk, Dv, seed=20)
    g = torch.Generator().manual_seed(2)
    dy, dS = torch.zeros(B, H, T, Dv), torch.zeros(B, H, Dk, Dv)
    dy[:, :, -4:] = torch.randn(B, H, 4, Dv, generator=g)
    dy = dy.bfloat16()
    got = la().delta_backward(*dev(*args[:4], dy), 2, *dev(args[4], args[5], dS), q_scale=0.25)
    gradients_near(got, args, dy, 2, dS, 0.25, [0, 3], torch.bfloat16)


def test_a_sequence_alone_and_in_a_batch():
    # 130 tokens alone take three planes, in a batch of 40 two: within both bars of one another
    args = make(40, 2, 1, 130, 64, 64, seed=21)
    dy = torch.randn(args[2].shape, generator=torch.Generator().manual_seed(3)).bfloat16()
    got = la().delta_backward(*dev(*args[:4], dy), 2, *dev(args[4], args[5]))
    one = [t[7:8].contiguous() for t in (*args[:4], dy, args[4], args[5])]
    alone = la().delta_backward(*dev(*one[:5]), 2, *dev(*one[5:]))
    gradients_near([t[7:8] for t in got], (*one[:4], *one[5:]), one[4], 2, torch.zeros(1, 2, 64, 64), 1.0, [0], torch.bfloat16)
    gradients_near(alone, (*one[:4], *one[5:]), one[4], 2, torch.zeros(1, 2, 64, 64), 1.0, [0], torch.bfloat16)
    y, S = la().delta_forward(*dev(*args[:4]), 2, *dev(args[4], args[5]))
    ya, Sa = la().delta_forward(*dev(*one[:4]), 2, *dev(*one[5:]))
    assert slice_err(y[7:8], f64(ya)) <= BAR16 and slice_err(S[7:8], f64(Sa)) <= 2 * BAR_STATE
