"""GPU parity of the gated delta rule (la_delta_*) against the float64 oracle,
which runs the recurrence token by token.

Bars, per (b, h) slice, ||x - ref|| / ||ref|| (2-norms), derived before the
first run from the roundings a value goes through:
  bf16 outputs      2^-8 (half a step) for the rounding of the output and as
                    much for the one rounded operand, the chunk's own scores: 2^-7.
  fp32 outputs of bf16 inputs (states): products of operands split in two bf16
                    planes drop at most 2^-16 of the operand; four such operands
                    follow one another in a chunk (state, right-hand side, errors,
                    update): 2^-14.
  fp32 inputs       three planes leave the fp32 sums' own roundings, at most
                    2^-24 for each of the 128 + 64 terms of the two sums that
                    follow one another: 192 2^-24 = 1.2e-5.
"""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

BAR16, BAR_STATE, BAR32 = 2.0 ** -7, 2.0 ** -14, 192 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    from retention_scan_b200 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield
    assert la().device_error() == 0, "a kernel gave up waiting on a barrier"


def la():
    import retention_scan_b200
    return retention_scan_b200


def slice_err(x, ref):
    """Worst (b, h) slice of ||x - ref|| / ||ref||; a slice of zeros has to be zeros."""
    x = x.detach().cpu().double().numpy() if hasattr(x, "detach") else np.asarray(x, np.float64)
    ref = np.asarray(ref, np.float64)
    assert x.shape == ref.shape
    lead = ref.shape[0] * (ref.shape[1] if ref.ndim > 1 else 1)
    worst = 0.0
    for a, r in zip(x.reshape(lead, -1), ref.reshape(lead, -1)):
        if not np.isfinite(a).all():
            return float("inf")
        n, d = np.linalg.norm(r), np.linalg.norm(a - r)
        worst = max(worst, d / n if n > 0 else d)
    return worst


def make(B, H, Hk, T, Dk, Dv, dtype=torch.bfloat16, kind=2, init=True, seed=0, correlated=0.0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    q = unit(rn(B, Hk, T, Dk)).to(dtype)
    k = unit(rn(B, Hk, T, Dk) + correlated * rn(B, Hk, 1, Dk)).to(dtype)
    v = rn(B, H, T, Dv).to(dtype)
    beta = torch.sigmoid(rn(B, H, T))
    lg = None
    if kind == 1:
        lg = torch.log1p(-torch.exp2(-5 - torch.arange(H, dtype=torch.float64))).float()
    elif kind == 2:
        lg = torch.nn.functional.logsigmoid(rn(B, H, T) + 3)
    S0 = 0.3 * rn(B, H, Dk, Dv) if init else None
    return q, k, v, beta, lg, S0


def dev(*ts):
    return [t.cuda() if t is not None else None for t in ts]


def check_forward(args, kind, scale=0.25, dtype=torch.bfloat16):
    q, k, v, beta, lg, S0 = args
    y, S = la().delta_forward(*dev(q, k, v, beta), kind, *dev(lg, S0), q_scale=scale)
    ry, rS = oracle.delta_forward(q, k, v, beta, kind, lg, S0, scale)
    assert slice_err(y, ry) <= (BAR16 if dtype == torch.bfloat16 else BAR32)
    assert slice_err(S, rS) <= (BAR_STATE if dtype == torch.bfloat16 else BAR32)
    return y, S


@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 130, 257])
@pytest.mark.parametrize("kind", [0, 1, 2])
def test_forward_lengths(T, kind):
    check_forward(make(2, 2, 2, T, 64, 64, kind=kind, seed=T), kind)


@pytest.mark.parametrize("Dk,Dv", [(16, 16), (32, 48), (48, 32), (64, 112), (80, 64), (96, 80), (112, 16), (128, 128)])
def test_forward_widths(Dk, Dv):
    check_forward(make(1, 3, 3, 150, Dk, Dv, seed=Dk + Dv), 2)


@pytest.mark.parametrize("Dk,Dv", [(1, 1), (3, 130 - 3), (17, 33), (40, 7), (64, 64), (100, 60), (128, 128)])
@pytest.mark.parametrize("T", [1, 70, 140])
def test_forward_fp32(Dk, Dv, T):
    check_forward(make(1, 2, 1, T, Dk, Dv, torch.float32, seed=Dk), 2, dtype=torch.float32)


@pytest.mark.parametrize("B,H,Hk", [(1, 1, 1), (2, 6, 2), (3, 8, 1), (1, 4, 4), (40, 4, 2), (150, 2, 1)])
def test_forward_head_layouts(B, H, Hk):
    check_forward(make(B, H, Hk, 100, 32, 64, seed=B + H), 2)


def test_forward_without_initial_state_and_correlated_keys():
    # keys close to one another: (I + A diag(beta)) is far from the identity
    check_forward(make(2, 2, 2, 200, 64, 64, init=False, correlated=2.0, seed=5), 2)
    check_forward(make(2, 2, 2, 200, 64, 64, torch.float32, init=False, correlated=2.0, seed=5), 2, dtype=torch.float32)


@pytest.mark.parametrize("value", [-50.0, -1e30, float("-inf")])
def test_forward_hard_resets(value):
    q, k, v, beta, lg, S0 = make(1, 2, 2, 150, 64, 64, seed=9)
    lg[:, :, [0, 70, 71, 128]] = value
    check_forward((q, k, v, beta, lg, S0), 2)


def test_padding_leaves_the_state_as_it_was():
    q, k, v, beta, lg, S0 = dev(*make(2, 4, 2, 200, 64, 64, seed=3))
    n = 137
    beta[:, :, n:] = 0
    lg[:, :, n:] = 0
    v[:, :, n:] = 1e30  # finite values behind the last token do not matter
    _, S = la().delta_forward(q, k, v, beta, 2, lg, S0)
    cut = [x[:, :, :n].contiguous() for x in (q, k, v, beta)]
    _, Sn = la().delta_forward(*cut, 2, lg[:, :, :n].contiguous(), S0)
    assert torch.equal(S, Sn)


def test_split_sequence_carries_on():
    args = dev(*make(2, 2, 2, 320, 64, 64, seed=4))
    q, k, v, beta, lg, S0 = args
    y, S = la().delta_forward(q, k, v, beta, 2, lg, S0)
    at = 192  # a chunk boundary: the same chunks, the same bits
    a = [x[:, :, :at].contiguous() for x in (q, k, v, beta, lg)]
    b = [x[:, :, at:].contiguous() for x in (q, k, v, beta, lg)]
    y1, S1 = la().delta_forward(*a[:4], 2, a[4], S0)
    y2, S2 = la().delta_forward(*b[:4], 2, b[4], S1)
    assert torch.equal(torch.cat([y1, y2], 2), y) and torch.equal(S2, S)


def test_empty_sequence_and_batch():
    q, k, v, beta, lg, S0 = dev(*make(2, 2, 2, 0, 64, 64))
    y, S = la().delta_forward(q, k, v, beta, 2, lg, S0)
    assert y.shape == (2, 2, 0, 64) and torch.equal(S, S0)
    y, S = la().delta_forward(q, k, v, beta, 2, lg)
    assert not S.any()
    y, S = la().delta_forward(*dev(*make(0, 2, 2, 9, 64, 64)[:4]))
    assert y.numel() == 0 and S.numel() == 0


def test_long_sequence_offsets_and_accuracy():
    # 32 heads of 20000 tokens (more than 2^31 bytes of workspace is reached by the products alone)
    q, k, v, beta, lg, S0 = make(1, 32, 32, 20000, 128, 128, seed=11)
    y, S = la().delta_forward(*dev(q, k, v, beta), 2, *dev(lg, S0))
    pick = [0, 31]
    ry, rS = oracle.delta_forward(*(x[:, pick] for x in (q, k, v, beta)), 2, lg[:, pick], S0[:, pick])
    assert slice_err(y[:, pick], ry) <= BAR16
    assert slice_err(S[:, pick], rS) <= BAR_STATE


def test_no_final_state_given_outputs_and_workspace():
    q, k, v, beta, lg, S0 = dev(*make(1, 2, 2, 90, 64, 64))
    y, S = la().delta_forward(q, k, v, beta, 2, lg, S0)
    y2, S2 = la().delta_forward(q, k, v, beta, 2, lg, S0, return_final=False)
    assert S2 is None and torch.equal(y, y2)
    out, fin = torch.empty_like(y), torch.empty_like(S)
    ws = torch.full((la().delta_workspace_size(1, 2, 90, 64, 64),), 255, dtype=torch.uint8, device="cuda")  # NaN patterns
    y3, S3 = la().delta_forward(q, k, v, beta, 2, lg, S0, out=out, final_state=fin, workspace=ws)
    assert y3 is out and S3 is fin and torch.equal(y3, y) and torch.equal(S3, S)


def test_forward_on_another_stream_and_in_a_graph():
    q, k, v, beta, lg, S0 = dev(*make(2, 2, 1, 130, 64, 64, seed=8))
    y, S = la().delta_forward(q, k, v, beta, 2, lg, S0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ys, Ss = la().delta_forward(q, k, v, beta, 2, lg, S0, stream=s)
    s.synchronize()
    assert torch.equal(ys, y) and torch.equal(Ss, S)
    out, fin = torch.empty_like(y), torch.empty_like(S)
    ws = torch.empty(la().delta_workspace_size(2, 2, 130, 64, 64, key_heads=1), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        la().delta_forward(q, k, v, beta, 2, lg, S0, out=out, final_state=fin, workspace=ws)
    for _ in range(2):
        v.neg_()
        ws.fill_(255)
        graph.replay()
        ye, Se = la().delta_forward(q, k, v, beta, 2, lg, S0)
        assert torch.equal(out, ye) and torch.equal(fin, Se)


# ------------------------------------------------------------------ gradients
# Bars: dq, dk, dv in bf16 carry their own rounding, 2^-8, next to fp32 sums of split
# operands.  An fp32 gradient of bf16 inputs goes through the forward's four split operands
# and the reverse scan's four: twice the states' bar.  d log g and dbeta are what is left of
# sums whose terms are larger than they are (k.dk of the rows that push a state and the rows
# that draw on it); they are held to the same bar against the 2-norm of those terms, which the
# oracle's own dq and dk give.  fp32 inputs: likewise, twice the forward's bar.
def check_backward(args, kind, scale=0.25, dtype=torch.bfloat16, d_final=True, seed=0):
    q, k, v, beta, lg, S0 = args
    g = torch.Generator().manual_seed(seed + 100)
    dy = torch.randn(v.shape, generator=g).to(dtype)
    B, H, Dk, Dv = v.shape[0], v.shape[1], q.shape[-1], v.shape[-1]
    dS = 0.3 * torch.randn(B, H, Dk, Dv, generator=g) if d_final else None
    got = la().delta_backward(*dev(q, k, v, beta, dy), kind, *dev(lg, S0, dS), q_scale=scale)
    want = oracle.delta_backward(q, k, v, beta, dy, kind, lg, S0, dS, scale)
    low = 2 * (BAR_STATE if dtype == torch.bfloat16 else BAR32)
    own = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    for name, x, r in zip(("dq", "dk", "dv"), got[:3], want[:3]):
        assert slice_err(x, r) <= own + low, name
    if S0 is not None:
        assert slice_err(got[5], want[5]) <= low, "d_init_state"
    rep = H // q.shape[1]
    f64 = lambda x: np.asarray(x.double().numpy()) if hasattr(x, "double") else np.asarray(x)  # noqa: E731
    qd = np.repeat((f64(q) * want[0]).sum(-1), rep, 1)
    kd = np.repeat(np.linalg.norm(f64(k), axis=-1) * np.linalg.norm(want[1], axis=-1), rep, 1)
    terms = np.abs(qd) + kd + np.linalg.norm(f64(v), axis=-1) * np.linalg.norm(want[2], axis=-1)
    size = np.sqrt((terms ** 2).sum(-1)) + 1e-30
    db = got[3].cpu().double().numpy()
    assert (np.linalg.norm(db - want[3], axis=-1) <= low * (size + np.linalg.norm(want[3], axis=-1))).all(), "dbeta"
    if kind == 2:
        dl = got[4].cpu().double().numpy()
        ends = np.linalg.norm(want[4], axis=-1)
        assert (np.linalg.norm(dl - want[4], axis=-1) <= low * (size + ends)).all(), "d_log_g"
    elif kind == 1:
        dl = got[4].cpu().double().numpy()
        assert (np.abs(dl - want[4]) <= low * (terms.sum((0, 2)) + np.abs(want[4]))).all(), "d_log_g per head"
    else:
        assert got[4] is None
    return dy, dS, got


@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 130, 257])
@pytest.mark.parametrize("kind", [0, 1, 2])
def test_backward_lengths(T, kind):
    check_backward(make(2, 2, 2, T, 64, 64, kind=kind, seed=T), kind)


@pytest.mark.parametrize("Dk,Dv", [(16, 16), (32, 48), (48, 32), (64, 112), (80, 64), (96, 80), (112, 16), (128, 128)])
def test_backward_widths(Dk, Dv):
    check_backward(make(1, 3, 3, 150, Dk, Dv, seed=Dk + Dv), 2)


@pytest.mark.parametrize("Dk,Dv", [(1, 1), (3, 127), (17, 33), (40, 7), (64, 64), (100, 60), (128, 128)])
@pytest.mark.parametrize("T", [1, 70, 140])
def test_backward_fp32(Dk, Dv, T):
    check_backward(make(1, 2, 1, T, Dk, Dv, torch.float32, seed=Dk), 2, dtype=torch.float32)


@pytest.mark.parametrize("B,H,Hk", [(1, 1, 1), (2, 6, 2), (3, 8, 1), (1, 4, 4), (40, 4, 2), (150, 2, 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_backward_head_layouts(B, H, Hk, dtype):
    check_backward(make(B, H, Hk, 100, 32, 64, dtype, seed=B + H), 2, dtype=dtype)


def test_backward_without_states_and_with_correlated_keys():
    check_backward(make(2, 2, 2, 200, 64, 64, init=False, correlated=2.0, seed=5), 2, d_final=False)
    check_backward(make(2, 2, 2, 200, 64, 64, kind=1, init=False, seed=6), 1, d_final=False)


@pytest.mark.parametrize("B,H,T,Dk,Dv", [(2, 2, 1057, 16, 32), (1, 2, 334, 128, 128), (3, 6, 200, 64, 48), (40, 8, 65, 32, 64)])
def test_a_heads_decay_keeps_its_digits(B, H, T, Dk, Dv):
    # a per-head decay's gradient is what is left of terms of both signs: with three planes an operand
    # they are fp32 sums', 192 2^-24 of their absolute sum (twice: the scan and its reverse) and no more
    args = make(B, H, H, T, Dk, Dv, kind=1, init=False, seed=T)
    q, k, v, beta, lg, _ = args
    dy = torch.randn(v.shape, generator=torch.Generator().manual_seed(5)).bfloat16()
    got = la().delta_backward(*dev(q, k, v, beta, dy), 1, *dev(lg), q_scale=Dk ** -0.5)[4].cpu().double().numpy()
    want = oracle.delta_backward(q, k, v, beta, dy, 1, lg, None, None, Dk ** -0.5)[4]
    per_step = lg[None, :, None].expand(B, H, T)
    terms = np.abs(oracle.delta_backward(q, k, v, beta, dy, 2, per_step, None, None, Dk ** -0.5)[4]).sum((0, 2))
    assert (np.abs(got - want) <= 2 * BAR32 * terms).all()
    assert np.linalg.norm(got - want) <= 1e-5 * np.linalg.norm(terms)


def test_backward_of_zero_beta_and_hard_resets():
    # beta = 0 writes nothing, but its gradient is the error it would have written
    q, k, v, beta, lg, S0 = make(1, 2, 2, 150, 64, 64, seed=9)
    beta[:, :, ::3] = 0
    lg[:, :, [0, 70, 71, 128]] = -1e30
    check_backward((q, k, v, beta, lg, S0), 2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_first_decay_of_nothing_has_no_gradient(dtype):
    # without an initial state the first token's decay multiplies zero: its gradient is 0, not a rounding
    for T in (1, 66):
        q, k, v, beta, lg, _ = make(2, 3, 3, T, 32, 48, dtype, init=False, seed=4)
        dy = torch.randn(v.shape, generator=torch.Generator().manual_seed(6)).to(dtype)
        d = la().delta_backward(*dev(q, k, v, beta, dy), 2, *dev(lg))[4]
        assert (d[:, :, 0] == 0).all() and (T == 1 or (d[:, :, 1:] != 0).all())
        d = la().delta_backward(*dev(q, k, v, beta, dy), 1, *dev(lg[0, :, 0]))[4]
        assert (d == 0).all() == (T == 1)


def test_backward_against_differences():
    # fp32, along a random direction of every input, by central differences of the library's forward
    q, k, v, beta, lg, S0 = make(1, 2, 1, 75, 24, 20, torch.float32, seed=21)
    dy, dS, got = check_backward((q, k, v, beta, lg, S0), 2, dtype=torch.float32, seed=3)
    g = torch.Generator().manual_seed(77)
    leaves = [q, k, v, beta, lg, S0]

    def loss(xs):
        y, S = oracle.delta_forward(*xs[:4], 2, xs[4], xs[5], 0.25)
        return float((y * dy.double().numpy()).sum() + (S * dS.double().numpy()).sum())
    for i, x in enumerate(leaves):
        d = torch.randn(x.shape, generator=g, dtype=torch.float64)
        h = 1e-5
        up = [t.double() + h * d if j == i else t.double() for j, t in enumerate(leaves)]
        dn = [t.double() - h * d if j == i else t.double() for j, t in enumerate(leaves)]
        slope = (loss(up) - loss(dn)) / (2 * h)
        mine = float((got[i].cpu().double() * d).sum())
        size = float(got[i].cpu().double().norm() * d.norm())
        # differences are off by h^2 and the forward's 64-bit noise / h; fp32 gradients by 2 BAR32
        assert abs(mine - slope) <= 2 * BAR32 * size + 1e-7 * size + 1e-8, i


def test_backward_padding_shared_outputs_and_determinism():
    q, k, v, beta, lg, S0 = dev(*make(2, 4, 2, 200, 64, 64, seed=3))
    n = 137
    beta[:, :, n:] = 0
    lg[:, :, n:] = 0
    dy = torch.randn(v.shape, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    dy[:, :, n:] = 0
    got = la().delta_backward(q, k, v, beta, dy, 2, lg, S0)
    cut = [x[:, :, :n].contiguous() for x in (q, k, v, beta, dy)]
    want = la().delta_backward(*cut, 2, lg[:, :, :n].contiguous(), S0)
    for a, b in zip(got[:3], want[:3]):
        assert torch.equal(a[:, :, :n], b)
    assert torch.equal(got[3][:, :, :n], want[3]) and torch.equal(got[5], want[5])
    assert not got[0][:, :, n:].any() and not got[2][:, :, n:].any()
    ws = torch.full((la().delta_backward_workspace_size(2, 4, 200, 64, 64, key_heads=2),), 255, dtype=torch.uint8, device="cuda")
    outs = tuple(torch.full_like(x, float("nan")) for x in got)
    again = la().delta_backward(q, k, v, beta, dy, 2, lg, S0, workspace=ws, out=outs)
    for a, b, o in zip(again, got, outs):
        assert a is o and torch.equal(a, b)
    some = la().delta_backward(q, k, v, beta, dy, 2, lg, S0, need_log_g=False, need_init_state=False)
    assert some[4] is None and some[5] is None and torch.equal(some[1], got[1])


def test_backward_empty():
    q, k, v, beta, lg, S0 = dev(*make(2, 2, 2, 0, 64, 64))
    got = la().delta_backward(q, k, v, beta, v, 2, lg, S0, S0)
    assert torch.equal(got[5], S0) and got[4].shape == (2, 2, 0)
    got = la().delta_backward(q, k, v, beta, v, 1, torch.zeros(2, device="cuda"), S0)
    assert not got[5].any() and not got[4].any()
    e = dev(*make(0, 2, 2, 9, 64, 64, kind=1))
    assert not la().delta_backward(e[0], e[1], e[2], e[3], e[2], 1, e[4])[4].any()


def test_backward_in_a_graph():
    q, k, v, beta, lg, S0 = dev(*make(2, 4, 2, 130, 64, 64, seed=8))
    dy = torch.randn(v.shape, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    outs = tuple(torch.empty_like(x) for x in (q, k, v, beta, lg, S0))
    ws = torch.empty(la().delta_backward_workspace_size(2, 4, 130, 64, 64, key_heads=2), dtype=torch.uint8, device="cuda")
    la().delta_backward(q, k, v, beta, dy, 2, lg, S0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        la().delta_backward(q, k, v, beta, dy, 2, lg, S0, S0, workspace=ws, out=outs)
    for _ in range(2):
        dy.neg_()
        ws.fill_(255)
        graph.replay()
        for a, b in zip(outs, la().delta_backward(q, k, v, beta, dy, 2, lg, S0, S0)):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ one token
@pytest.mark.parametrize("B,H,Hk", [(1, 1, 1), (3, 6, 2), (200, 4, 4)])
@pytest.mark.parametrize("Dk,Dv,dtype", [(16, 16, torch.bfloat16), (64, 80, torch.bfloat16), (128, 128, torch.bfloat16),
                                         (40, 36, torch.bfloat16), (7, 5, torch.float32), (128, 127, torch.float32),
                                         (100, 60, torch.float32), (1, 1, torch.bfloat16), (33, 128, torch.float32)])
@pytest.mark.parametrize("kind", [0, 1, 2])
def test_decode(B, H, Hk, Dk, Dv, dtype, kind):
    q, k, v, beta, lg, S0 = make(B, H, Hk, 1, Dk, Dv, dtype, kind=kind, seed=Dk + Dv)
    q, k, v, beta = (x[:, :, 0].contiguous() for x in (q, k, v, beta))
    lg = lg[:, :, 0].contiguous() if kind == 2 else lg
    state = S0.cuda()
    y = la().delta_decode_step(*dev(q, k, v, beta), state, kind, *dev(lg), q_scale=0.5)
    ry, rS = oracle.delta_decode_step(q, k, v, beta, S0, kind, lg, 0.5)
    # S' = g S - k (beta S^T k)^T + k (beta v)^T is a difference: with |k| <= 1 + 2^-8 and
    # beta, g <= 1 its terms are at most ||S|| and ||v||, and each of the fp32 roundings (a sum of
    # Dk terms, the difference, the update) is relative to those, not to what they leave.  y is
    # q^T of such a state: once more the same, times the scale, and its own rounding.
    terms = np.linalg.norm(S0.double().numpy(), axis=(2, 3)) + 2 * np.linalg.norm(v.double().numpy(), axis=2)
    bar = (Dk + 4) * 2.0 ** -24 * terms
    assert (np.linalg.norm(state.cpu().double().numpy() - rS, axis=(2, 3)) <= bar).all()
    off = np.linalg.norm(y.cpu().double().numpy() - ry, axis=2)
    assert (off <= bar + (2.0 ** -8 * np.linalg.norm(ry, axis=2) if dtype == torch.bfloat16 else 0)).all()


def test_decode_steps_equal_the_forward():
    q, k, v, beta, lg, S0 = dev(*make(2, 4, 2, 70, 64, 64, seed=2))
    y, S = la().delta_forward(q, k, v, beta, 2, lg, S0, q_scale=0.3)
    state = S0.clone()
    rows = [la().delta_decode_step(*(x[:, :, t].contiguous() for x in (q, k, v, beta)), state, 2,
                                   lg[:, :, t].contiguous(), q_scale=0.3) for t in range(70)]
    assert slice_err(state, S.cpu().double()) <= BAR_STATE
    assert slice_err(torch.stack(rows, 2), y.cpu().double()) <= 2 * BAR16


def test_decode_in_a_graph_moves_the_state_on_each_replay():
    q, k, v, beta, lg, S0 = dev(*make(2, 4, 2, 1, 64, 64, seed=6))
    q, k, v, beta, lg = (x[:, :, 0].contiguous() for x in (q, k, v, beta, lg))
    state, out = S0.clone(), torch.empty_like(v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        la().delta_decode_step(q, k, v, beta, state, 2, lg, out=out)
    want = S0.clone()
    for _ in range(3):
        graph.replay()
        y = la().delta_decode_step(q, k, v, beta, want, 2, lg)
        assert torch.equal(state, want) and torch.equal(out, y)


# ------------------------------------------------------------------ around the calls
def banded(shape, dtype, fill=0x5A):
    """A contiguous tensor inside a larger buffer of one byte pattern, and a check that the rest still has it."""
    n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
    pad = 4096
    raw = torch.full((n + 2 * pad,), fill, dtype=torch.uint8, device="cuda")
    t = raw[pad:pad + n].view(dtype).view(shape)

    def intact():
        return bool((raw[:pad] == fill).all() and (raw[pad + n:] == fill).all())
    return t, intact


@pytest.mark.parametrize("T,Dk,Dv,dtype", [(1, 16, 16, torch.bfloat16), (67, 48, 80, torch.bfloat16), (130, 128, 112, torch.bfloat16),
                                           (67, 33, 21, torch.float32), (65, 128, 127, torch.float32)])
def test_nothing_is_written_outside(T, Dk, Dv, dtype):
    B, H, Hk = 2, 4, 2
    q, k, v, beta, lg, S0 = dev(*make(B, H, Hk, T, Dk, Dv, dtype, seed=T))
    y, c1 = banded((B, H, T, Dv), dtype)
    S, c2 = banded((B, H, Dk, Dv), torch.float32)
    ws, c3 = banded((la().delta_workspace_size(B, H, T, Dk, Dv, dtype, key_heads=Hk),), torch.uint8)
    la().delta_forward(q, k, v, beta, 2, lg, S0, out=y, final_state=S, workspace=ws)
    outs, checks = zip(*(banded(t.shape, t.dtype) for t in (q, k, v, beta, lg, S0)))
    wb, c4 = banded((la().delta_backward_workspace_size(B, H, T, Dk, Dv, dtype, key_heads=Hk),), torch.uint8)
    la().delta_backward(q, k, v, beta, v, 2, lg, S0, S0, workspace=wb, out=outs)
    state, c5 = banded(S0.shape, torch.float32)
    state.copy_(S0)
    o, c6 = banded((B, H, Dv), dtype)
    la().delta_decode_step(*(x[:, :, 0].contiguous() for x in (q, k, v, beta)), state, 2, lg[:, :, 0].contiguous(), out=o)
    torch.cuda.synchronize()
    assert all(c() for c in (c1, c2, c3, c4, c5, c6, *checks))


def test_two_streams_at_once():
    a, b = (dev(*make(2, 8, 4, 300, 64, 64, seed=s)) for s in (1, 2))
    want = [la().delta_backward(*x[:4], x[2], 2, *x[4:]) for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, (s, x) in enumerate(zip(streams, (a, b))):
            got[i].append(la().delta_backward(*x[:4], x[2], 2, *x[4:], stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(p, q) for p, q in zip(r, want[i]))


def test_refusals_on_the_gpu():
    q, k, v, beta, lg, S0 = dev(*make(1, 4, 2, 5, 16, 16))
    f, m = la().delta_forward, la()
    for bad, error in [
        (lambda: f(q, k[:, :, :4], v, beta), ValueError), (lambda: f(q, k, v[:, :3], beta), ValueError),
        (lambda: f(q, k, v.float(), beta), TypeError), (lambda: f(q, k, v, beta.double()), TypeError),
        (lambda: f(q, k, v, beta.cpu()), ValueError), (lambda: f(q.transpose(2, 3), k, v, beta), ValueError),
        (lambda: f(q.half(), k.half(), v.half(), beta), TypeError), (lambda: f(q, k, v, beta, 2), ValueError),
        (lambda: f(q, k, v, beta, 7, lg), ValueError), (lambda: f(q, k, v, beta, 1, lg), ValueError),
        (lambda: f(q, k, v, beta, init_state=S0[:, :2]), ValueError), (lambda: f(q, k, v, None), ValueError),
        (lambda: f(q, k, v, beta, out=torch.empty_like(v).float()), TypeError),
        (lambda: f(q, k, v, beta, q_scale=float("nan")), m.LAError),
        (lambda: f(q, k, v, beta, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), m.LAError),
        (lambda: f(q, k, v, beta, workspace=torch.empty(1 << 20, device="cuda")), ValueError),
        (lambda: m.delta_backward(q, k, v, beta, None), ValueError),
        (lambda: m.delta_backward(q, k, v, beta, v[:, :, :3]), ValueError),
        (lambda: m.delta_backward(q, k, v, beta, v, out=(None,) * 6), ValueError),
        (lambda: m.delta_decode_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], beta[:, :, 0], S0), ValueError),
        (lambda: m.delta_decode_step(*(x[:, :, 0].contiguous() for x in (q, k, v, beta)), None), ValueError),
    ]:
        with pytest.raises(error):
            bad()


def test_systems_far_from_the_identity():
    # I + A diag(beta) for one key repeated: row sums up to 64 beta.  A solution's error is bounded by the
    # condition number times the operands' rounding: ||I + N|| <= 1 + 63 beta, and the inverse's columns are
    # beta (1 - beta)^n: ||inverse|| <= 1 + beta (beta = 1), 1 + 1.9 / (1 - 0.9) = 20 (beta = 1.9, sign of the
    # key alternating or not).  Four split operands in a row, as in BAR_STATE.
    for beta_value, sign, inverse in ((1.0, 1, 2.0), (1.9, 1, 20.0), (1.9, -1, 20.0)):
        for dtype, unit in ((torch.bfloat16, BAR_STATE), (torch.float32, BAR32)):
            q, k, v, beta, lg, S0 = make(1, 2, 2, 300, 64, 64, dtype, kind=0, seed=12)
            k = k[:, :, :1].expand_as(k).contiguous()
            k[:, :, ::2] *= sign
            beta[:] = beta_value
            y, S = la().delta_forward(*dev(q, k, v, beta), 0, None, *dev(S0))
            ry, rS = oracle.delta_forward(q, k, v, beta, 0, None, S0)
            assert slice_err(S, rS) <= (1 + 63 * beta_value) * inverse * unit
            assert slice_err(y, ry) <= (1 + 63 * beta_value) * inverse * unit + (BAR16 if dtype == torch.bfloat16 else 0)


def test_the_first_call_of_a_process_inside_a_capture():
    import subprocess
    import sys
    code = r'''
import torch, retention_scan_b200 as la
q = torch.nn.functional.normalize(torch.randn(1, 2, 100, 64, device="cuda"), dim=-1).bfloat16()
beta, out, fin = torch.rand(1, 2, 100, device="cuda"), torch.empty_like(q), torch.empty(1, 2, 64, 64, device="cuda")
ws = torch.empty(la.delta_workspace_size(1, 2, 100, 64, 64), dtype=torch.uint8, device="cuda")
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    la.delta_forward(q, q, q, beta, out=out, final_state=fin, workspace=ws)
g.replay()
y, S = la.delta_forward(q, q, q, beta)
torch.cuda.synchronize()
assert torch.equal(out, y) and torch.equal(fin, S) and la.device_error() == 0
print("same")
'''
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=root, timeout=120)
    assert r.stdout.strip().endswith("same"), r.stderr[-2000:]


# ------------------------------------------------------------------ keys and queries close to one another
@pytest.mark.parametrize("B,H", [(1, 2), (5, 4), (10, 4)])  # four and two warps a slice, one
@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 64), (32, 48)])
@pytest.mark.parametrize("noise,beta_value", [(0.5, 0.99), (0.1, 1.0), (0.5, 0.5)])
def test_outputs_of_scores_that_cancel(B, H, Dk, Dv, noise, beta_value):
    # Keys and queries around one direction: the chunk's scores are all about 1 and the errors they meet are
    # differences, so that P U is what is left of terms several times as large.  y has its own rounding, half a
    # step (2^-8 of each value), and the split operands' 2^-14 of those terms, at most 16 times y here (64 tokens,
    # whose errors fall off with beta): 2^-8 + 2^-10.  P rounded to bf16 (2^-9 of a term) would not hold it.
    g = torch.Generator().manual_seed(B + Dk)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    T = 150
    c = unit(rn(B, H, 1, Dk)) * Dk ** 0.5
    k, q = (unit(c + noise * rn(B, H, T, Dk)).bfloat16() for _ in range(2))
    v = rn(B, H, T, Dv).bfloat16()
    beta, lg = torch.full((B, H, T), beta_value), torch.full((B, H, T), -0.01)
    y, S = la().delta_forward(*dev(q, k, v, beta), 2, *dev(lg))
    ry, rS = oracle.delta_forward(q, k, v, beta, 2, lg)
    assert slice_err(y, ry) <= 2.0 ** -8 + 2.0 ** -10
    assert slice_err(S, rS) <= BAR_STATE


@pytest.mark.parametrize("dtype,unit", [(torch.float32, BAR32), (torch.bfloat16, BAR_STATE)])
@pytest.mark.parametrize("Dk,Dv", [(128, 32), (64, 16), (32, 16)])  # four and two warps a slice
def test_long_gradients_of_states_do_not_drift(Dk, Dv, dtype, unit):
    # No decay and small beta: the state's gradient is carried over 64 chunks.  Each chunk adds to it with two
    # rounded operations, at most half a step of 2^-23 each, and 128 half steps in all; products and operands
    # within a chunk as in BAR32 and BAR_STATE, for what that chunk adds.  All values positive, so that nothing cancels and a
    # one-sided error shows.  Its mean has a tenth of that bound from the roundings, which go either way, and from
    # the tensor core's truncations at most 24 additions (4 blocks, 6 pairs of planes) of 2^-24 each in a chunk's
    # own products; into the carried gradient they would make 64 times as many.
    q, k, v, beta, _, S0 = make(1, 2, 2, 4096, Dk, Dv, dtype, kind=0, seed=13)
    g = torch.Generator().manual_seed(14)
    beta, q, dy = 0.02 * beta, q.abs(), torch.randn(v.shape, generator=g).abs().to(dtype)
    dS = 10 * torch.randn(1, 2, Dk, Dv, generator=g).abs()
    got = la().delta_backward(*dev(q, k, v, beta, dy), 0, None, *dev(S0, dS))
    want = oracle.delta_backward(q, k, v, beta, dy, 0, None, S0, dS)
    bar = 128 * 2.0 ** -24
    assert slice_err(got[5], want[5]) <= bar + unit / 8
    bias = (got[5].cpu().double().numpy() - want[5]).mean() / np.abs(want[5]).mean()
    assert abs(bias) <= bar / 10 + 24 * 2.0 ** -24
    for x, r in zip(got[:3], want[:3]):
        assert slice_err(x, r) <= bar + unit + (2.0 ** -8 if dtype == torch.bfloat16 else 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_key_heads_that_serve_no_value_head(dtype):
    q, k, v, beta, lg, S0 = dev(*make(2, 4, 2, 70, 32, 16, dtype))
    none = [t[:, :0].contiguous() for t in (v, beta, lg, S0)]
    y, S = la().delta_forward(q, k, none[0], none[1], 2, none[2], none[3])
    assert y.shape == (2, 0, 70, 16) and S.shape == (2, 0, 32, 16)
    outs = (torch.full_like(q, 7.0), torch.full_like(k, 7.0), *(torch.empty_like(t) for t in none))
    got = la().delta_backward(q, k, none[0], none[1], none[0], 2, none[2], none[3], out=outs)
    assert got[0] is outs[0] and not got[0].any() and not got[1].any()
