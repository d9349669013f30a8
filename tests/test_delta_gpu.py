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
