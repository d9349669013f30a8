"""GPU parity of the gated norm, its gradients and rotary positions against
float64, and of a whole block's chain: rotary, L2 norm, the gated delta rule,
gated norm, and back.

Bars are elementwise and count roundings.  A bf16 result: 2^-8 of itself (half
a step).  What precedes that rounding is fp32: sums of D terms, (D + 16) 2^-24
of their terms; an exponential of z by the fast instruction, off by at most
2 + 1.173 |z| steps of 2^-23 by CUDA's table, used once in the gate.  Terms are
measured where they are largest: a difference (x - mean) by its operands."""
import itertools

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
KINDS, ACTS = ("rms", "layer", "l2"), ("none", "silu", "sigmoid")


@pytest.fixture(scope="module", autouse=True)
def built():
    from retention_scan_b200 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def la():
    import retention_scan_b200
    return retention_scan_b200


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def how(kind, act, **more):
    m = la()
    return dict(kind=KINDS.index(kind), activation=m.GATE_SIGMOID if act == "sigmoid" else m.GATE_SILU, **more)


def near(x, ref, terms, steps, dtype, name=""):
    """|x - ref| <= its own rounding + steps * 2^-24 of the terms."""
    x = f64(x)
    assert x.shape == ref.shape and np.isfinite(x).all(), name
    own = 2.0 ** -8 if dtype == torch.bfloat16 else U
    bad = np.abs(x - ref) - own * np.abs(ref) - steps * U * terms
    assert (bad <= 1e-37).all(), (name, float(bad.max()))


def norm_terms(x, gate, weight, kind, act, eps, scale):
    """What the normalised part's factors multiply up to, with x for x - mean, and the steps of its roundings."""
    D = x.shape[-1]
    c = x - x.mean(-1, keepdims=True) if kind == "layer" else x
    ss = (c * c).sum(-1, keepdims=True)
    r = 1 / np.sqrt((ss if kind == "l2" else ss / D) + eps)
    big = (np.abs(c) + (np.abs(x).mean(-1, keepdims=True) if kind == "layer" else 0)) * r
    w = np.abs(weight) if weight is not None else 1.0
    steps = D + 16.0
    a = 1.0
    if gate is not None:
        a = np.abs(oracle.block._activation(gate, act)[0])
        steps = steps + 2 * (2 + 1.173 * np.abs(gate)) + 8
    return abs(scale) * big * w * a, steps, r, big


def tensors(shape, dtype, seed, act, weight, residual, offset=0.0, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = (offset + spread * rn(*shape)).to(dtype).cuda()
    gate = (3 * rn(*shape)).to(dtype).cuda() if act != "none" else None
    w = (1 + 0.3 * rn(shape[-1])).cuda() if weight else None
    res = rn(*shape).to(dtype).cuda() if residual else None
    return x, gate, w, res, rn(*shape).to(dtype).cuda()


def check_norm(x, gate, w, res, kind, act, eps=1e-5, scale=1.0, out=None):
    y = la().gated_norm(x, gate, w, res, out=out, **how(kind, act, eps=eps, scale=scale))
    args = [f64(t) for t in (x, gate, w, res)]
    ref = oracle.gated_norm(*args, kind, act, eps, scale)
    terms, steps, _, _ = norm_terms(args[0], args[1], args[2], kind, act, eps, scale)
    if res is not None:
        terms = terms + np.abs(args[3]) * 2 / np.min(steps)
    near(y, ref, terms, steps, x.dtype, (kind, act, tuple(x.shape)))
    return y


def check_norm_backward(dout, x, gate, w, kind, act, eps=1e-5, scale=1.0):
    got = la().gated_norm_backward(dout, x, gate, w, **how(kind, act, eps=eps, scale=scale))
    d, xx, z, ww = (f64(t) for t in (dout, x, gate, w))
    ref = oracle.gated_norm_backward(d, xx, z, ww, kind, act, eps, scale)
    terms, steps, r, big = norm_terms(xx, z, ww, kind, act, eps, scale)
    D = xx.shape[-1]
    wa = 1.0 if ww is None else np.abs(ww)
    a, da = (np.ones(1), None) if z is None else oracle.block._activation(z, act)
    dn = np.abs(scale * d) * wa * np.abs(a)
    K = 1 if kind == "l2" else D
    inner = (dn * big).sum(-1, keepdims=True) / K
    t = r * (dn + big * inner + (dn.mean(-1, keepdims=True) if kind == "layer" else 0))
    worst = np.max(steps, axis=-1, keepdims=True) if np.ndim(steps) else steps
    near(got[0], ref[0], t, 3 * worst, x.dtype, "dx")
    if z is not None:
        # a' = s (1 + z (1 - s)): its terms, not what they leave
        s = oracle.block._activation(z, "sigmoid")[0]
        near(got[1], ref[1], np.abs(scale * d) * big * wa * (s * (1 + np.abs(z)) if act == "silu" else s), 2 * steps + 8,
             x.dtype, "dgate")
    if w is not None:
        rows = d.reshape(-1, D).shape[0]
        col = (np.abs(scale * d) * np.abs(a) * big * np.ones_like(xx)).reshape(-1, D).sum(0)
        near(got[2], ref[2], col, rows + np.max(steps), torch.float32, "dweight")
    else:
        assert got[2] is None
    assert (got[1] is None) == (gate is None)
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind,act", list(itertools.product(KINDS, ACTS)))
@pytest.mark.parametrize("shape", [(1, 1), (5, 7), (3, 2, 16), (2, 5, 3, 64), (2, 3, 9, 128)])
def test_norm_kinds(shape, kind, act, dtype):
    i = len(shape)
    x, gate, w, res, d = tensors(shape, dtype, i, act, i % 2 == 0, i % 3 == 0)
    check_norm(x, gate, w, res, kind, act, scale=0.7)
    check_norm_backward(d, x, gate, w, kind, act, scale=0.7)


# every team size and vector width, on both sides of their limits
@pytest.mark.parametrize("D", [2, 4, 5, 8, 9, 16, 31, 32, 33, 64, 65, 96, 100, 127, 129, 130, 255, 256, 257, 258, 260, 512, 520,
                               1000, 1023, 1024, 1026, 1032, 2048, 2049, 2050, 4096, 4100, 6000, 8191, 8192])
def test_norm_widths(D):
    for dtype in (torch.bfloat16, torch.float32):
        x, gate, w, res, d = tensors((3, 7, D), dtype, D, "silu", True, True)
        check_norm(x, gate, w, res, "layer", "silu")
        if D <= 2050:
            check_norm_backward(d, x, gate, w, "layer", "silu")
    if D > 2050:  # the oracle writes the whole Jacobian: one row
        x, gate, w, res, d = tensors((1, D), torch.bfloat16, D, "silu", True, True)
        check_norm_backward(d, x, gate, w, "rms", "silu")


@pytest.mark.parametrize("rows", [1, 2, 63, 64, 1183, 1185, 9473, 40000])
def test_norm_rows(rows):
    x, gate, w, res, d = tensors((rows, 32), torch.bfloat16, rows, "silu", True, False)
    check_norm(x, gate, w, res, "rms", "silu")
    check_norm_backward(d, x, gate, w, "rms", "silu")


def test_norm_heads_layout_and_other_views():
    x, gate, w, res, d = tensors((2, 4, 10, 64), torch.bfloat16, 1, "silu", True, True)  # [B,H,T,D]
    xt = x.transpose(1, 2)  # as [B,T,H,D]
    y = check_norm(xt, gate.transpose(1, 2).contiguous(), w, res.transpose(1, 2), "rms", "silu")
    assert y.is_contiguous() and y.shape == (2, 10, 4, 64)
    got = check_norm_backward(d.transpose(1, 2), xt, gate.transpose(1, 2), w, "rms", "silu")
    assert got[0].stride() == xt.stride()
    # a slice of a fused projection, an odd offset (2-byte alignment), a broadcast gate
    wide = torch.randn(3, 5, 3 * 64 + 1, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    check_norm(wide[..., 64:128], wide[..., 128:192], w, None, "layer", "sigmoid")
    check_norm(wide[..., 1:65], wide[..., 65:129], w, None, "layer", "sigmoid")
    one = wide[:1, :1, :64].expand(3, 5, 64)
    check_norm(wide[..., 64:128], one, w, wide[..., :64], "rms", "silu")
    got = la().gated_norm_backward(wide[..., :64], wide[..., 64:128], one, w)
    assert got[1].shape == (3, 5, 64) and got[1].stride(0) != 0


def test_norm_in_place_and_given_outputs():
    x, gate, w, res, d = tensors((6, 300), torch.bfloat16, 3, "silu", True, True)
    y = la().gated_norm(x, gate, w, res)
    for target in range(3):
        a = [x.clone(), gate.clone(), res.clone()]
        assert torch.equal(la().gated_norm(a[0], a[1], w, a[2], out=a[target]), y) and torch.equal(a[target], y)
    got = la().gated_norm_backward(d, x, gate, w)
    outs = tuple(torch.full_like(t, float("nan")) for t in got)
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
    again = la().gated_norm_backward(d, x, gate, w, out=outs, workspace=ws)
    for a, b, o in zip(again, got, outs):
        assert a is o and torch.equal(a, b)
    assert la().gated_norm_backward(d, x, gate, w, need_weight=False)[2] is None


def test_norm_extreme_values():
    # gates far out, a mean far above the spread, rows of zeros, infinities and NaN that stay in their rows
    g = torch.tensor([-1e4, -100.0, -88.0, -20.0, 0.0, 20.0, 100.0, 1e4]).repeat(4, 1).cuda()
    x = torch.randn(4, 8, generator=torch.Generator().manual_seed(1)).cuda()
    for act in ("silu", "sigmoid"):
        y = la().gated_norm(x, g, **how("rms", act))
        ref = oracle.gated_norm(x, g, None, None, "rms", act)
        assert np.isfinite(f64(y)).all() and np.abs(f64(y) - ref).max() <= 1e-5 * np.abs(ref).max()
        dx, dg, _ = la().gated_norm_backward(x, x, g, **how("rms", act))
        assert torch.isfinite(dx).all() and torch.isfinite(dg).all()
    x, _, w, _, d = tensors((8, 128), torch.float32, 4, "none", True, False, offset=1000.0)
    check_norm(x, None, w, None, "layer", "none")
    check_norm_backward(d, x, None, w, "layer", "none")
    z = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    for kind in KINDS:
        assert not la().gated_norm(z, **how(kind, "none")).any()
    assert torch.isnan(la().gated_norm(z, eps=0.0)).all()
    y0 = la().gated_norm(x)
    x[3, 5], x[6, 7] = float("inf"), float("nan")
    y = la().gated_norm(x)
    rows = [0, 1, 2, 4, 5, 7]
    assert torch.equal(y[rows], y0[rows]) and torch.isnan(y[6]).all() and torch.isnan(y[3, 5])


@pytest.mark.parametrize("rows,D", [(1, 128), (5, 128), (3, 64), (9, 100), (2, 2048), (300, 36)])
def test_teams_without_a_row_add_nothing(rows, D):
    # eps = 0: what a team behind the last row computes must not reach dweight
    x, gate, w, _, d = tensors((rows, D), torch.bfloat16, rows, "silu", True, False)
    check_norm_backward(d, x, gate, w, "rms", "silu", eps=0.0)
    check_norm_backward(d, x, None, w, "l2", "none", eps=0.0)


def test_norm_empty():
    x = torch.empty(0, 5, 64, device="cuda")
    assert la().gated_norm(x).shape == (0, 5, 64)
    w = torch.ones(64, device="cuda")
    dx, _, dw = la().gated_norm_backward(x, x, None, w)
    assert dx.numel() == 0 and not dw.any()


@pytest.mark.parametrize("kind,act", [("rms", "silu"), ("layer", "sigmoid"), ("l2", "none")])
def test_norm_gradients_against_differences(kind, act):
    x, gate, w, _, d = tensors((4, 24), torch.float32, 6, act, True, False)
    got = la().gated_norm_backward(d, x, gate, w, **how(kind, act, scale=0.6))
    leaves = [f64(t) for t in (x, gate, w)]
    g = np.random.RandomState(0)

    def loss(xs):
        return float((oracle.gated_norm(xs[0], xs[1], xs[2], None, kind, act, 1e-5, 0.6) * f64(d)).sum())
    for i, t in enumerate(leaves):
        if t is None:
            continue
        v = g.randn(*t.shape)
        up, dn = ([u + s * v if j == i else u for j, u in enumerate(leaves)] for s in (1e-6, -1e-6))
        slope = (loss(up) - loss(dn)) / 2e-6
        # fp32 roundings (the bars above allow 3 (D + 16) of them) and the differences' own h^2 and 64-bit noise / h
        size = np.linalg.norm(f64(got[i])) * np.linalg.norm(v)
        assert abs((f64(got[i]) * v).sum() - slope) <= (3 * 40 * U + 1e-8) * size + 1e-8


# ------------------------------------------------------------------ rotary
def check_rotary(x, x2, freq, pos, layout, mscale=1.0, start=0, backward=False, **more):
    got = la().rotary(x, freq, pos, x2, start=start, layout=0 if layout == "half" else 1, mscale=mscale, backward=backward,
                      **more)
    got = got if x2 is not None else (got,)
    where = f64(pos) if pos is not None else start + np.arange(x.shape[2])
    for t, y in zip((x, x2), got):
        if t is None:
            continue
        ref = oracle.rotary(t, freq, where, layout, mscale, backward)
        # pairs: the angle (rounded to fp32 below 2 pi: 2^-22), sine and cosine (2 steps), two products
        R = 2 * freq.shape[0]
        terms = np.zeros_like(ref)
        terms[..., :R] = abs(mscale) * np.abs(f64(t)[..., :R]).max(-1, keepdims=True)
        near(y, ref, terms, 24, t.dtype, (layout, tuple(t.shape), R))
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,R", [(2, 2), (3, 2), (7, 6), (8, 8), (16, 6), (64, 64), (100, 40), (128, 64), (128, 128), (256, 32), (130, 130)])
def test_rotary_widths(D, R, layout, dtype):
    g = torch.Generator().manual_seed(D + R)
    q = torch.randn(2, 3, 37, D, generator=g).to(dtype).cuda()
    k = torch.randn(2, 1, 37, D, generator=g).to(dtype).cuda()
    freq, _ = la().rotary_frequencies(R, device="cuda")
    for back in (False, True):
        check_rotary(q, k, freq, None, layout, mscale=1.3, backward=back)


@pytest.mark.parametrize("B,H,H2,T", [(1, 1, 0, 1), (1, 40, 8, 1), (64, 4, 2, 1), (3, 5, 2, 300), (1, 2, 2, 2049), (300, 1, 1, 3)])
def test_rotary_shapes(B, H, H2, T):
    g = torch.Generator().manual_seed(B + T)
    q = torch.randn(B, T, H, 64, generator=g).bfloat16().cuda().transpose(1, 2)
    k = torch.randn(B, T, H2, 64, generator=g).bfloat16().cuda().transpose(1, 2) if H2 else None
    freq, m = la().rotary_frequencies(48, scaling="yarn", factor=4.0, trained_length=2048, device="cuda")
    got = check_rotary(q, k, freq, None, "half", mscale=m, start=777)
    assert got[0].is_contiguous()


def test_rotary_far_positions():
    g = torch.Generator().manual_seed(1)
    q = torch.randn(4, 2, 3, 64, generator=g).cuda()
    freq, _ = la().rotary_frequencies(64, device="cuda")
    for base in (10 ** 6, 2 ** 31 + 11, 2 ** 40 + 3, -5):
        pos = base + torch.arange(12, device="cuda").reshape(4, 3) * 7
        check_rotary(q, None, freq, pos, "half")
        check_rotary(q, None, freq, pos[0], "interleaved")
    check_rotary(q, None, freq, None, "half", start=2 ** 33)
    # a slice of a longer table of positions: rows a stride apart
    table = torch.arange(40, device="cuda").reshape(4, 10)
    check_rotary(q, None, freq, table[:, 2:5], "half")


def test_rotary_in_place_inverse_and_odd_strides():
    g = torch.Generator().manual_seed(3)
    freq, _ = la().rotary_frequencies(32, device="cuda")
    wide = torch.randn(2, 9, 3, 129, generator=g).cuda()
    x = wide[..., 1:65].transpose(1, 2)  # 4-byte aligned rows an odd stride apart
    y = check_rotary(x, None, freq, None, "interleaved")[0]
    check_rotary(x, x, freq, None, "half")
    z = x.contiguous()
    assert la().rotary(z, freq, layout=1, out=z) is z and torch.equal(z, y)
    back = la().rotary(z, freq, layout=1, backward=True)
    assert (back - x).abs().max() <= 48 * U * x.abs().max()


def test_rotary_empty():
    freq, _ = la().rotary_frequencies(4, device="cuda")
    assert la().rotary(torch.empty(2, 3, 0, 8, device="cuda"), freq).shape == (2, 3, 0, 8)
    a, b = la().rotary(torch.ones(1, 0, 2, 8, device="cuda"), freq, None, torch.ones(1, 1, 2, 8, device="cuda"), start=1)
    assert a.numel() == 0 and b.shape == (1, 1, 2, 8)


def test_norm_and_rotary_on_another_stream_and_in_a_graph():
    x, gate, w, _, d = tensors((2, 4, 9, 64), torch.bfloat16, 5, "silu", True, False)
    freq, _ = la().rotary_frequencies(64, device="cuda")
    want = [la().gated_norm(x, gate, w), *la().gated_norm_backward(d, x, gate, w), la().rotary(x, freq, start=5)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [la().gated_norm(x, gate, w, stream=s), *la().gated_norm_backward(d, x, gate, w, stream=s),
           la().rotary(x, freq, start=5, stream=s)]
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    outs = [torch.zeros_like(t) for t in want]
    ws = torch.empty(1 << 18, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        la().gated_norm(x, gate, w, out=outs[0])
        la().gated_norm_backward(d, x, gate, w, out=tuple(outs[1:4]), workspace=ws)
        la().rotary(x, freq, start=5, out=outs[4])
    x.mul_(-0.5)
    ws.fill_(255)
    graph.replay()
    want = [la().gated_norm(x, gate, w), *la().gated_norm_backward(d, x, gate, w), la().rotary(x, freq, start=5)]
    for a, b in zip(outs, want):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ a block's chain
def chain_inputs(B=2, T=150, H=4, Hk=2, D=64, seed=0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(q=rn(B, T, Hk, D).bfloat16().cuda(), k=rn(B, T, Hk, D).bfloat16().cuda(), v=rn(B, H, T, D).bfloat16().cuda(),
                beta=torch.sigmoid(rn(B, H, T)).cuda(), lg=torch.nn.functional.logsigmoid(3 + rn(B, H, T)).cuda(),
                gate=rn(B, T, H, D).bfloat16().cuda(), w=(1 + 0.2 * rn(D)).cuda(), dout=rn(B, T, H, D).bfloat16().cuda())


def chain_forward(c, m, freq):
    """The projections' [B,T,H,D] to the output projection's [B,T,H,D], bf16 between the calls as in a bf16 model."""
    s = dict(c)
    s["qn"], s["kn"] = (m.gated_norm(c[n].transpose(1, 2), kind=m.NORM_L2) for n in ("q", "k"))
    s["qr"], s["kr"] = m.rotary(s["qn"], freq, None, s["kn"])
    s["y"], s["S"] = m.delta_forward(s["qr"], s["kr"], c["v"], c["beta"], m.DECAY_PER_STEP, c["lg"], q_scale=0.125)
    s["out"] = m.gated_norm(s["y"].transpose(1, 2), c["gate"], c["w"])
    return s


def chain_backward(s, m, freq):
    dy, dgate, dw = m.gated_norm_backward(s["dout"], s["y"].transpose(1, 2), s["gate"], s["w"])
    dqr, dkr, dv, dbeta, dlg, _ = m.delta_backward(s["qr"], s["kr"], s["v"], s["beta"], dy.transpose(1, 2), m.DECAY_PER_STEP,
                                                   s["lg"], q_scale=0.125)
    dqn, dkn = m.rotary(dqr, freq, None, dkr, backward=True)
    dq, dk = (m.gated_norm_backward(d, s[n].transpose(1, 2), kind=m.NORM_L2)[0].transpose(1, 2)
              for d, n in ((dqn, "q"), (dkn, "k")))
    return dict(q=dq, k=dk, v=dv, beta=dbeta, lg=dlg, gate=dgate, w=dw)


def test_block_chain_forward_backward_and_token_by_token():
    m = la()
    c = chain_inputs()
    T = c["v"].shape[2]
    freq, _ = m.rotary_frequencies(32, device="cuda")
    s = chain_forward(c, m, freq)
    got = chain_backward(s, m, freq)

    # the same chain in float64 from the same inputs, nothing rounded between
    qn, kn = (oracle.gated_norm(f64(c[n]).transpose(0, 2, 1, 3), kind="l2") for n in ("q", "k"))
    qr, kr = (oracle.rotary(x, freq, np.arange(T)) for x in (qn, kn))
    y, _ = oracle.delta_forward(qr, kr, c["v"], c["beta"], 2, c["lg"], None, 0.125)
    out = oracle.gated_norm(y.transpose(0, 2, 1, 3), c["gate"], c["w"])
    # three roundings to bf16 of keys and queries (norm, rotary), of y and of out; the delta rule's own 2^-7
    rel = lambda a, b: np.linalg.norm(f64(a) - b) / np.linalg.norm(b)  # noqa: E731
    assert rel(s["out"], out) <= 6 * 2.0 ** -8
    dy, dgate, dw = oracle.gated_norm_backward(c["dout"], y.transpose(0, 2, 1, 3), c["gate"], c["w"])
    dqr, dkr, dv, dbeta, dlg, _ = oracle.delta_backward(qr, kr, c["v"], c["beta"], dy.transpose(0, 2, 1, 3), 2, c["lg"], None,
                                                        None, 0.125)
    want = dict(v=dv, beta=dbeta, lg=dlg, gate=dgate, w=dw)
    for n, d in (("q", dqr), ("k", dkr)):
        d = oracle.rotary(d, freq, np.arange(T), backward=True)
        want[n] = oracle.gated_norm_backward(d, f64(c[n]).transpose(0, 2, 1, 3), kind="l2")[0].transpose(0, 2, 1, 3)
    for n, r in want.items():
        # the forward's six roundings, met again on the way back, and three more of the gradients
        assert rel(got[n], r) <= 15 * 2.0 ** -8, n

    # token by token: the serving path gives the same rows
    state = torch.zeros_like(s["S"])
    rows = []
    for t in range(T):
        at = slice(t, t + 1)
        qn, kn = (m.gated_norm(c[n][:, at].transpose(1, 2), kind=m.NORM_L2) for n in ("q", "k"))
        qr, kr = m.rotary(qn, freq, None, kn, start=t)
        y = m.delta_decode_step(qr[:, :, 0], kr[:, :, 0], c["v"][:, :, t].contiguous(), c["beta"][:, :, t].contiguous(), state,
                                m.DECAY_PER_STEP, c["lg"][:, :, t].contiguous(), q_scale=0.125)
        rows.append(m.gated_norm(y, c["gate"][:, t], c["w"]))
    assert rel(torch.stack(rows, 1), f64(s["out"])) <= 2 * 2.0 ** -7
    assert rel(state, f64(s["S"])) <= 2.0 ** -14


def test_refusals_on_the_gpu():
    m = la()
    x = torch.randn(2, 3, 5, 16, device="cuda")
    w, f = torch.ones(16, device="cuda"), torch.ones(4, device="cuda")
    for bad, error in [
        (lambda: m.gated_norm(x, x[:1]), ValueError), (lambda: m.gated_norm(x, x.bfloat16()), TypeError),
        (lambda: m.gated_norm(x.transpose(2, 3)), ValueError), (lambda: m.gated_norm(x, None, w[:8]), ValueError),
        (lambda: m.gated_norm(x, None, w.bfloat16()), TypeError), (lambda: m.gated_norm(x.half()), TypeError),
        (lambda: m.gated_norm(x, out=x[:1].expand(2, 3, 5, 16)), ValueError), (lambda: m.gated_norm(x, kind=4), m.LAError),
        (lambda: m.gated_norm(x, eps=-1.0), m.LAError), (lambda: m.gated_norm(x, x.cpu()), ValueError),
        (lambda: m.gated_norm(torch.zeros(2, 8200, device="cuda")), m.LAError),
        (lambda: m.gated_norm_backward(None, x), ValueError), (lambda: m.gated_norm_backward(x[:1], x), ValueError),
        (lambda: m.gated_norm_backward(x, x, out=(None, None, None)), ValueError),
        (lambda: m.gated_norm_backward(x, x, x, out=(x.clone(), None, None)), ValueError),
        (lambda: m.gated_norm_backward(x, x, None, w, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda")), m.LAError),
        (lambda: m.rotary(x, torch.ones(9, device="cuda")), ValueError), (lambda: m.rotary(x, f.double()), TypeError),
        (lambda: m.rotary(x[0], f), ValueError), (lambda: m.rotary(x, f, torch.zeros(4, dtype=torch.int64, device="cuda")), ValueError),
        (lambda: m.rotary(x, f, torch.zeros(5, dtype=torch.int32, device="cuda")), TypeError),
        (lambda: m.rotary(x, f, torch.zeros(5, dtype=torch.int64, device="cuda"), start=3), ValueError),
        (lambda: m.rotary(x, f, None, x[:1]), ValueError), (lambda: m.rotary(x, f, out2=x), ValueError),
        (lambda: m.rotary(x, f, layout=3), m.LAError), (lambda: m.rotary(x, f, mscale=float("inf")), m.LAError),
    ]:
        with pytest.raises(error):
            bad()


def test_rows_outside_a_view_stay_as_they_were():
    wide = torch.full((3, 7, 200), 7.0, device="cuda").bfloat16()
    x = torch.randn(3, 5, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    view = wide[:, 1:6, 65:129]
    la().gated_norm(x, out=view)
    assert torch.equal(view, la().gated_norm(x))
    mask = torch.ones_like(wide, dtype=torch.bool)
    mask[:, 1:6, 65:129] = False
    assert (wide[mask] == 7.0).all()
    freq, _ = la().rotary_frequencies(32, device="cuda")
    q = x.view(3, 1, 5, 64)
    la().rotary(q, freq, out=view.unsqueeze(1))
    assert torch.equal(view.unsqueeze(1), la().rotary(q, freq)) and (wide[mask] == 7.0).all()


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_fp32_gates_far_out_keep_their_digits(act):
    # Every value to (D + 16) steps of 2^-24 of itself, for gates down to where a(z) is 2^-122: the sum of D squares,
    # its root, the exponential (2 steps of 2^-23), a sum, a division and the products; no step grows with |z|.
    g = torch.Generator().manual_seed(8)
    D = 8
    x, d = (torch.randn(512, D, generator=g).cuda() for _ in range(2))
    z = torch.linspace(-84, 84, 512 * D)[torch.randperm(512 * D, generator=g)].view(512, D).cuda()
    y = f64(la().gated_norm(x, z, **how("rms", act)))
    ref = oracle.gated_norm(x, z, None, None, "rms", act)
    assert (np.abs(y - ref) <= (D + 16) * U * np.abs(ref)).all()
    # the gate's gradient from the same factors, where its two terms do not cancel: silu' = s + z s (1 - s), sigmoid' = s (1 - s)
    dg = f64(la().gated_norm_backward(d, x, z, **how("rms", act))[1])
    ref = oracle.gated_norm_backward(d, x, z, None, "rms", act)[1]
    far = f64(z) < -4
    assert (np.abs(dg - ref) <= 2 * (D + 16) * U * np.abs(ref))[far].all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_angles_up_to_2_to_the_53(layout):
    # frequencies of 24 bits: the angle's product has up to 77, and its rounding to 64 bits is 0.25 rad at 2^53
    q = torch.randn(1, 2, 6, 16, generator=torch.Generator().manual_seed(4)).cuda()
    freq = torch.tensor([1.0, 0.7131, 0.3333333, 1e-3, 2.0 ** -30, 3.1], device="cuda")
    for pos in ([2 ** 53 - 1, -(2 ** 53) + 1, 2 ** 52 + 1, 2 ** 50 + 7, 2 ** 48 - 5, 2 ** 47 + 9], [2 ** 45 + 1, 2 ** 44, 2 ** 42 - 1, 2 ** 40 + 3, 0, -1]):
        check_rotary(q, None, freq, torch.tensor(pos, device="cuda"), layout)
    check_rotary(q, None, freq, None, layout, start=2 ** 53 - 6)
    for start in (2 ** 53 - 5, -(2 ** 53) - 1, 2 ** 63, 2 ** 64 + 5, -(2 ** 70)):
        with pytest.raises(ValueError, match="start"):
            la().rotary(q, freq, start=start)


def test_norm_of_a_batch_far_apart():
    # sequences 2^32 elements and more apart (one layer of a long cache): offsets and strides beyond 32 bits
    m, apart = la(), 2 ** 32 + 64
    wide = torch.empty(apart + 8 * 64, dtype=torch.bfloat16, device="cuda")
    x = wide.as_strided((2, 3, 64), (apart, 128, 1))
    x.copy_(torch.randn(2, 3, 64, generator=torch.Generator().manual_seed(2)))
    near_by = x.contiguous()
    d = torch.randn(2, 3, 64, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    w = torch.ones(64, device="cuda")
    assert torch.equal(m.gated_norm(x, x, w), m.gated_norm(near_by, near_by, w))
    for a, b in zip(m.gated_norm_backward(d, x, x, w), m.gated_norm_backward(d, near_by, near_by, w)):
        assert torch.equal(a, b)
    want = m.gated_norm(near_by)
    assert torch.equal(m.gated_norm(x, out=x), want) and torch.equal(x, want)
    # four dimensions: the batch's stride may be any, the inner two are below 2^32
    q, freq = x.unsqueeze(1), m.rotary_frequencies(64, device="cuda")[0]
    assert torch.equal(m.rotary(q, freq), m.rotary(q.contiguous(), freq))


# ------------------------------------------------------------------ gradients over many rows a team
def closed_norm_backward(d, x, z, w, kind, act, eps, scale):
    """oracle.gated_norm_backward without the Jacobian: dx = r (dn - n <dn, n> / K - [layer] mean dn)."""
    D = x.shape[-1]
    n, r = oracle.block._normalised(x, kind, eps)
    w = np.ones(D) if w is None else w
    a, da = (1.0, None) if z is None else oracle.block._activation(z, act)
    m = scale * d
    dn = m * w * a
    dx = r * (dn - n * (dn * n).sum(-1, keepdims=True) / (1 if kind == "l2" else D)
              - (dn.mean(-1, keepdims=True) if kind == "layer" else 0))
    return dx, None if z is None else m * n * w * da, (m * a * n).reshape(-1, D).sum(0)


@pytest.mark.parametrize("kind,act", list(itertools.product(KINDS, ACTS)))
def test_closed_norm_gradients_are_the_oracles(kind, act):
    r = np.random.default_rng(1)
    d, x, w = r.standard_normal((2, 3, 9)), r.standard_normal((2, 3, 9)), r.standard_normal(9)
    z = r.standard_normal((2, 3, 9)) if act != "none" else None
    for a, b in zip(closed_norm_backward(d, x, z, w, kind, act, 1e-3, 0.7),
                    oracle.gated_norm_backward(d, x, z, w, kind, act, 1e-3, 0.7)):
        assert (a is None and b is None) or np.allclose(a, b, rtol=1e-12, atol=1e-13)


# rows: more than one a team for every team size (296 blocks of 256 threads), with an innermost size that
# wraps within a team's run, and block-wide teams of several rows
@pytest.mark.parametrize("dtype,shape", [
    (torch.bfloat16, (2, 1700, 7, 32)), (torch.bfloat16, (3, 1003, 7, 64)), (torch.bfloat16, (2, 1100, 5, 128)),
    (torch.bfloat16, (2, 700, 5, 256)), (torch.bfloat16, (2, 401, 7, 512)), (torch.bfloat16, (1, 903, 3, 1024)),
    (torch.bfloat16, (2, 167, 3, 2048)), (torch.bfloat16, (1, 301, 3, 4096)), (torch.bfloat16, (1, 201, 3, 8192)),
    (torch.bfloat16, (2, 1500, 3, 33)), (torch.bfloat16, (1, 301, 3, 2050)), (torch.bfloat16, (1, 301, 2, 4099)),
    (torch.float32, (2, 1700, 7, 32)), (torch.float32, (2, 700, 5, 128)), (torch.float32, (1, 903, 3, 512)),
    (torch.float32, (1, 301, 3, 1024)), (torch.float32, (1, 301, 3, 2052)), (torch.float32, (1, 301, 3, 4096)),
    (torch.float32, (1, 201, 3, 8192)), (torch.float32, (1, 301, 2, 2049)), (torch.float32, (1, 151, 2, 8191)),
])
def test_norm_gradients_of_many_rows(dtype, shape):
    x, gate, w, _, d = tensors(shape, dtype, shape[-1], "silu", True, False)
    x = x.transpose(1, 2).contiguous().transpose(1, 2)  # the scan's layout under the projection's
    D = shape[-1]
    for kind, act, z in (("layer", "silu", gate), ("rms", "sigmoid", gate), ("l2", "none", None)):
        got = la().gated_norm_backward(d, x, z, w, **how(kind, act, scale=0.7))
        dd, xx, zz, ww = (f64(t) for t in (d, x, z, w))
        ref = closed_norm_backward(dd, xx, zz, ww, kind, act, 1e-5, 0.7)
        # the bars of check_norm_backward
        terms, steps, r, big = norm_terms(xx, zz, ww, kind, act, 1e-5, 0.7)
        a = 1.0 if zz is None else np.abs(oracle.block._activation(zz, act)[0])
        dn = np.abs(0.7 * dd) * np.abs(ww) * a
        t = r * (dn + big * (dn * big).sum(-1, keepdims=True) / (1 if kind == "l2" else D)
                 + (dn.mean(-1, keepdims=True) if kind == "layer" else 0))
        worst = np.max(steps, axis=-1, keepdims=True) if np.ndim(steps) else steps
        near(got[0], ref[0], t, 3 * worst, dtype, "dx")
        if zz is not None:
            s = oracle.block._activation(zz, "sigmoid")[0]
            near(got[1], ref[1], np.abs(0.7 * dd) * big * np.abs(ww) * (s * (1 + np.abs(zz)) if act == "silu" else s), 2 * steps + 8,
                 dtype, "dgate")
        col = (np.abs(0.7 * dd) * a * big).reshape(-1, D).sum(0)
        near(got[2], ref[2], col, dd.reshape(-1, D).shape[0] + np.max(steps), torch.float32, "dweight")
        again = la().gated_norm_backward(d, x, z, w, **how(kind, act, scale=0.7))
        assert all(torch.equal(p, q) for p, q in zip(got, again) if p is not None)
