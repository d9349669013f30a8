"""The gated norm and rotary positions without a GPU: the oracle against
independent forms, frequencies, the C ABI's refusals (none reaches CUDA)."""
import ctypes
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
import retention_scan_b200 as la
from test_abi_cpu import L, ROOT  # noqa: F401  (fixture)


def test_oracle_norm_against_torch():
    g = torch.Generator().manual_seed(0)
    x, z, r = (torch.randn(3, 5, 12, generator=g, dtype=torch.float64) for _ in range(3))
    w = torch.randn(12, generator=g, dtype=torch.float64)
    F = torch.nn.functional
    assert np.allclose(oracle.gated_norm(x, None, w, r, "layer", eps=1e-3, scale=0.5),
                       r + 0.5 * F.layer_norm(x, (12,), w, None, 1e-3))
    assert np.allclose(oracle.gated_norm(x, z, w, None, "rms", "silu", 1e-3), F.rms_norm(x, (12,), w, 1e-3) * F.silu(z))
    assert np.allclose(oracle.gated_norm(x, z, None, None, "l2", "sigmoid", 0.0), F.normalize(x, dim=-1) * torch.sigmoid(z))


@pytest.mark.parametrize("kind", ["rms", "layer", "l2"])
@pytest.mark.parametrize("act", ["none", "silu", "sigmoid"])
def test_oracle_norm_gradients_against_differences(kind, act):
    r = np.random.default_rng(3)
    x, d, w = r.standard_normal((4, 9)), r.standard_normal((4, 9)), r.standard_normal(9)
    z = r.standard_normal((4, 9)) if act != "none" else None
    got = oracle.gated_norm_backward(d, x, z, w, kind, act, 1e-3, 0.7)
    for i, t in enumerate((x, z, w)):
        if t is None:
            assert got[i] is None
            continue
        v = r.standard_normal(t.shape)
        at = lambda s: [u + s * v if j == i else u for j, u in enumerate((x, z, w))]  # noqa: E731
        f = lambda a: (oracle.gated_norm(a[0], a[1], a[2], None, kind, act, 1e-3, 0.7) * d).sum()  # noqa: E731
        slope = (f(at(1e-6)) - f(at(-1e-6))) / 2e-6
        assert abs((got[i] * v).sum() - slope) <= 1e-7 * (1 + abs(slope))


def test_oracle_rotary():
    r = np.random.default_rng(1)
    x = r.standard_normal((2, 3, 5, 10))
    freq = np.array([1.0, 0.3, 0.05])
    y = oracle.rotary(x, freq, np.arange(5), "half", 1.0)
    assert np.array_equal(y[:, :, 0], x[:, :, 0]) and np.array_equal(y[..., 6:], x[..., 6:])
    # the pair (0, 3) by the angle t
    t = 4
    assert np.allclose(y[:, :, t, 0], x[:, :, t, 0] * math.cos(t) - x[:, :, t, 3] * math.sin(t))
    assert np.allclose(y[:, :, t, 3], x[:, :, t, 0] * math.sin(t) + x[:, :, t, 3] * math.cos(t))
    # interleaved is the half layout of reordered elements
    order = [0, 2, 4, 1, 3, 5, 6, 7, 8, 9]
    z = oracle.rotary(x[..., np.argsort(order)], freq, np.arange(5), "interleaved")
    assert np.allclose(z[..., order], y)
    # scores depend on distances alone; the transposed map undoes it
    a, b = (oracle.rotary(x[:, :, :1].repeat(5, 2), freq, p) for p in (np.arange(5), np.arange(5) + 7))
    assert np.allclose((a[:, :, 2] * a[:, :, 4]).sum(-1), (b[:, :, 2] * b[:, :, 4]).sum(-1))
    assert np.allclose(oracle.rotary(y, freq, np.arange(5), backward=True), x)


def test_frequencies():
    f, m = la.rotary_frequencies(8)
    assert m == 1.0 and f.dtype == torch.float32
    assert np.allclose(f.double(), 10000.0 ** (-np.arange(4) / 4), rtol=2.0 ** -24)
    assert np.allclose(la.rotary_frequencies(8, scaling="linear", factor=4.0)[0].double() * 4, f.double(), rtol=2.0 ** -23)
    n = la.rotary_frequencies(8, scaling="ntk", factor=4.0)[0].double()
    assert n[0] == 1.0 and math.isclose(float(f[3] / n[3]), 4.0, rel_tol=1e-6)
    y, m = la.rotary_frequencies(64, scaling="yarn", factor=4.0, trained_length=4096)
    base = la.rotary_frequencies(64)[0]
    turns = 4096 * base.double() / (2 * math.pi)
    assert math.isclose(m, 0.1 * math.log(4.0) + 1)
    assert torch.equal(y[turns >= 32], base[turns >= 32]) and torch.allclose(y[turns <= 1], base[turns <= 1] / 4)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and (y[mid] < base[mid]).all() and (y[mid] > base[mid] / 4).all()
    assert la.rotary_frequencies(2, scaling="ntk", factor=8.0)[0].tolist() == [1.0]
    for bad in (dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=8, factor=0.5), dict(rot_dim=8, base=-1.0),
                dict(rot_dim=8, scaling="yarn"), dict(rot_dim=8, scaling="yarn", trained_length=10, fast=1.0),
                dict(rot_dim=8, scaling="other")):
        with pytest.raises(ValueError):
            la.rotary_frequencies(**bad)


# ------------------------------------------------------------------ the C ABI's refusals
def view(data=64, s0=96, s1=32, s2=16):
    return la._View(data, s0, s1, s2)


def ref(v):
    return ctypes.addressof(v) if v is not None else None


def norm(lib, **over):
    a = dict(x=view(), gate=None, w=None, res=None, out=view(), n0=2, n1=3, n2=2, D=16, kind=0, act=0, eps=1e-5, scale=1.0,
             dtype=1)
    a.update(over)
    return lib.la_gated_norm(ref(a["x"]), ref(a["gate"]), a["w"], ref(a["res"]), ref(a["out"]), a["n0"], a["n1"], a["n2"],
                             a["D"], a["kind"], a["act"], a["eps"], a["scale"], a["dtype"], None)


def norm_bwd(lib, **over):
    a = dict(dout=view(), x=view(), gate=None, w=None, dx=view(), dgate=None, dw=None, n0=2, n1=3, n2=2, D=16, kind=0, act=0,
             eps=1e-5, scale=1.0, dtype=1, ws=None, nbytes=0)
    a.update(over)
    return lib.la_gated_norm_backward(ref(a["dout"]), ref(a["x"]), ref(a["gate"]), a["w"], ref(a["dx"]), ref(a["dgate"]),
                                      a["dw"], a["n0"], a["n1"], a["n2"], a["D"], a["kind"], a["act"], a["eps"], a["scale"],
                                      a["dtype"], a["ws"], a["nbytes"], None)


def rot(lib, **over):
    a = dict(x=view(), H=3, x2=None, H2=0, out=view(), out2=None, freq=64, pos=None, ps=0, start=0, B=2, T=2, D=16, R=8,
             layout=0, m=1.0, back=0, dtype=1)
    a.update(over)
    return lib.la_rotary(ref(a["x"]), a["H"], ref(a["x2"]), a["H2"], ref(a["out"]), ref(a["out2"]), a["freq"], a["pos"], a["ps"],
                         a["start"], a["B"], a["T"], a["D"], a["R"], a["layout"], a["m"], a["back"], a["dtype"], None)


NORM = [
    (dict(x=None), 1), (dict(x=view(None)), 1), (dict(x=view(65)), 1), (dict(x=view(s1=-1)), 1), (dict(x=view(s2=1 << 32)), 1),
    (dict(n0=-1), 1), (dict(D=0), 1), (dict(kind=3), 1), (dict(act=-1), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(dtype=2), 1), (dict(w=2), 1), (dict(D=8193), 2),
    (dict(n0=1 << 20, n1=1 << 20, n2=2), 2), (dict(n0=1 << 16, n1=1 << 16), 2),
]


@pytest.mark.parametrize("over,status", NORM + [
    (dict(out=None), 1), (dict(out=view(s0=0)), 1), (dict(out=view(s2=0)), 1), (dict(gate=view(1)), 1), (dict(res=view(1)), 1),
], ids=lambda o: ",".join(o) if isinstance(o, dict) else str(o))
def test_norm_refusals(L, over, status):  # noqa: F811
    assert norm(L, **over) == status


@pytest.mark.parametrize("over,status", NORM + [
    (dict(dout=None), 1), (dict(dx=None), 1), (dict(dx=view(s1=0)), 1), (dict(gate=view()), 1), (dict(dgate=view()), 1),
    (dict(gate=view(), dgate=view(s0=0)), 1), (dict(dw=64), 1), (dict(w=64, dw=2), 1), (dict(w=64, dw=64), 1),
    (dict(w=64, dw=64, ws=8, nbytes=1 << 20), 1), (dict(w=64, dw=64, ws=64, nbytes=16), 1),
], ids=lambda o: ",".join(o) if isinstance(o, dict) else str(o))
def test_norm_backward_refusals(L, over, status):  # noqa: F811
    assert norm_bwd(L, **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(x=None), 1), (dict(out=None), 1), (dict(x=view(65)), 1), (dict(out=view(s2=0)), 1), (dict(out=view(s1=0)), 1),
    (dict(H2=2), 1), (dict(x2=view(), H2=2), 1), (dict(freq=None), 1), (dict(freq=2), 1), (dict(pos=4), 1),
    (dict(pos=64, ps=-1), 1), (dict(B=-1), 1), (dict(T=-1), 1), (dict(H=-1), 1), (dict(R=0), 1), (dict(R=7), 1), (dict(R=18), 1),
    (dict(D=0), 1), (dict(layout=2), 1), (dict(m=float("nan")), 1), (dict(dtype=5), 1), (dict(D=9000), 2),
    (dict(T=1 << 30, B=4), 2), (dict(H=1 << 24), 2),
], ids=lambda o: ",".join(o) if isinstance(o, dict) else str(o))
def test_rotary_refusals(L, over, status):  # noqa: F811
    assert rot(L, **over) == status


def test_nothing_to_do(L):  # noqa: F811
    assert norm(L, n1=0, x=None, out=None) == 0
    assert norm_bwd(L, n2=0, x=None) == 0
    assert rot(L, B=0, x=None, freq=None) == 0 and rot(L, H=0) == 0
    assert int(L.la_gated_norm_backward_workspace_size(0, 3, 4, 16)) == 0
    assert int(L.la_gated_norm_backward_workspace_size(2, 3, 4, 100)) >= 2 * 3 * 4 * 400


def test_injected_launch_failure():
    code = r'''
import sys
sys.path[:0] = [%r, %r]
import test_block_cpu as t, retention_scan_b200 as la
lib = la.lib()
print(t.norm(lib), t.norm_bwd(lib), t.rot(lib))
''' % (ROOT, ROOT + "/tests")
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, check=True,
                         env=dict(os.environ, LA_FAULT_INJECT="launch"))
    assert out.stdout.split() == ["3", "3", "3"]


def test_binding_refuses_before_it_calls():
    x = torch.zeros(2, 3, 8)
    with pytest.raises(ValueError, match="CUDA"):
        la.gated_norm(x)
    with pytest.raises(ValueError, match="dimensions"):
        la.gated_norm(torch.zeros(1, 1, 1, 1, 8))
    with pytest.raises(ValueError, match="CUDA"):
        la.gated_norm_backward(x, x)
    with pytest.raises(ValueError, match="CUDA"):
        la.rotary(torch.zeros(1, 1, 2, 8), torch.zeros(4))


def test_oracle_angles_of_far_positions():
    # 2^53 - 1 turns of a frequency that is a whole number of 2^-24: the product has 77 bits.  By Euler's formula
    # the angle of p is that of its halves: exp(i p f) from exp(i 2^26 f) and the rest, in 64-bit steps small enough.
    f = np.array([1.0, 0.71310001611709595, 2.0 ** -20, 3.5])
    for p in (2 ** 53 - 1, 2 ** 45 + 1, 2 ** 40 + 3, -5, 2 ** 31 + 11):
        unit = np.exp(1j * f.astype(np.longdouble))
        z, n, w = np.ones(4, dtype=np.clongdouble), abs(p), unit
        while n:  # repeated squaring in 64-bit mantissas: p roundings of 2^-64 of the angle
            z, w, n = (z * w if n & 1 else z), w * w, n >> 1
        z = z if p > 0 else z.conj()
        got = np.exp(1j * oracle.block._angles(np.array([float(p)]), f)[0])
        assert np.abs(got - z.astype(complex)).max() <= abs(p) * 2.0 ** -62 + 1e-14, p


@pytest.mark.parametrize("over,status", [
    (dict(start=(1 << 53) - 1), 1), (dict(start=-(1 << 53) - 1), 1), (dict(start=(1 << 63) - 1), 1), (dict(start=-(1 << 63)), 1),
], ids=str)
def test_rotary_refuses_starts_beyond_exact_positions(L, over, status):  # noqa: F811
    assert rot(L, **over) == status


def test_yarn_values():
    # by hand: 64 / 2 pi = 10.19 turns of the first pair, 1.92 of the second (base 28.2), .36 of the third
    f, m = la.rotary_frequencies(6, base=28.2, scaling="yarn", factor=4.0, trained_length=64, fast=8.0, slow=1.5)
    b = [28.2 ** (-i / 3) for i in range(3)]
    turns = [64 * x / (2 * math.pi) for x in b]
    assert turns[0] > 8 and 1.5 < turns[1] < 8 and turns[2] < 1.5
    share = (turns[1] - 1.5) / (8 - 1.5)  # of the trained frequency; the rest of a quarter of it
    want = [b[0], b[1] * share + b[1] / 4 * (1 - share), b[2] / 4]
    assert np.allclose(f.double(), want, rtol=2.0 ** -23) and math.isclose(m, 0.1 * math.log(4.0) + 1)
