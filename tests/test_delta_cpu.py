"""The gated delta rule without a GPU: the oracle against closed forms and
differences, the C ABI's refusals (none reaches CUDA), workspace sizes."""
import ctypes
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
import retention_scan_b200 as la
from test_abi_cpu import L, ROOT  # noqa: F401  (fixture)


def rng_case(B=2, H=4, Hk=2, T=9, Dk=5, Dv=3, seed=0, kind=2):
    r = np.random.default_rng(seed)
    q, k = r.standard_normal((B, Hk, T, Dk)), r.standard_normal((B, Hk, T, Dk))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    v, beta = r.standard_normal((B, H, T, Dv)), r.uniform(0, 1, (B, H, T))
    lg = None if kind == 0 else -r.uniform(0, 1, (H,) if kind == 1 else (B, H, T))
    return q, k, v, beta, lg, r.standard_normal((B, H, Dk, Dv))


def test_oracle_one_token_by_hand():
    q, k, v, beta, lg, S0 = rng_case(1, 1, 1, 1, 4, 3)
    y, S = oracle.delta_forward(q, k, v, beta, 2, lg, S0, 0.5)
    g, kk, b = np.exp(lg[0, 0, 0]), k[0, 0, 0], beta[0, 0, 0]
    want = g * (np.eye(4) - b * np.outer(kk, kk)) @ S0[0, 0] + b * np.outer(kk, v[0, 0, 0])
    assert np.allclose(S[0, 0], want, atol=1e-14) and np.allclose(y[0, 0, 0], 0.5 * want.T @ q[0, 0, 0], atol=1e-14)


def test_oracle_orthonormal_keys_look_up_the_last_value():
    # beta = 1, g = 1, keys from an orthonormal basis: row j of the state is the last value written with key j
    r = np.random.default_rng(1)
    basis = np.linalg.qr(r.standard_normal((6, 6)))[0]
    idx = r.integers(0, 6, 20)
    k = basis[idx][None, None]
    v = r.standard_normal((1, 1, 20, 3))
    y, S = oracle.delta_forward(k, k, v, np.ones((1, 1, 20)))
    assert np.allclose(y, v, atol=1e-12)
    for j in set(idx):
        last = max(t for t in range(20) if idx[t] == j)
        assert np.allclose(basis[j] @ S[0, 0], v[0, 0, last], atol=1e-12)


def test_oracle_distinct_orthonormal_keys_are_linear_attention():
    # with no key met twice the prediction along it stays zero: beta v as the value of the plain recurrence
    q, k, v, beta, lg, _ = rng_case(1, 2, 2, 5, 5, 3)
    k[:] = np.linalg.qr(np.random.default_rng(2).standard_normal((5, 5)))[0]
    y, S = oracle.delta_forward(q, k, v, beta, 2, lg)
    yl, Sl, _ = oracle.forward(q, k, beta[..., None] * v, 2, lg)
    assert np.allclose(y, yl, atol=1e-12) and np.allclose(S, Sl, atol=1e-12)


def test_oracle_split_carry_shared_heads_and_padding():
    q, k, v, beta, lg, S0 = rng_case()
    y, S = oracle.delta_forward(q, k, v, beta, 2, lg, S0)
    cut = lambda a, b: [x[:, :, a:b] for x in (q, k, v, beta, lg)]  # noqa: E731
    a = cut(0, 4)
    y1, S1 = oracle.delta_forward(*a[:4], 2, a[4], S0)
    b = cut(4, 9)
    y2, S2 = oracle.delta_forward(*b[:4], 2, b[4], S1)
    assert np.allclose(np.concatenate([y1, y2], 2), y) and np.allclose(S2, S)
    ye, Se = oracle.delta_forward(q.repeat(2, 1), k.repeat(2, 1), v, beta, 2, lg, S0)
    assert np.array_equal(ye, y) and np.array_equal(Se, S)
    beta[:, :, 4:] = 0
    lg[:, :, 4:] = 0
    assert np.allclose(oracle.delta_forward(q, k, v, beta, 2, lg, S0)[1], S1)


def test_oracle_decode_is_the_forward():
    q, k, v, beta, lg, S = rng_case(T=6)
    y, Sf = oracle.delta_forward(q, k, v, beta, 2, lg, S, 0.3)
    for t in range(6):
        yt, S = oracle.delta_decode_step(*(x[:, :, t] for x in (q, k, v, beta)), S, 2, lg[:, :, t], 0.3)
        assert np.allclose(yt, y[:, :, t])
    assert np.allclose(S, Sf)


@pytest.mark.parametrize("kind", [0, 1, 2])
def test_oracle_gradients_against_differences(kind):
    q, k, v, beta, lg, S0 = rng_case(kind=kind, seed=kind)
    r = np.random.default_rng(9)
    dy, dS = r.standard_normal(v.shape), r.standard_normal(S0.shape)
    got = oracle.delta_backward(q, k, v, beta, dy, kind, lg, S0, dS, 0.7)
    leaves = [q, k, v, beta, lg, S0]

    def loss(xs):
        y, S = oracle.delta_forward(*xs[:4], kind, xs[4], xs[5], 0.7)
        return (y * dy).sum() + (S * dS).sum()
    for i, x in enumerate(leaves):
        if x is None:
            assert got[i] is None
            continue
        d = r.standard_normal(x.shape)
        up, dn = ([u + s * d if j == i else u for j, u in enumerate(leaves)] for s in (1e-5, -1e-5))
        slope = (loss(up) - loss(dn)) / 2e-5
        assert abs((got[i] * d).sum() - slope) <= 1e-7 * (1 + abs(slope)), i


# ------------------------------------------------------------------ the C ABI's refusals
def fwd(lib, **over):
    a = dict(q=16, k=16, v=16, beta=16, decay=None, scale=1.0, S0=None, out=16, Sf=None, B=1, H=4, Hk=2, T=4, Dk=16, Dv=16,
             dtype=1, ws=16, nbytes=1 << 30)
    a.update(over)
    vp, d = ctypes.c_void_p, a["decay"]
    return lib.la_delta_forward_ws(vp(a["q"]), vp(a["k"]), vp(a["v"]), vp(a["beta"]), ctypes.byref(d) if d else None,
                                   a["scale"], vp(a["S0"]), vp(a["out"]), vp(a["Sf"]), a["B"], a["H"], a["Hk"], a["T"],
                                   a["Dk"], a["Dv"], a["dtype"], vp(a["ws"]), a["nbytes"], None)


def bwd(lib, **over):
    a = dict(q=16, k=16, v=16, beta=16, decay=None, scale=1.0, S0=None, dy=16, dSf=None, dq=16, dk=16, dv=16, db=16, dlg=None,
             dS0=None, B=1, H=4, Hk=2, T=4, Dk=16, Dv=16, dtype=1, ws=16, nbytes=1 << 30)
    a.update(over)
    vp, d = ctypes.c_void_p, a["decay"]
    return lib.la_delta_backward_ws(
        vp(a["q"]), vp(a["k"]), vp(a["v"]), vp(a["beta"]), ctypes.byref(d) if d else None, a["scale"], vp(a["S0"]), vp(a["dy"]),
        vp(a["dSf"]), vp(a["dq"]), vp(a["dk"]), vp(a["dv"]), vp(a["db"]), vp(a["dlg"]), vp(a["dS0"]), a["B"], a["H"], a["Hk"],
        a["T"], a["Dk"], a["Dv"], a["dtype"], vp(a["ws"]), a["nbytes"], None)


def dec(lib, **over):
    a = dict(q=16, k=16, v=16, beta=16, decay=None, scale=1.0, state=16, out=16, B=1, H=4, Hk=2, Dk=16, Dv=16, dtype=1)
    a.update(over)
    vp, d = ctypes.c_void_p, a["decay"]
    return lib.la_delta_decode_step(vp(a["q"]), vp(a["k"]), vp(a["v"]), vp(a["beta"]), ctypes.byref(d) if d else None,
                                    a["scale"], vp(a["state"]), vp(a["out"]), a["B"], a["H"], a["Hk"], a["Dk"], a["Dv"],
                                    a["dtype"], None)


SHARED = [
    (dict(q=None), 1), (dict(k=8), 1), (dict(v=None), 1), (dict(beta=None), 1), (dict(beta=2), 1), (dict(out=None), 1),
    (dict(B=-1), 1), (dict(H=-4), 1), (dict(Hk=0), 1), (dict(Hk=3), 1), (dict(Hk=-2), 1), (dict(Dk=0), 1), (dict(Dv=0), 1),
    (dict(dtype=7), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(decay=la._Decay(5, 64)), 1), (dict(decay=la._Decay(1, None)), 1), (dict(decay=la._Decay(2, 2)), 1),
    (dict(Dk=144, dtype=0), 2), (dict(Dv=129, dtype=0), 2),
]


@pytest.mark.parametrize("over,status", SHARED + [
    (dict(S0=8), 1), (dict(Sf=4), 1), (dict(T=-1), 1), (dict(ws=None), 1), (dict(ws=8), 1), (dict(nbytes=64), 1),
    (dict(Dk=24), 2), (dict(Dv=40), 2), (dict(B=1 << 14, T=1 << 20), 2),
], ids=str)
def test_forward_refusals(L, over, status):  # noqa: F811
    assert fwd(L, **over) == status


@pytest.mark.parametrize("over,status", [x for x in SHARED if "out" not in x[0]] + [
    (dict(dy=None), 1), (dict(dq=None), 1), (dict(dk=8), 1), (dict(dv=None), 1), (dict(db=None), 1), (dict(db=2), 1),
    (dict(dlg=16), 1), (dict(dlg=2, decay=la._Decay(2, 64)), 1), (dict(dSf=8), 1), (dict(dS0=4), 1), (dict(S0=4), 1),
    (dict(ws=None), 1), (dict(nbytes=64), 1), (dict(T=-1), 1), (dict(Dk=24), 2),
], ids=str)
def test_backward_refusals(L, over, status):  # noqa: F811
    assert bwd(L, **over) == status


@pytest.mark.parametrize("over,status", SHARED + [(dict(state=None), 1), (dict(state=8), 1), (dict(out=8), 1)], ids=str)
def test_decode_refusals(L, over, status):  # noqa: F811
    assert dec(L, **over) == status


def test_nothing_to_do(L):  # noqa: F811
    assert fwd(L, B=0, q=None, k=None, v=None, out=None, ws=None, nbytes=0) == 0
    assert fwd(L, H=0, Hk=0) == 0
    assert bwd(L, B=0, q=None, dq=None, ws=None) == 0
    assert dec(L, B=0, state=None) == 0
    # an empty per-step log_g may have no address; an unknown kind stays refused
    assert fwd(L, B=0, decay=la._Decay(2, None)) == 0
    assert fwd(L, B=0, decay=la._Decay(9, None)) == 1


def test_workspace_sizes(L):  # noqa: F811
    size = lambda *a: int(L.la_delta_workspace_size(*a))  # noqa: E731
    back = lambda *a, kind=2: int(L.la_delta_backward_workspace_size(*a, kind))  # noqa: E731
    rec = 8192 * 3 + 5 * 64 * 4  # two planes of the inverse, one of the scores, the factors
    assert size(2, 4, 2, 65, 64, 64, 1) == -(-2 * 4 * 2 * rec // 256) * 256
    assert size(2, 4, 2, 0, 64, 64, 1) == size(0, 4, 2, 65, 64, 64, 1) == 0
    assert size(2, 4, 3, 65, 64, 64, 1) == 0 and size(2, 4, 2, 65, 40, 64, 1) == 0
    assert back(2, 4, 2, 65, 64, 64, 1) > size(2, 4, 2, 65, 64, 64, 1)
    assert back(2, 4, 2, 65, 64, 64, 1) > back(2, 4, 4, 65, 64, 64, 1)  # partial sums of shared heads
    # a third plane: a decay per head, Dk <= 32, fewer than 4096 tokens times heads
    assert back(2, 4, 2, 512, 64, 64, 1, kind=1) > back(2, 4, 2, 512, 64, 64, 1) == back(2, 4, 2, 512, 64, 64, 1, kind=0)
    assert back(2, 4, 2, 511, 64, 64, 1, kind=1) == back(2, 4, 2, 511, 64, 64, 1) > back(2, 4, 2, 512, 64, 64, 1)
    assert back(2, 4, 2, 512, 32, 64, 1, kind=1) == back(2, 4, 2, 512, 32, 64, 1)
    assert back(2, 4, 2, 512, 64, 64, 0, kind=1) == back(2, 4, 2, 512, 64, 64, 0)
    assert size(1, 32, 32, 1 << 20, 128, 128, 1) == 32 * (1 << 14) * rec  # beyond 2^33: no 32-bit size


def test_injected_launch_failure():
    code = r'''
import sys
sys.path[:0] = [%r, %r]
import test_delta_cpu as t, retention_scan_b200 as la
lib = la.lib()
print(t.fwd(lib), t.bwd(lib), t.dec(lib))
''' % (ROOT, ROOT + "/tests")
    import os
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, check=True,
                         env=dict(os.environ, LA_FAULT_INJECT="launch"))
    assert out.stdout.split() == ["3", "3", "3"]


def test_binding_refuses_before_it_calls():
    z = torch.zeros
    ok = dict(q=z(1, 2, 3, 16), k=z(1, 2, 3, 16), v=z(1, 4, 3, 16), beta=z(1, 4, 3))
    with pytest.raises(ValueError, match="CUDA"):
        la.delta_forward(**ok)
    with pytest.raises(ValueError, match="dimensions"):
        la.delta_forward(**dict(ok, q=z(2, 3, 16)))
    with pytest.raises(ValueError, match="CUDA"):
        la.delta_decode_step(z(1, 2, 16), z(1, 2, 16), z(1, 4, 16), z(1, 4), z(1, 4, 16, 16))


def test_key_heads_without_value_heads(L):  # noqa: F811
    # their gradients are written (zeros), so they have to have an address
    assert bwd(L, H=0, dq=None) == 1 and bwd(L, H=0, dk=8) == 1
    assert bwd(L, H=0, Hk=0, dq=None, dk=None) == 0 and bwd(L, H=0, T=0, dq=None) == 0 and bwd(L, H=0, B=0, dq=None) == 0
    assert bwd(L, H=0, B=1 << 20, Hk=1 << 20) == 2 and bwd(L, H=0, B=1 << 30, T=1 << 30) == 2
