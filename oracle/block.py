"""The gated norm, its gradients and rotary positions in float64 numpy, from
their definitions."""
import numpy as np


def _f64(a):
    if a is None:
        return None
    if hasattr(a, "detach"):
        a = a.detach().to("cpu").double().numpy()
    return np.asarray(a, dtype=np.float64)


def _activation(z, name):
    """a(z) and a'(z), without overflow for any finite z."""
    s = np.where(z >= 0, 1 / (1 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))))
    return (z * s, s * (1 + z * (1 - s))) if name == "silu" else (s, s * (1 - s))


def _normalised(x, kind, eps):
    if kind == "layer":
        x = x - x.mean(-1, keepdims=True)
    ss = (x * x).sum(-1, keepdims=True)
    r = 1 / np.sqrt((ss if kind == "l2" else ss / x.shape[-1]) + eps)
    return x * r, r


def gated_norm(x, gate=None, weight=None, residual=None, kind="rms", activation="silu", eps=1e-5, scale=1.0):
    x, gate, weight, residual = (_f64(t) for t in (x, gate, weight, residual))
    y = scale * _normalised(x, kind, eps)[0]
    if weight is not None:
        y = y * weight
    if gate is not None:
        y = y * _activation(gate, activation)[0]
    return y if residual is None else residual + y


def gated_norm_backward(dout, x, gate=None, weight=None, kind="rms", activation="silu", eps=1e-5, scale=1.0):
    """(dx, dgate or None, dweight or None): the Jacobian of the norm written out,
    d n_i / d x_j = r (P_ij - n_i n_j / K) with P the centring of the layer norm."""
    dout, x, gate, weight = (_f64(t) for t in (dout, x, gate, weight))
    D = x.shape[-1]
    n, r = _normalised(x, kind, eps)
    w = np.ones(D) if weight is None else weight
    a, da = (np.ones(1), None) if gate is None else _activation(gate, activation)
    J = np.eye(D) - (1 / D if kind == "layer" else 0) - n[..., :, None] * n[..., None, :] / (1 if kind == "l2" else D)
    dx = r * np.einsum("...ij,...i->...j", J, scale * dout * w * a)
    dgate = None if gate is None else scale * dout * n * w * da
    dweight = None if weight is None else (scale * dout * a * n).reshape(-1, D).sum(0)
    return dx, dgate, dweight


_SHIFT = 240
_TWO_PI = int("6283185307179586476925286766559005768394338798750211641949889184615632812572417997256") * (1 << _SHIFT) // 10 ** 84


def _angles(positions, freq):
    """positions[..., None] * freq modulo 2 pi: far positions in whole numbers, since a
    64-bit product at 2^45 is off by 2^-9 already."""
    if np.abs(positions).max(initial=0) * np.abs(freq).max() < 2 ** 20:
        return positions[..., None] * freq
    out = np.empty(positions.shape + freq.shape)
    for j, f in enumerate(freq):
        m, d = float(f).as_integer_ratio()
        for at in np.ndindex(positions.shape):
            turns = (int(positions[at]) * m << _SHIFT) // d % _TWO_PI
            out[at + (j,)] = float(turns >> (_SHIFT - 60)) / 2.0 ** 60
    return out


def rotary(x, freq, positions, layout="half", mscale=1.0, backward=False):
    """x [B,H,T,D], freq [R/2], positions broadcastable to [B,T]; pairs as complex numbers."""
    x, freq = _f64(x), _f64(freq)
    B, _, T, _ = x.shape
    R = 2 * freq.shape[0]
    angle = _angles(np.broadcast_to(np.asarray(positions, dtype=np.float64), (B, T)), freq)[:, None]
    turn = mscale * np.exp((-1j if backward else 1j) * angle)
    out = x.copy()
    a, b = (slice(0, R // 2), slice(R // 2, R)) if layout == "half" else (slice(0, R, 2), slice(1, R, 2))
    z = (x[..., a] + 1j * x[..., b]) * turn
    out[..., a], out[..., b] = z.real, z.imag
    return out
