"""The gated delta rule in float64 numpy, token by token from its definition,
and its gradients by the chain rule through the same steps.

    S' = g_t S_{t-1}    e_t = v_t - S'^T k_t    S_t = S' + k_t (beta_t e_t)^T    y_t = scale S_t^T q_t
"""
import numpy as np


def _f64(a):
    if a is None:
        return None
    if hasattr(a, "detach"):
        a = a.detach().to("cpu").double().numpy()
    return np.ascontiguousarray(a, dtype=np.float64)


def _inputs(q, k, v, beta, kind, log_g, init_state):
    q, k, v, beta, log_g = (_f64(x) for x in (q, k, v, beta, log_g))
    B, H, T, Dv = v.shape
    rep = H // q.shape[1]
    q, k = np.repeat(q, rep, 1), np.repeat(k, rep, 1)
    lg = np.zeros((B, H, T))
    if kind == 1:
        lg = np.broadcast_to(log_g[None, :, None], (B, H, T))
    elif kind == 2:
        lg = log_g
    S = np.zeros((B, H, q.shape[-1], Dv)) if init_state is None else _f64(init_state).copy()
    return q, k, v, beta, np.exp(lg), S, rep


def delta_forward(q, k, v, beta, kind=0, log_g=None, init_state=None, scale=1.0):
    """q, k [B,Hk,T,Dk]; v [B,H,T,Dv]; beta [B,H,T].  Returns (y, final_state)."""
    q, k, v, beta, g, S, _ = _inputs(q, k, v, beta, kind, log_g, init_state)
    y = np.zeros_like(v)
    for t in range(v.shape[2]):
        S = g[:, :, t, None, None] * S
        e = v[:, :, t] - np.einsum("bhij,bhi->bhj", S, k[:, :, t])
        S = S + k[:, :, t, :, None] * (beta[:, :, t, None] * e)[:, :, None, :]
        y[:, :, t] = scale * np.einsum("bhij,bhi->bhj", S, q[:, :, t])
    return y, S


def delta_backward(q, k, v, beta, dy, kind=0, log_g=None, init_state=None, d_final_state=None, scale=1.0):
    """Gradients of sum(dy y) + <d_final_state, S_T>: (dq, dk, dv, dbeta,
    d_log_g or None, d_init_state), dq and dk summed over shared heads."""
    q, k, v, beta, g, S, rep = _inputs(q, k, v, beta, kind, log_g, init_state)
    dy = _f64(dy)
    T = v.shape[2]
    decayed, errors = [], []
    for t in range(T):
        S = g[:, :, t, None, None] * S
        e = v[:, :, t] - np.einsum("bhij,bhi->bhj", S, k[:, :, t])
        decayed.append(S)
        errors.append(e)
        S = S + k[:, :, t, :, None] * (beta[:, :, t, None] * e)[:, :, None, :]
    dq, dk, dv, dbeta, dlog = (np.zeros_like(x) for x in (q, k, v, beta, beta))
    G = np.zeros_like(S) if d_final_state is None else _f64(d_final_state).copy()
    for t in range(T - 1, -1, -1):
        kt, e, bt = k[:, :, t], errors[t], beta[:, :, t, None]
        St = decayed[t] + kt[..., None] * (bt * e)[:, :, None, :]
        dq[:, :, t] = scale * np.einsum("bhij,bhj->bhi", St, dy[:, :, t])
        G = G + scale * q[:, :, t, :, None] * dy[:, :, t, None, :]
        du = np.einsum("bhij,bhi->bhj", G, kt)
        dbeta[:, :, t] = (du * e).sum(-1)
        de = bt * du
        dv[:, :, t] = de
        dk[:, :, t] = np.einsum("bhij,bhj->bhi", G, bt * e) - np.einsum("bhij,bhj->bhi", decayed[t], de)
        G = G - kt[..., None] * de[:, :, None, :]
        dlog[:, :, t] = (G * decayed[t]).sum((-1, -2))
        G = g[:, :, t, None, None] * G
    if rep > 1:
        dq, dk = (x.reshape(x.shape[0], -1, rep, *x.shape[2:]).sum(2) for x in (dq, dk))
    d_log_g = None if kind == 0 else dlog.sum((0, 2)) if kind == 1 else dlog
    return dq, dk, dv, dbeta, d_log_g, G


def delta_decode_step(q, k, v, beta, state, kind=0, log_g=None, scale=1.0):
    """One token; q, k [B,Hk,Dk], v [B,H,Dv], beta [B,H].  Returns (y, new_state)."""
    if kind == 2:
        log_g = _f64(log_g)[:, :, None]
    y, S = delta_forward(*(_f64(x)[:, :, None] for x in (q, k, v, beta)), kind, log_g, state, scale)
    return y[:, :, 0], S
