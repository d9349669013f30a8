"""The gated delta rule: whole sequence, gradients, one token (include/la.h,
la_delta_*).  Argument checks and output allocation only; every step runs in
the library's kernels.

    S' = g_t S_{t-1}    e_t = v_t - S'^T k_t    S_t = S' + k_t (beta_t e_t)^T    y_t = q_scale S_t^T q_t
"""
import ctypes
import functools

import torch

from . import (DECAY_NONE, DECAY_PER_HEAD, DECAY_PER_STEP, _check, _decay, _device, _dtype_code, _need, _raw_stream, lib)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _heads(q, k, v, beta, decay_kind, log_g, token):
    """Sizes (B, H, Hk, T, Dk, Dv) after the shape, dtype and device checks;
    token: one-token tensors, without the T dimension."""
    want = 3 if token else 4
    if q.dim() != want or k.dim() != want or v.dim() != want:
        raise ValueError(f"q, k, v: expected {want} dimensions, got {tuple(q.shape)}, {tuple(k.shape)}, {tuple(v.shape)}")
    if not q.is_cuda:
        raise ValueError(f"q: expected a CUDA tensor, got {q.device}")
    if beta is None:
        raise ValueError("beta is required")
    shape, vshape, dev, dtype = q.shape, v.shape, q.device, q.dtype
    B, Hk, Dk = shape[0], shape[1], shape[-1]
    H, Dv = vshape[1], vshape[-1]
    if H and (Hk == 0 or H % Hk):
        raise ValueError(f"v has {H} heads, which is not a multiple of q's {Hk}")
    _dtype_code(dtype)
    per_token = vshape[:-1]
    _need(q, "q", shape, dtype, dev)
    _need(k, "k", shape, dtype, dev)
    _need(v, "v", (B, H, Dv) if token else (B, H, shape[2], Dv), dtype, dev)
    _need(beta, "beta", per_token, torch.float32, dev)
    if decay_kind != DECAY_NONE:
        if log_g is None:
            raise ValueError("log_g is required for a per-head or per-step decay")
        if decay_kind == DECAY_PER_STEP:
            _need(log_g, "log_g", per_token, torch.float32, dev)
        elif decay_kind == DECAY_PER_HEAD:
            _need(log_g, "log_g", (H,), torch.float32, dev)
        else:
            raise ValueError(f"unknown decay kind {decay_kind}")
    return B, H, Hk, (1 if token else shape[2]), Dk, Dv


def _scratch(workspace, nbytes, dev):
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace: expected a contiguous uint8 tensor on the inputs' device")
    return workspace


@functools.lru_cache(maxsize=256)
def _size(backward, *sizes):
    L = lib()
    return int((L.la_delta_backward_workspace_size if backward else L.la_delta_workspace_size)(*sizes))


def delta_workspace_size(B, H, T, Dk, Dv, dtype=torch.bfloat16, key_heads=None):
    """Scratch bytes delta_forward needs (la_delta_workspace_size)."""
    return _size(False, B, H, key_heads or H, T, Dk, Dv, _dtype_code(dtype))


def delta_forward(q, k, v, beta, decay_kind=DECAY_NONE, log_g=None, init_state=None, q_scale=1.0, out=None,
                  final_state=None, return_final=True, stream=None, workspace=None):
    """Whole-sequence gated delta rule (la_delta_forward_ws).

    q, k: [B,Hk,T,Dk]; v: [B,H,T,Dv], H a multiple of Hk (key head j serves
    value heads j H / Hk and the ones after it); float32 or bfloat16 CUDA
    tensors.  beta [B,H,T] fp32; decay_kind / log_g as chunk_forward;
    init_state [B,H,Dk,Dv] fp32 or None.  Returns (out [B,H,T,Dv],
    final_state or None).  stream: None, the current one, or a stream that the
    caller has ordered behind the inputs; the call runs and allocates on it, and
    tensors may be dropped while it runs.  workspace: None allocates it with
    torch on that stream, or a CUDA uint8 tensor of at least
    delta_workspace_size(...) bytes."""
    B, H, Hk, T, Dk, Dv = _heads(q, k, v, beta, decay_kind, log_g, token=False)
    dev = q.device
    _need(init_state, "init_state", (B, H, Dk, Dv), torch.float32, dev)
    _need(out, "out", v.shape, q.dtype, dev)
    _need(final_state, "final_state", (B, H, Dk, Dv), torch.float32, dev)
    d = _decay(decay_kind, log_g)
    with _device(dev, stream, (q, k, v, beta, log_g, init_state, out, final_state, workspace)) as output:
        if out is None:
            out = output(torch.empty_like(v))
        if final_state is None and return_final:
            final_state = output(torch.empty((B, H, Dk, Dv), dtype=torch.float32, device=dev))
        workspace = _scratch(workspace, delta_workspace_size(B, H, T, Dk, Dv, q.dtype, Hk), dev)
        _check(lib().la_delta_forward_ws(
            _ptr(q), _ptr(k), _ptr(v), _ptr(beta), ctypes.byref(d) if d is not None else None, float(q_scale),
            _ptr(init_state), _ptr(out), _ptr(final_state), B, H, Hk, T, Dk, Dv, _dtype_code(q.dtype),
            _ptr(workspace), workspace.numel(), _raw_stream(stream, dev)))
    return out, final_state


def delta_backward_workspace_size(B, H, T, Dk, Dv, dtype=torch.bfloat16, key_heads=None,
                                  decay_kind=DECAY_PER_HEAD):
    """Scratch bytes delta_backward needs (la_delta_backward_workspace_size): by default for any decay."""
    return _size(True, B, H, key_heads or H, T, Dk, Dv, _dtype_code(dtype), decay_kind)


def delta_backward(q, k, v, beta, dy, decay_kind=DECAY_NONE, log_g=None, init_state=None, d_final_state=None,
                   q_scale=1.0, need_log_g=True, need_init_state=True, stream=None, workspace=None, out=None):
    """Gradients of delta_forward (la_delta_backward_ws) for the loss
    sum(dy * y) + sum(d_final_state * final_state).

    Arguments as delta_forward, plus dy [B,H,T,Dv] in the inputs' dtype and
    d_final_state [B,H,Dk,Dv] fp32 or None.  Returns (dq, dk, dv, dbeta,
    d_log_g, d_init_state): dq, dk (summed over shared heads) and dv in the
    input dtype, dbeta fp32, d_log_g fp32 with log_g's shape (None without a
    decay or need_log_g=False), d_init_state fp32 (None with
    need_init_state=False).  workspace: None, or a CUDA uint8 tensor of at
    least delta_backward_workspace_size(...) bytes.  out: None, or a tuple of
    the six outputs preallocated (the last two may be None to skip them)."""
    B, H, Hk, T, Dk, Dv = _heads(q, k, v, beta, decay_kind, log_g, token=False)
    dev = q.device
    if dy is None:
        raise ValueError("dy is required")
    _need(dy, "dy", (B, H, T, Dv), q.dtype, dev)
    _need(init_state, "init_state", (B, H, Dk, Dv), torch.float32, dev)
    _need(d_final_state, "d_final_state", (B, H, Dk, Dv), torch.float32, dev)
    if out is not None:
        dq, dk, dv, dbeta, d_log_g, d_init = out
        if any(x is None for x in (dq, dk, dv, dbeta)):
            raise ValueError("out: dq, dk, dv and dbeta are always written")
        if d_log_g is not None and decay_kind == DECAY_NONE:
            raise ValueError("d_log_g: there is no decay")
        _need(dq, "dq", (B, Hk, T, Dk), q.dtype, dev)
        _need(dk, "dk", (B, Hk, T, Dk), q.dtype, dev)
        _need(dv, "dv", (B, H, T, Dv), q.dtype, dev)
        _need(dbeta, "dbeta", (B, H, T), torch.float32, dev)
        if d_log_g is not None:
            _need(d_log_g, "d_log_g", tuple(log_g.shape), torch.float32, dev)
        _need(d_init, "d_init_state", (B, H, Dk, Dv), torch.float32, dev)
    d = _decay(decay_kind, log_g)
    with _device(dev, stream, (q, k, v, beta, dy, log_g, init_state, d_final_state, workspace, *(out or ()))) as output:
        if out is None:
            dq, dk, dv, dbeta = (output(torch.empty_like(x)) for x in (q, k, v, beta))
            d_log_g = output(torch.empty_like(log_g)) if decay_kind != DECAY_NONE and need_log_g else None
            d_init = output(torch.empty((B, H, Dk, Dv), dtype=torch.float32, device=dev)) if need_init_state else None
        workspace = _scratch(workspace, delta_backward_workspace_size(B, H, T, Dk, Dv, q.dtype, Hk, decay_kind), dev)
        _check(lib().la_delta_backward_ws(
            _ptr(q), _ptr(k), _ptr(v), _ptr(beta), ctypes.byref(d) if d is not None else None, float(q_scale),
            _ptr(init_state), _ptr(dy), _ptr(d_final_state), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dbeta), _ptr(d_log_g),
            _ptr(d_init), B, H, Hk, T, Dk, Dv, _dtype_code(q.dtype), _ptr(workspace), workspace.numel(),
            _raw_stream(stream, dev)))
    return dq, dk, dv, dbeta, d_log_g, d_init


def delta_decode_step(q, k, v, beta, state, decay_kind=DECAY_NONE, log_g=None, q_scale=1.0, out=None, stream=None):
    """One token of the gated delta rule (la_delta_decode_step); state
    [B,H,Dk,Dv] fp32 is updated in place.  q, k: [B,Hk,Dk]; v: [B,H,Dv];
    beta [B,H] fp32; log_g [H] or [B,H].  Returns out [B,H,Dv]."""
    B, H, Hk, _, Dk, Dv = _heads(q, k, v, beta, decay_kind, log_g, token=True)
    dev = q.device
    if state is None:
        raise ValueError("state is required")
    _need(state, "state", (B, H, Dk, Dv), torch.float32, dev)
    _need(out, "out", v.shape, q.dtype, dev)
    d = _decay(decay_kind, log_g)
    with _device(dev, stream, (q, k, v, beta, log_g, state, out)) as output:
        if out is None:
            out = output(torch.empty_like(v))
        _check(lib().la_delta_decode_step(
            _ptr(q), _ptr(k), _ptr(v), _ptr(beta), ctypes.byref(d) if d is not None else None, float(q_scale),
            _ptr(state), _ptr(out), B, H, Hk, Dk, Dv, _dtype_code(q.dtype), _raw_stream(stream, dev)))
    return out
