"""What stands before and after a scan in a block: rotary positions of queries
and keys, and the norm with its gate and residual (include/la.h, la_rotary and
la_gated_norm).  Argument checks and output allocation only; every step runs
in the library's kernels.

Tensors are read and written through their strides (the last dimension dense),
so queries and keys go from projections laid out [B,T,H,D] to the scans'
[B,H,T,D], and the scan's output back, without a copy: pass x.transpose(1, 2).
The scans themselves take contiguous [B,H,T,D]: values, beta, log g and the
gradient of the output are the caller's to lay out.

stream (every call): None, the current one, or a stream that the caller has
ordered behind the inputs; the call runs and allocates on it, and tensors may
be dropped while it runs.
"""
import array
import functools
import math

import torch

from . import (GATE_SIGMOID, GATE_SILU, NORM_L2, NORM_LAYER, NORM_RMS, ROTARY_HALF, ROTARY_INTERLEAVED, _check, _device,
               _dtype_code, _need, _raw_stream, lib)

def _ptr(t):
    return None if t is None else t.data_ptr()


def _check_view(t, name, shape, dtype, device, output=False):
    """The tensor's strides, after the checks that make it a view of rows."""
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name}: expected device {device}, got {t.device}")
    lead = t.stride()
    if lead[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}: the last dimension must be dense")
    if output and 0 in lead and any(k > 1 and s == 0 for k, s in zip(shape[:-1], lead)):
        raise ValueError(f"{name}: an output's rows must not share memory")
    return lead


class _Views:
    """la_view records of a call's tensors, side by side in one buffer (a
    structure object each took as long as the checks)."""

    def __init__(self, shape, dtype, device):
        self.shape, self.dtype, self.device, self.words, self.at = shape, dtype, device, [], []

    def add(self, t, name, output=False, shape=None):
        if t is None:
            self.at.append(None)
            return
        shape = shape if shape is not None else self.shape
        lead = _check_view(t, name, shape, self.dtype, self.device, output)
        self.at.append(len(self.words))
        n = len(shape)
        if n == 4:
            self.words += (t.data_ptr(), lead[0], lead[1], lead[2])
        elif n == 3:  # a batch of rows: its stride may be any, as the first of three
            self.words += (t.data_ptr(), lead[0], 0, lead[1])
        else:
            self.words += (t.data_ptr(), 0, 0, lead[0] if n == 2 else 0)

    def addresses(self):
        """Addresses of the records in the order they were added (None: absent); the buffer lives as long as self."""
        self.buffer = array.array("q", self.words)
        base = self.buffer.buffer_info()[0]
        return [None if i is None else base + 8 * i for i in self.at]


def _rows(x, name="x"):
    if not 1 <= x.dim() <= 4:
        raise ValueError(f"{name}: expected 1 to 4 dimensions, got shape {tuple(x.shape)}")
    if not x.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor, got {x.device}")
    if x.shape[-1] < 1:
        raise ValueError(f"{name}: the last dimension is empty")
    lead = tuple(x.shape[:-1])
    return lead if len(lead) == 3 else (lead[0], 1, lead[1]) if len(lead) == 2 else (1, 1, *lead) if lead else (1, 1, 1)


def gated_norm(x, gate=None, weight=None, residual=None, kind=NORM_RMS, activation=GATE_SILU, eps=1e-5, scale=1.0,
               out=None, stream=None):
    """residual + scale * n(x) * weight * a(gate) over rows of the last
    dimension (la_gated_norm), in fp32 and rounded once.

    x: 1 to 4 dimensions, float32 or bfloat16, any strides with a dense last
    dimension of at most 8192; gate, residual: x's shape and dtype, or None;
    weight: fp32 [D] or None.  kind: NORM_RMS, NORM_LAYER or NORM_L2;
    activation of the gate: GATE_SILU or GATE_SIGMOID.  Returns out (a
    contiguous tensor of x's shape unless given; it may be x, gate or residual
    itself)."""
    n = _rows(x)
    dev, shape, dtype = x.device, x.shape, x.dtype
    D, code = shape[-1], _dtype_code(dtype)
    views = _Views(shape, dtype, dev)
    views.add(x, "x")
    views.add(gate, "gate")
    views.add(residual, "residual")
    _need(weight, "weight", (D,), torch.float32, dev)
    with _device(dev, stream, (x, gate, weight, residual, out)) as output:
        if out is None:
            out = output(torch.empty_like(x, memory_format=torch.contiguous_format))
        views.add(out, "out", True)
        xv, gv, rv, ov = views.addresses()
        _check(lib().la_gated_norm(xv, gv, _ptr(weight), rv, ov, *n, D, kind, activation, eps, scale, code,
                                   _raw_stream(stream, dev)))
    return out


@functools.lru_cache(maxsize=256)
def _norm_workspace_size(n, D):
    return int(lib().la_gated_norm_backward_workspace_size(*n, D))


def gated_norm_backward(dout, x, gate=None, weight=None, kind=NORM_RMS, activation=GATE_SILU, eps=1e-5, scale=1.0,
                        need_weight=True, out=None, stream=None, workspace=None):
    """Gradients of gated_norm for the loss sum(dout * out)
    (la_gated_norm_backward).  Arguments as gated_norm; dout of x's shape and
    dtype.  Returns (dx, dgate, dweight): dx and dgate in x's and the gate's
    shape, dtype and memory order, dweight fp32 [D], summed over the rows;
    dgate is None without a gate, dweight without a weight or
    need_weight=False.  The residual's gradient is dout itself.  out: None,
    or the tuple of outputs preallocated."""
    n = _rows(x)
    dev, shape, dtype = x.device, x.shape, x.dtype
    D, code = shape[-1], _dtype_code(dtype)
    if dout is None:
        raise ValueError("dout is required")
    if out is not None:
        dx, dgate, dweight = out
        if dx is None or (dgate is None) != (gate is None) or (dweight is not None and weight is None):
            raise ValueError("out: dx and, with a gate, dgate are always written; dweight needs a weight")
    views = _Views(shape, dtype, dev)
    views.add(dout, "dout")
    views.add(x, "x")
    views.add(gate, "gate")
    _need(weight, "weight", (D,), torch.float32, dev)
    with _device(dev, stream, (dout, x, gate, weight, workspace, *(out or ()))) as output:
        if out is None:
            dx = output(torch.empty_like(x))
            dgate = output(torch.empty_like(gate)) if gate is not None else None
            dweight = output(torch.empty_like(weight)) if weight is not None and need_weight else None
        views.add(dx, "dx", True)
        views.add(dgate, "dgate", True)
        dv, xv, gv, dxv, dgv = views.addresses()
        _need(dweight, "dweight", (D,), torch.float32, dev)
        if workspace is not None:
            if workspace.device != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
                raise ValueError("workspace: expected a contiguous uint8 tensor on the inputs' device")
        elif dweight is not None:
            workspace = torch.empty(max(_norm_workspace_size(n, D), 1), dtype=torch.uint8, device=dev)
        _check(lib().la_gated_norm_backward(
            dv, xv, gv, _ptr(weight), dxv, dgv, _ptr(dweight), *n, D, kind, activation, eps, scale, code, _ptr(workspace),
            0 if workspace is None else workspace.numel(), _raw_stream(stream, dev)))
    return dx, dgate, dweight


def rotary(x, freq, positions=None, x2=None, start=0, layout=ROTARY_HALF, mscale=1.0, backward=False, out=None, out2=None,
           stream=None):
    """Rotary positions (la_rotary) of x [B,H,T,D] and, in the same launch, of
    x2 [B,H2,T,D] (queries and keys); float32 or bfloat16, any strides with a
    dense last dimension.

    freq: fp32 [R/2], the pairs' inverse frequencies (rotary_frequencies); the
    first R elements of each row turn, the rest is copied.  positions: None
    (token t is at start + t), or int64 [T] or [B,T], up to 2^53 either way.  layout: ROTARY_HALF or
    ROTARY_INTERLEAVED.  mscale: factor of the rotated part.  backward: the
    transposed map, which takes the outputs' gradients to the inputs'.
    Returns out, or (out, out2) with x2: contiguous unless given; each may be
    its input itself."""
    if x.dim() != 4 or not x.is_cuda:
        raise ValueError(f"x: expected a [B,H,T,D] CUDA tensor, got {tuple(x.shape)} on {x.device}")
    B, H, T, D = x.shape
    dev, code = x.device, _dtype_code(x.dtype)
    if freq.dim() != 1:
        raise ValueError(f"freq: expected one dimension, got shape {tuple(freq.shape)}")
    R = 2 * freq.shape[0]
    if not 2 <= R <= D:
        raise ValueError(f"freq: {freq.shape[0]} pairs do not fit rows of {D}")
    _need(freq, "freq", (R // 2,), torch.float32, dev)
    H2 = 0
    if x2 is not None:
        if x2.dim() != 4:
            raise ValueError(f"x2: expected [B,H2,T,D], got {tuple(x2.shape)}")
        H2 = x2.shape[1]
    elif out2 is not None:
        raise ValueError("out2 without x2")
    pstride = 0
    if positions is not None:
        if positions.shape != (B, T) and positions.shape != (T,):
            raise ValueError(f"positions: expected shape {(T,)} or {(B, T)}, got {tuple(positions.shape)}")
        if positions.dtype != torch.int64:
            raise TypeError(f"positions: expected int64, got {positions.dtype}")
        if positions.device != dev:
            raise ValueError(f"positions: expected device {dev}, got {positions.device}")
        if T > 1 and positions.stride(-1) != 1:
            raise ValueError("positions: the last dimension must be dense")
        if start != 0:
            raise ValueError("start applies only without positions")
        pstride = positions.stride(0) if positions.dim() == 2 and B > 1 else 0
    elif not -(1 << 53) <= start <= (1 << 53) - T:
        raise ValueError(f"start: positions {start} .. {start} + {T} exceed 2^53")
    shape, shape2, dtype = (B, H, T, D), (B, H2, T, D), x.dtype
    views = _Views(shape, dtype, dev)
    views.add(x, "x")
    views.add(x2, "x2", shape=shape2)
    with _device(dev, stream, (x, x2, freq, positions, out, out2)) as output:
        if out is None:
            out = output(torch.empty_like(x, memory_format=torch.contiguous_format))
        if out2 is None and x2 is not None:
            out2 = output(torch.empty_like(x2, memory_format=torch.contiguous_format))
        views.add(out, "out", True)
        views.add(out2, "out2", True, shape2)
        xv, xv2, ov, ov2 = views.addresses()
        _check(lib().la_rotary(xv, H, xv2, H2, ov, ov2, freq.data_ptr(), _ptr(positions), pstride, start, B, T, D, R, layout,
                               mscale, 1 if backward else 0, code, _raw_stream(stream, dev)))
    return (out, out2) if x2 is not None else out


def rotary_frequencies(rot_dim, base=10000.0, scaling="none", factor=1.0, trained_length=None, fast=32.0, slow=1.0,
                       device=None):
    """Inverse frequencies base^(-2 i / rot_dim) of the rot_dim / 2 pairs, and
    the magnitude factor for rotary's mscale, for contexts up to `factor`
    times the trained length:

      "none"    as trained.
      "linear"  every frequency divided by factor (positions interpolated).
      "ntk"     the base raised to base * factor^(rot_dim / (rot_dim - 2)): the
                fastest pair unchanged, the slowest stretched by factor.
      "yarn"    per pair: at least `fast` turns within trained_length keep their
                frequency, at most `slow` turns take frequency / factor, a linear
                ramp between; magnitude 0.1 ln(factor) + 1.

    Computed in 64 bits, rounded once.  Returns (freq fp32 [rot_dim / 2], mscale)."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError(f"rot_dim: expected an even number of at least 2, got {rot_dim}")
    if base <= 0 or factor < 1:
        raise ValueError("base must be positive and factor at least 1")
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    if scaling == "ntk":
        # a single pair has frequency 1 whatever the base
        base = base * factor ** (rot_dim / (rot_dim - 2)) if rot_dim > 2 else base
    freq, mscale = base ** (-2 * i / rot_dim), 1.0
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "yarn":
        if trained_length is None or trained_length <= 0 or not fast > slow:
            raise ValueError("yarn needs the trained length, and fast above slow")
        keep = ((trained_length * freq / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        freq = freq / factor * (1 - keep) + freq * keep
        mscale = 0.1 * math.log(factor) + 1.0
    elif scaling not in ("none", "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return freq.float().to(device), mscale
