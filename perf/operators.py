"""The operators that surround and replace the decayed scan in a linear-attention
block, as they are measured: the gated delta rule (whole sequence, its gradients,
one token), the norm with gate and residual that follows the scan, and the rotary
positions that precede it.

`listed()` and `draw()` give cases, `prepare()` what a program has in hand before
the call, `run()` one call: elementary torch operations where `own` is false, the
library's calls where it is true.  `exact()` evaluates each operator from its
definition, token by token, in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # Long-context prefill of one sequence: few heads, all the parallelism along T.
        dict(name="delta_prefill_t65536", op="delta", dtype="bf16", B=1, H=32, Hk=32, T=65536, Dk=128, Dv=128,
             decay="step", init=False, pad=0),
        # A serving batch that continues from a carried state, two value heads to a key head.
        dict(name="delta_batch_t4096_grouped", op="delta", dtype="bf16", B=8, H=16, Hk=8, T=4096, Dk=128, Dv=128,
             decay="step", init=True, pad=0),
        # A short odd fp32 sequence with odd widths, retention's decay per head.
        dict(name="delta_odd_f32_t777", op="delta", dtype="f32", B=2, H=4, Hk=4, T=777, Dk=60, Dv=52,
             decay="head", init=True, pad=0),
        # The training step's gradients at the usual training length.
        dict(name="delta_grad_t4096", op="delta_grad", dtype="bf16", B=2, H=16, Hk=16, T=4096, Dk=128, Dv=128,
             decay="step", init=False, pad=0),
        # Gradients of a padded ragged batch with shared key heads and gradients of both states.
        dict(name="delta_grad_ragged_t501", op="delta_grad", dtype="bf16", B=3, H=6, Hk=2, T=501, Dk=64, Dv=80,
             decay="step", init=True, pad=37),
        # One token for a full serving batch: the fp32 states cross HBM once each way.
        dict(name="delta_decode_b256", op="delta_decode", dtype="bf16", B=256, H=32, Hk=32, Dk=128, Dv=128, decay="head"),
        # One token of one user: the smallest call, where latency counts.
        dict(name="delta_decode_b1", op="delta_decode", dtype="bf16", B=1, H=8, Hk=4, Dk=64, Dv=64, decay="step"),
        # The scan's output [B,H,T,D], normalised per head and gated, laid out [B,T,H,D] for the output projection.
        dict(name="norm_heads_t4096", op="norm", dtype="bf16", shape="heads", B=8, H=16, T=4096, D=128, kind="rms",
             act="silu", weight=True, residual=False),
        # Its gradients in a training step.
        dict(name="norm_heads_grad_t4096", op="norm_grad", dtype="bf16", shape="heads", B=4, H=16, T=4096, D=128,
             kind="rms", act="silu", weight=True, residual=False),
        # The norm after a block over the model width, fused with the scaled residual.
        dict(name="norm_wide_residual", op="norm", dtype="bf16", shape="rows", B=3, H=1, T=1023, D=2048, kind="layer",
             act="none", weight=True, residual=True),
        # Queries and keys of a training batch, rotated on their way from the projections' layout to the scan's.
        dict(name="rotary_t4096", op="rotary", dtype="bf16", B=8, H=16, Hk=16, T=4096, D=128, R=128, layout="half",
             where="arange", scaling="none"),
        # One far token each for a serving batch: positions per sequence, half of the head rotated, scaled frequencies.
        dict(name="rotary_token_far", op="rotary", dtype="bf16", B=64, H=32, Hk=8, T=1, D=128, R=64,
             layout="interleaved", where="far", scaling="yarn"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["delta", "delta", "delta_grad", "delta_grad", "delta_decode", "norm", "norm_grad", "rotary"])
    if op.startswith("delta"):
        dtype = "f32" if rng.random() < 0.25 else "bf16"
        Hk = rng.choice([1, 2, 3, 4, 8, 16])
        H = Hk * rng.choice([1, 1, 2, 3])
        width = (lambda: rng.choice([16, 32, 48, 64, 80, 96, 112, 128, 128])) if dtype == "bf16" else \
            (lambda: rng.randint(12, 128))
        c = dict(op=op, dtype=dtype, H=H, Hk=Hk, Dk=width(), Dv=width(), decay=rng.choice(["none", "head", "step", "step"]))
        if op == "delta_decode":
            return dict(c, B=_log_int(rng, 1, max(1, 4096 // H)))
        most = (1 << 17 if dtype == "bf16" else 1 << 14) * (4 if op == "delta" else 1)
        c["B"] = rng.randint(1, 4)
        c["T"] = _log_int(rng, 1, min(4096 if op == "delta_grad" else 16384, most // (c["B"] * H)))
        c["init"] = rng.random() < 0.5
        c["pad"] = rng.randint(0, c["T"] // 4)
        return c
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("norm"):
        c = dict(op=op, dtype=dtype, kind=rng.choice(["rms", "layer", "l2"]), act=rng.choice(["none", "silu", "sigmoid"]),
                 weight=rng.random() < 0.7, residual=rng.random() < 0.4)
        if rng.random() < 0.6:
            return dict(c, shape="heads", B=rng.randint(1, 4), H=rng.randint(1, 20), T=_log_int(rng, 1, 4096),
                        D=rng.randint(8, 128))
        return dict(c, shape="rows", B=rng.randint(1, 4), H=1, T=_log_int(rng, 1, 2048), D=_log_int(rng, 64, 8192))
    D = 2 * rng.randint(4, 64)
    return dict(op=op, dtype=dtype, B=rng.randint(1, 8), H=rng.randint(1, 16), Hk=rng.randint(1, 16),
                T=_log_int(rng, 1, 4096), D=D, R=2 * rng.randint(1, D // 2), layout=rng.choice(["half", "interleaved"]),
                where=rng.choice(["arange", "far", "offset"]), scaling=rng.choice(["none", "linear", "ntk", "yarn"]))


# ------------------------------------------------------------------ inputs
def _frequencies(R, scaling):
    """Inverse frequencies of the rotated pairs (fp32) and the magnitude factor
    of the rotated part: the usual powers of 10000, and the three usual ways to
    stretch them to 8 times the trained length of 4096."""
    i = torch.arange(R // 2, dtype=torch.float64)
    base, factor, trained = 10000.0, 8.0, 4096.0
    if scaling == "ntk":
        base = base * factor ** (R / (R - 2)) if R > 2 else base
    freq, mscale = base ** (-2 * i / R), 1.0
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "yarn":
        turns = trained * freq / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        freq = freq / factor * (1 - keep) + freq * keep
        mscale = 0.1 * math.log(factor) + 1.0
    return freq.float(), mscale


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    c, op = case, case["op"]
    s = dict(case=dict(case))
    if op.startswith("delta"):
        T = (c["T"],) if "T" in c else ()
        B, H, Hk, Dk, Dv = c["B"], c["H"], c["Hk"], c["Dk"], c["Dv"]
        s["q"], s["k"] = (torch.nn.functional.normalize(randn(B, Hk, *T, Dk), dim=-1).to(dt) for _ in range(2))
        s["v"] = randn(B, H, *T, Dv).to(dt)
        beta = torch.sigmoid(randn(B, H, *T))
        s["log_g"] = None
        if c["decay"] == "step":
            s["log_g"] = torch.nn.functional.logsigmoid(4 + randn(B, H, *T))
        elif c["decay"] == "head":
            s["log_g"] = torch.log1p(-torch.exp2(-5 - torch.arange(H, device=DEV, dtype=torch.float64))).float()
        if c.get("pad"):  # a padded tail: it must neither write to the state nor decay it
            beta[..., c["T"] - c["pad"]:] = 0
            if c["decay"] == "step":
                s["log_g"][..., c["T"] - c["pad"]:] = 0
        s["beta"] = beta
        s["scale"] = Dk ** -0.5
        if op == "delta_decode":
            s["state"] = 0.1 * randn(B, H, Dk, Dv)
        else:
            s["init"] = 0.1 * randn(B, H, Dk, Dv) if c["init"] else None
        if op == "delta_grad":
            s["dy"] = randn(B, H, *T, Dv).to(dt)
            s["d_final"] = 0.1 * randn(B, H, Dk, Dv) if c["init"] else None
    elif op.startswith("norm"):
        B, H, Tn, D = c["B"], c["H"], c["T"], c["D"]
        if c["shape"] == "heads":
            x, shape = randn(B, H, Tn, D).to(dt).transpose(1, 2), (B, Tn, H, D)
        else:
            shape = (B, Tn, D)
            x = randn(*shape).to(dt)
        s["x"] = x
        s["gate"] = randn(*shape).to(dt) if c["act"] != "none" else None
        s["weight"] = 1 + 0.2 * randn(D) if c["weight"] else None
        s["residual"] = randn(*shape).to(dt) if c["residual"] else None
        s["eps"], s["scale"] = 1e-5, 0.7 if c["residual"] else 1.0
        if op == "norm_grad":
            s["dout"] = randn(*shape).to(dt)
    else:
        B, H, Hk, Tn, D = c["B"], c["H"], c["Hk"], c["T"], c["D"]
        s["q"] = randn(B, Tn, H, D).to(dt).transpose(1, 2)
        s["k"] = randn(B, Tn, Hk, D).to(dt).transpose(1, 2)
        freq, s["mscale"] = _frequencies(c["R"], c["scaling"])
        s["freq"] = freq.to(DEV)
        if c["where"] == "far":  # each sequence at its own place in a long context
            start = torch.randint(0, 1 << 20, (B, 1), generator=g, device=DEV)
            s["pos"], s["start"] = start + torch.arange(Tn, device=DEV), 0
        else:
            s["pos"], s["start"] = None, 100_000 if c["where"] == "offset" else 0
    return s


# ------------------------------------------------------------------ the calls of the library
def _run_own(s):
    import retention_scan_b200 as la
    c, op = s["case"], s["case"]["op"]
    decay = {"none": la.DECAY_NONE, "head": la.DECAY_PER_HEAD, "step": la.DECAY_PER_STEP}
    if op == "delta":
        return la.delta_forward(s["q"], s["k"], s["v"], s["beta"], decay[c["decay"]], s["log_g"], init_state=s["init"],
                                q_scale=s["scale"])
    if op == "delta_grad":
        return la.delta_backward(s["q"], s["k"], s["v"], s["beta"], s["dy"], decay[c["decay"]], s["log_g"],
                                 init_state=s["init"], d_final_state=s["d_final"], q_scale=s["scale"])
    if op == "delta_decode":
        out = la.delta_decode_step(s["q"], s["k"], s["v"], s["beta"], s["state"], decay[c["decay"]], s["log_g"],
                                   q_scale=s["scale"])
        return out, s["state"]
    if op.startswith("norm"):
        how = dict(kind={"rms": la.NORM_RMS, "layer": la.NORM_LAYER, "l2": la.NORM_L2}[c["kind"]],
                   activation=la.GATE_SIGMOID if c["act"] == "sigmoid" else la.GATE_SILU, eps=s["eps"], scale=s["scale"])
        if op == "norm":
            return la.gated_norm(s["x"], s["gate"], s["weight"], s["residual"], **how)
        return la.gated_norm_backward(s["dout"], s["x"], s["gate"], s["weight"], **how)
    return la.rotary(s["q"], s["freq"], s["pos"], s["k"], start=s["start"], mscale=s["mscale"],
                     layout=la.ROTARY_HALF if c["layout"] == "half" else la.ROTARY_INTERLEAVED)


def run(state):
    if own:
        return _run_own(state)
    return {"delta": _plain_delta, "delta_grad": _plain_delta_grad, "delta_decode": _plain_decode,
            "norm": _plain_norm, "norm_grad": _plain_norm_grad, "rotary": _plain_rotary}[state["case"]["op"]](state)


# ------------------------------------------------------------------ plain forms
CHUNK = 64


def _heads(x, H):
    """[B,Hk,...] -> [B,H,...]: every key head serves H / Hk consecutive value heads."""
    return x.repeat_interleave(H // x.shape[1], 1) if x.shape[1] != H else x


def _chunks(x, n):
    """[B,H,T,...] -> fp32 [B,H,n,CHUNK,...], zeros behind the last token."""
    x = x.float()
    out = x.new_zeros(x.shape[:2] + (n * CHUNK,) + x.shape[3:])
    out[:, :, :x.shape[2]] = x
    return out.reshape(x.shape[:2] + (n, CHUNK) + x.shape[3:])


class _Chunked:
    """What both directions of the plain delta rule share: the operands in
    chunks, the decays within a chunk, and E = (I + A B)^-1 as a matrix, with
    A_ts = exp(L_t - L_s) k_t.k_s below the diagonal and B = diag(beta)."""

    def __init__(self, s):
        q, k, v = s["q"], s["k"], s["v"]
        B, H, T, Dv = v.shape
        n = (T + CHUNK - 1) // CHUNK
        self.n, self.T, self.shape = n, T, (B, H, k.shape[-1], Dv)
        log_g = s["log_g"]
        if log_g is None:
            log_g = v.new_zeros((B, H, T), dtype=torch.float32)
        elif log_g.dim() == 1:
            log_g = log_g[None, :, None].expand(B, H, T)
        self.q, self.k, self.v = _chunks(_heads(q, H), n), _chunks(_heads(k, H), n), _chunks(v, n)
        self.beta = _chunks(s["beta"], n)
        L = _chunks(log_g, n).double().cumsum(-1)  # a difference of long sums: in 64 bits
        self.gamma = L.exp().float()
        self.rest = (L[..., -1:] - L).exp().float()
        self.total = self.gamma[..., -1, None, None]
        lower = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=v.device).tril()
        self.strict = lower.tril(-1)
        D = (L[..., :, None] - L[..., None, :]).masked_fill(~lower, -torch.inf).exp().float()
        self.D = D
        self.kk = self.k @ self.k.transpose(-1, -2)
        self.P = (self.q @ self.k.transpose(-1, -2)) * D * s["scale"]
        self.A = self.kk * D * self.strict
        N = self.A * self.beta[..., None, :]
        E = torch.eye(CHUNK, device=v.device).expand_as(N).contiguous()
        for t in range(1, CHUNK):  # forward substitution, a row at a time
            E[..., t, :t] = -(N[..., t, None, :t] @ E[..., :t, :t]).squeeze(-2)
        self.E = E

    def flat(self, x):
        return x.reshape(x.shape[:2] + (self.n * CHUNK,) + x.shape[4:])[:, :, :self.T]


def _scan_states(c, init):
    """The chunks' incoming states, their prediction errors and the last state."""
    S = init.clone() if init is not None else c.v.new_zeros(c.shape)
    states, errors = [], []
    for i in range(c.n):
        states.append(S)
        e = c.E[:, :, i] @ (c.v[:, :, i] - c.gamma[:, :, i, :, None] * (c.k[:, :, i] @ S))
        errors.append(e)
        S = c.total[:, :, i] * S + (c.k[:, :, i] * c.rest[:, :, i, :, None]).transpose(-1, -2) @ \
            (c.beta[:, :, i, :, None] * e)
    return states, errors, S


def _plain_delta(s):
    c = _Chunked(s)
    S = s["init"].clone() if s["init"] is not None else c.v.new_zeros(c.shape)
    y = torch.empty_like(c.v)
    for i in range(c.n):
        u = c.E[:, :, i] @ (c.v[:, :, i] - c.gamma[:, :, i, :, None] * (c.k[:, :, i] @ S)) * c.beta[:, :, i, :, None]
        y[:, :, i] = s["scale"] * c.gamma[:, :, i, :, None] * (c.q[:, :, i] @ S) + c.P[:, :, i] @ u
        S = c.total[:, :, i] * S + (c.k[:, :, i] * c.rest[:, :, i, :, None]).transpose(-1, -2) @ u
    return c.flat(y).to(s["v"].dtype), S


def _plain_delta_grad(s):
    c = _Chunked(s)
    H, Hk = s["v"].shape[1], s["q"].shape[1]
    states, errors, S_end = _scan_states(c, s["init"])
    dy = _chunks(s["dy"], c.n)
    dS = s["d_final"].clone() if s["d_final"] is not None else torch.zeros_like(S_end)
    ends, dus, des = [None] * c.n, [None] * c.n, [None] * c.n
    for i in reversed(range(c.n)):
        ends[i] = dS
        du = c.P[:, :, i].transpose(-1, -2) @ dy[:, :, i] + c.rest[:, :, i, :, None] * (c.k[:, :, i] @ dS)
        de = c.E[:, :, i].transpose(-1, -2) @ (c.beta[:, :, i, :, None] * du)
        dus[i], des[i] = du, de
        g = c.gamma[:, :, i, :, None]
        dS = c.total[:, :, i] * dS + (c.q[:, :, i] * (g * s["scale"])).transpose(-1, -2) @ dy[:, :, i] \
            - (c.k[:, :, i] * g).transpose(-1, -2) @ de
    S, dSe, e, du, de = (torch.stack(x, 2) for x in (states, ends, errors, dus, des))
    u = c.beta[..., None] * e
    dP = (dy @ u.transpose(-1, -2)) * c.D * s["scale"]
    dN = -(de @ e.transpose(-1, -2)) * c.strict  # gradient of A B
    dA = dN * c.D * c.beta[..., None, :]
    dq = s["scale"] * c.gamma[..., None] * (dy @ S.transpose(-1, -2)) + dP @ c.k
    dk_row = dA @ c.k - c.gamma[..., None] * (de @ S.transpose(-1, -2))
    dk_col = dP.transpose(-1, -2) @ c.q + dA.transpose(-1, -2) @ c.k + c.rest[..., None] * (u @ dSe.transpose(-1, -2))
    dbeta = (e * du).sum(-1) + (dN * c.A).sum(-2)
    dlog = None
    if s["log_g"] is not None:
        dL = ((c.q * dq).sum(-1) + (c.k * (dk_row - dk_col)).sum(-1)).double()
        after = torch.cat([S[:, :, 1:], S_end[:, :, None]], 2)  # the chunks' outgoing states
        dL[..., -1] += (after.double() * dSe.double()).sum((-1, -2))
        dlog = c.flat(dL.flip(-1).cumsum(-1).flip(-1))
        dlog = (dlog.sum((0, 2)) if s["log_g"].dim() == 1 else dlog).float()
    dq, dk = (c.flat(x).unflatten(1, (Hk, H // Hk)).sum(2).to(s["q"].dtype) for x in (dq, dk_row + dk_col))
    return dq, dk, c.flat(de).to(s["v"].dtype), c.flat(dbeta), dlog, dS


def _plain_decode(s):
    H = s["v"].shape[1]
    q, k, v = _heads(s["q"].float(), H), _heads(s["k"].float(), H), s["v"].float()
    S = s["state"]
    if s["log_g"] is not None:
        S.mul_(s["log_g"].exp()[..., None, None])
    e = v - (k[..., None] * S).sum(-2)
    S.add_(k[..., None] * (s["beta"][..., None] * e)[..., None, :])
    return (s["scale"] * (q[..., None] * S).sum(-2)).to(s["v"].dtype), S


def _plain_norm_parts(s):
    x, kind = s["x"].float(), s["case"]["kind"]
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    ss = x.square().sum(-1, keepdim=True) if kind == "l2" else x.square().mean(-1, keepdim=True)
    r = (ss + s["eps"]).rsqrt()
    n = x * r
    w = s["weight"] if s["weight"] is not None else torch.ones((), device=x.device)
    if s["gate"] is None:
        return n, r, w, torch.ones((), device=x.device), None
    z = s["gate"].float()
    sig = 1 / (1 + (-z).exp())
    return (n, r, w, z * sig, sig * (1 + z * (1 - sig))) if s["case"]["act"] == "silu" else (n, r, w, sig, sig * (1 - sig))


def _plain_norm(s):
    n, _, w, a, _ = _plain_norm_parts(s)
    out = s["scale"] * n * w * a
    return (out + s["residual"].float() if s["residual"] is not None else out).to(s["x"].dtype)


def _plain_norm_grad(s):
    n, r, w, a, da = _plain_norm_parts(s)
    kind, dt = s["case"]["kind"], s["x"].dtype
    m = s["scale"] * s["dout"].float()
    dn = m * a * w
    inner = (dn * n).sum(-1, keepdim=True) if kind == "l2" else (dn * n).mean(-1, keepdim=True)
    dx = r * (dn - n * inner - (dn.mean(-1, keepdim=True) if kind == "layer" else 0))
    dw = (m * a * n).flatten(0, -2).double().sum(0).float() if s["weight"] is not None else None
    dgate = (m * n * w * da).to(dt) if da is not None else None
    return dx.to(dt), dgate, dw


def _plain_rotary(s):
    c = s["case"]
    B, H, T, D = s["q"].shape
    R = c["R"]
    pos = s["pos"] if s["pos"] is not None else (s["start"] + torch.arange(T, device=DEV))[None]
    angle = pos[:, None, :, None].double() * s["freq"].double()  # far positions: in 64 bits
    cos, sin = (s["mscale"] * angle.cos()).float(), (s["mscale"] * angle.sin()).float()

    def turn(x):
        out = x.float().clone(memory_format=torch.contiguous_format)
        x = x.float()
        at = (slice(0, R // 2), slice(R // 2, R)) if c["layout"] == "half" else (slice(0, R, 2), slice(1, R, 2))
        a, b = x[..., at[0]], x[..., at[1]]
        out[..., at[0]], out[..., at[1]] = a * cos - b * sin, a * sin + b * cos
        return out.to(s["q"].dtype)

    return turn(s["q"]), turn(s["k"])


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c, op = case, case["op"]
    es = 2 if c["dtype"] == "bf16" else 4
    if op.startswith("delta"):
        T = c.get("T", 1)
        keys, vals, state = c["B"] * c["Hk"] * T * c["Dk"] * es, c["B"] * c["H"] * T * c["Dv"] * es, \
            4 * c["B"] * c["H"] * c["Dk"] * c["Dv"]
        per_token = 4 * c["B"] * c["H"] * T
        decay = {"none": 0, "head": 4 * c["H"], "step": per_token}[c["decay"]]
        tok = c["B"] * c["H"] * T * c["Dk"] * c["Dv"]
        if op == "delta":
            return dict(bytes=2 * keys + 2 * vals + per_token + decay + state * (2 if c["init"] else 1), flops=6 * tok)
        if op == "delta_decode":
            return dict(bytes=2 * keys + 2 * vals + per_token + decay + 2 * state, flops=6 * tok)
        return dict(bytes=4 * keys + 3 * vals + 2 * per_token + 2 * decay + state * (3 if c["init"] else 1), flops=18 * tok)
    if op.startswith("norm"):
        n = c["B"] * c["H"] * c["T"] * c["D"]
        gate, w = c["act"] != "none", 4 * c["D"] * c["weight"]
        if op == "norm":
            return dict(bytes=n * es * (2 + gate + c["residual"]) + w, flops=n * (6 + 4 * gate))
        return dict(bytes=n * es * (3 + 2 * gate) + 2 * w, flops=n * (14 + 10 * gate))
    n = c["B"] * (c["H"] + c["Hk"]) * c["T"]
    return dict(bytes=2 * n * c["D"] * es + 2 * c["R"] + (8 * c["B"] * c["T"] if c["where"] == "far" else 0), flops=3 * n * c["R"])


# ------------------------------------------------------------------ the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("delta"):
        return _exact_delta(s)
    if op.startswith("norm"):
        return _exact_norm(s)
    c = s["case"]
    T, R = s["q"].shape[2], c["R"]
    pos = s["pos"] if s["pos"] is not None else (s["start"] + torch.arange(T, device=DEV))[None]
    angle = pos[:, None, :, None].double() * s["freq"].double()
    unit = torch.polar(torch.full_like(angle, s["mscale"]), angle)

    def turn(x):
        rot, rest = x[..., :R].double(), x[..., R:].double()
        if c["layout"] == "half":
            z = torch.complex(rot[..., :R // 2], rot[..., R // 2:]) * unit
            return torch.cat([z.real, z.imag, rest], -1)
        z = torch.view_as_complex(rot.unflatten(-1, (R // 2, 2)).contiguous()) * unit
        return torch.cat([torch.view_as_real(z).flatten(-2), rest], -1)

    return turn(s["q"]), turn(s["k"])


def _exact_norm(s):
    c = s["case"]
    grad = c["op"] == "norm_grad"
    leaf = {n: s[n].double().requires_grad_(grad) for n in ("x", "gate", "weight") if s[n] is not None}
    x = leaf["x"]
    if c["kind"] == "layer":
        n = (x - x.mean(-1, keepdim=True)) / (x.var(-1, unbiased=False, keepdim=True) + s["eps"]).sqrt()
    else:
        p = (x * x).sum(-1, keepdim=True)
        n = x / ((p if c["kind"] == "l2" else p / x.shape[-1]) + s["eps"]).sqrt()
    if "weight" in leaf:
        n = n * leaf["weight"]
    if "gate" in leaf:
        n = n * torch.sigmoid(leaf["gate"]) * (leaf["gate"] if c["act"] == "silu" else 1)
    n = s["scale"] * n
    if not grad:
        return n + s["residual"].double() if s["residual"] is not None else n
    got = dict(zip(leaf, torch.autograd.grad(n, list(leaf.values()), s["dout"].double())))
    return got["x"], got.get("gate"), got.get("weight")


def _exact_delta(s):
    """Token by token: S' = g S, e = v - S'^T k, S = S' + k (beta e)^T, y = scale S^T q, and the chain rule back."""
    c, scale = s["case"], s["scale"]
    one = c["op"] == "delta_decode"
    at = (lambda x: x.unsqueeze(2)) if one else (lambda x: x)
    v, beta = at(s["v"]).double(), at(s["beta"]).double()
    B, H, T, Dv = v.shape
    rep = H // s["q"].shape[1]
    q, k = (at(x).double().repeat_interleave(rep, 1) for x in (s["q"], s["k"]))
    Dk = q.shape[-1]
    grad = c["op"] == "delta_grad"
    if grad and B * H * T * Dk * Dv * 8 > 24e9:
        return None
    lg = s["log_g"]
    lg = torch.zeros_like(beta) if lg is None else lg.double()[None, :, None].expand(B, H, T) if lg.dim() == 1 else at(lg).double()
    g = lg.exp()
    S = s["state"] if one else s["init"]
    S = S.double() if S is not None else v.new_zeros((B, H, Dk, Dv))
    y, before, errs = torch.empty_like(v), [], []
    for t in range(T):
        kt = k[:, :, t, :, None]
        Sd = g[:, :, t, None, None] * S
        e = v[:, :, t] - (Sd * kt).sum(-2)
        S = Sd + kt * (beta[:, :, t, None] * e)[..., None, :]
        if grad:
            before.append(Sd)
            errs.append(e)
        else:
            y[:, :, t] = scale * (S * q[:, :, t, :, None]).sum(-2)
    if not grad:
        return (y[:, :, 0] if one else y), S
    dy = s["dy"].double()
    G = s["d_final"].double() if s["d_final"] is not None else torch.zeros_like(S)
    dq, dk, dv, dbeta, dlg = (torch.empty_like(x) for x in (q, k, v, beta, beta))
    for t in reversed(range(T)):
        kt, Sd, e = k[:, :, t], before[t], errs[t]
        u = beta[:, :, t, None] * e
        St = Sd + kt[..., None] * u[..., None, :]
        dq[:, :, t] = scale * (St * dy[:, :, t, None, :]).sum(-1)
        G = G + scale * q[:, :, t, :, None] * dy[:, :, t, None, :]
        du = (G * kt[..., None]).sum(-2)
        dbeta[:, :, t] = (du * e).sum(-1)
        de = beta[:, :, t, None] * du
        dv[:, :, t] = de
        dk[:, :, t] = (G * u[..., None, :]).sum(-1) - (Sd * de[..., None, :]).sum(-1)
        G = G - kt[..., None] * de[..., None, :]
        dlg[:, :, t] = (G * Sd).sum((-1, -2))
        G = g[:, :, t, None, None] * G
    dq, dk = (x.unflatten(1, (H // rep, rep)).sum(2) for x in (dq, dk))
    dlg = None if s["log_g"] is None else dlg.sum((0, 2)) if s["log_g"].dim() == 1 else dlg
    return dq, dk, dv, dbeta, dlg, G
