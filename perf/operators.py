"""Cases of the gated delta rule (whole sequences, gradients, single tokens) and of the
norms around a block, each in a plain form and through the library.

* ``delta_fwd``:  S_t = e^{a_t} S_{t-1} + beta_t (v_t - e^{a_t} S_{t-1} k_t) k_t^T,
  y_t = scale S_t q_t, over a whole sequence; y and the final state.
* ``delta_bwd``:  the gradients of all inputs from those of y and the final state.
* ``delta_step``: K tokens on a kept state (K = 1: decoding), the state after the
  accepted ones.
* ``norm_gate``:  the norm after the mixer with its gate; and its gradients.
* ``norm_add``:   the residual sum with a per-channel scale and the norm of the next
  block; and its gradients.

``run`` computes them from elementary torch operations in 32 bits, or (``own``) with the
library's calls.  ``exact`` follows the definitions token by token in 64 bits.
"""
import math

import torch

own = False

DEVICE = "cuda"
CHUNK = 64          # tokens per chunk of the plain form
EPS = 1e-5          # of every norm here


# ------------------------------------------------------------------------- cases
def listed():
    return [
        # a short prompt with a kept state: one chunk and a part of the next
        dict(name="delta_fwd_short_bf16", op="delta_fwd", io="bf16", b=1, L=77, H=8, G=2, P=64, N=64, init=True),
        # a training layer: 4 sequences of 2048 tokens, 32 heads on 8 groups of keys
        dict(name="delta_fwd_layer_bf16", op="delta_fwd", io="bf16", b=4, L=2048, H=32, G=8, P=128, N=128, init=False),
        # one long document (prefill), from a kept state
        dict(name="delta_fwd_long_bf16", op="delta_fwd", io="bf16", b=1, L=16384, H=32, G=8, P=128, N=128, init=True),
        # full-precision run of a small model, ragged length
        dict(name="delta_fwd_ragged_f32", op="delta_fwd", io="f32", b=2, L=1337, H=12, G=4, P=64, N=64, init=True),
        # backward of the training layer
        dict(name="delta_bwd_layer_bf16", op="delta_bwd", io="bf16", b=4, L=2048, H=32, G=8, P=128, N=128, init=False),
        # backward in full precision, ragged length, kept state
        dict(name="delta_bwd_ragged_f32", op="delta_bwd", io="f32", b=2, L=777, H=6, G=3, P=32, N=64, init=True),
        # decoding one token for 64 sequences
        dict(name="delta_step_decode_bf16", op="delta_step", io="bf16", b=64, K=1, H=32, G=8, P=128, N=128),
        # verifying 5 draft tokens of 3 sequences
        dict(name="delta_step_verify_f32", op="delta_step", io="f32", b=3, K=5, H=16, G=16, P=64, N=128),
        # gated norm of a decode batch: latency
        dict(name="norm_gate_fwd_decode_bf16", op="norm_gate", io="bf16", bwd=False, rows=5, D=5120, group=5120, gate_first=True),
        # gradients of the gated norm of a training layer, one group per head
        dict(name="norm_gate_bwd_layer_bf16", op="norm_gate", io="bf16", bwd=True, rows=8192, D=4096, group=128, gate_first=False),
        # residual sum and norm of a training layer, residual kept in 32 bits
        dict(name="norm_add_fwd_layer_bf16", op="norm_add", io="bf16", bwd=False, rows=8192, D=2560, res="f32", scaled=True),
        # its gradients in full precision, ragged
        dict(name="norm_add_bwd_ragged_f32", op="norm_add", io="f32", bwd=True, rows=2677, D=1288, res="f32", scaled=True),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["delta_fwd", "delta_fwd", "delta_bwd", "delta_bwd", "delta_step", "norm_gate", "norm_add"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op in ("delta_fwd", "delta_bwd"):
        P = rng.choice([16, 32, 48, 64, 96, 128])
        N = rng.choice([32, 64, 128] if io == "f32" or op == "delta_bwd" else [32, 64, 128, 256])
        G = rng.choice([1, 2, 3, 4, 8])
        H = G * rng.choice([1, 2, 3, 4])
        b = rng.choice([1, 1, 2, 3, 4])
        most = (1 << 32) if op == "delta_fwd" else (1 << 30)
        L = _log_uniform(rng, 1, max(2, min(16384 if op == "delta_fwd" else 2048, most // (b * H * P * N))))
        return dict(op=op, io=io, b=b, L=L, H=H, G=G, P=P, N=N, init=rng.random() < 0.5)
    if op == "delta_step":
        G = rng.choice([1, 2, 4, 8])
        return dict(op=op, io=io, b=_log_uniform(rng, 1, 48), K=rng.choice([1, 1, 2, 3, 5, 8]), H=G * rng.choice([1, 2, 4]), G=G,
                    P=rng.choice([16, 40, 64, 100, 128]), N=rng.choice([32, 64, 128, 256]))
    bwd, rows = rng.random() < 0.5, _log_uniform(rng, 1, 4096)
    if op == "norm_gate":
        group = 8 * _log_uniform(rng, 2, 512)
        D = group * rng.choice([1, 1, 2, 4] if group <= 1024 else [1])
        return dict(op=op, io=io, bwd=bwd, rows=rows, D=D, group=group, gate_first=rng.random() < 0.5)
    return dict(op=op, io=io, bwd=bwd, rows=rows, D=8 * _log_uniform(rng, 2, 640), res=rng.choice(["f32", io]), scaled=rng.random() < 0.7)


def _dtype(io):
    return torch.bfloat16 if io == "bf16" else torch.float32


# ------------------------------------------------------------------------ inputs
def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    t = _dtype(c["io"])

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEVICE)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=DEVICE)

    if c["op"].startswith("delta"):
        b, H, G, P, N = c["b"], c["H"], c["G"], c["P"], c["N"]
        L = c["K"] if c["op"] == "delta_step" else c["L"]
        c["scale"] = N ** -0.5
        # unit queries and keys, gates of a softplus step times a rate per head
        c["q"] = torch.nn.functional.normalize(normal(b, L, G, N), dim=-1).to(t)
        c["k"] = torch.nn.functional.normalize(normal(b, L, G, N), dim=-1).to(t)
        c["v"] = normal(b, L, H, P).to(t)
        rate = torch.exp(uniform(H) * math.log(16.0))
        dt = torch.nn.functional.softplus(normal(b, L, H) - 4.6).clamp(1e-3, 1e-1)
        c["a"] = -dt * rate
        c["beta"] = torch.sigmoid(normal(b, L, H))
        if c["op"] == "delta_step":
            c["state"] = 0.1 * normal(b, H, P, N)
            c["accept_len"] = torch.randint(0, L + 1, (b,), generator=gen, device=DEVICE, dtype=torch.int32) if L > 1 else None
        else:
            c["init_state"] = 0.1 * normal(b, H, P, N) if c["init"] else None
        if c["op"] == "delta_bwd":
            c["dy"] = normal(b, L, H, P).to(t)
            c["d_final"] = normal(b, H, P, N)
        return c
    rows, D = c["rows"], c["D"]
    c["x"] = normal(rows, D).to(t)
    c["w"] = 1.0 + 0.1 * normal(D)
    if c["op"] == "norm_gate":
        c["z"] = normal(rows, D).to(t)
    else:
        c["residual"] = (2.0 * normal(rows, D)).to(_dtype(c["res"]))
        c["ls"] = 0.5 + 0.1 * normal(D) if c["scaled"] else None
        if c["bwd"]:
            # the forward pass's sum, kept for the backward pass as a model keeps it
            s = c["x"].float() if c["ls"] is None else c["x"].float() * c["ls"]
            c["sum"] = (c["residual"].float() + s).to(_dtype(c["res"]))
            c["d_sum"] = normal(rows, D).to(_dtype(c["res"]))
    if c["bwd"]:
        c["dy"] = normal(rows, D).to(t)
    return c


# -------------------------------------------------------------------- plain forms
def _delta_chunks(q, k, v, a, beta, init_state, scale):
    """The chunked form: within a chunk the token updates are a triangular system, from
    chunk to chunk the state is passed on.  All 32 bits but the gate sums (64)."""
    b, L, H, P = v.shape
    G, N = k.shape[2:]
    pad = -L % CHUNK
    nc = (L + pad) // CHUNK

    def chunks(x):     # [b, L, heads, ...] -> [b, heads, nc, CHUNK, ...]
        x = torch.nn.functional.pad(x, (0, 0) * (x.dim() - 2) + (0, pad))
        return x.reshape(b, nc, CHUNK, *x.shape[2:]).movedim(3, 1)

    def heads(x):      # one copy of a group's rows per head
        return chunks(x).repeat_interleave(H // G, dim=1)

    q, k, v, a, beta = heads(q), heads(k), chunks(v), chunks(a), chunks(beta)
    cum = torch.cumsum(a.double(), -1)
    keep = torch.tril(torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=v.device))
    decay = torch.exp((cum[..., :, None] - cum[..., None, :]).masked_fill(~keep, -math.inf)).float()
    from_start, to_end = torch.exp(cum).float(), torch.exp(cum[..., -1:] - cum).float()
    kt = k.transpose(-1, -2).contiguous()
    lower = torch.tril(beta[..., :, None] * torch.matmul(k, kt) * decay, -1)
    # (I + lower)^-1 = (I - lower)(I + lower^2)(I + lower^4) ...: lower^64 = 0
    eye = torch.eye(CHUNK, device=v.device)
    power, inverse = -lower, eye - lower
    for _ in range(5):
        power = torch.matmul(power, power)
        inverse = inverse + torch.matmul(inverse, power)
    u = torch.matmul(inverse, beta[..., None] * v)
    w = torch.matmul(inverse, (beta * from_start)[..., None] * k)
    scores = scale * torch.matmul(q, kt) * decay
    q = scale * from_start[..., None] * q
    k = to_end[..., None] * k
    S = torch.zeros(b, H, P, N, device=v.device) if init_state is None else init_state
    ys = []
    for c in range(nc):
        st = S.transpose(-1, -2)
        new = u[:, :, c] - torch.matmul(w[:, :, c], st)
        ys.append(torch.matmul(q[:, :, c], st) + torch.matmul(scores[:, :, c], new))
        S = from_start[:, :, c, -1, None, None] * S + torch.matmul(new.transpose(-1, -2), k[:, :, c])
    y = torch.stack(ys, 2).movedim(1, 3).reshape(b, nc * CHUNK, H, P)[:, :L]
    return y, S


def _delta_fwd(c):
    y, S = _delta_chunks(c["q"].float(), c["k"].float(), c["v"].float(), c["a"], c["beta"], c["init_state"], c["scale"])
    return y.to(c["v"].dtype), S.contiguous()


def _delta_bwd(c):
    b, L, H, P = c["v"].shape
    init = torch.zeros(b, H, P, c["k"].shape[3], device=DEVICE) if c["init_state"] is None else c["init_state"]
    leaves = [x.float().detach().requires_grad_() for x in (c["q"], c["k"], c["v"], c["a"], c["beta"], init)]
    with torch.enable_grad():
        y, S = _delta_chunks(*leaves, c["scale"])
        dq, dk, dv, da, dbeta, d_init = torch.autograd.grad((y, S), leaves, (c["dy"].float(), c["d_final"]))
    t = c["v"].dtype
    return dq.to(t), dk.to(t), dv.to(t), da, dbeta, d_init


def _delta_step(c):
    b, K, H, P = c["v"].shape
    r = H // c["k"].shape[2]
    q, k = (c[n].float().repeat_interleave(r, dim=2) for n in ("q", "k"))
    v, beta, alpha = c["v"].float(), c["beta"], torch.exp(c["a"])
    S = kept = c["state"]
    ys = []
    for t in range(K):
        S = alpha[:, t, :, None, None] * S
        u = beta[:, t, :, None] * (v[:, t] - (S * k[:, t, :, None, :]).sum(-1))
        S = S + u[..., None] * k[:, t, :, None, :]
        ys.append(c["scale"] * (S * q[:, t, :, None, :]).sum(-1))
        if c["accept_len"] is not None:
            kept = torch.where((c["accept_len"] > t)[:, None, None, None], S, kept)
    return torch.stack(ys, 1).to(c["v"].dtype), S if c["accept_len"] is None else kept


def _norm_gate(c):
    x, z, w, g = c["x"].float(), c["z"].float(), c["w"], c["group"]
    t, rows, D = c["x"].dtype, c["rows"], c["D"]
    sig = torch.sigmoid(z)
    act = z * sig
    u = x * act if c["gate_first"] else x
    r = torch.rsqrt(u.view(rows, -1, g).square().mean(-1, keepdim=True) + EPS)
    n = (u.view(rows, -1, g) * r).view(rows, D)
    if not c["bwd"]:
        return ((n * w) if c["gate_first"] else (n * w * act)).to(t)
    dy = c["dy"].float()
    dact = sig * (1.0 + z * (1.0 - sig))
    up = dy if c["gate_first"] else dy * act
    dn = (up * w).view(rows, -1, g)
    du = ((dn - n.view(rows, -1, g) * (dn * n.view(rows, -1, g)).mean(-1, keepdim=True)) * r).view(rows, D)
    dw = (up * n).sum(0)
    if c["gate_first"]:
        return (du * act).to(t), (du * x * dact).to(t), dw
    return du.to(t), (dy * n * w * dact).to(t), dw


def _norm_add(c):
    x, w, t, tr = c["x"].float(), c["w"], c["x"].dtype, c["residual"].dtype
    if not c["bwd"]:
        s = c["residual"].float() + (x if c["ls"] is None else x * c["ls"])
        s = s.to(tr)
        f = s.float()
        return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS) * w).to(t), s
    s, dy = c["sum"].float(), c["dy"].float()
    r = torch.rsqrt(s.square().mean(-1, keepdim=True) + EPS)
    n = s * r
    dn = dy * w
    ds = c["d_sum"].float() + r * (dn - n * (dn * n).mean(-1, keepdim=True))
    dw = (dy * n).sum(0)
    if c["ls"] is None:
        return ds.to(t), ds.to(tr), dw
    return (ds * c["ls"]).to(t), ds.to(tr), dw, (ds * x).sum(0)


# ---------------------------------------------------------------- the library's calls
def _library(c):
    from selective_state_space_ssd_amd import binding as bd
    op = c["op"]
    if op == "delta_fwd":
        return bd.gated_delta_fwd(c["q"], c["k"], c["v"], c["a"], c["beta"], c["scale"], init_state=c["init_state"])
    if op == "delta_bwd":
        return bd.gated_delta_bwd(c["q"], c["k"], c["v"], c["a"], c["beta"], c["scale"], c["dy"], init_state=c["init_state"], d_final=c["d_final"])
    if op == "delta_step":
        return bd.gated_delta_step(c["state"], c["q"], c["k"], c["v"], c["a"], c["beta"], c["scale"], accept_len=c["accept_len"])
    if op == "norm_gate":
        if c["bwd"]:
            return bd.norm_gate_bwd(c["x"], c["z"], c["w"], c["dy"], c["group"], EPS, gate_first=c["gate_first"])
        return bd.norm_gate_fwd(c["x"], c["z"], c["w"], c["group"], EPS, gate_first=c["gate_first"])
    if not c["bwd"]:
        return bd.norm_add_fwd(c["x"], c["residual"], c["w"], EPS, scale=c["ls"])
    dx, d_res, dw, d_scale = bd.norm_add_bwd(c["x"], c["sum"], c["w"], c["dy"], c["d_sum"], EPS, scale=c["ls"])
    return (dx, d_res, dw) if d_scale is None else (dx, d_res, dw, d_scale)


def run(state):
    if own:
        return _library(state)
    return {"delta_fwd": _delta_fwd, "delta_bwd": _delta_bwd, "delta_step": _delta_step, "norm_gate": _norm_gate,
            "norm_add": _norm_add}[state["op"]](state)


# -------------------------------------------------------------------------- work
def work(case):
    """Bytes: every input once and every output once.  Operations of the delta rule: the
    recurrence itself (per token, head and state element: decay, S k, the update, S q)."""
    c = case
    e = 2 if c["io"] == "bf16" else 4
    if c["op"].startswith("delta"):
        b, H, G, P, N = c["b"], c["H"], c["G"], c["P"], c["N"]
        L = c["K"] if c["op"] == "delta_step" else c["L"]
        qk, vy, gates, st = b * L * G * N * e * 2, b * L * H * P * e, b * L * H * 4 * 2, b * H * P * N * 4
        cells = b * L * H * P * N
        if c["op"] == "delta_step":
            return {"bytes": qk + 2 * vy + gates + 2 * st, "flops": 7 * cells}
        held = st if c["init"] else 0
        if c["op"] == "delta_fwd":
            return {"bytes": qk + 2 * vy + gates + held + st, "flops": 7 * cells}
        # backward: states again, then dq, the two parts of dS, du, two parts of dk, dS', the gate
        return {"bytes": 2 * qk + 3 * vy + 2 * gates + held + 2 * st, "flops": 21 * cells}
    n, D = c["rows"] * c["D"], c["D"]
    if c["op"] == "norm_gate":
        return {"bytes": 5 * n * e + 8 * D, "flops": 20 * n} if c["bwd"] else {"bytes": 3 * n * e + 4 * D, "flops": 10 * n}
    r = 2 if c["res"] == "bf16" else 4
    if c["bwd"]:
        x = n * e + 8 * D if c["scaled"] else 0     # x is read for the scale's gradient alone
        return {"bytes": x + 2 * n * e + 3 * n * r + 8 * D, "flops": 14 * n}
    return {"bytes": 2 * n * e + 2 * n * r + 8 * D, "flops": 6 * n}


# ------------------------------------------------------------------------- exact
def _exact_delta(c):
    """Token by token in 64 bits; the backward pass walks the kept states in reverse."""
    q, k, v, a, beta = (c[n].double() for n in ("q", "k", "v", "a", "beta"))
    b, L, H, P = v.shape
    G, N = k.shape[2:]
    head_group = torch.arange(H, device=DEVICE) // (H // G)
    q, k = q[:, :, head_group], k[:, :, head_group]
    scale, bwd, step = c["scale"], c["op"] == "delta_bwd", c["op"] == "delta_step"
    S0 = c["state"] if step else c["init_state"]
    S = torch.zeros(b, H, P, N, dtype=torch.float64, device=DEVICE) if S0 is None else S0.double()
    y = torch.zeros_like(v)
    kept = S.clone()
    before, e = [], torch.zeros_like(v)
    alpha = a.exp()
    for t in range(L):
        S = S * alpha[:, t, :, None, None]
        if bwd:
            before.append(S)
        kc = k[:, t, :, :, None]
        e[:, t] = v[:, t] - (S @ kc)[..., 0]
        S = S + (beta[:, t, :, None] * e[:, t])[..., None] * k[:, t, :, None, :]
        y[:, t] = scale * (S @ q[:, t, :, :, None])[..., 0]
        if step and c["accept_len"] is not None:
            kept = torch.where((c["accept_len"] > t).view(b, 1, 1, 1), S, kept)
    if step:
        return y, S if c["accept_len"] is None else kept
    if not bwd:
        return y, S
    dy, dS = c["dy"].double(), c["d_final"].double()
    dq, dk = torch.zeros_like(q), torch.zeros_like(k)
    dv, da, dbeta = torch.zeros_like(v), torch.zeros_like(a), torch.zeros_like(beta)
    for t in reversed(range(L)):
        Sb = before.pop()
        u = beta[:, t, :, None] * e[:, t]
        qr, kr = q[:, t, :, None, :], k[:, t, :, None, :]
        after = Sb + u[..., None] * kr
        dq[:, t] = scale * (dy[:, t, :, None, :] @ after)[..., 0, :]
        dS = dS + scale * dy[:, t, :, :, None] * qr
        du = (dS @ k[:, t, :, :, None])[..., 0]
        dbeta[:, t] = (du * e[:, t]).sum(-1)
        de = beta[:, t, :, None] * du
        dv[:, t] = de
        dk[:, t] = (u[..., None, :] @ dS)[..., 0, :] - (de[..., None, :] @ Sb)[..., 0, :]
        dS = dS - de[..., None] * kr
        da[:, t] = (dS * Sb).sum((-1, -2))
        dS = dS * alpha[:, t, :, None, None]

    def groups(x):
        return x.view(b, L, G, H // G, N).sum(3)
    return groups(dq), groups(dk), dv, da, dbeta, dS


def _exact_norm(c):
    x, w = c["x"].double(), c["w"].double()
    if c["op"] == "norm_gate":
        rows, D, g = c["rows"], c["D"], c["group"]
        z = c["z"].double()
        act = z / (1 + torch.exp(-z))
        inner = (x * act if c["gate_first"] else x).reshape(rows * (D // g), g)
        inv = 1 / torch.sqrt((inner * inner).sum(1) / g + EPS)
        hat = (inner * inv[:, None]).reshape(rows, D)
        if not c["bwd"]:
            return hat * w if c["gate_first"] else hat * w * act
        dy = c["dy"].double()
        slope = torch.exp(-z) * z / (1 + torch.exp(-z)) ** 2 + 1 / (1 + torch.exp(-z))
        into = dy if c["gate_first"] else dy * act
        dhat = (into * w).reshape(rows * (D // g), g)
        h2 = hat.reshape(rows * (D // g), g)
        dinner = (inv[:, None] * (dhat - h2 * (dhat * h2).sum(1, keepdim=True) / g)).reshape(rows, D)
        dw = (into * hat).sum(0)
        return (dinner * act, dinner * x * slope, dw) if c["gate_first"] else (dinner, dy * hat * w * slope, dw)
    ls = 1.0 if c["ls"] is None else c["ls"].double()
    D = c["D"]
    if not c["bwd"]:
        total = c["residual"].double() + ls * x
        held = total if c["res"] == "f32" else total.float().to(torch.bfloat16).double()
        return held / torch.sqrt((held * held).sum(1, keepdim=True) / D + EPS) * w, total
    total, dy = c["sum"].double(), c["dy"].double()
    inv = 1 / torch.sqrt((total * total).sum(1, keepdim=True) / D + EPS)
    hat = total * inv
    d_total = c["d_sum"].double() + inv * (dy * w - hat * (dy * w * hat).sum(1, keepdim=True) / D)
    out = (d_total * ls, d_total, (dy * hat).sum(0))
    return out if c["ls"] is None else out + ((d_total * x).sum(0),)


def exact(case, seed):
    c = prepare(case, seed)
    if not c["op"].startswith("delta"):
        return _exact_norm(c)
    return _exact_delta(c)
