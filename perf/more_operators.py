"""Cases of the gated scan (whole sequences, gradients, single tokens) and of two forms of the
norm before a block, each in a plain form and through the library.

* ``scan_fwd``:  h_t = alpha_t h_{t-1} + u_t per channel, y_t = h_t; alpha = e^a and u = x, or
  (``sigmoid``) alpha = 1 / (1 + e^-a) and u = (1 - alpha) x; y and the final state.
* ``scan_bwd``:  the gradients of x, a and the initial state from those of y and the final state.
* ``scan_step``: K tokens on a kept state (K = 1: decoding), the state after the accepted ones.
* ``norm_drop``: the residual sum with dropout on what is added, and its norm; and the gradients.
  The mask comes from a counter-based generator, Philox4x32-10 (Salmon, Moraes, Dror and Shaw,
  "Parallel random numbers: as easy as 1, 2, 3", 2011), whose seed and offset are inputs.
* ``norm_q8``:   the residual sum and its norm in 8 bits (e4m3), one scale per group of channels.

``run`` computes them from elementary torch operations in 32 bits, or (``own``) with the
library's calls.  ``exact`` follows the definitions in 64 bits, the recurrence token by token.
"""
import math

import torch

own = False

DEVICE = "cuda"
EPS = 1e-5          # of every norm here
KEPT = 32           # the forward pass keeps the state before every 32nd token
E4M3_MAX = 448.0
TINY = 2.0 ** -126  # the least scale of a group


# ------------------------------------------------------------------------- cases
def listed():
    return [
        # a short prompt with a kept state
        dict(name="scan_fwd_prompt_bf16", op="scan_fwd", io="bf16", a_io="bf16", b=1, L=77, D=512, sigmoid=False, init=True),
        # a training layer: 4 sequences of 2048 tokens, gates straight from their projection
        dict(name="scan_fwd_layer_bf16", op="scan_fwd", io="bf16", a_io="bf16", b=4, L=2048, D=5120, sigmoid=True, init=False),
        # one long document (prefill) from a kept state, decays in 32 bits
        dict(name="scan_fwd_long_bf16", op="scan_fwd", io="bf16", a_io="f32", b=1, L=16384, D=2560, sigmoid=False, init=True),
        # full-precision run of a small model, ragged length
        dict(name="scan_fwd_ragged_f32", op="scan_fwd", io="f32", a_io="f32", b=2, L=1337, D=1288, sigmoid=False, init=True),
        # backward of the training layer
        dict(name="scan_bwd_layer_bf16", op="scan_bwd", io="bf16", a_io="bf16", b=4, L=2048, D=5120, sigmoid=True, init=False),
        # backward in full precision, ragged length and channels, kept state
        dict(name="scan_bwd_ragged_f32", op="scan_bwd", io="f32", a_io="f32", b=2, L=777, D=645, sigmoid=False, init=True),
        # decoding one token for 64 sequences
        dict(name="scan_step_decode_bf16", op="scan_step", io="bf16", a_io="bf16", b=64, K=1, D=5120, sigmoid=True),
        # verifying 5 draft tokens of 3 sequences
        dict(name="scan_step_verify_f32", op="scan_step", io="f32", a_io="f32", b=3, K=5, D=1288, sigmoid=False),
        # residual sum with dropout and norm of a training layer, residual kept in 32 bits
        dict(name="norm_drop_fwd_layer_bf16", op="norm_drop", io="bf16", bwd=False, rows=8192, D=2560, res="f32", scaled=False, p=0.1),
        # its gradients, with a scale per channel
        dict(name="norm_drop_bwd_layer_bf16", op="norm_drop", io="bf16", bwd=True, rows=8192, D=2560, res="f32", scaled=True, p=0.1),
        # what the next projection of a decode batch reads: latency
        dict(name="norm_q8_decode_bf16", op="norm_q8", io="bf16", rows=5, D=5120, group=5120, res="bf16", scaled=False),
        # the same of a prefill, a scale per 128 channels
        dict(name="norm_q8_prefill_bf16", op="norm_q8", io="bf16", rows=8192, D=2560, group=128, res="f32", scaled=True),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_fwd", "scan_bwd", "scan_bwd", "scan_step", "norm_drop", "norm_drop", "norm_q8", "norm_q8"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("scan"):
        D = _log_uniform(rng, 16, 5120)
        D = D if rng.random() < 0.3 else 8 * max(1, D // 8)
        c = dict(op=op, io=io, a_io=rng.choice([io, "f32"]), D=D, sigmoid=rng.random() < 0.5)
        if op == "scan_step":
            return dict(c, b=_log_uniform(rng, 1, 64), K=rng.choice([1, 1, 2, 3, 5, 8]))
        b = rng.choice([1, 1, 2, 3, 4])
        most = (1 << 25) if io == "bf16" else (1 << 24)
        return dict(c, b=b, L=_log_uniform(rng, 1, max(2, min(16384 if op == "scan_fwd" else 2048, most // (b * D)))), init=rng.random() < 0.5)
    rows, res = _log_uniform(rng, 1, 4096), rng.choice(["f32", io])
    if op == "norm_q8":
        group = rng.choice([32, 64, 128, 0])
        D = _log_uniform(rng, 16, 5120) if not group else group * _log_uniform(rng, 1, 5120 // group)
        return dict(op=op, io=io, rows=rows, D=D, group=group or D, res=res, scaled=rng.random() < 0.5)
    D = _log_uniform(rng, 16, 5120)
    D = D if rng.random() < 0.3 else 8 * max(1, D // 8)
    return dict(op=op, io=io, bwd=rng.random() < 0.5, rows=rows, D=D, res=res, scaled=rng.random() < 0.5, p=rng.choice([0.05, 0.1, 0.25, 0.5]))


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

    if c["op"].startswith("scan"):
        b, D = c["b"], c["D"]
        L = c["K"] if c["op"] == "scan_step" else c["L"]
        c["x"] = normal(b, L, D).to(t)
        if c["sigmoid"]:
            # gates open to different lengths of memory, a bias per channel
            a = normal(b, L, D) + 5.0 * uniform(D)
        else:
            # a softplus step times a rate per channel
            a = -torch.nn.functional.softplus(normal(b, L, D) - 4.6).clamp(1e-3, 1e-1) * torch.exp(uniform(D) * math.log(16.0))
        c["a"] = a.to(_dtype(c["a_io"]))
        if c["op"] == "scan_step":
            c["state"] = normal(b, D)
            c["accept_len"] = torch.randint(0, L + 1, (b,), generator=gen, device=DEVICE, dtype=torch.int32) if L > 1 else None
            return c
        c["init_state"] = normal(b, D) if c["init"] else None
        if c["op"] == "scan_bwd":
            # what the forward pass kept for the backward pass: the state before tokens 0, 32, 64, ...
            alpha, u = _gates(c["x"].float(), c["a"].float(), c["sigmoid"])[:2]
            h = _scan(alpha, u, c["init_state"])
            first = torch.zeros(b, 1, D, device=DEVICE) if c["init_state"] is None else c["init_state"][:, None]
            c["states"] = torch.cat((first, h[:, KEPT - 1:L - 1:KEPT]), 1).contiguous()
            c["dy"] = normal(b, L, D).to(t)
            c["d_final"] = normal(b, D)
        return c
    rows, D = c["rows"], c["D"]
    c["x"] = normal(rows, D).to(t)
    c["w"] = 1.0 + 0.1 * normal(D)
    c["residual"] = (2.0 * normal(rows, D)).to(_dtype(c["res"]))
    c["ls"] = 0.5 + 0.1 * normal(D) if c["scaled"] else None
    if c["op"] == "norm_drop":
        # the generator's state: a seed, and the offset that a training step counts on
        c["rng"] = torch.tensor([seed * 0x9E3779B97F4A7C15 % (1 << 63), 1000003 * (seed + 1)], device=DEVICE)
        if c["bwd"]:
            # the forward pass's sum, kept for the backward pass as a model keeps it
            keep, up = _mask(c)
            s = torch.where(keep, c["x"].float() * up, 0.0)
            c["sum"] = (c["residual"].float() + (s if c["ls"] is None else s * c["ls"])).to(_dtype(c["res"]))
            c["dy"] = normal(rows, D).to(t)
            c["d_sum"] = normal(rows, D).to(_dtype(c["res"]))
            del c["residual"]
    return c


# -------------------------------------------------------------------- plain forms
def _gates(x, a, sigmoid):
    """(decay, what enters the state, its factor)."""
    if not sigmoid:
        return torch.exp(a), x, None
    beta = 1.0 / (1.0 + torch.exp(a))
    return 1.0 / (1.0 + torch.exp(-a)), beta * x, beta


def _scan(alpha, u, init):
    """h_t = alpha_t h_{t-1} + u_t over dim 1, in log2(L) steps of doubled reach."""
    h, p = u.clone(), alpha
    if init is not None:
        h[:, 0] += alpha[:, 0] * init
    reach = 1
    while reach < h.shape[1]:
        h = torch.cat((h[:, :reach], h[:, reach:] + p[:, reach:] * h[:, :-reach]), 1)
        p = torch.cat((p[:, :reach], p[:, reach:] * p[:, :-reach]), 1)
        reach *= 2
    return h


def _scan_fwd(c):
    alpha, u, _ = _gates(c["x"].float(), c["a"].float(), c["sigmoid"])
    h = _scan(alpha, u, c["init_state"])
    return h.to(c["x"].dtype), h[:, -1].clone()


def _scan_bwd(c):
    x, dy = c["x"].float(), c["dy"].float()
    alpha, u, beta = _gates(x, c["a"].float(), c["sigmoid"])
    h = _scan(alpha, u, c["init_state"])
    first = torch.zeros_like(h[:, :1]) if c["init_state"] is None else c["init_state"][:, None]
    before = torch.cat((first, h[:, :-1]), 1)
    # the gradient's recurrence runs from the last token to the first
    dy = torch.cat((dy[:, :-1], dy[:, -1:] + c["d_final"][:, None]), 1)
    later = torch.cat((alpha[:, 1:], torch.zeros_like(alpha[:, :1])), 1)
    lam = _scan(later.flip(1), dy.flip(1), None).flip(1)
    if c["sigmoid"]:
        dx, da = lam * beta, lam * alpha * beta * (before - x)
    else:
        dx, da = lam, lam * alpha * before
    return dx.to(c["x"].dtype), da.to(c["a"].dtype), alpha[:, 0] * lam[:, 0]


def _scan_step(c):
    alpha, u, _ = _gates(c["x"].float(), c["a"].float(), c["sigmoid"])
    h = kept = c["state"]
    ys = []
    for t in range(c["K"]):
        h = alpha[:, t] * h + u[:, t]
        ys.append(h)
        if c["accept_len"] is not None:
            kept = torch.where((c["accept_len"] > t)[:, None], h, kept)
    return torch.stack(ys, 1).to(c["x"].dtype), h if c["accept_len"] is None else kept


def _philox(counters, offset, seed):
    """The four words of every counter: 64-bit products, of which the low and the high half
    of the bits are right although the sign is not."""
    m = 0xFFFFFFFF
    c = [counters & m, counters >> 32 & m, (offset & m).expand_as(counters), (offset >> 32 & m).expand_as(counters)]
    k0, k1 = seed & m, seed >> 32 & m
    for _ in range(10):
        p, q = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [q >> 32 & m ^ c[1] ^ k0, q & m, p >> 32 & m ^ c[3] ^ k1, p & m]
        k0, k1 = k0 + 0x9E3779B9 & m, k1 + 0xBB67AE85 & m
    return c


def _p32(p):
    """p as the library takes it, in 32 bits."""
    return float(torch.tensor(p, dtype=torch.float32))


def _mask(c):
    rows, D, p = c["rows"], c["D"], _p32(c["p"])
    quads = torch.arange((rows * D + 3) // 4, device=DEVICE)
    words = torch.stack(_philox(quads, c["rng"][1], c["rng"][0]), 1).reshape(-1)[:rows * D]
    return (words >= int(p * 2.0 ** 32)).reshape(rows, D), 1.0 / (1.0 - p)


def _norm_drop(c):
    keep, up = _mask(c)
    x = torch.where(keep, c["x"].float() * up, 0.0)
    w, t = c["w"], c["x"].dtype
    if not c["bwd"]:
        s = (c["residual"].float() + (x if c["ls"] is None else x * c["ls"])).to(c["residual"].dtype)
        f = s.float()
        return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS) * w).to(t), s
    s, dy = c["sum"].float(), c["dy"].float()
    r = torch.rsqrt(s.square().mean(-1, keepdim=True) + EPS)
    n = s * r
    dn = dy * w
    ds = c["d_sum"].float() + r * (dn - n * (dn * n).mean(-1, keepdim=True))
    dx = torch.where(keep, ds * up if c["ls"] is None else ds * c["ls"] * up, 0.0)
    out = dx.to(t), ds.to(c["sum"].dtype), (dy * n).sum(0)
    return out if c["ls"] is None else out + ((ds * x).sum(0),)


def _norm_q8(c):
    x, D = c["x"].float(), c["D"]
    s = (c["residual"].float() + (x if c["ls"] is None else x * c["ls"])).to(c["residual"].dtype)
    f = s.float()
    y = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS) * c["w"]
    g = y.view(c["rows"], D // c["group"], c["group"])
    scale = (g.abs().amax(-1) / E4M3_MAX).clamp_min(TINY)
    return (g / scale[..., None]).reshape(c["rows"], D).to(torch.float8_e4m3fn), scale, s


# ---------------------------------------------------------------- the library's calls
def _library(c):
    from selective_state_space_ssd_amd import binding as bd
    op = c["op"]
    if op == "scan_fwd":
        return bd.gated_scan_fwd(c["x"], c["a"], sigmoid=c["sigmoid"], init_state=c["init_state"])
    if op == "scan_bwd":
        return bd.gated_scan_bwd(c["x"], c["a"], c["dy"], sigmoid=c["sigmoid"], init_state=c["init_state"], d_final=c["d_final"], states=c["states"])
    if op == "scan_step":
        return bd.gated_scan_step(c["state"], c["x"], c["a"], sigmoid=c["sigmoid"], accept_len=c["accept_len"])
    if op == "norm_q8":
        return bd.norm_add_q8_fwd(c["x"], c["residual"], c["w"], EPS, group=c["group"], scale=c["ls"])
    if not c["bwd"]:
        return bd.norm_add_drop_fwd(c["x"], c["residual"], c["w"], EPS, c["p"], c["rng"], scale=c["ls"])
    dx, d_res, dw, d_scale = bd.norm_add_drop_bwd(c["x"], c["sum"], c["w"], c["dy"], c["d_sum"], EPS, c["p"], c["rng"], scale=c["ls"])
    return (dx, d_res, dw) if d_scale is None else (dx, d_res, dw, d_scale)


def run(state):
    if own:
        return _library(state)
    return {"scan_fwd": _scan_fwd, "scan_bwd": _scan_bwd, "scan_step": _scan_step, "norm_drop": _norm_drop, "norm_q8": _norm_q8}[state["op"]](state)


# -------------------------------------------------------------------------- work
def work(case):
    """Bytes: every input once and every output once."""
    c = case
    e = 2 if c["io"] == "bf16" else 4
    if c["op"].startswith("scan"):
        ea, b, D = 2 if c["a_io"] == "bf16" else 4, c["b"], c["D"]
        L = c["K"] if c["op"] == "scan_step" else c["L"]
        n, st = b * L * D, b * D * 4
        if c["op"] == "scan_step":
            return {"bytes": n * (2 * e + ea) + 2 * st, "flops": 4 * n}
        held = st if c["init"] else 0
        if c["op"] == "scan_fwd":
            return {"bytes": n * (2 * e + ea) + held + st, "flops": 4 * n}
        return {"bytes": n * (3 * e + 2 * ea) + -(-L // KEPT) * st + 2 * st, "flops": 10 * n}
    n, D = c["rows"] * c["D"], c["D"]
    r = 2 if c["res"] == "bf16" else 4
    params = 4 * D * (2 if c["scaled"] else 1)
    if c["op"] == "norm_q8":
        return {"bytes": n * (e + 2 * r + 1) + 4 * c["rows"] * (D // c["group"]) + params, "flops": 8 * n}
    if c["bwd"]:
        return {"bytes": n * ((3 if c["scaled"] else 2) * e + 3 * r) + 2 * params, "flops": 40 * n}
    return {"bytes": n * (2 * e + 2 * r) + params, "flops": 32 * n}


# ------------------------------------------------------------------------- exact
def _exact_scan(c):
    x, a = c["x"].double(), c["a"].double()
    step, bwd = c["op"] == "scan_step", c["op"] == "scan_bwd"
    L = x.shape[1]
    alpha = torch.sigmoid(a) if c["sigmoid"] else a.exp()
    share = torch.sigmoid(-a) if c["sigmoid"] else torch.ones_like(a)
    start = c["state"] if step else c["init_state"]
    h = torch.zeros(x.shape[0], x.shape[2], dtype=torch.float64, device=DEVICE) if start is None else start.double()
    kept, y, before = h, torch.empty_like(x), torch.empty_like(x)
    for t in range(L):
        before[:, t] = h
        h = alpha[:, t] * h + share[:, t] * x[:, t]
        y[:, t] = h
        if step and c["accept_len"] is not None:
            kept = torch.where((c["accept_len"] > t).view(-1, 1), h, kept)
    if step:
        return y, h if c["accept_len"] is None else kept
    if not bwd:
        return y, h
    g, dx, da = c["d_final"].double(), torch.empty_like(x), torch.empty_like(x)
    for t in reversed(range(L)):
        g = g + c["dy"][:, t].double()
        dx[:, t] = g * share[:, t]
        da[:, t] = g * alpha[:, t] * ((before[:, t] - x[:, t]) * share[:, t] if c["sigmoid"] else before[:, t])
        g = g * alpha[:, t]
    return dx, da, g


def _wide(m, v):
    """High and low word of the constant m times v, in halves of 16 bits."""
    lo, hi = (m & 0xFFFF) * v, (m >> 16) * v            # 48 bits each
    low = lo + ((hi & 0xFFFF) << 16)
    return (hi >> 16) + (low >> 32), low & 0xFFFFFFFF


def _exact_keep(c):
    n = c["rows"] * c["D"]
    seed, offset = (int(v) for v in c["rng"])
    i = torch.arange(n, device=DEVICE)
    words = torch.empty(n, dtype=torch.int64, device=DEVICE)
    at = torch.arange(0, n, 4, device=DEVICE) // 4
    w = [at % (1 << 32), at // (1 << 32), torch.full_like(at, offset % (1 << 32)), torch.full_like(at, offset // (1 << 32))]
    for r in range(10):
        key0, key1 = (seed + r * 0x9E3779B9) % (1 << 32), (seed // (1 << 32) + r * 0xBB67AE85) % (1 << 32)
        (h0, l0), (h1, l1) = _wide(0xD2511F53, w[0]), _wide(0xCD9E8D57, w[2])
        w = [h1 ^ w[1] ^ key0, l1, h0 ^ w[3] ^ key1, l0]
    for j in range(4):
        words[j::4] = w[j][:len(words[j::4])]
    return (words[i] >= math.floor(_p32(c["p"]) * 4294967296)).view(c["rows"], c["D"]).double() / (1 - _p32(c["p"]))


def _exact_norm(c):
    x, w, D = c["x"].double(), c["w"].double(), c["D"]
    ls = 1.0 if c["ls"] is None else c["ls"].double()
    keep = _exact_keep(c) if c["op"] == "norm_drop" else 1.0
    if c["op"] == "norm_drop" and c["bwd"]:
        total, dy = c["sum"].double(), c["dy"].double()
        inv = 1 / torch.sqrt((total * total).sum(1, keepdim=True) / D + EPS)
        hat = total * inv
        d_total = c["d_sum"].double() + inv * (dy * w - hat * (dy * w * hat).sum(1, keepdim=True) / D)
        out = (d_total * ls * keep, d_total, (dy * hat).sum(0))
        return out if c["ls"] is None else out + ((d_total * x * keep).sum(0),)
    total = c["residual"].double() + ls * x * keep
    held = total if c["res"] == "f32" else total.float().to(torch.bfloat16).double()
    y = held / torch.sqrt((held * held).sum(1, keepdim=True) / D + EPS) * w
    if c["op"] == "norm_drop":
        return y, total
    g = y.reshape(c["rows"], -1, c["group"])
    scale = torch.clamp_min(g.abs().max(2).values / E4M3_MAX, TINY)
    return (g / scale.unsqueeze(2)).reshape(c["rows"], D), scale, total


def exact(case, seed):
    c = prepare(case, seed)
    return _exact_scan(c) if c["op"].startswith("scan") else _exact_norm(c)
