"""Plain fp64 forms of the state space layer's operators, token by token, and
the error bounds that the tests hold the kernels to.

Token tensors are flat ([T, ...]); `spans` lists each sequence's (start, length).

The scan's bounds come from running, beside the recurrence, the recurrence of
its absolute values and that of a first-order bound of the rounding errors:
    |h|:  H_t = a_t H_{t-1} + |b_t|
    err:  E_t = a_t E_{t-1} + e_a a_t H_{t-1} + e_b |b_t| + U H_t
with U = 2^-24 the rounding of one fp32 operation, e_b = 2^-19 the relative
error of b = dt u B (dt from an exponential, a division and a short series, each
a few ulp) and e_a that of the decay exp(dt A) as computed: 2^-21 for the
approximate exponential and |dt A| (e_dt + 4 U) for its argument.
"""
import torch

U = 2.0 ** -24
E_DT = 2.0 ** -20
E_B = 2.0 ** -19
E_GATE = 2.0 ** -19  # z sigmoid(z) and its derivative: exponential, division, products


def spans_of(lens):
    out, at = [], 0
    for n in lens:
        out.append((at, n))
        at += n
    return out


def softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _steps(p):
    raw = p["delta"] + (p["delta_bias"] if p.get("delta_bias") is not None else 0.0)
    return raw, (softplus(raw) if p["softplus"] else raw)


def _grp(x, D):
    return x.repeat_interleave(D // x.shape[-2], dim=-2)


def scan(p, spans, state_in=None):
    """p: dict of fp64 u, delta [T, D], A [D, n], B, C [T, G, n], optional D, z,
    delta_bias, and softplus. Returns y, state_out, the bounds of both, and all h."""
    T, D = p["u"].shape
    n = p["A"].shape[1]
    raw, dt = _steps(p)
    B, C = _grp(p["B"], D), _grp(p["C"], D)
    a = torch.exp(dt[..., None] * p["A"])
    b = (dt * p["u"])[..., None] * B
    ea = 2.0 ** -21 + (dt[..., None] * p["A"]).abs() * (E_DT + 4 * U)
    hs, Hs, Es = [], [], []
    out_h, out_E = [], []
    zero = torch.zeros((D, n), dtype=torch.float64)
    for i, (at, length) in enumerate(spans):
        h = state_in[i] if state_in is not None else zero
        H, E = h.abs(), zero
        for t in range(at, at + length):
            E = a[t] * E + ea[t] * a[t] * H + E_B * b[t].abs()
            h = a[t] * h + b[t]
            H = a[t] * H + b[t].abs()
            E = E + U * H
            hs.append(h), Hs.append(H), Es.append(E)
        out_h.append(h), out_E.append(E)
    state = torch.stack(out_h) if out_h else zero.new_zeros((0, D, n))
    bound_state = torch.stack(out_E) if out_h else state
    if T == 0:
        return p["u"] * 0, state, p["u"] * 0, bound_state, zero.new_zeros((0, D, n))
    h, H, E = torch.stack(hs), torch.stack(Hs), torch.stack(Es)
    y = (C * h).sum(-1)
    size, err = (C.abs() * H).sum(-1), (C.abs() * E).sum(-1)
    if p.get("D") is not None:
        y = y + p["D"] * p["u"]
        size = size + (p["D"] * p["u"]).abs()
    err = err + (n + 2) * U * size
    if p.get("z") is not None:
        gate = p["z"] * torch.sigmoid(p["z"])
        y = y * gate
        err = (err + E_GATE * size) * gate.abs() + U * 8
    return y, state, 2 * err, 2 * bound_state, h


def scan_backward(p, spans, h, dy, state_in=None, dstate_out=None, size=False):
    """The gradients by their formulas. With `size`, each is the sum of the
    absolute values of its terms instead (inputs must then be absolute values,
    but for A, delta and delta_bias): the scale of its rounding errors."""
    T, D = p["u"].shape
    n, G = p["A"].shape[1], p["B"].shape[1]
    raw, dt = _steps(p)
    B, C = _grp(p["B"], D), _grp(p["C"], D)
    a = torch.exp(dt[..., None] * p["A"])
    A = p["A"].abs() if size else p["A"]
    if size:
        dt = dt.abs()
    Dw = p["D"] if p.get("D") is not None else torch.zeros(D, dtype=torch.float64)
    y = (C * h).sum(-1) + Dw * p["u"]
    out = {}
    w = dy
    if p.get("z") is not None:
        z = p["z_signed"] if size else p["z"]
        sg = torch.sigmoid(z)
        slope = sg * (1 + z * (1 - sg))
        gate = z * sg
        # The slope is a sum of two terms, sg and z sg (1 - sg), which cancel near
        # z = -1.28: each is rounded by itself, so the scale is that of both
        # together, sg + |z| sg (1 - sg), and not the sum's own size.
        out["dz"] = dy * y * (sg * (1 + z.abs() * (1 - sg)) if size else slope)
        w = dy * (gate.abs() if size else gate)
    out["dD"] = (w * p["u"]).sum(0)
    du, ddt = torch.zeros_like(w), torch.zeros_like(w)
    dB, dC = torch.zeros_like(p["B"]), torch.zeros_like(p["C"])
    dA = torch.zeros_like(p["A"])
    dst = []
    zero = torch.zeros((D, n), dtype=torch.float64)
    for i, (at, length) in enumerate(spans):
        carry = dstate_out[i] if dstate_out is not None else zero
        for t in range(at + length - 1, at - 1, -1):
            g = C[t] * w[t, :, None] + carry
            before = h[t - 1] if t > at else (state_in[i] if state_in is not None else zero)
            carry = a[t] * g
            dC[t] = (w[t, :, None] * h[t]).reshape(G, D // G, n).sum(1)
            dB[t] = (g * (dt[t] * p["u"][t])[:, None]).reshape(G, D // G, n).sum(1)
            gb = (g * B[t]).sum(-1)
            du[t] = Dw * w[t] + dt[t] * gb
            ddt[t] = (A * carry * before).sum(-1) + p["u"][t] * gb
            dA += dt[t][:, None] * carry * before
        dst.append(carry)
    out.update(du=du, dB=dB, dC=dC, dA=dA)
    out["ddelta"] = ddt * torch.sigmoid(raw) if p["softplus"] else ddt
    out["ddelta_bias"] = out["ddelta"].sum(0)
    out["dstate_in"] = torch.stack(dst) if dst else zero.new_zeros((0, D, n))
    return out


def scan_backward_bounds(p, spans, dy, state_in=None, dstate_out=None):
    """Bounds of the gradients' errors: the sum of their terms' absolute values
    times the relative error that a product of a state and a gradient of a state
    can have gathered: over L tokens each, L (2^-21 + max|dt A| (e_dt + 4 U) + U)
    on either side, and some constant ones (gate, dt, the sums)."""
    q = {k: (v.abs() if isinstance(v, torch.Tensor) and k not in ("A", "delta", "delta_bias") else v)
         for k, v in p.items()}
    q["z_signed"] = p.get("z")
    st = None if state_in is None else state_in.abs()
    h = scan(q, spans, st)[4]
    sizes = scan_backward(q, spans, h, dy.abs(), st, None if dstate_out is None else dstate_out.abs(),
                          size=True)
    _, dt = _steps(p)
    L = max([n for _, n in spans] + [1])
    arg = float((dt[..., None] * p["A"]).abs().max()) if dt.numel() else 0.0
    rel = 2 * L * (2.0 ** -21 + arg * (E_DT + 4 * U) + U) + 8 * E_GATE
    T = p["u"].shape[0]
    terms = {"dD": T, "dA": T, "ddelta_bias": T, "dB": p["u"].shape[1], "dC": p["u"].shape[1]}
    return {k: v.abs() * (rel + U * terms.get(k, 2 * p["A"].shape[1])) for k, v in sizes.items()}


def conv(x, weight, bias, silu, spans, state_in=None):
    """x [T, D], weight [D, W]. Returns y, state_out [S, W-1, D] and y's bound."""
    D, W = weight.shape
    y, bound, states = torch.zeros_like(x), torch.zeros_like(x), []
    b = bias if bias is not None else torch.zeros(D, dtype=torch.float64)
    for i, (at, length) in enumerate(spans):
        old = state_in[i] if state_in is not None else torch.zeros((W - 1, D), dtype=torch.float64)
        line = torch.cat((old, x[at:at + length]))
        for t in range(length):
            win = line[t:t + W].t()
            pre = (win * weight).sum(-1) + b
            err = (W + 1) * U * ((win * weight).abs().sum(-1) + b.abs())
            y[at + t] = pre * torch.sigmoid(pre) if silu else pre
            # |silu'| <= 1.1
            bound[at + t] = 1.1 * err + E_GATE * y[at + t].abs() if silu else err
        states.append(line[length:])
    state = torch.stack(states) if states else x.new_zeros((0, W - 1, D))
    return y, state, 2 * bound + 2.0 ** -60


def conv_backward(dy, x, weight, bias, silu, spans, state_in=None, dstate_out=None):
    """Gradients by their formulas, and the bounds of their errors."""
    D, W = weight.shape
    b = bias if bias is not None else torch.zeros(D, dtype=torch.float64)
    dx, sx = torch.zeros_like(x), torch.zeros_like(x)
    dw, sw = torch.zeros_like(weight), torch.zeros_like(weight)
    db, sb = torch.zeros_like(b), torch.zeros_like(b)
    ds, ss = [], []
    for i, (at, length) in enumerate(spans):
        old = state_in[i] if state_in is not None else torch.zeros((W - 1, D), dtype=torch.float64)
        line = torch.cat((old, x[at:at + length]))
        dline, sline = torch.zeros_like(line), torch.zeros_like(line)
        for t in range(length):
            win = line[t:t + W].t()
            pre = (win * weight).sum(-1) + b
            mag = (win * weight).abs().sum(-1) + b.abs()
            q, eq = dy[at + t], torch.zeros_like(b)
            if silu:
                sg = torch.sigmoid(pre)
                # |silu''| <= 1/2
                eq = q.abs() * (0.5 * (W + 1) * U * mag + 1.1 * E_GATE)
                q = q * sg * (1 + pre * (1 - sg))
            for j in range(W):
                dline[t + j] += weight[:, j] * q
                sline[t + j] += weight[:, j].abs() * (eq + 2 * W * U * q.abs())
            dw += q[:, None] * win
            sw += (eq + (x.shape[0] + 2) * U * q.abs())[:, None] * win.abs()
            db += q
            sb += eq + (x.shape[0] + 2) * U * q.abs()
        if dstate_out is not None:
            dline[length:] += dstate_out[i]
            sline[length:] += 2 * W * U * dstate_out[i].abs()
        dx[at:at + length], sx[at:at + length] = dline[W - 1:], sline[W - 1:]
        ds.append(dline[:W - 1]), ss.append(sline[:W - 1])
    none = x.new_zeros((0, W - 1, D))
    grads = {"dx": dx, "dweight": dw, "dbias": db, "dstate_in": torch.stack(ds) if ds else none}
    sizes = {"dx": sx, "dweight": sw, "dbias": sb, "dstate_in": torch.stack(ss) if ss else none}
    return grads, {k: 2 * v + 2.0 ** -60 for k, v in sizes.items()}


def layer_norm(x, weight, bias, eps):
    """y, mean, rstd and the bounds of their errors: each sum over F terms adds
    less than F roundings (pairwise in practice), rsqrt and the products a few."""
    F = x.shape[-1]
    mean = x.mean(-1)
    c = x - mean[:, None]
    var = c.square().mean(-1)
    rstd = 1 / torch.sqrt(var + eps)
    n = c * rstd[:, None]
    y = n * weight + (bias if bias is not None else 0.0)
    depth = F / 32 + 64  # longest chain of additions
    e_mean = depth * U * x.abs().mean(-1)
    # d rstd = -rstd^3 / 2 d var; the centred squares move by 2 |c| e_mean at most
    e_var = (depth + 4) * U * var + 2 * c.abs().mean(-1) * e_mean
    e_rstd = 0.5 * rstd ** 3 * e_var + 4 * U * rstd
    e_n = (e_mean[:, None] + 2 * U * (x.abs() + mean.abs()[:, None])) * rstd[:, None] + \
        c.abs() * e_rstd[:, None]
    e_y = e_n * weight.abs() + 4 * U * (n * weight).abs() + 2 * U * y.abs()
    return y, mean, rstd, 2 * e_y, 2 * e_mean, 2 * e_rstd


def layer_norm_backward(dy, x, weight, mean, rstd):
    """Gradients for the given fp32 mean and rstd, and the bounds of their errors."""
    F, R = x.shape[-1], x.shape[0]
    n = (x - mean[:, None]) * rstd[:, None]
    e_n = 3 * U * (x.abs() + mean.abs()[:, None]) * rstd[:, None]
    e = dy * weight
    dx = rstd[:, None] * (e - e.mean(-1, keepdim=True) - n * (e * n).mean(-1, keepdim=True))
    depth = F / 32 + 64
    m1 = e.abs().mean(-1, keepdim=True)
    m2 = (e * n).abs().mean(-1, keepdim=True)
    e_m2 = (depth + 4) * U * m2 + (e.abs() * e_n).mean(-1, keepdim=True)
    s = rstd[:, None] * (4 * U * e.abs() + (depth + 4) * U * m1 + n.abs() * e_m2 + (e_n + 4 * U * n.abs()) * m2)
    dw, db = (dy * n).sum(0), dy.sum(0)
    sw = (dy.abs() * (e_n + (R + 4) * U * n.abs())).sum(0)
    sb = (R + 4) * U * dy.abs().sum(0)
    return (dx, dw, db), (2 * s, 2 * sw, 2 * sb)


def check(got, want, bound, what):
    """|got - want| <= bound + half a step of got's type, elementwise."""
    g = got.detach().cpu().double()
    assert g.shape == want.shape, f"{what}: {tuple(g.shape)} instead of {tuple(want.shape)}"
    step = torch.finfo(got.dtype).eps / 2
    limit = bound * (1 + step) + step * want.abs() + 2.0 ** -126
    bad = ~((g - want).abs() <= limit)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} values off, the worst by "
                           f"{float(((g - want).abs() / limit)[bad].max()):.3g} times the bound")
