"""The scan and its gradients in fp64 with bounds of the kernels' rounding errors
that follow the errors themselves: beside each recurrence run that of its terms'
absolute values and that of a first-order bound of its error, forward for the
state h and in reverse for its gradient g, so that an error decays as its state
does. On any device; the convolution in fp64 without a loop over tokens.

Relative errors of one operation, U = 2^-24 the rounding of an fp32 one:
    E_DT + U |raw|   of dt = softplus(raw) and of its slope. The exponential has
                     2^-22 = 4 U, the reciprocal 2 U, the polynomial and the
                     products and sums around them 7 U, less than E_DT = 16 U;
                     raw = delta + bias is rounded, which moves dt by U |raw| dt
                     at most
    ea               of the decay exp(dt A): 2^-21 = 8 U for the exponential, and
                     its argument's error |dt A| (e_dt + 4 U). Where the kernel
                     takes the decay of m tokens as exp(A sum dt), the sum's m U
                     |A| sum dt stands against the 8 m U that m decays have here
    E_GATE           of z sigmoid(z): |z| 2.2 U for the exponent, 8 U for the rest,
                     less than 32 U up to |z| = 10
A sum of terms along a chain of k additions is off by k U times the sum of their
absolute values. Every bound is doubled, for products of errors and for the sums
of dt where they pass what the decays have.
"""
import torch

from tests.ssm_reference import E_DT, E_GATE, U, softplus


def scan(p, spans, chunk, dy=None, state_in=None, dstate_out=None):
    """(values, bounds) of y and state, and with dy of every gradient, as dicts.
    `chunk`: tokens that the backward kernel walks from zero before it joins them."""
    dev = p["u"].device
    f = dict(dtype=torch.float64, device=dev)
    T, D = p["u"].shape
    n, G = p["A"].shape[1], p["B"].shape[1]
    bias = p["delta_bias"] if p.get("delta_bias") is not None else torch.zeros(D, **f)
    raw = p["delta"] + bias
    dt = softplus(raw) if p["softplus"] else raw
    e_dt = E_DT + U * raw.abs()
    Dw = p["D"] if p.get("D") is not None else torch.zeros(D, **f)
    A, u = p["A"], p["u"]
    wide = lambda x: x.repeat_interleave(D // G, dim=0)  # noqa: E731
    zero = torch.zeros((D, n), **f)

    def token(t):
        a = torch.exp(dt[t, :, None] * A)
        ea = 2.0 ** -21 + (dt[t, :, None] * A).abs() * (e_dt[t, :, None] + 4 * U)
        return a, ea, wide(p["B"][t]), wide(p["C"][t])

    h_all, E_all = torch.zeros((T, D, n), **f), torch.zeros((T, D, n), **f)
    pre, e_pre = torch.zeros((T, D), **f), torch.zeros((T, D), **f)
    states, e_states = torch.zeros((len(spans), D, n), **f), torch.zeros((len(spans), D, n), **f)
    for i, (at, length) in enumerate(spans):
        h = state_in[i] if state_in is not None else zero
        H, E = h.abs(), zero
        for t in range(at, at + length):
            a, ea, B, C = token(t)
            b = (dt[t] * u[t])[:, None] * B
            E = a * (E + ea * H) + (e_dt[t, :, None] + 4 * U) * b.abs()
            h, H = a * h + b, a * H + b.abs()
            E = E + U * H
            h_all[t], E_all[t] = h, E
            pre[t] = (C * h).sum(-1) + Dw * u[t]
            e_pre[t] = (C.abs() * E).sum(-1) + (n + 4) * U * ((C * h).abs().sum(-1) + (Dw * u[t]).abs())
        states[i], e_states[i] = h, E
    gate, slope, e_slope = torch.ones((T, D), **f), None, None
    if p.get("z") is not None:
        sg = torch.sigmoid(p["z"])
        gate, slope = p["z"] * sg, sg * (1 + p["z"] * (1 - sg))
        # sg and z sg (1 - sg) cancel near z = -1.28, each with its own rounding
        e_slope = E_GATE * sg * (1 + p["z"].abs() * (1 - sg))
    y = pre * gate
    value = {"y": y, "state": states}
    bound = {"y": e_pre * gate.abs() + E_GATE * y.abs(), "state": e_states}
    if dy is not None:
        w = dy * gate
        ew = E_GATE if slope is not None else 0.0
        du, ddelta = torch.zeros((T, D), **f), torch.zeros((T, D), **f)
        e_du, e_dd = torch.zeros((T, D), **f), torch.zeros((T, D), **f)
        dB, dC = torch.zeros((T, G, n), **f), torch.zeros((T, G, n), **f)
        e_dB, e_dC = torch.zeros((T, G, n), **f), torch.zeros((T, G, n), **f)
        dA, e_dA, s_dA = zero.clone(), zero.clone(), zero.clone()
        d_in, e_in = torch.zeros((len(spans), D, n), **f), torch.zeros((len(spans), D, n), **f)
        over_channels = D // G / 16 + 16   # a CTA has 16 channels at least
        over_tokens = chunk + T // chunk + len(spans) + 16
        group = lambda x: x.reshape(G, D // G, n).sum(1)  # noqa: E731
        for i, (at, length) in enumerate(spans):
            c = dstate_out[i] if dstate_out is not None else zero
            Cm, Ce = c.abs(), zero
            for t in range(at + length - 1, at - 1, -1):
                a, ea, B, C = token(t)
                h, E = h_all[t], E_all[t]
                if t > at:
                    before, Eb = h_all[t - 1], E_all[t - 1]
                else:
                    before, Eb = (state_in[i] if state_in is not None else zero), zero
                wt = w[t, :, None]
                g = C * wt + c
                Gm = (C * wt).abs() + Cm
                Ge = (C * wt).abs() * (ew + 2 * U) + Ce + U * Gm
                dC[t] = group(wt * h)
                size = (wt * h).abs()
                e_dC[t] = group(wt.abs() * E + size * (ew + 2 * U)) + over_channels * U * group(size)
                add = (dt[t] * u[t])[:, None]
                dB[t] = group(g * add)
                size = (g * add).abs()
                e_dB[t] = group(add.abs() * Ge + size * (e_dt[t, :, None] + 4 * U)) + over_channels * U * group(size)
                gb = (g * B).sum(-1)
                e_gb = (B.abs() * Ge).sum(-1) + (n + 4) * U * (g * B).abs().sum(-1)
                du[t] = Dw * w[t] + dt[t] * gb
                e_du[t] = ((Dw * w[t]).abs() * (ew + 4 * U) + dt[t].abs() * e_gb +
                           (dt[t] * gb).abs() * (e_dt[t] + 4 * U))
                c, Cm, Ce = a * g, a * Gm, a * (Ge + (ea + U) * Gm)
                left = c * before
                e_left = Ce * before.abs() + c.abs() * Eb + Ce * Eb
                ddt = (A * left).sum(-1) + u[t] * gb
                e_ddt = ((A.abs() * e_left).sum(-1) + (n + 8) * U * (A * left).abs().sum(-1) +
                         u[t].abs() * e_gb + 4 * U * (u[t] * gb).abs())
                sl = torch.sigmoid(raw[t]) if p["softplus"] else torch.ones_like(raw[t])
                ddelta[t] = ddt * sl
                e_dd[t] = sl * (e_ddt + ddt.abs() * (e_dt[t] if p["softplus"] else U))
                dA += dt[t, :, None] * left
                size = (dt[t, :, None] * left).abs()
                s_dA += size
                e_dA += dt[t, :, None].abs() * e_left + size * (e_dt[t, :, None] + 4 * U)
                if (t - at) % chunk == 0:
                    # the chunk's own share of g was summed from its first token on
                    Ce = Ce + chunk * U * Cm
            d_in[i], e_in[i] = c, Ce
        value.update(du=du, ddelta=ddelta, dB=dB, dC=dC, dA=dA, dD=(w * u).sum(0), ddelta_bias=ddelta.sum(0),
                     dstate_in=d_in)
        bound.update(du=e_du, ddelta=e_dd, dB=e_dB, dC=e_dC, dA=e_dA + over_tokens * U * s_dA,
                     dD=(ew + (over_tokens + 2) * U) * (w * u).abs().sum(0),
                     ddelta_bias=e_dd.sum(0) + over_tokens * U * ddelta.abs().sum(0), dstate_in=e_in)
        if slope is not None:
            value["dz"] = dy * pre * slope
            bound["dz"] = dy.abs() * (e_pre * slope.abs() + pre.abs() * e_slope) + 4 * U * value["dz"].abs()
    # 1e-36: what is below fp32's normal range counts as 0
    return value, {k: 2 * v + 1e-36 for k, v in bound.items()}


def conv(x, weight, bias, silu, lens, state_in=None, dy=None, dstate_out=None, chain=0):
    """(values, bounds) of y and state, with dy of the gradients. `chain`: most
    additions in a row of the sums over tokens (0: the number of tokens)."""
    f = dict(dtype=torch.float64, device=x.device)
    D, W = weight.shape
    T, S = x.shape[0], len(lens)
    b = bias if bias is not None else torch.zeros(D, **f)
    # each sequence's W - 1 earlier inputs, then its own
    ln = torch.tensor(lens, device=x.device)
    seq = torch.repeat_interleave(torch.arange(S, device=x.device), ln)
    own = torch.arange(T, device=x.device) + (seq + 1) * (W - 1)
    first = torch.cumsum(ln, 0) - ln + torch.arange(S, device=x.device) * (W - 1)
    head = (first[:, None] + torch.arange(W - 1, device=x.device)).flatten()
    tail = (first[:, None] + ln[:, None] + torch.arange(W - 1, device=x.device)).flatten()
    line = torch.zeros((T + S * (W - 1), D), **f)
    line[own] = x
    if state_in is not None:
        line[head] = state_in.flatten(0, 1)
    pre, mag = b.expand(T, D).clone(), b.abs().expand(T, D).clone()
    for j in range(W):
        term = line[own - (W - 1) + j] * weight[:, j]
        pre += term
        mag += term.abs()
    e_pre = (W + 1) * U * mag
    y = pre * torch.sigmoid(pre) if silu else pre
    value = {"y": y, "state": line[tail].unflatten(0, (S, W - 1))}
    # |silu'| <= 1.1
    bound = {"y": 1.1 * e_pre + E_GATE * y.abs() if silu else e_pre, "state": torch.zeros_like(value["state"])}
    if dy is not None:
        q, e_q = dy, torch.zeros_like(dy)
        if silu:
            sg = torch.sigmoid(pre)
            q = dy * sg * (1 + pre * (1 - sg))
            e_q = dy.abs() * (0.5 * e_pre + 1.1 * E_GATE)  # |silu''| <= 1/2
        chain = chain or T
        dline, e_line = torch.zeros_like(line), torch.zeros_like(line)
        dw, e_dw = torch.zeros_like(weight), torch.zeros_like(weight)
        for j in range(W):
            at = own - (W - 1) + j
            dline.index_add_(0, at, weight[:, j] * q)
            e_line.index_add_(0, at, weight[:, j].abs() * (e_q + 2 * W * U * q.abs()))
            dw[:, j] = (q * line[at]).sum(0)
            e_dw[:, j] = ((e_q + (chain + 2) * U * q.abs()) * line[at].abs()).sum(0)
        if dstate_out is not None:
            dline.index_add_(0, tail, dstate_out.flatten(0, 1))
            e_line.index_add_(0, tail, 2 * W * U * dstate_out.abs().flatten(0, 1))
        value.update(dx=dline[own], dweight=dw, dbias=q.sum(0), dstate_in=dline[head].unflatten(0, (S, W - 1)))
        bound.update(dx=e_line[own], dweight=e_dw, dbias=(e_q + (chain + 2) * U * q.abs()).sum(0),
                     dstate_in=e_line[head].unflatten(0, (S, W - 1)))
    return value, {k: 2 * v + 1e-36 for k, v in bound.items()}
