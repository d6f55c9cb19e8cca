"""Cases of the state space layer's operators: the selective scan, the short
causal convolution before it and the layer norm around them, each over prompts,
for single tokens and backward.

With ``own`` false, ``run`` computes an operator by its formula in elementary
torch operations, in fp32 (rounded once at the end); with ``own`` true it makes
the library's calls. ``exact`` computes the same in fp64, token by token.

Layouts are those of the library: token-major rows. Dense inputs are [B, N, ...]
and packed ones [T, ...] with int32 cu_seqlens; a case with "lens" is packed.
As in a layer, the convolution's input and the scan's gate z are the two halves
of one projection [.., 2 D], and B and C are slices of another [.., r + 2 G n].

    scan:  dt = softplus(delta + bias),  h_t = exp(dt A) h_{t-1} + dt u B_t,
           y_t = (C_t . h_t + D u) z sigmoid(z)
    conv:  y_t = silu(bias + sum_j w_j x_{t - (W-1) + j})
    norm:  y = (x - mean) / sqrt(var + eps) w + b
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5


def listed():
    return [
        # One generated token for a handful of sequences: latency counts.
        {"name": "scan step, 8 sequences", "op": "scan_step", "B": 8, "D": 8192, "G": 1, "n": 16, "dtype": "bf16"},
        # One generated token for a full decode batch: the states' stream from memory.
        {"name": "scan step, 256 sequences", "op": "scan_step", "B": 256, "D": 8192, "G": 1, "n": 16, "dtype": "bf16"},
        # A long prompt through a wide layer.
        {"name": "scan, 8K prompt", "op": "scan", "B": 1, "N": 8192, "D": 8192, "G": 1, "n": 16, "dtype": "bf16", "state": False},
        # Packed prompts that continue cached ones, one of them long, in a narrow layer: little to do at once but time.
        {"name": "scan, packed, fp32", "op": "scan", "lens": "40001,2500,1,517,0,2000", "D": 1024, "G": 2, "n": 16, "dtype": "f32", "state": True},
        # The gradients of a training step.
        {"name": "scan backward", "op": "scan_bwd", "B": 2, "N": 4096, "D": 4096, "G": 1, "n": 16, "dtype": "bf16", "state": False},
        # The gradients of a small ragged fp32 batch with odd sizes.
        {"name": "scan backward, packed, fp32", "op": "scan_bwd", "lens": "700,1,0,333,64,65", "D": 1001, "G": 1, "n": 10, "dtype": "f32", "state": True},
        # Prompts through the convolution.
        {"name": "conv, 4 x 8K prompts", "op": "conv", "B": 4, "N": 8192, "D": 8192, "W": 4, "dtype": "bf16", "state": False},
        # Its gradients in a training step.
        {"name": "conv backward", "op": "conv_bwd", "B": 2, "N": 8192, "D": 8192, "W": 4, "dtype": "bf16", "state": False},
        # One generated token for a decode batch.
        {"name": "conv step, 64 sequences", "op": "conv_step", "B": 64, "D": 8192, "W": 4, "dtype": "bf16"},
        # The norm of a long prompt.
        {"name": "norm, 32K rows", "op": "norm", "rows": 32768, "F": 8192, "dtype": "bf16"},
        # Its gradients in a training step, the weight's summed over all rows.
        {"name": "norm backward, 16K rows", "op": "norm_bwd", "rows": 16384, "F": 8192, "dtype": "bf16"},
        # Odd sizes in fp32.
        {"name": "norm backward, odd, fp32", "op": "norm_bwd", "rows": 517, "F": 5003, "dtype": "f32"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A number of features: a multiple of 64 mostly, any number otherwise."""
    n = _log_int(rng, lo, hi)
    return n if rng.random() < 0.3 else max(64, n // 64 * 64)


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_bwd", "scan_bwd", "scan_step", "conv", "conv_bwd", "conv_step", "norm", "norm_bwd"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op in ("norm", "norm_bwd"):
        F = _width(rng, 64, 16384)
        return {**c, "rows": _log_int(rng, 1, min(32768, (1 << 27) // F)), "F": F}
    D = _width(rng, 64, 8192)
    if op.startswith("scan"):
        c["n"] = rng.choice([4, 8, 16, 16, 16, 32, 64, rng.randint(1, 64)])
        c["G"] = rng.choice([1, 1, 1, 2, 4])
        D -= D % c["G"]
        most = (1 << 25) // (D * max(c["n"], 4) // 16)  # tokens
    else:
        c["W"] = rng.randint(2, 4)
        most = (1 << 27) // D
    c["D"] = D
    if op.endswith("_step"):
        return {**c, "B": _log_int(rng, 1, min(256, most))}
    most = min(most, 40000)
    c["state"] = rng.random() < 0.5
    if rng.random() < 0.5:
        B = _log_int(rng, 1, 16)
        return {**c, "B": B, "N": _log_int(rng, 1, max(1, most // B))}
    lens, left = [], most
    for _ in range(rng.randint(1, 10)):
        n = rng.choice([0, 1, 2, 3]) if rng.random() < 0.25 else _log_int(rng, 1, max(1, left))
        n = min(n, left)
        lens.append(n)
        left -= n
    if sum(lens) == 0:
        lens.append(1)
    return {**c, "lens": ",".join(map(str, lens))}


# ---------------------------------------------------------------- inputs

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def _lead(case):
    """Leading shape of the token tensors, and the number of sequences."""
    if "lens" in case:
        lens = _lens(case)
        return (sum(lens),), len(lens)
    if "N" in case:
        return (case["B"], case["N"]), case["B"]
    return (case["B"],), case["B"]


def _cu(case):
    if "lens" not in case:
        return None
    cu = [0]
    for n in _lens(case):
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def rnd(*shape, dtype=torch.float32, scale=1.0):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(scale).to(dtype)

    op, t = case["op"], _dtype(case)
    s = {"op": op}
    if op in ("norm", "norm_bwd"):
        rows, F = case["rows"], case["F"]
        s["x"] = rnd(rows, F, dtype=t).add_(0.3)
        s["weight"] = 1 + 0.2 * rnd(F)
        s["bias"] = 0.2 * rnd(F)
        if op == "norm_bwd":
            s["dy"] = rnd(rows, F, dtype=t)
            x = s["x"].double()  # kept by the forward pass of a training step
            s["mean"] = x.mean(-1)
            s["rstd"] = ((x - s["mean"][:, None]).square().mean(-1) + EPS).rsqrt().float()
            s["mean"] = s["mean"].float()
        return s
    lead, seqs = _lead(case)
    D = case["D"]
    s["cu"] = _cu(case)
    if op.startswith("conv"):
        W = case["W"]
        s["x"] = rnd(*lead, 2 * D, dtype=t)[..., :D]
        s["weight"] = rnd(D, W, scale=W ** -0.5)
        s["bias"] = rnd(D, scale=0.1)
        if op == "conv_step" or case.get("state"):
            s["state"] = rnd(seqs, W - 1, D, dtype=t)
        if op == "conv_bwd":
            s["dy"] = rnd(*lead, D, dtype=t)
        return s
    G, n = case["G"], case["n"]
    r = max(8, D // 16 // 8 * 8)
    s["u"] = rnd(*lead, D, dtype=t)
    s["delta"] = rnd(*lead, D, dtype=t, scale=0.5)
    s["z"] = rnd(*lead, 2 * D, dtype=t)[..., D:]
    proj = rnd(*lead, r + 2 * G * n, dtype=t)
    s["B"] = proj[..., r:r + G * n].unflatten(-1, (G, n))
    s["C"] = proj[..., r + G * n:].unflatten(-1, (G, n))
    s["A"] = -torch.arange(1, n + 1, device=DEV, dtype=torch.float32).expand(D, n) * (1 + 0.1 * torch.rand((D, n), generator=g, device=DEV))
    s["D"] = 1 + 0.1 * rnd(D)
    # steps of 1e-3 to 1e-1, spread over their logarithm: softplus(bias) = dt
    dt = torch.exp(torch.rand(D, generator=g, device=DEV) * math.log(100.0) + math.log(1e-3))
    s["delta_bias"] = dt + torch.log(-torch.expm1(-dt))
    if op == "scan_step" or case.get("state"):
        s["state"] = rnd(seqs, D, n, scale=0.2)
    if op == "scan_bwd":
        s["dy"] = rnd(*lead, D, dtype=t)
        if case.get("state"):
            s["dstate"] = rnd(seqs, D, n, scale=0.2)
    return s


# ---------------------------------------------------------------- plain forms

def _first(s, lead):
    """Per token: the index of its sequence and its place in it, as flat tensors."""
    if s["cu"] is None:
        seq = torch.arange(lead[0], device=DEV).repeat_interleave(lead[1])
        return seq, torch.arange(lead[1], device=DEV).repeat(lead[0])
    lens = (s["cu"][1:] - s["cu"][:-1]).long()
    seq = torch.arange(lens.numel(), device=DEV).repeat_interleave(lens, output_size=lead[0])
    return seq, torch.arange(lead[0], device=DEV) - s["cu"].long()[seq]


def _lengths(s, lead):
    return torch.full((lead[0],), lead[1], device=DEV) if s["cu"] is None else (s["cu"][1:] - s["cu"][:-1]).long()


def _flat(x, lead):
    return x.reshape((-1,) + tuple(x.shape[len(lead):])).float()


def _cum(a, b):
    """h_t = a_t h_{t-1} + b_t from h_{-1} = 0 along the first axis, by doubling."""
    step = 1
    while step < a.shape[0]:
        b = torch.cat((b[:step], torch.addcmul(b[step:], a[step:], b[:-step])))
        a = torch.cat((a[:step], a[step:] * a[:-step]))
        step *= 2
    return b


def _per_channel(x, D):
    """[.., G, n] to [.., D, n]: group g serves the channels g D/G to (g + 1) D/G - 1."""
    return x.repeat_interleave(D // x.shape[-2], dim=-2)


def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _scan_states(s, lead, seqs):
    """u, dt, B, C, a = exp(dt A) and all h, flat over tokens, with each token's sequence and place."""
    D = s["A"].shape[0]
    u, B, C = _flat(s["u"], lead), _per_channel(_flat(s["B"], lead), D), _per_channel(_flat(s["C"], lead), D)
    dt = _softplus(_flat(s["delta"], lead) + s["delta_bias"])
    a = torch.exp(dt[..., None] * s["A"])
    b = (dt * u)[..., None] * B
    seq, place = _first(s, lead)
    start = place == 0
    if "state" in s:
        b[start] += a[start] * s["state"][seq[start]]
    h = _cum(a.masked_fill(start[:, None, None], 0.0), b)
    return u, dt, B, C, a, h, seq, place


def _final(s, h, lead, seqs):
    """The state after each sequence's last token; an empty sequence keeps its own."""
    last = _lengths(s, lead)
    end = last.cumsum(0) - 1
    out = h[end.clamp(min=0)] if h.shape[0] else h.new_zeros((seqs,) + tuple(h.shape[1:]))
    keep = s["state"] if "state" in s else torch.zeros_like(out)
    return torch.where((last > 0)[:, None, None], out, keep)


def _plain_scan(s):
    lead = tuple(s["u"].shape[:-1])
    seqs = lead[0] if s["cu"] is None else s["cu"].numel() - 1
    u, _, _, C, _, h, _, _ = _scan_states(s, lead, seqs)
    z = _flat(s["z"], lead)
    y = ((C * h).sum(-1) + s["D"] * u) * z * torch.sigmoid(z)
    return y.to(s["u"].dtype).reshape(s["u"].shape), _final(s, h, lead, seqs)


def _plain_scan_step(s):
    D = s["A"].shape[0]
    u, z = s["u"].float(), s["z"].float()
    dt = _softplus(s["delta"].float() + s["delta_bias"])
    s["state"].mul_(torch.exp(dt[..., None] * s["A"])).add_((dt * u)[..., None] * _per_channel(s["B"].float(), D))
    y = ((_per_channel(s["C"].float(), D) * s["state"]).sum(-1) + s["D"] * u) * z * torch.sigmoid(z)
    return y.to(s["u"].dtype), s["state"]


def _plain_scan_bwd(s):
    lead, t = tuple(s["u"].shape[:-1]), s["u"].dtype
    D, n, G = s["A"].shape[0], s["A"].shape[1], s["B"].shape[-2]
    seqs = lead[0] if s["cu"] is None else s["cu"].numel() - 1
    u, dt, B, C, a, h, seq, place = _scan_states(s, lead, seqs)
    z, dy = _flat(s["z"], lead), _flat(s["dy"], lead)
    sig = torch.sigmoid(z)
    dz = dy * ((C * h).sum(-1) + s["D"] * u) * sig * (1 + z * (1 - sig))
    dy = dy * z * sig
    # g_t = C_t dy_t + a_{t+1} g_{t+1}: the same recurrence in reversed time
    lens = _lengths(s, lead)
    end = place == lens[seq] - 1
    g = C * dy[..., None]
    if "dstate" in s:
        g[end] += s["dstate"][seq[end]]
    coef = torch.cat((a[1:], torch.zeros_like(a[:1]))).masked_fill(end[:, None, None], 0.0)
    g = _cum(coef.flip(0), g.flip(0)).flip(0)
    before = torch.cat((torch.zeros_like(h[:1]), h[:-1])).masked_fill((place == 0)[:, None, None], 0.0)
    if "state" in s:
        before[place == 0] = s["state"][seq[place == 0]]
    dC = (h * dy[..., None]).reshape(-1, G, D // G, n).sum(2)
    dB = (g * (dt * u)[..., None]).reshape(-1, G, D // G, n).sum(2)
    gB = (g * B).sum(-1)
    ga = g * a * before
    ddt = (ga * s["A"]).sum(-1) + u * gB
    ddelta = ddt * torch.sigmoid(_flat(s["delta"], lead) + s["delta_bias"])
    out = {"du": (s["D"] * dy + dt * gB).to(t).reshape(s["u"].shape), "ddelta": ddelta.to(t).reshape(s["u"].shape),
           "dz": dz.to(t).reshape(s["u"].shape), "dB": dB.to(t).reshape(s["B"].shape), "dC": dC.to(t).reshape(s["C"].shape),
           "dA": (ga * dt[..., None]).sum(0), "dD": (dy * u).sum(0), "ddelta_bias": ddelta.sum(0)}
    if "state" in s:
        keep = s["dstate"] if "dstate" in s else torch.zeros_like(s["state"])
        begin = (lens.cumsum(0) - lens).clamp(max=max(0, a.shape[0] - 1))
        out["dstate_in"] = torch.where((lens > 0)[:, None, None], (a * g)[begin], keep)
    return out


def _taps(s, lead):
    """The W inputs under each token's window, fp32, oldest first, flat over tokens."""
    x, W = _flat(s["x"], lead), s["weight"].shape[1]
    seq, place = _first(s, lead)
    if "state" in s:
        old = s["state"].float()
    else:
        old = x.new_zeros((int(lead[0]) if s["cu"] is None else s["cu"].numel() - 1, W - 1, x.shape[-1]))
    taps = []
    for j in range(W):
        back = W - 1 - j
        tap = torch.cat((x.new_zeros((back,) + tuple(x.shape[1:])), x))[:x.shape[0]]
        early = place < back
        tap[early] = old[seq[early], (place + j)[early]]
        taps.append(tap)
    return taps, seq, place


def _plain_conv(s):
    lead = tuple(s["x"].shape[:-1])
    taps, seq, place = _taps(s, lead)
    W = len(taps)
    pre = s["bias"].expand_as(taps[0])
    for j in range(W):
        pre = torch.addcmul(pre, taps[j], s["weight"][:, j])
    y = (pre * torch.sigmoid(pre)).to(s["x"].dtype).reshape(s["x"].shape)
    # the last W - 1 inputs of each sequence
    x, lens = _flat(s["x"], lead), _lengths(s, lead)
    begin = lens.cumsum(0) - lens
    at = lens[:, None] - (W - 1) + torch.arange(W - 1, device=DEV)
    state = x[(begin[:, None] + at).clamp(0, max(0, x.shape[0] - 1))]
    older = at < 0
    state[older] = 0.0
    if "state" in s:
        seqs = torch.arange(lens.numel(), device=DEV)[:, None].expand_as(at)
        state[older] = s["state"].float()[seqs[older], (at + W - 1)[older]]
    return y, state.to(s["x"].dtype)


def _plain_conv_step(s):
    x, st = s["x"], s["state"]
    window = torch.cat((st, x[:, None]), 1)
    pre = s["bias"] + (window.float() * s["weight"].t()).sum(1)
    st.copy_(window[:, 1:])
    return (pre * torch.sigmoid(pre)).to(x.dtype), st


def _plain_conv_bwd(s):
    lead, t = tuple(s["x"].shape[:-1]), s["x"].dtype
    taps, seq, place = _taps(s, lead)
    W = len(taps)
    pre = s["bias"].expand_as(taps[0])
    for j in range(W):
        pre = torch.addcmul(pre, taps[j], s["weight"][:, j])
    sig = torch.sigmoid(pre)
    g = _flat(s["dy"], lead) * sig * (1 + pre * (1 - sig))
    left = _lengths(s, lead)[seq] - 1 - place
    dx = torch.zeros_like(g)
    for j in range(W):
        ahead = W - 1 - j
        part = torch.cat((g, g.new_zeros((ahead, g.shape[1]))))[ahead:].masked_fill((left < ahead)[:, None], 0.0)
        dx = torch.addcmul(dx, part, s["weight"][:, j])
    out = {"dx": dx.to(t).reshape(s["x"].shape), "dweight": torch.stack([(g * x).sum(0) for x in taps], 1), "dbias": g.sum(0)}
    if "state" in s:
        dst = torch.zeros_like(s["state"], dtype=torch.float32)
        for j in range(W):  # token place p with p < W - 1 - j reads row p + j of the old inputs
            early = place < W - 1 - j
            dst.index_put_((seq[early], (place + j)[early]), g[early] * s["weight"][:, j], accumulate=True)
        out["dstate_in"] = dst.to(t)
    return out


def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(-1)
    c = x - mean[:, None]
    rstd = (c.square().mean(-1) + EPS).rsqrt()
    return (c * rstd[:, None] * s["weight"] + s["bias"]).to(s["x"].dtype), mean, rstd


def _plain_norm_bwd(s):
    n = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["weight"]
    dx = (g - g.mean(-1, keepdim=True) - n * (g * n).mean(-1, keepdim=True)) * s["rstd"][:, None]
    return dx.to(s["x"].dtype), (dy * n).sum(0), dy.sum(0)


_PLAIN = {"scan": _plain_scan, "scan_step": _plain_scan_step, "scan_bwd": _plain_scan_bwd, "conv": _plain_conv, "conv_step": _plain_conv_step,
          "conv_bwd": _plain_conv_bwd, "norm": _plain_norm, "norm_bwd": _plain_norm_bwd}


# ---------------------------------------------------------------- the library's calls

def _own(s):
    from long_context_02_b200 import binding as L

    op = s["op"]
    if op == "scan":
        return L.selective_scan(s["u"], s["delta"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], delta_bias=s["delta_bias"], softplus=True,
                                state_in=s.get("state"), cu_seqlens=s["cu"])
    if op == "scan_step":
        y = L.selective_scan_step(s["u"], s["delta"], s["A"], s["B"], s["C"], s["state"], D=s["D"], z=s["z"], delta_bias=s["delta_bias"], softplus=True)
        return y, s["state"]
    if op == "scan_bwd":
        return L.selective_scan_backward(s["dy"], s["u"], s["delta"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], delta_bias=s["delta_bias"],
                                         softplus=True, state_in=s.get("state"), dstate_out=s.get("dstate"), cu_seqlens=s["cu"])
    if op == "conv":
        return L.short_conv(s["x"], s["weight"], s["bias"], silu=True, state_in=s.get("state"), cu_seqlens=s["cu"], want_state=True)
    if op == "conv_step":
        return L.short_conv_step(s["x"], s["weight"], s["bias"], s["state"], silu=True), s["state"]
    if op == "conv_bwd":
        return L.short_conv_backward(s["dy"], s["x"], s["weight"], s["bias"], silu=True, state_in=s.get("state"), cu_seqlens=s["cu"])
    if op == "norm":
        return L.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)
    return L.layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"])


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op in ("norm", "norm_bwd"):
        x, F = case["rows"] * case["F"], case["F"]
        if op == "norm":
            return {"bytes": 2 * e * x + 8 * F + 8 * case["rows"], "flops": 8 * x}
        return {"bytes": 3 * e * x + 12 * F + 8 * case["rows"], "flops": 14 * x}
    lead, seqs = _lead(case)
    tokens, D = math.prod(lead), case["D"]
    x = tokens * D
    if op.startswith("conv"):
        W = case["W"]
        states = seqs * (W - 1) * D * e * ((1 if op == "conv" else 0) + (1 if "state" in case and case["state"] or op == "conv_step" else 0))
        if op == "conv_step":
            return {"bytes": 2 * e * x + 2 * seqs * (W - 1) * D * e + 4 * D * (W + 1), "flops": x * (2 * W + 5)}
        if op == "conv":
            return {"bytes": 2 * e * x + states + 4 * D * (W + 1), "flops": x * (2 * W + 5)}
        return {"bytes": 3 * e * x + 2 * states + 8 * D * (W + 1), "flops": x * (6 * W + 10)}
    G, n = case["G"], case["n"]
    bc = 2 * tokens * G * n * e
    held = seqs * D * n * 4
    weights = D * n * 4 + 8 * D
    if op == "scan_step":
        return {"bytes": 4 * e * x + bc + 2 * held + weights, "flops": x * (7 * n + 16)}
    more = held if case.get("state") else 0
    if op == "scan":
        return {"bytes": 4 * e * x + bc + held + more + weights, "flops": x * (7 * n + 16)}
    return {"bytes": 7 * e * x + 2 * bc + 3 * more + 2 * weights, "flops": x * (21 * n + 40)}


# ---------------------------------------------------------------- fp64, token by token

def _sequences(case):
    """(first flat token, length) of each sequence."""
    if "lens" in case:
        out, at = [], 0
        for n in _lens(case):
            out.append((at, n))
            at += n
        return out
    return [(b * case["N"], case["N"]) for b in range(case["B"])]


def _exact_scan(case, s):
    back = case["op"] == "scan_bwd"
    D, n, G = case["D"], case["n"], case["G"]
    f = lambda x: x.double().reshape(-1, *x.shape[(1 if "lens" in case or "N" not in case else 2):])  # noqa: E731
    u, z, A, Dw = f(s["u"]), f(s["z"]), s["A"].double(), s["D"].double()
    raw = f(s["delta"]) + s["delta_bias"].double()
    dt = torch.nn.functional.softplus(raw, threshold=60.0)
    Bm, Cm = f(s["B"]), f(s["C"])
    dtu = dt * u
    group = torch.arange(D, device=DEV) // (D // G)
    y, out_state = torch.empty_like(u), []
    hs = torch.empty((u.shape[0], D, n), dtype=torch.float64, device=DEV) if back else None
    spans = _sequences(case)
    for i, (at, length) in enumerate(spans):
        h = s["state"][i].double() if "state" in s else torch.zeros((D, n), dtype=torch.float64, device=DEV)
        for t in range(at, at + length):
            h = torch.exp(dt[t, :, None] * A) * h + dtu[t, :, None] * Bm[t][group]
            y[t] = (Cm[t][group] * h).sum(-1)
            if back:
                hs[t] = h
        out_state.append(h)
    gate = z / (1 + torch.exp(-z))
    if not back:
        return ((y + Dw * u) * gate).reshape(s["u"].shape), torch.stack(out_state)
    dy = f(s["dy"])
    sg = 1 / (1 + torch.exp(-z))
    dz = dy * (y + Dw * u) * (sg + gate * (1 - sg))
    dy = dy * gate
    dB, dC = torch.zeros_like(Bm), torch.zeros_like(Cm)
    du, ddt = torch.empty_like(u), torch.empty_like(u)
    dA, dst = torch.zeros_like(A), []
    zero = torch.zeros((D, n), dtype=torch.float64, device=DEV)
    for i, (at, length) in enumerate(spans):
        carry = s["dstate"][i].double() if "dstate" in s else zero
        for t in range(at + length - 1, at - 1, -1):
            g = carry + Cm[t][group] * dy[t, :, None]
            prev = hs[t - 1] if t > at else (s["state"][i].double() if "state" in s else zero)
            carry = g * torch.exp(dt[t, :, None] * A)
            dC[t] = (hs[t] * dy[t, :, None]).reshape(G, D // G, n).sum(1)
            dB[t] = (g * dtu[t, :, None]).reshape(G, D // G, n).sum(1)
            gb = (g * Bm[t][group]).sum(-1)
            du[t] = Dw * dy[t] + dt[t] * gb
            w = carry * prev
            ddt[t] = (w * A).sum(-1) + u[t] * gb
            dA += w * dt[t, :, None]
        dst.append(carry)
    dd = ddt / (1 + torch.exp(-raw))
    shape = s["u"].shape
    out = {"du": du.reshape(shape), "ddelta": dd.reshape(shape), "dz": dz.reshape(shape), "dB": dB.reshape(s["B"].shape), "dC": dC.reshape(s["C"].shape),
           "dA": dA, "dD": (dy * u).sum(0), "ddelta_bias": dd.sum(0)}
    if "state" in s:
        out["dstate_in"] = torch.stack(dst)
    return out


def _exact_conv(case, s):
    W, D = case["W"], case["D"]
    w, b = s["weight"].double(), s["bias"].double()
    back = case["op"] == "conv_bwd"
    flat = s["x"].reshape(-1, D).double()
    dy = s["dy"].reshape(-1, D).double() if back else None
    y, dx = torch.empty_like(flat), torch.empty_like(flat)
    states, dstates, dw, db = [], [], torch.zeros_like(w), torch.zeros_like(b)
    for i, (at, length) in enumerate(_sequences(case)):
        old = s["state"][i].double() if "state" in s else flat.new_zeros((W - 1, D))
        line = torch.cat((old, flat[at:at + length]))
        states.append(line[length:])
        windows = line.unfold(0, W, 1)  # [length, D, W]
        pre = (windows * w).sum(-1) + b
        sg = 1 / (1 + torch.exp(-pre))
        y[at:at + length] = pre * sg
        if back:
            g = dy[at:at + length] * (sg + pre * sg * (1 - sg))
            dline = torch.zeros_like(line)
            for j in range(W):
                dline[j:j + length] += g * w[:, j]
            dw += (windows * g[..., None]).sum(0)
            db += g.sum(0)
            dx[at:at + length] = dline[W - 1:]
            dstates.append(dline[:W - 1])
    if not back:
        return y.reshape(s["x"].shape), torch.stack(states)
    out = {"dx": dx.reshape(s["x"].shape), "dweight": dw, "dbias": db}
    if "state" in s:
        out["dstate_in"] = torch.stack(dstates)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("scan", "scan_bwd"):
        return _exact_scan(case, s)
    if op in ("conv", "conv_bwd"):
        return _exact_conv(case, s)
    if op == "scan_step":
        group = torch.arange(case["D"], device=DEV) // (case["D"] // case["G"])
        dt = torch.nn.functional.softplus(s["delta"].double() + s["delta_bias"].double(), threshold=60.0)
        h = torch.exp(dt[..., None] * s["A"].double()) * s["state"].double() + dt[..., None] * s["u"].double()[..., None] * s["B"].double()[:, group]
        z = s["z"].double()
        y = (torch.einsum("bdn,bdn->bd", s["C"].double()[:, group], h) + s["D"].double() * s["u"].double()) * z / (1 + torch.exp(-z))
        return y, h
    if op == "conv_step":
        line = torch.cat((s["state"].double(), s["x"].double()[:, None]), 1)
        pre = torch.einsum("bwd,dw->bd", line, s["weight"].double()) + s["bias"].double()
        return pre / (1 + torch.exp(-pre)), line[:, 1:]
    x = s["x"].double()
    if op == "norm":
        var, mean = torch.var_mean(x, dim=-1, unbiased=False)
        rstd = 1 / torch.sqrt(var + EPS)
        return (x - mean[:, None]) * rstd[:, None] * s["weight"].double() + s["bias"].double(), mean, rstd
    dy, rstd = s["dy"].double(), s["rstd"].double()[:, None]
    n = (x - s["mean"].double()[:, None]) * rstd
    g = dy * s["weight"].double()
    inner = torch.einsum("rf,rf->r", g, n) / x.shape[1]
    return rstd * (g - g.mean(1, keepdim=True) - inner[:, None] * n), torch.einsum("rf,rf->f", dy, n), dy.sum(0)
