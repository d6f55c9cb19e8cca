"""The bounds of tests/ssm_bounds.py on the CPU: its values are those of the plain
fp64 forms, an fp32 walk in the kernels' order stays within the bounds, and the
mistakes that they are to find do not."""
import pytest
import torch

from tests import ssm_bounds as S
from tests import ssm_reference as R

f32, f64 = torch.float32, torch.float64
LENS = [200, 0, 1, 75]


def _problem(D=12, G=2, n=6, seed=0, softplus=True, gate=True):
    T = sum(LENS)
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    p = {"u": r(T, D), "delta": r(T, D) * 0.5 if softplus else r(T, D).abs() * 0.1,
         "A": -torch.rand((D, n), generator=g) * 4 - 0.01, "B": r(T, G, n), "C": r(T, G, n), "D": r(D),
         "z": r(T, D) if gate else None, "delta_bias": r(D) - 2 if softplus else None, "softplus": softplus}
    return p, r(T, D), r(len(LENS), D, n), r(len(LENS), D, n)


def _f64(p):
    return {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in p.items()}


def _walk(p, dy, state_in, dstate_out, chunk, spoil=None):
    """The scan and its gradients in fp32, the gradient chunk by chunk. `spoil`
    maps (name, value) to the value that goes on: a planted mistake."""
    spoil = spoil or (lambda name, v: v)
    T, D = p["u"].shape
    n, G = p["A"].shape[1], p["B"].shape[1]
    raw = p["delta"] + p["delta_bias"] if p["delta_bias"] is not None else p["delta"]
    dt = torch.nn.functional.softplus(raw) if p["softplus"] else raw
    wide = lambda x: x.repeat_interleave(D // G, dim=-2)  # noqa: E731
    B, C = wide(p["B"]), wide(p["C"])
    a = torch.exp(dt[..., None] * p["A"])
    gate = p["z"] * torch.sigmoid(p["z"]) if p["z"] is not None else torch.ones_like(dt)
    w = dy * gate
    h = torch.empty((T, D, n))
    out = {k: torch.empty(s) for k, s in dict(du=(T, D), ddelta=(T, D), dB=(T, G, n), dC=(T, G, n)).items()}
    dA, states, d_in = torch.zeros_like(p["A"]), [], []
    for i, (at, length) in enumerate(R.spans_of(LENS)):
        x = state_in[i]
        for t in range(at, at + length):
            x = spoil("state", a[t] * x + (dt[t] * p["u"][t])[:, None] * B[t]) if (t - at) % 8 == 7 else \
                a[t] * x + (dt[t] * p["u"][t])[:, None] * B[t]
            h[t] = x
        states.append(x)
        carry = dstate_out[i]
        for t in range(at + length - 1, at - 1, -1):
            g = C[t] * w[t, :, None] + carry
            carry = a[t] * g
            if (t - at) % chunk == 0:
                carry = spoil("carry", carry)
            before = h[t - 1] if t > at else state_in[i]
            out["dC"][t] = (w[t, :, None] * h[t]).reshape(G, D // G, n).sum(1)
            out["dB"][t] = (g * (dt[t] * p["u"][t])[:, None]).reshape(G, D // G, n).sum(1)
            gb = (g * B[t]).sum(-1)
            out["du"][t] = p["D"] * w[t] + dt[t] * gb
            ddt = (p["A"] * carry * before).sum(-1) + p["u"][t] * gb
            out["ddelta"][t] = ddt * torch.sigmoid(raw[t]) if p["softplus"] else ddt
            dA += dt[t][:, None] * carry * before
        d_in.append(carry)
    pre = (C * h).sum(-1) + p["D"] * p["u"]
    out.update(y=pre * gate, state=torch.stack(states), dA=spoil("dA", dA), dD=(w * p["u"]).sum(0),
               ddelta_bias=out["ddelta"].sum(0), dstate_in=torch.stack(d_in))
    if p["z"] is not None:
        sg = torch.sigmoid(p["z"])
        out["dz"] = dy * pre * sg * (1 + p["z"] * (1 - sg))
    return out


def _outside(got, want, bounds):
    bad = set()
    for k, v in got.items():
        try:
            R.check(v, want[k], bounds[k], k)
        except AssertionError:
            bad.add(k)
    return bad


@pytest.mark.parametrize("softplus,gate", [(True, True), (False, False)])
def test_values_and_an_fp32_walk(softplus, gate):
    p, dy, st, ds = _problem(softplus=softplus, gate=gate)
    q, spans = _f64(p), R.spans_of(LENS)
    want, bounds = S.scan(q, spans, 32, dy.double(), st.double(), ds.double())
    y, state, _, _, h = R.scan(q, spans, st.double())
    plain = {"y": y, "state": state, **R.scan_backward(q, spans, h, dy.double(), st.double(), ds.double())}
    assert set(plain) == set(want) == set(bounds)
    for k, v in plain.items():
        torch.testing.assert_close(want[k], v, rtol=1e-11, atol=1e-11)
    assert not _outside(_walk(p, dy, st, ds, 32), want, bounds)


def test_what_the_bounds_find():
    """A state or a gradient of a state held in bf16 between blocks or chunks, an
    infinitesimal share of a gradient lost, in the longest sequence only."""
    p, dy, st, ds = _problem()
    want, bounds = S.scan(_f64(p), R.spans_of(LENS), 32, dy.double(), st.double(), ds.double())
    low = lambda v: v.bfloat16().float()  # noqa: E731
    state = _outside(_walk(p, dy, st, ds, 32, lambda k, v: low(v) if k == "state" else v), want, bounds)
    assert {"y", "dC", "dA", "ddelta", "dz"} <= state
    carry = _outside(_walk(p, dy, st, ds, 32, lambda k, v: low(v) if k == "carry" else v), want, bounds)
    assert {"du", "dB", "ddelta", "dA", "dstate_in"} <= carry
    assert _outside(_walk(p, dy, st, ds, 32, lambda k, v: v * (1 + 2 ** -12) if k == "dA" else v), want, bounds) == {"dA"}


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("silu", [True, False])
def test_convolution_without_a_loop(W, silu):
    lens = [0, 9, 1, 0, 2, 30]
    g = torch.Generator().manual_seed(W)
    r = lambda *s: torch.randn(s, generator=g, dtype=f64)  # noqa: E731
    x, dy, w, b, st, ds = r(42, 5), r(42, 5), r(5, W), r(5), r(6, W - 1, 5), r(6, W - 1, 5)
    spans = R.spans_of(lens)
    value, bound = S.conv(x, w, b, silu, lens, st, dy, ds)
    y, state, by = R.conv(x, w, b, silu, spans, st)
    grads, bounds = R.conv_backward(dy, x, w, b, silu, spans, st, ds)
    torch.testing.assert_close(value["y"], y)
    torch.testing.assert_close(value["state"], state)
    torch.testing.assert_close(bound["y"], by)
    for k, v in grads.items():
        torch.testing.assert_close(value[k], v)
        torch.testing.assert_close(bound[k], bounds[k])
