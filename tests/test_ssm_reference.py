"""The plain fp64 forms that the state space layer's kernels are tested
against: worked by hand, their gradients against automatic differentiation and
against differences."""
import math

import pytest
import torch

from tests import ssm_reference as R

f64 = torch.float64


def _problem(T, D, G, n, seed, softplus=True, gate=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, dtype=f64)  # noqa: E731
    return {"u": r(T, D), "delta": r(T, D) if softplus else r(T, D).abs() * 0.3, "A": -r(D, n).abs(),
            "B": r(T, G, n), "C": r(T, G, n), "D": r(D), "z": r(T, D) if gate else None,
            "delta_bias": r(D) if softplus else None, "softplus": softplus}


def test_scan_by_hand():
    """One channel, one state, two tokens: dt = 1, 2; a = e^-1, e^-2."""
    t = lambda x: torch.tensor(x, dtype=f64)  # noqa: E731
    p = {"u": t([[3.0], [5.0]]), "delta": t([[1.0], [2.0]]), "A": t([[-1.0]]), "B": t([[[2.0]], [[7.0]]]),
         "C": t([[[1.0]], [[10.0]]]), "D": t([0.5]), "z": None, "delta_bias": None, "softplus": False}
    y, st, _, _, _ = R.scan(p, [(0, 2)], t([[[4.0]]]))
    h1 = 4 * math.exp(-1) + 6
    h2 = h1 * math.exp(-2) + 70
    assert abs(float(y[0]) - (h1 + 1.5)) < 1e-12 and abs(float(y[1]) - (10 * h2 + 2.5)) < 1e-11
    assert abs(float(st) - h2) < 1e-11
    assert abs(float(R.softplus(t(0.0))) - math.log(2)) < 1e-15


@pytest.mark.parametrize("softplus,gate", [(True, True), (False, False)])
def test_scan_gradients(softplus, gate):
    spans = R.spans_of([5, 0, 1, 7])
    p = _problem(13, 4, 2, 3, 0, softplus, gate)
    g = torch.Generator().manual_seed(1)
    st = torch.randn((4, 4, 3), generator=g, dtype=f64)
    dy, ds = torch.randn((13, 4), generator=g, dtype=f64), torch.randn((4, 4, 3), generator=g, dtype=f64)
    names = [k for k in ("u", "delta", "A", "B", "C", "D", "z", "delta_bias") if p[k] is not None]

    def loss(q, s):
        y, out, _, _, _ = R.scan(q, spans, s)
        return (y * dy).sum() + (out * ds).sum()

    grads = R.scan_backward(p, spans, R.scan(p, spans, st)[4], dy, st, ds)
    q = {**p, **{k: p[k].clone().requires_grad_() for k in names}}
    s = st.clone().requires_grad_()
    loss(q, s).backward()
    for k in names:
        torch.testing.assert_close(grads["d" + k], q[k].grad, rtol=1e-10, atol=1e-10)
    torch.testing.assert_close(grads["dstate_in"], s.grad, rtol=1e-10, atol=1e-10)
    eps = 1e-5
    for k in names:
        v = torch.randn(p[k].shape, generator=g, dtype=f64)
        diff = (loss({**p, k: p[k] + eps * v}, st) - loss({**p, k: p[k] - eps * v}, st)) / (2 * eps)
        assert abs(float(diff - (grads["d" + k] * v).sum())) <= 1e-7 * max(1.0, abs(float(diff)))


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("silu", [True, False])
def test_conv_against_the_library_convolution_and_gradients(W, silu):
    spans = R.spans_of([6, 0, 1, 2, 9])
    g = torch.Generator().manual_seed(W)
    r = lambda *s: torch.randn(s, generator=g, dtype=f64)  # noqa: E731
    x, w, b, st, dy, ds = r(18, 5), r(5, W), r(5), r(5, W - 1, 5), r(18, 5), r(5, W - 1, 5)
    y, out, _ = R.conv(x, w, b, silu, spans, st)
    for i, (at, n) in enumerate(spans):
        line = torch.cat((st[i], x[at:at + n]))
        if n:
            pre = torch.nn.functional.conv1d(line.t()[None], w[:, None], b, groups=5)[0].t()
            torch.testing.assert_close(y[at:at + n], torch.nn.functional.silu(pre) if silu else pre)
        torch.testing.assert_close(out[i], line[n:])
    leaves = [t.clone().requires_grad_() for t in (x, w, b, st)]
    yy, oo, _ = R.conv(leaves[0], leaves[1], leaves[2], silu, spans, leaves[3])
    ((yy * dy).sum() + (oo * ds).sum()).backward()
    grads, _ = R.conv_backward(dy, x, w, b, silu, spans, st, ds)
    for k, t in zip(("dx", "dweight", "dbias", "dstate_in"), leaves):
        torch.testing.assert_close(grads[k], t.grad, rtol=1e-10, atol=1e-10)


def test_norm_gradients():
    g = torch.Generator().manual_seed(3)
    x, w, b, dy = (torch.randn(s, generator=g, dtype=f64) for s in ((7, 11), (11,), (11,), (7, 11)))
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    torch.nn.functional.layer_norm(leaves[0], (11,), leaves[1], leaves[2], 1e-5).backward(dy)
    y, mean, rstd, _, _, _ = R.layer_norm(x, w, b, 1e-5)
    torch.testing.assert_close(y, torch.nn.functional.layer_norm(x, (11,), w, b, 1e-5))
    grads, _ = R.layer_norm_backward(dy, x, w, mean, rstd)
    for got, t in zip(grads, leaves):
        torch.testing.assert_close(got, t.grad, rtol=1e-10, atol=1e-10)
