"""The state space layer on the GPU against its plain fp64 forms
(tests/ssm_reference.py), whose error bounds are the tolerances: selective
scan, short convolution and layer norm, over prompts, for single tokens and
backward; then the calls together, as a layer makes them."""
import ctypes

import pytest
import torch

from long_context_02_b200 import binding as L
from tests import ssm_reference as R

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def _rnd(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def _f64(t):
    return None if t is None else t.detach().cpu().double()


def _scan_problem(lens, D, G, n, dtype, seed, gate=True, skip=True, bias=True, softplus=True,
                  sliced=True):
    """CPU tensors [T, ...] in the kernel's dtypes; z, B and C as slices of wider ones."""
    T = sum(lens)
    g = torch.Generator().manual_seed(seed)
    p = {"u": _rnd(g, T, D, dtype=dtype),
         "delta": _rnd(g, T, D, dtype=dtype, scale=0.5) if softplus else _rnd(g, T, D, dtype=dtype).abs() * 0.1,
         "A": -torch.rand((D, n), generator=g) * 4 - 0.1, "softplus": softplus,
         "D": _rnd(g, D) if skip else None, "delta_bias": _rnd(g, D) - 2 if bias else None}
    wide = _rnd(g, T, 2 * D, dtype=dtype)
    p["z"] = (wide[:, D:] if sliced else wide[:, D:].contiguous()) if gate else None
    proj = _rnd(g, T, 5 + 2 * G * n, dtype=dtype)
    p["B"], p["C"] = proj[:, 5:5 + G * n].unflatten(-1, (G, n)), proj[:, 5 + G * n:].unflatten(-1, (G, n))
    return p


def _to(p, dev=DEV):
    """To the GPU, slices staying slices."""
    out = {}
    for k, v in p.items():
        if isinstance(v, torch.Tensor) and not v.is_contiguous():
            base = v._base.to(dev)
            out[k] = base.as_strided(v.shape, v.stride(), v.storage_offset())
        else:
            out[k] = v.to(dev) if isinstance(v, torch.Tensor) else v
    return out


def _cu(lens):
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def _args(p):
    return [p[k] for k in ("u", "delta", "A", "B", "C")], {k: p[k] for k in ("D", "z", "delta_bias", "softplus")}


def _dense(p, B):
    """The same tensors as [B, N, ...]."""
    return {k: (v.unflatten(0, (B, -1)) if k in ("u", "delta", "z", "B", "C") and v is not None else v)
            for k, v in p.items()}


SCANS = [
    # lens, D, G, n, dtype, gate, skip, bias, softplus, state
    ([1], 1, 1, 1, F32, True, True, True, True, True),
    ([37], 40, 1, 16, BF, True, True, True, True, False),
    ([0, 5, 1, 130, 0, 64], 70, 2, 16, BF, True, True, True, True, True),
    ([300, 290], 33, 1, 16, F32, True, True, True, True, True),        # cut into chunks
    ([33, 2], 200, 4, 3, F32, False, True, True, True, True),
    ([9, 31, 33], 130, 1, 8, BF, True, False, False, False, True),
    ([65], 50, 5, 10, F32, True, False, True, True, True),
    ([40, 41], 24, 1, 32, BF, True, True, False, True, True),
    ([17, 64], 19, 1, 33, F32, False, False, False, False, False),
    ([70], 12, 3, 64, F32, True, True, True, True, True),
    ([2] * 40, 150, 1, 16, F32, True, True, True, True, True),         # one chunk each
    ([400], 16, 1, 4, BF, True, True, True, True, True),
]


@pytest.mark.parametrize("lens,D,G,n,dtype,gate,skip,bias,softplus,state", SCANS)
def test_scan(lens, D, G, n, dtype, gate, skip, bias, softplus, state):
    p = _scan_problem(lens, D, G, n, dtype, len(lens) + D, gate, skip, bias, softplus)
    st = _rnd(torch.Generator().manual_seed(5), len(lens), D, n) if state else None
    args, kw = _args(_to(p))
    y, out = L.selective_scan(*args, **kw, state_in=None if st is None else st.to(DEV),
                              cu_seqlens=_cu(lens), out_dtype=F32)
    q = {k: _f64(v) if isinstance(v, torch.Tensor) else v for k, v in p.items()}
    want, ws, by, bs, _ = R.scan(q, R.spans_of(lens), _f64(st))
    R.check(y, want, by, "y")
    R.check(out, ws, bs, "state")
    # the same sequences as a dense batch, where they have one length
    if len(set(lens)) == 1 and lens[0] > 0:
        d = _dense(_to(p), len(lens))
        args, kw = _args(d)
        y2, out2 = L.selective_scan(*args, **kw, state_in=None if st is None else st.to(DEV))
        R.check(y2.flatten(0, 1), want, by, "dense y")
        R.check(out2, ws, bs, "dense state")


@pytest.mark.parametrize("lens,D,G,n,dtype,gate,skip,bias,softplus,state", SCANS)
def test_scan_backward(lens, D, G, n, dtype, gate, skip, bias, softplus, state):
    p = _scan_problem(lens, D, G, n, dtype, len(lens) + D, gate, skip, bias, softplus)
    g = torch.Generator().manual_seed(6)
    st = _rnd(g, len(lens), D, n) if state else None
    ds = _rnd(g, len(lens), D, n) if state else None
    dy = _rnd(g, sum(lens), D, dtype=dtype)
    args, kw = _args(_to(p))
    opt = {} if st is None else {"state_in": st.to(DEV), "dstate_out": ds.to(DEV)}
    got = L.selective_scan_backward(dy.to(DEV), *args, **kw, **opt, cu_seqlens=_cu(lens), out_dtype=F32)
    q = {k: _f64(v) if isinstance(v, torch.Tensor) else v for k, v in p.items()}
    spans = R.spans_of(lens)
    h = R.scan(q, spans, _f64(st))[4]
    want = R.scan_backward(q, spans, h, _f64(dy), _f64(st), _f64(ds))
    bounds = R.scan_backward_bounds(q, spans, _f64(dy), _f64(st), _f64(ds))
    assert ("dz" in got, "dD" in got, "ddelta_bias" in got, "dstate_in" in got) == (gate, skip, bias, state)
    for k, v in got.items():
        R.check(v, want[k], bounds[k], k)
    # bf16 outputs are the fp32 ones rounded, and a second call gives the same bits
    if dtype == BF:
        low = L.selective_scan_backward(dy.to(DEV), *args, **kw, **opt, cu_seqlens=_cu(lens))
        for k, v in low.items():
            assert torch.equal(v, got[k].to(v.dtype)), k


def test_scan_gradient_against_differences():
    """The kernel's gradients along random directions against central
    differences of the fp64 form; the difference's own error is below 1e-7."""
    lens, D, n = [150, 20], 24, 16
    p = _scan_problem(lens, D, 2, n, F32, 3)
    g = torch.Generator().manual_seed(4)
    dy = _rnd(g, sum(lens), D)
    args, kw = _args(_to(p))
    got = L.selective_scan_backward(dy.to(DEV), *args, **kw, cu_seqlens=_cu(lens))
    q = {k: _f64(v) if isinstance(v, torch.Tensor) else v for k, v in p.items()}
    spans = R.spans_of(lens)
    bounds = R.scan_backward_bounds(q, spans, _f64(dy))
    for k in ("u", "delta", "A", "B", "C", "D", "z", "delta_bias"):
        v = torch.randn(q[k].shape, generator=g, dtype=torch.float64)
        at = lambda e: float((R.scan({**q, k: q[k] + e * v}, spans)[0] * _f64(dy)).sum())  # noqa: E731,B023
        diff = (at(1e-5) - at(-1e-5)) / 2e-5
        mine = float((_f64(got["d" + k]) * v).sum())
        limit = float((bounds["d" + k] * v.abs()).sum()) + 1e-6 * (abs(diff) + 1)
        assert abs(mine - diff) <= limit, (k, mine, diff, limit)


@pytest.mark.parametrize("B,D,G,n,dtype", [(1, 1, 1, 1, F32), (3, 200, 2, 16, BF), (5, 67, 1, 7, F32),
                                           (2, 48, 1, 64, BF), (4, 130, 1, 4, BF), (3, 90, 3, 32, F32)])
def test_scan_prompt_then_steps(B, D, G, n, dtype):
    """A prompt, then single tokens from its state, against one scan of all."""
    N, more = 21, 3
    p = _dense(_scan_problem([(N + more) * B], D, G, n, dtype, 8), B)
    d = {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in p.items()}
    tok = ("u", "delta", "z", "B", "C")
    first = {k: (v[:, :N].contiguous() if k in tok else v) for k, v in d.items()}
    args, kw = _args(first)
    _, st = L.selective_scan(*args, **kw)
    ys = []
    for t in range(N, N + more):
        args, kw = _args({k: (v[:, t] if k in tok else v) for k, v in d.items()})
        ys.append(L.selective_scan_step(*args[:5], st, **kw, out_dtype=F32))
    flat = {k: _f64(v.flatten(0, 1)) if k in tok else (_f64(v) if isinstance(v, torch.Tensor) else v)
            for k, v in p.items()}
    want, ws, by, bs, _ = R.scan(flat, R.spans_of([N + more] * B))
    pick = lambda x: x.unflatten(0, (B, N + more))[:, N:]  # noqa: E731
    R.check(torch.stack(ys, 1), pick(want), pick(by), "y of the steps")
    R.check(st, ws, bs, "state")


def test_scan_in_place_state_and_rows_behind_the_last_sequence():
    """state_in and state_out as one array, cut into chunks; rows behind the last
    sequence keep what they held, forward and backward."""
    lens, D, n = [200, 150], 20, 16
    p = _scan_problem(lens + [9], D, 1, n, F32, 11, sliced=False)
    st = _rnd(torch.Generator().manual_seed(1), 2, D, n)
    for k in ("u", "delta", "z", "B", "C"):  # what is behind the last sequence is not read either
        p[k] = p[k].clone()
        p[k][sum(lens):] = float("nan")
    d = {k: (v.contiguous().to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in p.items()}
    cu, T = _cu(lens), sum(lens) + 9
    s = L.SCAN_INPUTS.pack(*[d[k].data_ptr() for k in ("u", "delta", "z", "B", "C")], D, D, D, n, n,
                           *[d[k].data_ptr() for k in ("A", "D", "delta_bias")], 1)
    need = L.la_workspace_bytes(L.LA_OP_SCAN, 1, D, T, n, 2, F32)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    state, y = st.to(DEV), torch.full((T, D), 7.0, device=DEV)
    stream = torch.cuda.current_stream().cuda_stream
    assert L.lib().la_selective_scan(cu.data_ptr(), 2, s, state.data_ptr(), y.data_ptr(), state.data_ptr(),
                                     T, D, 1, n, 1, 1, ws.data_ptr(), need, stream) == L.LA_OK
    q = {k: (_f64(v[:sum(lens)]) if k in ("u", "delta", "z", "B", "C") else
             _f64(v) if isinstance(v, torch.Tensor) else v) for k, v in p.items()}
    want, wst, by, bs, _ = R.scan(q, R.spans_of(lens), _f64(st))
    R.check(y[:sum(lens)], want, by, "y")
    R.check(state, wst, bs, "state in place")
    assert (y[sum(lens):] == 7.0).all()
    names = ["du", "ddelta", "dz", "dB", "dC", "dA", "dD", "ddelta_bias", "dstate_in"]
    shape = {"dB": (T, 1, n), "dC": (T, 1, n), "dA": (D, n), "dD": (D,), "ddelta_bias": (D,),
             "dstate_in": (2, D, n)}
    out = {f: torch.full(shape.get(f, (T, D)), 7.0, device=DEV) for f in names}
    need = L.la_workspace_bytes(L.LA_OP_SCAN_BACKWARD, 1, D, T, n, 2, F32)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)  # NaN wherever it is read unwritten
    dy = torch.ones((T, D), device=DEV)
    assert L.lib().la_selective_scan_backward(
        cu.data_ptr(), 2, s, None, dy.data_ptr(), D, None, L.SCAN_GRADS.pack(*[out[f].data_ptr() for f in names]),
        T, D, 1, n, 1, 1, ws.data_ptr(), need, stream) == L.LA_OK
    one = torch.ones((sum(lens), D), dtype=torch.float64)
    spans = R.spans_of(lens)
    want = R.scan_backward(q, spans, R.scan(q, spans)[4], one)
    bounds = R.scan_backward_bounds(q, spans, one)
    for f in names:
        v = out[f][:sum(lens)] if f in ("du", "ddelta", "dz", "dB", "dC") else out[f]
        R.check(v, want[f], bounds[f], f)
        if f in ("du", "ddelta", "dz", "dB", "dC"):
            assert (out[f][sum(lens):] == 7.0).all(), f


def test_scan_many_short_sequences():
    """5000 packed sequences of 0 to 3 tokens, and one long one among them that is
    cut into chunks: the table of chunks spans several rounds of its CTA."""
    g = torch.Generator().manual_seed(0)
    lens = torch.randint(0, 4, (5000,), generator=g).tolist()
    lens[2500] = 500
    D, n = 6, 4
    p = _scan_problem(lens, D, 1, n, F32, 1)
    st = _rnd(g, len(lens), D, n)
    dy, ds = _rnd(g, sum(lens), D), _rnd(g, len(lens), D, n)
    args, kw = _args(_to(p))
    q = {k: _f64(v) if isinstance(v, torch.Tensor) else v for k, v in p.items()}
    spans = R.spans_of(lens)
    y, out = L.selective_scan(*args, **kw, state_in=st.to(DEV), cu_seqlens=_cu(lens))
    want, ws, by, bs, h = R.scan(q, spans, _f64(st))
    R.check(y, want, by, "y")
    R.check(out, ws, bs, "state")
    got = L.selective_scan_backward(dy.to(DEV), *args, **kw, state_in=st.to(DEV), dstate_out=ds.to(DEV),
                                    cu_seqlens=_cu(lens))
    want = R.scan_backward(q, spans, h, _f64(dy), _f64(st), _f64(ds))
    bounds = R.scan_backward_bounds(q, spans, _f64(dy), _f64(st), _f64(ds))
    for k, v in got.items():
        R.check(v, want[k], bounds[k], k)


def test_scan_one_group_per_channel_and_strided_gradient():
    """G = D, and dy as a slice of a wider tensor."""
    lens, D, n = [40], 9, 5
    p = _scan_problem(lens, D, D, n, BF, 13)
    wide = _rnd(torch.Generator().manual_seed(1), 40, 30, dtype=BF)
    args, kw = _args(_to(p))
    q = {k: _f64(v) if isinstance(v, torch.Tensor) else v for k, v in p.items()}
    y, _ = L.selective_scan(*args, **kw, cu_seqlens=_cu(lens), out_dtype=F32)
    want, _, by, _, h = R.scan(q, [(0, 40)])
    R.check(y, want, by, "y")
    got = L.selective_scan_backward(wide.to(DEV)[:, 3:12], *args, **kw, cu_seqlens=_cu(lens), out_dtype=F32)
    dy = _f64(wide[:, 3:12])
    want, bounds = R.scan_backward(q, [(0, 40)], h, dy), R.scan_backward_bounds(q, [(0, 40)], dy)
    for k, v in got.items():
        R.check(v, want[k], bounds[k], k)


def test_scan_non_finite_inputs_stay_in_their_channel():
    lens, D, n = [90], 40, 16
    p = _scan_problem(lens, D, 1, n, F32, 12)
    p["u"][50, 3] = float("nan")
    p["delta"][20, 7] = float("inf")
    args, kw = _args(_to(p))
    y, st = L.selective_scan(*args, **kw, cu_seqlens=_cu(lens))
    q = {k: _f64(v) if isinstance(v, torch.Tensor) else v for k, v in p.items()}
    want, ws, by, bs, _ = R.scan(q, R.spans_of(lens))
    fine = torch.tensor([c not in (3, 7) for c in range(D)])
    R.check(y[:, fine.to(DEV)], want[:, fine], by[:, fine], "other channels")
    R.check(st[:, fine.to(DEV)], ws[:, fine], bs[:, fine], "other states")
    R.check(y[:50, 3], want[:50, 3], by[:50, 3], "tokens before the NaN")
    assert torch.isnan(y[50:, 3]).all()
    R.check(y[:20, 7], want[:20, 7], by[:20, 7], "tokens before the infinity")


@pytest.mark.parametrize("D,n", [(41, 10), (40, 10), (41, 16), (40, 3)])
def test_scan_backward_of_an_infinite_step(D, n):
    """An infinite dt forgets the state, so that the tokens before it get the
    finite gradients of a sequence that ends there, in its channel too, and
    dB stays finite everywhere else. The sums that remain are a part of those
    without the infinity, whose bounds therefore hold."""
    lens, at, ch = [90], 60, D - 1
    p = _scan_problem(lens, D, 1, n, F32, 21)
    q = {k: _f64(v) if isinstance(v, torch.Tensor) else v for k, v in p.items()}
    spans = R.spans_of(lens)
    dy = _rnd(torch.Generator().manual_seed(22), sum(lens), D)
    bounds = R.scan_backward_bounds(q, spans, _f64(dy))
    p["delta"][at, ch] = q["delta"][at, ch] = float("inf")
    want = R.scan_backward(q, spans, R.scan(q, spans)[4], _f64(dy))
    args, kw = _args(_to(p))
    got = L.selective_scan_backward(dy.to(DEV), *args, **kw, cu_seqlens=_cu(lens))
    for k in ("du", "ddelta", "dz", "dB", "dC"):
        assert torch.isfinite(want[k][:at]).all()
        R.check(got[k][:at], want[k][:at], bounds[k][:at], k)
    R.check(got["dB"][at + 1:], want["dB"][at + 1:], bounds["dB"][at + 1:], "dB behind it")
    for k in ("du", "ddelta", "dz"):
        R.check(got[k][:, :ch], want[k][:, :ch], bounds[k][:, :ch], f"{k} of the others")
    R.check(got["dA"][:ch], want["dA"][:ch], bounds["dA"][:ch], "dA of the others")


def test_scan_forgets_at_once_where_a_is_infinite():
    """A state with A = -inf is dt u B of its own token; the gradients that its
    formula leaves finite (all but ddelta of its channel) agree, packed with an
    empty sequence and lengths that end inside a block. The bounds are those of
    A = -40: they grow with sums of absolute values, whose terms a decay above 0
    only adds to."""
    lens, D, n, ch, m = [45, 0, 13], 24, 16, 5, 2
    p = _scan_problem(lens, D, 1, n, F32, 23)
    q = {k: _f64(v) if isinstance(v, torch.Tensor) else v for k, v in p.items()}
    g = torch.Generator().manual_seed(24)
    st, dy = _rnd(g, 3, D, n), _rnd(g, sum(lens), D)
    spans = R.spans_of(lens)
    q["A"][ch, m] = -40.0
    _, _, by, bs, _ = R.scan(q, spans, _f64(st))
    bounds = R.scan_backward_bounds(q, spans, _f64(dy), _f64(st))
    p["A"][ch, m] = q["A"][ch, m] = float("-inf")
    want, ws, _, _, h = R.scan(q, spans, _f64(st))
    args, kw = _args(_to(p))
    y, out = L.selective_scan(*args, **kw, state_in=st.to(DEV), cu_seqlens=_cu(lens))
    R.check(y, want, by, "y")
    R.check(out, ws, bs, "state")
    grads = R.scan_backward(q, spans, h, _f64(dy), _f64(st))
    got = L.selective_scan_backward(dy.to(DEV), *args, **kw, state_in=st.to(DEV), cu_seqlens=_cu(lens))
    rest = torch.arange(D) != ch
    for k in ("du", "dz", "dB", "dC", "dA", "dstate_in"):
        R.check(got[k], grads[k], bounds[k], k)
    R.check(got["ddelta"][:, rest.to(DEV)], grads["ddelta"][:, rest], bounds["ddelta"][:, rest], "ddelta")


def test_scan_empty():
    t = lambda *s: torch.zeros(s, device=DEV)  # noqa: E731
    st = torch.randn((3, 8, 16), device=DEV)
    y, out = L.selective_scan(t(3, 0, 8), t(3, 0, 8), t(8, 16), t(3, 0, 1, 16), t(3, 0, 1, 16), state_in=st)
    assert y.shape == (3, 0, 8) and torch.equal(out, st)
    g = L.selective_scan_backward(t(3, 0, 8), t(3, 0, 8), t(3, 0, 8), t(8, 16), t(3, 0, 1, 16),
                                  t(3, 0, 1, 16), state_in=st, dstate_out=2 * st)
    assert torch.equal(g["dstate_in"], 2 * st) and not g["dA"].any()
    y, out = L.selective_scan(t(0, 8), t(0, 8), t(8, 16), t(0, 1, 16), t(0, 1, 16), cu_seqlens=_cu([]))
    assert y.shape == (0, 8) and out.shape == (0, 8, 16)
    g = L.selective_scan_backward(t(0, 8), t(0, 8), t(0, 8), t(8, 16), t(0, 1, 16), t(0, 1, 16),
                                  cu_seqlens=_cu([]))
    assert not g["dA"].any()
    y, out = L.selective_scan(t(0, 7, 8), t(0, 7, 8), t(8, 16), t(0, 7, 1, 16), t(0, 7, 1, 16))
    assert y.shape == (0, 7, 8) and out.shape == (0, 8, 16)
    w = torch.ones((8, 4), device=DEV)
    assert L.short_conv(t(0, 7, 8), w)[0].shape == (0, 7, 8)
    assert not L.short_conv_backward(t(0, 7, 8), t(0, 7, 8), w)["dweight"].any()
    assert L.short_conv_step(t(0, 8), w, None, t(0, 3, 8)).shape == (0, 8)
    assert L.selective_scan_step(t(0, 8), t(0, 8), t(8, 16), t(0, 1, 16), t(0, 1, 16), t(0, 8, 16)).shape == (0, 8)


def test_scan_long_sequence_offsets():
    """70,000 tokens in one narrow sequence (many chunks) and, on the same
    inputs, 64-token pieces continued from state to state by single-chunk calls
    at the sequence's end: both within the other's bound of rounding."""
    T, D, n = 70_000, 48, 16
    g = torch.Generator(device=DEV).manual_seed(2)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    u, dl, z, B, C = r(1, T, D), r(1, T, D), r(1, T, D), r(1, T, 1, n), r(1, T, 1, n)
    A, Dw, b = -torch.rand((D, n), generator=g, device=DEV) - 0.05, r(D), r(D) - 2
    y, st = L.selective_scan(u, dl, A, B, C, Dw, z, b)
    cut = T - 640
    part, state = [], None
    _, state = L.selective_scan(u[:, :cut], dl[:, :cut], A, B[:, :cut], C[:, :cut], Dw, z[:, :cut], b)
    for t in range(cut, T, 64):
        sl = slice(t, t + 64)
        o, state = L.selective_scan(u[:, sl], dl[:, sl], A, B[:, sl], C[:, sl], Dw, z[:, sl], b, state_in=state)
        part.append(o)
    flat = {"u": u, "delta": dl, "z": z, "B": B, "C": C}
    q = {k: _f64(v[0, cut:]) for k, v in flat.items()}
    q.update(A=_f64(A), D=_f64(Dw), delta_bias=_f64(b), softplus=True)
    # from a state 640 tokens back the rest is a small share: e^{-dt |A| 640} of the state
    start = L.selective_scan(u[:, :cut], dl[:, :cut], A, B[:, :cut], C[:, :cut], Dw, z[:, :cut], b)[1]
    want, ws, by, bs, _ = R.scan(q, [(0, 640)], _f64(start))
    R.check(y[0, cut:], want, 2 * by + 1e-5 * want.abs(), "last rows")
    R.check(torch.cat(part, 1)[0], want, by, "rows of the pieces")
    R.check(state, ws, bs, "state of the pieces")
    R.check(st, ws, 2 * bs + 1e-5 * ws.abs(), "state")


# ---------------------------------------------------------------- convolution

CONVS = [
    ([1], 1, 2, F32, True, True), ([50], 64, 4, BF, True, False), ([0, 1, 2, 3, 0, 130], 72, 4, BF, True, True),
    ([64, 65, 63], 37, 3, F32, False, True), ([5, 0, 1], 1032, 4, F32, True, True),
    ([200], 2056, 2, BF, False, True), ([1, 1, 1, 1, 2], 24, 4, BF, True, True), ([0], 16, 4, F32, True, True),
    ([129, 127], 9, 3, BF, True, False),
]


@pytest.mark.parametrize("sliced", [True, False])
@pytest.mark.parametrize("lens,D,W,dtype,silu,state", CONVS)
def test_conv_and_backward(lens, D, W, dtype, silu, state, sliced):
    T = sum(lens)
    g = torch.Generator().manual_seed(D + W)
    wide = _rnd(g, T, 2 * D, dtype=dtype)
    x = wide.to(DEV)[:, :D] if sliced else wide[:, :D].contiguous().to(DEV)
    w, b = _rnd(g, D, W), _rnd(g, D) if silu else None
    st = _rnd(g, len(lens), W - 1, D, dtype=dtype) if state else None
    dy, ds = _rnd(g, T, D, dtype=dtype), _rnd(g, len(lens), W - 1, D, dtype=dtype) if state else None
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    y, out = L.short_conv(x, dev(w), dev(b), silu, dev(st), _cu(lens), out_dtype=F32)
    spans = R.spans_of(lens)
    want, ws, by = R.conv(_f64(x), _f64(w), _f64(b), silu, spans, _f64(st))
    R.check(y, want, by, "y")
    assert torch.equal(out.cpu().double(), ws)
    got = L.short_conv_backward(dev(dy), x, dev(w), dev(b), silu, dev(st), dev(ds), _cu(lens), out_dtype=F32)
    want, bounds = R.conv_backward(_f64(dy), _f64(x), _f64(w), _f64(b), silu, spans, _f64(st), _f64(ds))
    assert ("dbias" in got, "dstate_in" in got) == (b is not None, state)
    for k, v in got.items():
        R.check(v, want[k], bounds[k], k)
    if dtype == BF:
        assert torch.equal(L.short_conv(x, dev(w), dev(b), silu, dev(st), _cu(lens))[0], y.to(BF))
        low = L.short_conv_backward(dev(dy), x, dev(w), dev(b), silu, dev(st), dev(ds), _cu(lens))
        for k, v in low.items():
            assert torch.equal(v, got[k].to(v.dtype)), k
    if len(lens) == 1 and T:
        y2, out2 = L.short_conv(x[None], dev(w), dev(b), silu, dev(st), out_dtype=F32)
        assert torch.equal(y2[0], y) and torch.equal(out2, out)


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("D,dtype", [(40, BF), (13, F32), (1500, BF)])
def test_conv_prompt_then_steps(W, D, dtype):
    B, N = 3, 7
    g = torch.Generator().manual_seed(W)
    x, w, b = _rnd(g, B, N + 5, D, dtype=dtype).to(DEV), _rnd(g, D, W).to(DEV), _rnd(g, D).to(DEV)
    whole, last = L.short_conv(x, w, b)
    _, st = L.short_conv(x[:, :N].contiguous(), w, b)
    for t in range(N, N + 5):
        assert torch.equal(L.short_conv_step(x[:, t], w, b, st), whole[:, t])
    assert torch.equal(st, last)


def test_conv_rows_behind_the_last_sequence():
    lens, D = [70, 3], 16
    T = sum(lens) + 90
    x, w = torch.randn((T, D), device=DEV), torch.randn((D, 4), device=DEV)
    y = torch.full((T, D), 7.0, device=DEV)
    s = torch.cuda.current_stream().cuda_stream
    assert L.lib().la_short_conv(_cu(lens).data_ptr(), 2, x.data_ptr(), D, w.data_ptr(), None, None,
                                 y.data_ptr(), None, T, D, 4, 1, 1, 1, s) == L.LA_OK
    assert (y[sum(lens):] == 7.0).all() and torch.isfinite(y).all()
    dx, dw = torch.full((T, D), 7.0, device=DEV), torch.empty((D, 4), device=DEV)
    need = L.la_workspace_bytes(L.LA_OP_CONV_BACKWARD, 1, D, T, 4, 2, F32)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    dy = torch.randn((T, D), device=DEV)
    assert L.lib().la_short_conv_backward(_cu(lens).data_ptr(), 2, dy.data_ptr(), D, x.data_ptr(), D, w.data_ptr(),
                                          None, None, None, dx.data_ptr(), dw.data_ptr(), None, None, T, D, 4, 1,
                                          1, 1, ws.data_ptr(), need, s) == L.LA_OK
    n = sum(lens)
    want, bounds = R.conv_backward(_f64(dy[:n]), _f64(x[:n]), _f64(w), None, True, R.spans_of(lens))
    R.check(dx[:n], want["dx"], bounds["dx"], "dx")
    R.check(dw, want["dweight"], bounds["dweight"], "dweight")
    assert (dx[n:] == 7.0).all()


def test_offsets_beyond_32_bits():
    """2.3e9 elements per tensor: the last rows of the convolution and of the
    norm are those of the same rows alone."""
    T, D = 290_000, 8192
    x = torch.empty((1, T, D), dtype=BF, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(0)
    for i in range(0, T, 29_000):
        x[0, i:i + 29_000] = torch.randn((29_000, D), generator=g, device=DEV)
    w, b = torch.randn((D, 4), device=DEV), torch.randn(D, device=DEV)
    y, st = L.short_conv(x, w, b)
    assert torch.equal(y[:, -200:], L.short_conv(x[:, -203:].contiguous(), w, b)[0][:, 3:])
    assert torch.equal(st[0], x[0, -3:])
    del y
    n, mean, _ = L.layer_norm(x[0], b, b)
    assert torch.equal(n[-100:], L.layer_norm(x[0, -100:].contiguous(), b, b)[0])
    del n, x
    torch.cuda.empty_cache()


def test_scan_offsets_beyond_32_bits():
    """2.3e9 elements per tensor: the last 64 rows are those of the same rows
    continued from the state before them, to the bit (a whole number of tiles)."""
    T, D, n = 70_016, 32_768, 16
    g = torch.Generator(device=DEV).manual_seed(0)
    u, dl = (torch.empty((1, T, D), dtype=BF, device=DEV) for _ in range(2))
    for i in range(0, T, 4376):
        u[0, i:i + 4376] = torch.randn((4376, D), generator=g, device=DEV)
        dl[0, i:i + 4376] = torch.randn((4376, D), generator=g, device=DEV)
    B, C = (torch.randn((1, T, 1, n), generator=g, device=DEV).to(BF) for _ in range(2))
    A, b = -torch.rand((D, n), generator=g, device=DEV) * 4, torch.randn(D, device=DEV) - 3
    y, st = L.selective_scan(u, dl, A, B, C, delta_bias=b)
    cut = T - 64
    last = y[:, cut:].clone()
    del y
    _, mid = L.selective_scan(u[:, :cut], dl[:, :cut], A, B[:, :cut], C[:, :cut], delta_bias=b)
    torch.cuda.empty_cache()
    y2, st2 = L.selective_scan(u[:, cut:], dl[:, cut:], A, B[:, cut:], C[:, cut:], delta_bias=b, state_in=mid)
    assert torch.equal(y2, last) and torch.equal(st2, st)
    del u, dl
    torch.cuda.empty_cache()


# ---------------------------------------------------------------- layer norm

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,F", [(1, 1), (1, 8), (5, 7), (33, 64), (7, 513), (3, 1024), (9, 1025), (5, 2048),
                                    (300, 2056), (4, 4100), (3, 8192), (2, 8191), (4, 16384), (2, 16383),
                                    (1300, 1032), (1187, 2056), (1185, 4104), (1186, 8200), (1200, 1031)])
def test_layer_norm(rows, F, dtype):
    g = torch.Generator().manual_seed(rows + F)
    x = (_rnd(g, rows, F) + 3).to(dtype)
    w, b, dy = _rnd(g, F), _rnd(g, F), _rnd(g, rows, F, dtype=dtype)
    xd, wd, bd, dyd = (t.to(DEV) for t in (x, w, b, dy))
    y, mean, rstd = L.layer_norm(xd, wd, bd, 1e-5, out_dtype=F32)
    want, wm, wr, by, bm, br = R.layer_norm(_f64(x), _f64(w), _f64(b), 1e-5)
    R.check(mean, wm, bm, "mean")
    R.check(rstd, wr, br, "rstd")
    R.check(y, want, by, "y")
    low = L.layer_norm(xd, wd, None, 1e-5, want_stats=False)
    assert low[1] is None and low[0].dtype == dtype
    R.check(low[0], want - _f64(b), by, "y without bias")
    dx, dw, db = L.layer_norm_backward(dyd, xd, wd, mean, rstd, out_dtype=F32)
    (gx, gw, gb), (sx, sw, sb) = R.layer_norm_backward(_f64(dy), _f64(x), _f64(w), _f64(mean), _f64(rstd))
    R.check(dx, gx, sx, "dx")
    R.check(dw, gw, sw, "dweight")
    R.check(db, gb, sb, "dbias")
    assert L.layer_norm_backward(dyd, xd, wd, mean, rstd, want_bias=False)[2] is None


def test_layer_norm_large_offset_constant_rows_and_in_place():
    x = torch.full((4, 1000), 1e4, device=DEV)
    x[1] += torch.arange(1000, device=DEV) * 0.01
    w, b = torch.ones(1000, device=DEV), torch.zeros(1000, device=DEV)
    y, mean, rstd = L.layer_norm(x, w, b)
    want, wm, wr, by, bm, br = R.layer_norm(_f64(x), _f64(w), _f64(b), 1e-5)
    R.check(y[:2], want[:2], by[:2], "y")
    z = x.clone()
    s = torch.cuda.current_stream().cuda_stream
    assert L.lib().la_layer_norm(z.data_ptr(), w.data_ptr(), b.data_ptr(), 1e-5, z.data_ptr(), None, None, 4,
                                 1000, 1, 1, s) == L.LA_OK
    assert torch.equal(z, y)
    e = torch.empty((0, 1000), device=DEV)
    _, dw, db = L.layer_norm_backward(e, e, w, e[:, 0].contiguous(), e[:, 0].contiguous())
    assert not dw.any() and not db.any()


# ---------------------------------------------------------------- together

def _layer(dtype, D=64, n=16, seed=0):
    g = torch.Generator().manual_seed(seed)
    return {"nw": 1 + 0.1 * _rnd(g, D), "nb": 0.1 * _rnd(g, D), "cw": _rnd(g, D, 4, scale=0.5), "cb": _rnd(g, D),
            "A": -torch.rand((D, n), generator=g) * 3 - 0.2, "D": _rnd(g, D), "bias": _rnd(g, D) - 2,
            "wz": _rnd(g, D, 2 * D, scale=D ** -0.5), "wd": _rnd(g, D, D + 2 * n, scale=D ** -0.5)}


def _forward(p, x, cu=None, states=None):
    """norm -> projection -> convolution -> projection -> gated scan."""
    v, mean, rstd = L.layer_norm(x, p["nw"], p["nb"])
    xz = v @ p["wz"]
    D = x.shape[-1]
    c, cs = L.short_conv(xz[..., :D], p["cw"], p["cb"], state_in=states[0] if states else None, cu_seqlens=cu)
    pr = c @ p["wd"]
    n = p["A"].shape[1]
    B, C = pr[..., D:D + n].unsqueeze(-2), pr[..., D + n:].unsqueeze(-2)
    y, hs = L.selective_scan(c, pr[..., :D], p["A"], B, C, p["D"], xz[..., D:], p["bias"],
                             state_in=states[1] if states else None, cu_seqlens=cu)
    return y, (cs, hs), (v, mean, rstd, xz, c, pr, B, C)


def test_layer_of_all_three_with_gradients():
    """The three operators with projections between them, forward and backward,
    against the same layer in fp64 with automatic differentiation."""
    D, n, lens = 64, 16, [70, 1, 29]
    p = _layer(F32)
    g = torch.Generator().manual_seed(9)
    x, dy = _rnd(g, 100, D), _rnd(g, 100, D)
    d = {k: t.to(DEV) for k, t in p.items()}
    cu = _cu(lens)
    y, _, (v, mean, rstd, xz, c, pr, B, C) = _forward(d, x.to(DEV), cu)
    gs = L.selective_scan_backward(dy.to(DEV), c, pr[:, :D], d["A"], B, C, d["D"], xz[:, D:], d["bias"], cu_seqlens=cu)
    dpr = torch.cat((gs["ddelta"], gs["dB"].flatten(1), gs["dC"].flatten(1)), 1)
    dc = gs["du"] + dpr @ d["wd"].t()
    gc = L.short_conv_backward(dc, xz[:, :D], d["cw"], d["cb"], cu_seqlens=cu)
    dxz = torch.cat((gc["dx"], gs["dz"]), 1)
    dx, dnw, dnb = L.layer_norm_backward(dxz @ d["wz"].t(), x.to(DEV), d["nw"], mean, rstd)
    q = {k: t.double().requires_grad_() for k, t in p.items()}
    xq = x.double().requires_grad_()
    vq = torch.nn.functional.layer_norm(xq, (D,), q["nw"], q["nb"], 1e-5)
    xzq = vq @ q["wz"]
    spans = R.spans_of(lens)
    cq = R.conv(xzq[:, :D], q["cw"], q["cb"], True, spans)[0]
    prq = cq @ q["wd"]
    sq = {"u": cq, "delta": prq[:, :D], "A": q["A"], "B": prq[:, None, D:D + n], "C": prq[:, None, D + n:],
          "D": q["D"], "z": xzq[:, D:], "delta_bias": q["bias"], "softplus": True}
    yq = R.scan(sq, spans)[0]
    (yq * dy.double()).sum().backward()
    # fp32 through two matrix products of 64 to 96 terms and some ten more roundings
    # each: a relative error of 2^-24 sqrt(100) per stage and six stages, with a factor
    # of 16 for cancellation, in the norm of each result
    tol = 2.0 ** -24 * 10 * 6 * 16

    def near(a, b, what):
        off = float((a.detach().cpu().double() - b).norm() / b.norm())
        assert off <= tol, f"{what}: {off:.2e} > {tol:.2e}"

    near(y, yq.detach(), "y")
    for got, want, what in ((dx, xq, "x"), (dnw, q["nw"], "norm weight"), (dnb, q["nb"], "norm bias"),
                            (gc["dweight"], q["cw"], "conv weight"), (gc["dbias"], q["cb"], "conv bias"),
                            (gs["dA"], q["A"], "A"), (gs["dD"], q["D"], "D"),
                            (gs["ddelta_bias"], q["bias"], "delta bias")):
        near(got, want.grad, what)


def test_layer_prompt_then_single_tokens_captured():
    """A prompt, then single tokens through a captured graph that advances the
    cached states in place, against the prompt with those tokens appended."""
    D, n, Bt, N, more = 64, 16, 3, 33, 4
    p = {k: t.to(DEV) for k, t in _layer(F32).items()}
    x = torch.randn((Bt, N + more, D), generator=torch.Generator().manual_seed(2)).to(DEV)
    whole, (cs_all, hs_all), _ = _forward(p, x)
    _, (cs, hs), _ = _forward(p, x[:, :N].contiguous())
    tok = torch.empty((Bt, D), device=DEV)

    def step():
        v = L.layer_norm(tok, p["nw"], p["nb"], want_stats=False)[0]
        xz = v @ p["wz"]
        c = L.short_conv_step(xz[:, :D], p["cw"], p["cb"], cs)
        pr = c @ p["wd"]
        return L.selective_scan_step(c, pr[:, :D], p["A"], pr[:, None, D:D + n], pr[:, None, D + n:], hs,
                                     p["D"], xz[:, D:], p["bias"])

    keep = cs.clone(), hs.clone()
    tok.copy_(x[:, N])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    cs.copy_(keep[0]), hs.copy_(keep[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    cs.copy_(keep[0]), hs.copy_(keep[1])
    # matrix products of other shapes may sum in another order: 64 roundings of 2^-24 each, six stages
    for t in range(N, N + more):
        tok.copy_(x[:, t])
        graph.replay()
        torch.testing.assert_close(out, whole[:, t], rtol=2.0 ** -14, atol=2.0 ** -14)
    torch.testing.assert_close(hs, hs_all, rtol=2.0 ** -14, atol=2.0 ** -14)
    torch.testing.assert_close(cs, cs_all, rtol=2.0 ** -14, atol=2.0 ** -14)


def test_captured_prompt_and_backward_and_other_streams():
    """Chunked scan, its backward, convolution and norm backward inside a graph,
    replayed on new inputs, and on a stream passed by argument: the eager bits."""
    lens, D, n = [400, 57], 40, 16
    p, q = (_to(_scan_problem(lens, D, 1, n, F32, s)) for s in (1, 2))
    dy = torch.randn((sum(lens), D), device=DEV)
    w, b = torch.randn((D, 4), device=DEV), torch.randn(D, device=DEV)
    cu = _cu(lens)

    def run(p, **kw):
        args, opt = _args(p)
        y, st = L.selective_scan(*args, **opt, cu_seqlens=cu, **kw)
        g = L.selective_scan_backward(dy, *args, **opt, cu_seqlens=cu, **kw)
        c = L.short_conv_backward(dy, p["u"], w, b, cu_seqlens=cu, **kw)
        v, m, r = L.layer_norm(p["u"], b, b, **kw)
        return [y, st, *[g[k] for k in sorted(g)], *[c[k] for k in sorted(c)], v,
                *L.layer_norm_backward(dy, p["u"], b, m, r, **kw)]

    first, second = [t.clone() for t in run(p)], [t.clone() for t in run(q)]
    live = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in p.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(live)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(live)
    for src, want in ((q, second), (p, first), (q, second)):
        for k, v in src.items():
            if isinstance(v, torch.Tensor):
                live[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want))
    torch.cuda.synchronize()
    got = run(p, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, first))


def test_two_streams_at_once():
    """Two calls in flight on two streams, each with its own workspace."""
    p, q = (_to(_scan_problem([600], 24, 1, 16, F32, s)) for s in (3, 4))
    want = []
    for x in (p, q):
        args, kw = _args(x)
        want.append(L.selective_scan(*args, **kw, cu_seqlens=_cu([600])))
    cu = _cu([600])
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(5):
        for x, s in ((p, s1), (q, s2)):
            args, kw = _args(x)
            got.append(L.selective_scan(*args, **kw, cu_seqlens=cu, stream=s))
    torch.cuda.synchronize()
    for i, (y, st) in enumerate(got):
        assert torch.equal(y, want[i % 2][0]) and torch.equal(st, want[i % 2][1])


def test_launch_counts():
    D = 40
    x = torch.randn((1, 10, D), device=DEV)
    w = torch.randn((D, 4), device=DEV)
    L.short_conv(x, w)
    assert L.la_last_launch_count() == 1
    assert L.lib().la_short_conv_step(ctypes.c_void_p(0), D, w.data_ptr(), None, None, None, 1, D, 4, 1, 1, 1,
                                      None) == L.LA_ERR_INVALID_ARG
    assert L.la_last_launch_count() == 0


def test_slices_of_stacked_tensors_of_odd_widths():
    """Tensors that start inside a larger one (x[1:], a layer's weights in a stack
    of them), where their width leaves them aligned to their elements only: the
    bits of aligned copies."""
    g = torch.Generator(device=DEV).manual_seed(0)

    def inner(*shape, dtype=F32):
        return torch.randn((2, *shape), generator=g, device=DEV).to(dtype)[1]

    def both(fn, *args, **kw):
        def flat(v):
            vs = v.values() if isinstance(v, dict) else v if isinstance(v, tuple) else (v,)
            return [t for t in vs if t is not None]

        copy = lambda v: v.clone() if isinstance(v, torch.Tensor) else v  # noqa: E731
        clones = [copy(a) for a in args], {k: copy(v) for k, v in kw.items()}
        first, second = flat(fn(*args, **kw)), flat(fn(*clones[0], **clones[1]))
        assert all(torch.equal(a, b) for a, b in zip(first, second, strict=True)), fn.__name__
        # the states that a step advances in place
        for a, b in zip(args, clones[0]):
            assert not isinstance(a, torch.Tensor) or torch.equal(a, b), fn.__name__

    offsets = set()
    for dtype in (BF, F32):
        for D, n, N in ((41, 5, 33), (42, 3, 700), (45, 6, 33)):
            B = 1 if N > 100 else 3
            tok = lambda: inner(B, N, D, dtype=dtype)  # noqa: E731,B023
            bc = lambda: inner(B, N, 1, n, dtype=dtype)  # noqa: E731,B023
            u, z, dy, A = tok(), tok(), tok(), inner(D, n)
            A.copy_(-A.abs() - 0.1)
            args = (u, tok(), A, bc(), bc(), inner(D), z, inner(D))
            offsets.add(A.data_ptr() % 16)
            both(L.selective_scan, *args, state_in=inner(B, D, n))
            both(L.selective_scan_backward, dy, *args, state_in=inner(B, D, n), dstate_out=inner(B, D, n))
            one = [a[:, 0].contiguous() if a.shape[:2] == (B, N) else a for a in args]
            both(lambda s, *a: L.selective_scan_step(*a[:5], s, *a[5:]), inner(B, D, n), *one)
        for D, W in ((41, 4), (42, 3), (44, 2)):
            x, dy, w, b = inner(3, 50, D, dtype=dtype), inner(3, 50, D, dtype=dtype), inner(D, W), inner(D)
            st, ds = inner(3, W - 1, D, dtype=dtype), inner(3, W - 1, D, dtype=dtype)
            both(L.short_conv, x, w, b, state_in=st)
            both(L.short_conv_backward, dy, x, w, b, state_in=st, dstate_out=ds)
            both(lambda s, *a: L.short_conv_step(*a, s), st, x[:, 0].contiguous(), w, b)
        for rows, F in ((3, 41), (5, 1031), (3, 5003), (1, 9001)):
            x, dy, w, b = inner(rows, F, dtype=dtype), inner(rows, F, dtype=dtype), inner(F), inner(F)
            offsets.add(x.data_ptr() % 16)
            both(L.layer_norm, x, w, b)
            _, mean, rstd = L.layer_norm(x, w, b)
            both(L.layer_norm_backward, dy, x, w, mean, rstd)
            # and as an output, in place
            want, at = L.layer_norm(x, w, b)[0], inner(rows, F, dtype=dtype)
            at.copy_(x)
            s, t = torch.cuda.current_stream().cuda_stream, int(dtype == F32)
            assert L.lib().la_layer_norm(at.data_ptr(), w.data_ptr(), b.data_ptr(), 1e-5, at.data_ptr(), None,
                                         None, rows, F, t, t, s) == L.LA_OK
            assert torch.equal(at, want)
    assert any(o % 4 for o in offsets) and any(o % 8 for o in offsets)


def test_scan_forgets_at_small_steps_where_a_is_infinite():
    """From dt = 3.7e-37 on a state with A = -inf is gone after its next token,
    without and with a softplus (of -83), packed, chunked and as a single token."""
    D, n = 6, 4
    g = torch.Generator(device=DEV).manual_seed(0)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    A = -torch.rand((D, n), generator=g, device=DEV) - 0.1
    A[2, 1] = A[4] = float("-inf")
    gone = torch.isinf(A)
    for N in (1, 5, 300):
        for dt, softplus in ((3.8e-37, False), (-83.0, True)):
            u, B, C, st = r(1, N, D), r(1, N, 1, n), r(1, N, 1, n), r(1, D, n)
            delta = torch.full((1, N, D), dt, device=DEV)
            y, out = L.selective_scan(u, delta, A, B, C, softplus=softplus, state_in=st)
            # 1e-30: what 300 tokens of dt u B can bring
            assert (out[0][gone].abs() < 1e-30).all() and torch.equal(out[0][~gone], st[0][~gone])
            assert (y[0, :, 4].abs() < 1e-30).all()
            if N == 1:
                one = L.selective_scan_step(u[:, 0], delta[:, 0], A, B[:, 0], C[:, 0], st, softplus=softplus)
                assert torch.equal(st, out)
                # the four products of a channel, below 25 in all, are added in another order
                assert ((one - y[:, 0]).abs() <= 6 * 2.0 ** -24 * 25).all()
