"""The state space layer's entry points refuse bad arguments before any CUDA
call, so every check here runs without a GPU."""
import ctypes

import pytest
import torch

from long_context_02_b200 import binding as L

P = ctypes.c_void_p
X = 256  # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    from long_context_02_b200 import build
    build.build()
    return L.lib()


def _inputs(**kw):
    a = dict(u=X, delta=X, z=X, B=X, C=X, ld_u=128, ld_delta=128, ld_z=128, ld_b=16, ld_c=16, A=X,
             D=X, delta_bias=X, softplus=1)
    a.update(kw)
    return L.SCAN_INPUTS.pack(*a.values())


def _scan(lib, cu=0, seqs=2, st=0, y=X, out=0, total=64, D=128, G=1, n=16, it=0, ot=0, ws=X,
          wsb=1 << 40, **kw):
    return lib.la_selective_scan(P(cu) if cu else None, seqs, _inputs(**kw), P(st) if st else None,
                                 P(y) if y else None, P(out) if out else None, total, D, G, n, it,
                                 ot, P(ws) if ws else None, wsb, None)


BAD_SCAN = [
    (dict(seqs=-1), L.LA_ERR_INVALID_ARG), (dict(total=-1), L.LA_ERR_INVALID_ARG),
    (dict(seqs=0), L.LA_ERR_INVALID_ARG),            # rows of no sequence
    (dict(total=63), L.LA_ERR_INVALID_ARG),          # dense: not a multiple of the sequences
    (dict(D=0), L.LA_ERR_INVALID_ARG), (dict(G=0), L.LA_ERR_INVALID_ARG),
    (dict(G=3), L.LA_ERR_INVALID_ARG),               # groups do not divide the channels
    (dict(n=0), L.LA_ERR_INVALID_ARG), (dict(n=65), L.LA_ERR_UNSUPPORTED),
    (dict(it=2), L.LA_ERR_INVALID_ARG), (dict(it=1, ot=0), L.LA_ERR_UNSUPPORTED),
    (dict(u=0), L.LA_ERR_INVALID_ARG), (dict(delta=0), L.LA_ERR_INVALID_ARG),
    (dict(A=0), L.LA_ERR_INVALID_ARG), (dict(B=0), L.LA_ERR_INVALID_ARG),
    (dict(C=0), L.LA_ERR_INVALID_ARG), (dict(y=0), L.LA_ERR_INVALID_ARG),
    (dict(u=X + 1), L.LA_ERR_INVALID_ARG),           # not aligned to its elements
    (dict(u=X + 2, it=1, ot=1), L.LA_ERR_INVALID_ARG),
    (dict(A=X + 4), L.LA_ERR_INVALID_ARG), (dict(y=X + 8), L.LA_ERR_INVALID_ARG),
    (dict(st=X + 4), L.LA_ERR_INVALID_ARG), (dict(cu=X + 2), L.LA_ERR_INVALID_ARG),
    (dict(ld_u=127), L.LA_ERR_INVALID_ARG), (dict(ld_z=0), L.LA_ERR_INVALID_ARG),
    (dict(ld_b=15), L.LA_ERR_INVALID_ARG),
    (dict(total=(1 << 31) - 2), L.LA_ERR_UNSUPPORTED),
    (dict(ld_u=(1 << 24) + 1), L.LA_ERR_UNSUPPORTED), (dict(ld_c=1 << 25), L.LA_ERR_UNSUPPORTED),
    (dict(seqs=1 << 25, total=0), L.LA_ERR_UNSUPPORTED),
    # a long prompt in a narrow layer is cut into chunks and needs a workspace
    (dict(total=1 << 16, ws=0), L.LA_ERR_WORKSPACE), (dict(total=1 << 16, wsb=64), L.LA_ERR_WORKSPACE),
]


@pytest.mark.parametrize("kw,status", BAD_SCAN)
def test_scan_refuses(lib, kw, status):
    assert _scan(lib, **kw) == status


def test_scan_takes_null_inputs_without_rows(lib):
    # no sequences: nothing to do, nothing launched
    assert _scan(lib, seqs=0, total=0, u=0, delta=0, z=0, B=0, C=0, y=0, ws=0, wsb=0) == L.LA_OK
    assert L.la_last_launch_count() == 0


def _step(lib, B=4, D=128, G=1, n=16, st=X, y=X, it=0, ot=0, **kw):
    return lib.la_selective_scan_step(_inputs(**kw), P(st) if st else None, P(y) if y else None, B, D,
                                      G, n, it, ot, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), L.LA_ERR_INVALID_ARG), (dict(st=0), L.LA_ERR_INVALID_ARG),
    (dict(y=0), L.LA_ERR_INVALID_ARG), (dict(st=X + 4), L.LA_ERR_INVALID_ARG),
    (dict(n=65), L.LA_ERR_UNSUPPORTED), (dict(G=7), L.LA_ERR_INVALID_ARG),
    (dict(ld_c=3), L.LA_ERR_INVALID_ARG), (dict(it=1), L.LA_ERR_UNSUPPORTED),
    (dict(B=0), L.LA_OK)])
def test_scan_step_refuses(lib, kw, status):
    assert _step(lib, **kw) == status


def _scan_back(lib, dy=X, ld_dy=128, total=64, ws=X, wsb=1 << 40, grads=None, **kw):
    g = dict(du=X, ddelta=X, dz=X, dB=X, dC=X, dA=X, dD=X, ddelta_bias=X, dstate_in=X)
    g.update(grads or {})
    out = L.SCAN_GRADS.pack(*g.values())
    return lib.la_selective_scan_backward(None, 2, _inputs(**kw), None, P(dy) if dy else None, ld_dy,
                                          None, out, total, 128, 1, 16, 0, 0, P(ws) if ws else None,
                                          wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=0), L.LA_ERR_INVALID_ARG), (dict(ld_dy=100), L.LA_ERR_INVALID_ARG),
    (dict(ld_dy=1 << 25), L.LA_ERR_UNSUPPORTED),
    (dict(grads=dict(dA=0)), L.LA_ERR_INVALID_ARG), (dict(grads=dict(du=0)), L.LA_ERR_INVALID_ARG),
    (dict(grads=dict(dz=0)), L.LA_ERR_INVALID_ARG),   # a gate without its gradient
    (dict(z=0), L.LA_ERR_INVALID_ARG),                # and the reverse
    (dict(grads=dict(dB=X + 2)), L.LA_ERR_INVALID_ARG),
    (dict(ws=0), L.LA_ERR_WORKSPACE), (dict(wsb=1000), L.LA_ERR_WORKSPACE)])
def test_scan_backward_refuses(lib, kw, status):
    assert _scan_back(lib, **kw) == status


def _conv(lib, cu=0, seqs=2, x=X, ld=64, w=X, b=X, st=0, y=X, out=0, total=32, D=64, W=4, it=0, ot=0):
    return lib.la_short_conv(P(cu) if cu else None, seqs, P(x) if x else None, ld, P(w) if w else None,
                             P(b) if b else None, P(st) if st else None, P(y) if y else None,
                             P(out) if out else None, total, D, W, 1, it, ot, None)


@pytest.mark.parametrize("kw,status", [
    (dict(W=0), L.LA_ERR_INVALID_ARG), (dict(W=1), L.LA_ERR_UNSUPPORTED),
    (dict(W=5), L.LA_ERR_UNSUPPORTED), (dict(x=0), L.LA_ERR_INVALID_ARG),
    (dict(w=0), L.LA_ERR_INVALID_ARG), (dict(y=0), L.LA_ERR_INVALID_ARG),
    (dict(ld=63), L.LA_ERR_INVALID_ARG), (dict(x=X + 1), L.LA_ERR_INVALID_ARG),
    (dict(w=X + 4), L.LA_ERR_INVALID_ARG), (dict(total=31), L.LA_ERR_INVALID_ARG),
    (dict(seqs=0), L.LA_ERR_INVALID_ARG), (dict(it=3), L.LA_ERR_INVALID_ARG),
    (dict(st=X, out=X), L.LA_ERR_INVALID_ARG)])       # the states may not be one array
def test_conv_refuses(lib, kw, status):
    assert _conv(lib, **kw) == status


def test_conv_step_and_backward_refuse(lib):
    x = P(X)
    step = lambda **k: lib.la_short_conv_step(*{**dict(x=x, ld=64, w=x, b=x, s=x, y=x, B=2, D=64, W=4, a=1, i=0, o=0, st=None), **k}.values())  # noqa: E731,E501
    assert step(s=None) == L.LA_ERR_INVALID_ARG
    assert step(B=-2) == L.LA_ERR_INVALID_ARG
    assert step(W=6) == L.LA_ERR_UNSUPPORTED
    assert step(B=0) == L.LA_OK
    back = lambda **k: lib.la_short_conv_backward(*{**dict(cu=None, s=2, dy=x, ldy=64, x=x, ld=64, w=x, b=x, si=None, so=None, dx=x, dw=x, db=x, ds=None, t=32, D=64, W=4, a=1, i=0, o=0, ws=x, n=1 << 30, st=None), **k}.values())  # noqa: E731,E501
    assert back(dy=None) == L.LA_ERR_INVALID_ARG
    assert back(dw=None) == L.LA_ERR_INVALID_ARG
    assert back(ldy=8) == L.LA_ERR_INVALID_ARG
    assert back(ws=None) == L.LA_ERR_WORKSPACE
    assert back(n=16) == L.LA_ERR_WORKSPACE


def test_norm_refuses(lib):
    x = P(X)
    f = lambda **k: lib.la_layer_norm(*{**dict(x=x, w=x, b=x, e=1e-5, y=x, m=x, r=x, rows=4, F=64, i=0, o=0, st=None), **k}.values())  # noqa: E731,E501
    assert f(F=0) == L.LA_ERR_INVALID_ARG
    assert f(rows=-1) == L.LA_ERR_INVALID_ARG
    assert f(F=16385) == L.LA_ERR_UNSUPPORTED
    assert f(e=-1.0) == L.LA_ERR_INVALID_ARG
    assert f(e=float("nan")) == L.LA_ERR_INVALID_ARG
    assert f(e=float("inf")) == L.LA_ERR_INVALID_ARG
    assert f(m=None) == L.LA_ERR_INVALID_ARG          # both statistics or neither
    assert f(w=None) == L.LA_ERR_INVALID_ARG
    assert f(x=P(X + 2)) == L.LA_ERR_INVALID_ARG
    assert f(o=1) == L.LA_ERR_INVALID_ARG             # in place only in the same dtype
    assert f(rows=0) == L.LA_OK
    g = lambda **k: lib.la_layer_norm_backward(*{**dict(dy=x, x=x, w=x, m=x, r=x, dx=x, dw=x, db=x, rows=4, F=64, i=0, o=0, ws=x, n=1 << 30, st=None), **k}.values())  # noqa: E731,E501
    assert g(dy=None) == L.LA_ERR_INVALID_ARG
    assert g(m=None) == L.LA_ERR_INVALID_ARG
    assert g(dw=None) == L.LA_ERR_INVALID_ARG
    assert g(F=20000) == L.LA_ERR_UNSUPPORTED
    assert g(n=8) == L.LA_ERR_WORKSPACE


def test_workspace_sizes(lib):
    size = L.la_workspace_bytes
    assert size(L.LA_OP_SCAN, 1, 8192, 8192, 16, 4) == 0            # wide enough: one pass
    assert size(L.LA_OP_SCAN, 1, 1024, 65536, 16, 1) > 0
    assert size(L.LA_OP_SCAN, 3, 1024, 65536, 16, 1) == 0           # invalid: G does not divide D
    assert size(L.LA_OP_SCAN_BACKWARD, 1, 1024, 4096, 65, 1) == 0
    assert size(L.LA_OP_SCAN_BACKWARD, 1, 1024, 4096, 64, 1) > 2 * 32 * 1024 * 64 * 4
    assert size(L.LA_OP_CONV_BACKWARD, 1, 100, 0, 4, 3) == 0        # no rows: no partial sums
    assert size(L.LA_OP_CONV_BACKWARD, 1, 100, 10, 5, 3) == 0
    assert size(L.LA_OP_NORM_BACKWARD, 1, 100, 7, 0, 0) >= 2 * 7 * 100 * 4
    assert size(L.LA_OP_NORM_BACKWARD, 1, 100000, 7, 0, 0) == 0


def test_binding_refuses(lib):
    """Shapes, dtypes and layouts that the binding turns down by itself."""
    x = torch.zeros((2, 8, 64))
    w = torch.zeros((64, 4))
    with pytest.raises(ValueError, match="GPU"):
        L.short_conv(x, w)
    with pytest.raises(ValueError, match="GPU"):
        L.layer_norm(x, w[:, 0].contiguous())
    with pytest.raises(ValueError, match="without cu_seqlens"):
        L.selective_scan(x[0], x[0], w, x, x)
    with pytest.raises(ValueError, match="int32"):
        L.short_conv(x[0], w, cu_seqlens=torch.zeros(3, dtype=torch.int64))
    z = torch.zeros
    assert L._rows(z((2, 8, 128))[..., 64:], (2, 8, 64), 2, 64, "x")[1] == 128
    assert L._rows(z((2, 8, 100))[..., 4:36].unflatten(-1, (2, 16)), (2, 8, 2, 16), 2, 32, "B")[1] == 100
    assert L._rows(z((1, 1, 64)), (1, 1, 64), 2, 64, "x")[1] == 64
    assert L._rows(z((5, 128))[:, :64], (5, 64), 1, 64, "x")[1] == 128
    with pytest.raises(ValueError, match="contiguous"):
        L._rows(z((2, 8, 128))[..., ::2], (2, 8, 64), 2, 64, "x")
    with pytest.raises(ValueError, match="evenly spaced"):
        L._rows(z((2, 16, 64))[:, :8], (2, 8, 64), 2, 64, "x")
    with pytest.raises(ValueError, match="expected"):
        L._rows(z((2, 8, 63)), (2, 8, 64), 2, 64, "x")


def test_sizes_beyond_31_bits_are_refused(lib):
    """More features than LA_MAX_LD, or more than 2^30 states, in calls that no stride refuses."""
    wide, many = (1 << 24) + 128, (1 << 30) + 2
    x = P(X)
    assert _scan(lib, total=1, seqs=1, D=wide) == L.LA_ERR_UNSUPPORTED
    assert _scan(lib, total=0, seqs=many, D=1, n=1) == L.LA_ERR_UNSUPPORTED
    assert _step(lib, B=1, D=wide) == L.LA_ERR_UNSUPPORTED
    assert _step(lib, B=many, D=1, ld_u=1, ld_delta=1, ld_z=1, n=1, ld_b=1, ld_c=1) == L.LA_ERR_UNSUPPORTED
    grads = L.SCAN_GRADS.pack(*[X] * 9)
    assert lib.la_selective_scan_backward(None, 1, _inputs(), None, x, wide, None, grads, 1, wide, 1,
                                          16, 0, 0, x, 1 << 60, None) == L.LA_ERR_UNSUPPORTED
    assert _conv(lib, total=1, seqs=1, D=(1 << 31) - 1) == L.LA_ERR_UNSUPPORTED
    assert _conv(lib, total=0, seqs=many, D=1, ld=1) == L.LA_ERR_UNSUPPORTED
    assert lib.la_short_conv_step(x, wide, x, x, x, x, 1, wide, 4, 1, 0, 0, None) == L.LA_ERR_UNSUPPORTED
    size = L.la_workspace_bytes
    assert size(L.LA_OP_SCAN_BACKWARD, 1, wide, 1, 16, 1) == 0
    assert size(L.LA_OP_SCAN_BACKWARD, 1, 1, 0, 1, many) == 0
    assert size(L.LA_OP_SCAN, 1, 1, 1 << 20, 1, many) == 0
    assert size(L.LA_OP_CONV_BACKWARD, 1, (1 << 31) - 1, 1, 4, 1) == 0


def test_binding_refuses_norm_of_a_scalar(lib, monkeypatch):
    monkeypatch.setattr(L, "_on", lambda *a: (0, None, 0))
    one = torch.zeros(())
    with pytest.raises(ValueError, match="no dimension"):
        L.layer_norm(one, torch.zeros(1))
    with pytest.raises(ValueError, match="no dimension"):
        L.layer_norm_backward(one, one, torch.zeros(1), one, one)


def test_slices_of_odd_widths_are_taken(lib):
    """A slice x[1:] of an aligned tensor whose rows allow no vectors is aligned to
    its elements only. None of these calls launches: they have no rows, or end at
    the check of the workspace, behind the tensors'."""
    x, o2, o4, o8 = P(X), P(X + 2), P(X + 4), P(X + 8)
    norm = lambda **k: lib.la_layer_norm(*{**dict(x=x, w=x, b=x, e=1e-5, y=x, m=x, r=x, rows=0, F=5003, i=1, o=1, st=None), **k}.values())  # noqa: E731,E501
    assert norm(x=o4, w=o4, b=o8) == L.LA_OK
    assert norm(x=o2, i=0) == L.LA_OK
    assert norm(x=o8, F=5002) == L.LA_OK
    assert norm(x=o4, F=5002) == L.LA_ERR_INVALID_ARG
    assert norm(w=P(X + 1)) == L.LA_ERR_INVALID_ARG
    back = lambda **k: lib.la_layer_norm_backward(*{**dict(dy=x, x=x, w=x, m=x, r=x, dx=x, dw=x, db=x, rows=4, F=5003, i=1, o=1, ws=None, n=0, st=None), **k}.values())  # noqa: E731,E501
    assert back(dy=o4, x=o4, w=o4, dx=o4, dw=o4, db=o4) == L.LA_ERR_WORKSPACE
    assert back(dx=o8, F=5004) == L.LA_ERR_INVALID_ARG
    odd = dict(total=1 << 16, D=127, n=5, ws=0)
    assert _scan(lib, **odd, A=X + 4, delta_bias=X + 4, st=X + 4, out=X + 4, y=X + 2) == L.LA_ERR_WORKSPACE
    assert _scan(lib, **odd, y=X + 2, ot=1) == L.LA_ERR_INVALID_ARG
    assert _scan(lib, **{**odd, "n": 16}, st=X + 4) == L.LA_ERR_INVALID_ARG
    assert _scan(lib, **{**odd, "D": 126}, y=X + 2) == L.LA_ERR_INVALID_ARG
    o = X + 4
    grads = L.SCAN_GRADS.pack(X + 2, X + 2, X + 2, X + 2, X + 2, o, o, o, o)
    args = [_inputs(A=o, D=o, delta_bias=o), P(o), x, 128, P(o), grads, 64, 127, 1, 5, 0, 0, None, 0, None]
    assert lib.la_selective_scan_backward(None, 2, *args) == L.LA_ERR_WORKSPACE
    args[6 + 1] = 128  # a width of whole vectors
    assert lib.la_selective_scan_backward(None, 2, *args) == L.LA_ERR_INVALID_ARG
    none = dict(seqs=0, total=0)
    assert _conv(lib, **none, D=13, W=3, w=X + 4, b=X + 4, y=X + 2, st=X + 8, out=X + 4) == L.LA_OK
    assert _conv(lib, **none, D=13, W=3, st=X + 2) == L.LA_ERR_INVALID_ARG  # two rows of 13: 52 bytes
    assert _conv(lib, **none, D=12, W=3, w=X + 4) == L.LA_ERR_INVALID_ARG
    assert _conv(lib, **none, D=12, W=2, st=X + 8) == L.LA_OK
    assert _conv(lib, **none, D=12, W=2, st=X + 4) == L.LA_ERR_INVALID_ARG
    conv = lambda **k: lib.la_short_conv_backward(*{**dict(cu=None, s=2, dy=x, ldy=64, x=x, ld=64, w=x, b=x, si=None, so=None, dx=x, dw=x, db=x, ds=None, t=32, D=63, W=4, a=1, i=0, o=0, ws=None, n=0, st=None), **k}.values())  # noqa: E731,E501
    assert conv(w=o8, b=o4, si=o2, so=o2, dx=o2, dw=o8, db=o4, ds=o2) == L.LA_ERR_INVALID_ARG  # weight: 63 * 16 bytes
    assert conv(W=3, w=o4, b=o4, si=o4, so=o4, dx=o2, dw=o4, db=o4, ds=o4) == L.LA_ERR_WORKSPACE
