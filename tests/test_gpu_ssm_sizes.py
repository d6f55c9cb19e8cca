"""The state space layer's kernels in the forms that large calls take, against
fp64 (tests/ssm_bounds.py): the scan with more CTAs than SMs and cut into chunks
for every number of lanes, its backward with every chunk length, single tokens in
vectors, the convolution's long tiles, and rings of the norm that go round more
than once. The rules that choose a form are restated here, so that a case that no
longer reaches its form fails."""
import pytest
import torch

from long_context_02_b200 import binding as L
from tests import ssm_bounds as S
from tests import ssm_reference as R
from tests import test_gpu_ssm as small

pytestmark = pytest.mark.gpu

DEV, BF, F32 = "cuda", torch.bfloat16, torch.float32
SMS = 148
TOKEN = ("u", "delta", "z", "B", "C")


def _near(got, want, bound, what):
    R.check(got, want.cpu(), bound.cpu(), what)


def _cu(lens):
    return torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device=DEV)


def _lanes(n):
    return 1 if n <= 4 else 2 if n <= 8 else 4 if n <= 16 else 8 if n <= 32 else 16


def _forward_ctas(lens, D, G, n):
    """(CTAs of the scan, chunk length or 0) of a packed batch."""
    CC, total = 256 // _lanes(n), sum(lens)
    ctas = G * -(-(D // G) // CC)
    if ctas * 2 > SMS:
        return ctas * len(lens), 0
    want = min(2 * SMS // ctas, 64)
    length = max(-(--(-total // want) // 32) * 32, 64)
    if total <= 2 * length:
        return ctas * len(lens), 0
    return ctas * (total // length + len(lens)), length


def _backward_chunk(lens, D, G, n):
    blocks = G * -(-(D // G) // (256 // max(_lanes(n), 2)))
    length = 128
    while length > 32 and (sum(lens) // length + 1) * blocks < 3 * SMS:
        length //= 2
    return length


def _problem(lens, D, G, n, dtype, gate=True):
    T = sum(lens)
    g = torch.Generator(device=DEV).manual_seed(D + n)
    r = lambda *s, dtype=F32: torch.randn(s, generator=g, device=DEV).to(dtype)  # noqa: E731
    proj = r(T, 8 + 2 * G * n, dtype=dtype)
    # slow and fast states: what an error does over the length shows in the slow ones
    p = {"u": r(T, D, dtype=dtype), "delta": (r(T, D) * 0.5).to(dtype), "B": proj[:, 8:8 + G * n].unflatten(-1, (G, n)),
         "C": proj[:, 8 + G * n:].unflatten(-1, (G, n)), "z": r(T, 2 * D, dtype=dtype)[:, D:] if gate else None,
         "A": -torch.rand((D, n), generator=g, device=DEV) * 4 - 0.01, "D": r(D), "delta_bias": r(D) - 2,
         "softplus": True}
    return p, r(T, D, dtype=dtype), r(len(lens), D, n), r(len(lens), D, n)


def _call(p):
    return [p[k] for k in ("u", "delta", "A", "B", "C")], {k: p[k] for k in ("D", "z", "delta_bias", "softplus")}


def _f64(p):
    return {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in p.items()}


MANY = [37, 0, 1, 64, 33, 9, 31, 32, 40, 5, 65, 2, 17, 70, 8, 16]
WIDE = [  # 10 channel blocks each
    (4, 2560, 2), (5, 1280, 1), (8, 1280, 1), (12, 640, 2), (16, 640, 1), (20, 320, 1), (32, 320, 2), (50, 160, 1),
    (64, 160, 1)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,D,G", WIDE)
def test_scan_with_more_ctas_than_sms(n, D, G, dtype):
    """16 sequences, packed (cut into chunks, as one long sequence would be) and as
    a dense batch (one pass)."""
    ctas, length = _forward_ctas(MANY, D, G, n)
    assert ctas > SMS and length > 0 and D // G % 2 == 0
    p, _, st, _ = _problem(MANY, D, G, n, dtype, gate=n != 12)
    args, kw = _call(p)
    want, bound = S.scan(_f64(p), R.spans_of(MANY), 32, state_in=st.double())
    y, out = L.selective_scan(*args, **kw, state_in=st, cu_seqlens=_cu(MANY), out_dtype=F32)
    assert L.la_last_launch_count() == 3
    _near(y, want["y"], bound["y"], "y")
    _near(out, want["state"], bound["state"], "state")
    if dtype == BF:
        assert torch.equal(L.selective_scan(*args, **kw, state_in=st, cu_seqlens=_cu(MANY))[0], y.to(BF))
    B, N = 16, 37
    assert B * 10 > SMS
    p, _, st, _ = _problem([N] * B, D, G, n, dtype, gate=n != 12)
    want, bound = S.scan(_f64(p), R.spans_of([N] * B), 32, state_in=st.double())
    args, kw = _call({k: v.unflatten(0, (B, N)) if k in TOKEN and v is not None else v for k, v in p.items()})
    y, out = L.selective_scan(*args, **kw, state_in=st, out_dtype=F32)
    assert L.la_last_launch_count() == 1
    _near(y.flatten(0, 1), want["y"], bound["y"], "dense y")
    _near(out, want["state"], bound["state"], "dense state")


CUT = [  # tokens, channel blocks, fewer channels than those: with more CTAs than SMs, fewer, without vectors
    ([2500, 0, 1, 499], 4, 0), ([300], 1, 0), ([170, 230], 2, 0), ([300, 3], 1, 3)]


@pytest.mark.parametrize("n", [3, 8, 16, 24, 32, 64])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens,blocks,less", CUT)
def test_scan_in_chunks(lens, blocks, less, n, dtype):
    D = blocks * (256 // _lanes(n)) - less
    ctas, length = _forward_ctas(lens, D, 1, n)
    assert length > 0 and (ctas > SMS) == (len(lens) == 4)
    p, _, st, _ = _problem(lens, D, 1, n, dtype)
    args, kw = _call(p)
    want, bound = S.scan(_f64(p), R.spans_of(lens), 32, state_in=st.double())
    y, out = L.selective_scan(*args, **kw, state_in=st, cu_seqlens=_cu(lens), out_dtype=F32)
    assert L.la_last_launch_count() == 3  # the table of chunks, their states, the outputs
    _near(y, want["y"], bound["y"], "y")
    _near(out, want["state"], bound["state"], "state")


def test_scan_in_chunks_of_a_dense_batch():
    B, N, D, n = 2, 700, 256, 16
    p, _, st, _ = _problem([N] * B, D, 1, n, BF)
    want, bound = S.scan(_f64(p), R.spans_of([N] * B), 32, state_in=st.double())
    args, kw = _call({k: v.unflatten(0, (B, N)) if k in TOKEN else v for k, v in p.items()})
    y, out = L.selective_scan(*args, **kw, state_in=st, out_dtype=F32)
    assert L.la_last_launch_count() == 2
    _near(y.flatten(0, 1), want["y"], bound["y"], "y")
    _near(out, want["state"], bound["state"], "state")


BACK = [  # n, channels per block, blocks in all, groups, fewer channels per group, dtype
    # chunks of 128
    (16, 64, 56, 1, 0, BF), (16, 64, 56, 2, 0, F32), (16, 64, 56, 1, 1, BF), (8, 128, 56, 1, 0, F32),
    (3, 128, 56, 1, 0, BF), (32, 32, 56, 1, 0, BF), (64, 16, 56, 1, 0, F32), (33, 16, 56, 1, 1, BF),
    # chunks of 64
    (16, 64, 28, 1, 0, BF), (16, 64, 28, 1, 1, F32), (5, 128, 28, 1, 0, BF), (24, 32, 28, 2, 0, F32),
    (64, 16, 28, 1, 0, BF),
    # chunks of 32
    (16, 64, 8, 1, 0, BF), (8, 128, 6, 1, 1, F32), (64, 16, 6, 2, 0, F32)]


@pytest.mark.parametrize("n,CC,blocks,G,less,dtype", BACK)
def test_scan_backward_by_chunk_length(n, CC, blocks, G, less, dtype):
    lens = [700, 0, 1, 249, 50]
    D = blocks * CC - less * G
    chunk = _backward_chunk(lens, D, G, n)
    assert chunk == {56: 128, 28: 64}.get(blocks, 32)
    p, dy, st, ds = _problem(lens, D, G, n, dtype)
    args, kw = _call(p)
    opt = dict(state_in=st, dstate_out=ds, cu_seqlens=_cu(lens))
    got = L.selective_scan_backward(dy, *args, **kw, **opt, out_dtype=F32)
    want, bound = S.scan(_f64(p), R.spans_of(lens), chunk, dy.double(), st.double(), ds.double())
    assert set(got) == set(want) - {"y", "state"}
    for k, v in got.items():
        _near(v, want[k], bound[k], k)
    if dtype == BF:
        for k, v in L.selective_scan_backward(dy, *args, **kw, **opt).items():
            assert torch.equal(v, got[k].to(v.dtype)), k


@pytest.mark.parametrize("lens,D,G,n,dtype,gate,skip,bias,softplus,state", small.SCANS)
def test_scan_backward_of_small_cases(lens, D, G, n, dtype, gate, skip, bias, softplus, state):
    """The cases of test_gpu_ssm.py within bounds that follow the errors."""
    p = small._to(small._scan_problem(lens, D, G, n, dtype, len(lens) + D, gate, skip, bias, softplus))
    g = torch.Generator(device=DEV).manual_seed(6)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    dy = r(sum(lens), D).to(dtype)
    st, ds = (r(len(lens), D, n), r(len(lens), D, n)) if state else (None, None)
    args, kw = _call(p)
    got = L.selective_scan_backward(dy, *args, **kw, state_in=st, dstate_out=ds, cu_seqlens=_cu(lens), out_dtype=F32)
    double = lambda t: None if t is None else t.double()  # noqa: E731
    want, bound = S.scan(_f64(p), R.spans_of(lens), _backward_chunk(lens, D, G, n), dy.double(), double(st), double(ds))
    for k, v in got.items():
        _near(v, want[k], bound[k], k)


def test_scan_backward_of_a_dense_batch_in_long_chunks():
    """Without states, a gate or a skip; the last chunk of each sequence is not whole."""
    B, N, D, n = 3, 331, 3584, 16
    p, dy, _, _ = _problem([N] * B, D, 1, n, BF, gate=False)
    p["D"] = None
    assert _backward_chunk([N] * B, D, 1, n) == 128
    want, bound = S.scan(_f64(p), R.spans_of([N] * B), 128, dy.double())
    args, kw = _call({k: v.unflatten(0, (B, N)) if k in TOKEN and v is not None else v for k, v in p.items()})
    got = L.selective_scan_backward(dy.unflatten(0, (B, N)), *args, **kw, out_dtype=F32)
    for k, v in got.items():
        _near(v.flatten(0, 1) if v.shape[:2] == (B, N) else v, want[k], bound[k], k)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,D,G,odd", [(4, 260, 1, 0), (8, 130, 2, 0), (16, 96, 3, 0), (32, 70, 1, 0), (64, 40, 2, 0),
                                       (16, 96, 1, 1), (64, 33, 1, 2), (9, 50, 1, 0)])
def test_scan_step_of_many_sequences(n, D, G, odd, dtype):
    """Whole vectors of states for every number of lanes, with B and C on vectors
    and (`odd` elements off) not, more sequences than a CTA takes."""
    B = 9
    g = torch.Generator(device=DEV).manual_seed(n)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    pick = lambda: r(B, odd + G * n + 4).to(dtype)[:, odd:odd + G * n].unflatten(-1, (G, n))  # noqa: E731
    p = {"u": r(B, D).to(dtype), "delta": r(B, D).to(dtype), "A": -torch.rand((D, n), generator=g, device=DEV) * 4,
         "B": pick(), "C": pick(), "D": r(D), "z": r(B, 2 * D).to(dtype)[:, D:], "delta_bias": r(D) - 2,
         "softplus": True}
    st = r(B, D, n)
    want, bound = S.scan(_f64(p), R.spans_of([1] * B), 32, state_in=st.double())
    args, kw = _call(p)
    y = L.selective_scan_step(*args, st, **kw, out_dtype=F32)
    _near(y, want["y"], bound["y"], "y")
    _near(st, want["state"], bound["state"], "state")


def _tile(total, D, wide, back):
    """Rows per CTA of the convolution."""
    blocks = -(-D // (512 if wide else 128))
    rows = total * blocks
    if not back:
        return 64 if rows >= SMS * 8 * 64 else 32 if rows >= SMS * 8 * 32 else 16
    waves = max((rows + SMS * 4 * 64) // (SMS * 4 * 128), 1)
    return max(-(-rows // (SMS * 4 * waves)), 16)


@pytest.mark.parametrize("W,dtype,silu", [(4, BF, True), (4, F32, True), (3, F32, False), (2, BF, False), (3, BF, True)])
@pytest.mark.parametrize("total,D", [(40_000, 64), (40_003, 37), (90_000, 40), (80_005, 27)])
def test_conv_in_long_tiles(total, D, W, dtype, silu):
    lens = [total // 2, 0, 1, 3, 700, 2, 129]
    lens.append(total - sum(lens))
    wide = D % 4 == 0
    assert _tile(total, D, wide, False) == (64 if total > 75_776 else 32) and _tile(total, D, wide, True) > 64
    g = torch.Generator(device=DEV).manual_seed(D + W)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    x, dy = r(total, 2 * D).to(dtype)[:, D:], r(total, D).to(dtype)
    w, b = r(D, W), r(D)
    st, ds = r(len(lens), W - 1, D).to(dtype), r(len(lens), W - 1, D).to(dtype)
    y, out = L.short_conv(x, w, b, silu, st, _cu(lens), out_dtype=F32)
    tile = _tile(total, D, wide, True)
    want, bound = S.conv(x.double(), w.double(), b.double(), silu, lens, st.double(), dy.double(), ds.double(),
                         chain=tile + -(-total // tile))
    _near(y, want["y"], bound["y"], "y")
    assert torch.equal(out.double(), want["state"])
    got = L.short_conv_backward(dy, x, w, b, silu, st, ds, _cu(lens), out_dtype=F32)
    for k, v in got.items():
        _near(v, want[k], bound[k], k)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,F", [(9001, 1032), (6003, 2056), (3001, 4104), (9001, 515)])
def test_layer_norm_rings_that_go_round(rows, F, dtype):
    """More rows than the resident CTAs hold in one turn of their rings."""
    g = torch.Generator(device=DEV).manual_seed(F)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    x, dy, w, b = (r(rows, F) + 3).to(dtype), r(rows, F).to(dtype), r(F), r(F)
    y, mean, rstd = L.layer_norm(x, w, b, out_dtype=F32)
    want, wm, wr, by, bm, br = R.layer_norm(x.double(), w.double(), b.double(), 1e-5)
    _near(mean, wm, bm, "mean")
    _near(rstd, wr, br, "rstd")
    _near(y, want, by, "y")
    got = L.layer_norm_backward(dy, x, w, mean, rstd, out_dtype=F32)
    want, bound = R.layer_norm_backward(dy.double(), x.double(), w.double(), mean.double(), rstd.double())
    for v, a, e, k in zip(got, want, bound, ("dx", "dweight", "dbias")):
        _near(v, a, e, k)
