"""Layer normalisation's kernels against the FP64 formulas."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU-only machines
    pytest.skip("needs a CUDA device", allow_module_level=True)

import causal_depthwise_conv1d_gb300 as ccv  # noqa: E402
from tests import mixer_ref as ref  # noqa: E402

DT = ref.DT
SIZES = [(1, 1), (3, 7), (5, 128), (1, 256), (9, 264), (33, 1000), (700, 64), (17, 1001), (4, 5120), (3, 8192),
         (2, 16384), (2, 40000), (1300, 512), (7, 130), (4, 9001)]


def case(N, D, dtype, wdtype, seed=0, mean=3.0):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    return ((rnd(N, D) + mean * rnd(1, D)).to(DT[dtype]), (1 + 0.3 * rnd(D)).to(DT[wdtype]),
            (0.3 * rnd(D)).to(DT[wdtype]), rnd(N, D).to(DT[dtype]))


def chain(D):
    """Longest FP32 addition chain of a row's sum, generously: 40 terms a
    thread or D over 512 threads, then the exchanges."""
    return 48 + D / 512


def fwd_bound(x, w, y, xh, r, dtype):
    D = x.shape[1]
    g = chain(D) * 2.0 ** -24
    # the mean is off by at most g mean|x|, the spread by g: through xh, then a few roundings
    dm = g * x.double().abs().mean(-1, keepdim=True) * r
    wa = 1.0 if w is None else w.double().abs()
    return ref.rounding(y, dtype) + wa * (dm * (1 + xh.abs()) + 2 * g * xh.abs()) + 4 * 2.0 ** -24 * y.abs() + \
        4 * 2.0 ** -24 * wa * xh.abs()


@pytest.mark.parametrize("dtype,wdtype", [("f32", "f32"), ("f16", "f32"), ("bf16", "bf16"), ("f16", "bf16")])
@pytest.mark.parametrize("N,D", SIZES)
def test_forward(N, D, dtype, wdtype):
    x, w, b, _ = case(N, D, dtype, wdtype)
    y, xh, r = ref.ln_fwd(x, w, b)
    got = ccv.layer_norm_fwd(x.cuda(), w.cuda(), b.cuda())
    assert ccv.ccv_last_kernel() == "ln_fwd"
    assert ref.worst(got, y, fwd_bound(x, w, y, xh, r, dtype) + 2.0 ** -23 * b.double().abs()) <= 1
    y0, xh, r = ref.ln_fwd(x, None, None)
    assert ref.worst(ccv.layer_norm_fwd(x.cuda()), y0, fwd_bound(x, None, y0, xh, r, dtype)) <= 1


def bwd_bounds(x, w, dy, dtype, wdtype):
    N, D = x.shape
    dx, dw, db = ref.ln_bwd(x, w, dy)
    _, xh, r = ref.ln_fwd(x, None, None)
    g = chain(D) * 2.0 ** -24
    d = dy.double().abs() * w.double().abs()
    dm = g * x.double().abs().mean(-1, keepdim=True) * r     # error of xh from the mean
    exh = dm * (1 + xh.abs()) + 2 * g * xh.abs()
    m1, m2 = d.mean(-1, keepdim=True), (d * xh.abs()).mean(-1, keepdim=True)
    bx = ref.rounding(dx, dtype) + r * (4 * g * (d + m1 + 2 * xh.abs() * m2) +
                                        exh * m2 + xh.abs() * (d * exh).mean(-1, keepdim=True) +
                                        (dm + 2 * g) * (d + m1 + xh.abs() * m2))
    gn = (N + 16) * 2.0 ** -24
    bw = ref.rounding(dw, wdtype) + (dy.double().abs() * (exh + gn * xh.abs())).sum(0)
    bb = ref.rounding(db, wdtype) + gn * dy.double().abs().sum(0)
    return (dx, bx), (dw, bw), (db, bb)


@pytest.mark.parametrize("dtype,wdtype", [("f32", "f32"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f16")])
@pytest.mark.parametrize("N,D", SIZES)
def test_backward(N, D, dtype, wdtype):
    x, w, b, dy = case(N, D, dtype, wdtype, seed=1)
    got = ccv.layer_norm_bwd(x.cuda(), w.cuda(), dy.cuda(), b.cuda())
    assert ccv.ccv_last_kernel() == "ln_bwd"
    for name, a, (e, bound) in zip(("dx", "dweight", "dbias"), got, bwd_bounds(x, w, dy, dtype, wdtype)):
        assert ref.worst(a, e, bound) <= 1, name
    again = ccv.layer_norm_bwd(x.cuda(), w.cuda(), dy.cuda(), b.cuda())
    assert all(torch.equal(p, q) for p, q in zip(got, again))  # fixed order
    only = ccv.layer_norm_bwd(x.cuda(), None, dy.cuda())
    assert only[1] is None and only[2] is None
    (e, bound), _, _ = bwd_bounds(x, torch.ones(D, dtype=DT[wdtype]), dy, dtype, wdtype)
    assert ref.worst(only[0], e, bound) <= 1


def test_gradient_against_differences():
    x, w, b, dy = (t.cuda() for t in case(5, 24, "f32", "f32", seed=2, mean=0.5))
    dx, dw, db = ccv.layer_norm_bwd(x, w, dy, b)
    h = 2.0 ** -7
    f = lambda *a: float((ccv.layer_norm_fwd(*a).double() * dy.double()).sum())  # noqa: E731
    for i, j in ((0, 0), (2, 5), (4, 23)):
        e = torch.zeros_like(x)
        e[i, j] = h
        # central difference: h^2 of a third derivative of a few units, rounding 1e-5
        assert abs((f(x + e, w, b) - f(x - e, w, b)) / (2 * h) - float(dx[i, j])) < 5e-3
    e = torch.zeros_like(w)
    e[7] = h
    assert abs((f(x, w + e, b) - f(x, w - e, b)) / (2 * h) - float(dw[7])) < 2e-3  # linear in w and b
    assert abs((f(x, w, b + e) - f(x, w, b - e)) / (2 * h) - float(db[7])) < 2e-3


def test_views_and_leading_dimensions():
    x, w, b, dy = case(48, 128, "bf16", "f32", seed=3)
    y = ccv.layer_norm_fwd(x.cuda(), w.cuda(), b.cuda())
    x3 = x.cuda().view(4, 12, 128)
    assert torch.equal(ccv.layer_norm_fwd(x3, w.cuda(), b.cuda()).view(48, 128), y)
    wide = torch.zeros(48, 400, dtype=x.dtype, device="cuda")
    wide[:, 136:264] = x.cuda()          # aligned slice of a wider row
    assert torch.equal(ccv.layer_norm_fwd(wide[:, 136:264], w.cuda(), b.cuda()), y)
    wide.zero_()
    wide[:, 3:131] = x.cuda()            # unaligned slice
    y0, xh, r = ref.ln_fwd(x, w, b)
    bound = fwd_bound(x, w, y0, xh, r, "bf16") + 2.0 ** -23 * b.double().abs()
    assert ref.worst(ccv.layer_norm_fwd(wide[:, 3:131], w.cuda(), b.cuda()), y0, bound) <= 1
    t = x.cuda().t().contiguous().t()    # feature stride N
    w2 = torch.stack([w, w], 1).cuda()[:, 0]  # strided weight
    out = torch.empty_like(t)
    assert ref.worst(ccv.layer_norm_fwd(t, w2, b.cuda(), out=out), y0, bound) <= 1
    for a, (e, bd) in zip(ccv.layer_norm_bwd(t, w2, dy.cuda(), b.cuda()), bwd_bounds(x, w, dy, "bf16", "f32")):
        assert ref.worst(a, e, bd) <= 1


def test_constant_rows_large_means_and_no_rows():
    x = torch.full((3, 512), 7.0, device="cuda")
    w, b = torch.ones(512, device="cuda"), torch.full((512,), 0.5, device="cuda")
    assert torch.equal(ccv.layer_norm_fwd(x, w, b), torch.full_like(x, 0.5))
    big = torch.randn(4, 1024, dtype=torch.float64) + 3000
    y, xh, r = ref.ln_fwd(big.float(), None, None)
    got = ccv.layer_norm_fwd(big.float().cuda())
    assert ref.worst(got, y, fwd_bound(big.float(), None, y, xh, r, "f32")) <= 1
    e = torch.empty((0, 512), device="cuda")
    assert ccv.layer_norm_fwd(e, w, b).shape == (0, 512)
    dx, dw, db = ccv.layer_norm_bwd(e, w, e, b)
    assert dx.shape == (0, 512) and not dw.any() and not db.any()


def test_non_finite_rows_stay_in_their_rows():
    x, w, b, dy = (t.cuda() for t in case(20, 256, "f16", "f32", seed=4))
    y = ccv.layer_norm_fwd(x, w, b)
    dx = ccv.layer_norm_bwd(x, w, dy, b)[0]
    x2 = x.clone()
    x2[7, 3], x2[11, 0] = float("nan"), float("inf")
    good = [i for i in range(20) if i not in (7, 11)]
    y2 = ccv.layer_norm_fwd(x2, w, b)
    assert torch.equal(y2[good], y[good]) and bool(torch.isnan(y2[7]).all())
    assert torch.equal(ccv.layer_norm_bwd(x2, w, dy, b)[0][good], dx[good])


def test_other_stream():
    x, w, b, dy = (t.cuda() for t in case(300, 1024, "bf16", "bf16", seed=5))
    want = ccv.layer_norm_bwd(x, w, dy, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ccv.layer_norm_bwd(x, w, dy, b, stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
