"""Group normalisation's kernels against the FP64 formulas."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU-only machines
    pytest.skip("needs a CUDA device", allow_module_level=True)

import causal_depthwise_conv1d_gb300 as ccv  # noqa: E402
from tests import rec_ref as ref  # noqa: E402

SIZES = [(1, 1, 1, 1), (3, 1, 8, 2), (700, 1, 512, 4), (9, 1, 1000, 8), (5, 1, 640, 4), (33, 1, 4096, 2),
         (2, 7, 24, 3), (3, 77, 200, 8), (2, 300, 256, 4), (1, 1000, 320, 2), (1, 2000, 640, 1), (2, 65, 96, 96),
         (40, 3, 64, 1), (1, 5000, 16, 1), (2, 1, 5120, 1), (1, 3, 12000, 2), (1, 700, 2080, 1), (600, 2, 64, 8),
         # slabs of unaligned groups, narrow rows, groups beyond a cluster, clusters of sixteen, samples in turn
         (1, 3000, 21, 1), (2, 1500, 35, 5), (300, 1, 7, 1), (129, 1, 60, 12), (70, 1, 201, 3), (1, 9000, 512, 1),
         (1, 5000, 128, 1), (64, 40, 64, 8), (3, 1100, 384, 2)]
TYPES = [("f32", "f32", True), ("f16", "f32", False), ("bf16", "bf16", True), ("f16", "bf16", True)]


def tol(e, bound, dtype):
    return bound + ref.rounding(e, dtype) + 1e-30


def shaped(x):
    return x[:, 0] if x.shape[1] == 1 else x


@pytest.mark.parametrize("dtype,wdtype,silu", TYPES)
@pytest.mark.parametrize("N,S,C,G", SIZES)
def test_forward(N, S, C, G, dtype, wdtype, silu):
    x, w, b, _ = ref.gn_inputs(1, N, S, C, dtype, wdtype)
    act = "silu" if silu else None
    got = ccv.group_norm_fwd(shaped(x).cuda(), G, w.cuda(), b.cuda(), activation=act)
    assert ccv.ccv_last_kernel() == "gn_fwd" and got.shape == shaped(x).shape
    e, bound = ref.gn_fwd(x, G, w, b, silu=silu)
    assert ref.worst(got.view(N, S, C), e, tol(e, bound, dtype)) <= 1
    assert torch.equal(got, ccv.group_norm_fwd(shaped(x).cuda(), G, w.cuda(), b.cuda(), activation=act))
    e, bound = ref.gn_fwd(x, G, None, None, silu=silu)
    assert ref.worst(ccv.group_norm_fwd(x.cuda(), G, activation=act), e, tol(e, bound, dtype)) <= 1


@pytest.mark.parametrize("dtype,wdtype,silu", TYPES)
@pytest.mark.parametrize("N,S,C,G", SIZES)
def test_backward(N, S, C, G, dtype, wdtype, silu):
    x, w, b, dy = ref.gn_inputs(2, N, S, C, dtype, wdtype)
    act = "silu" if silu else None
    arg = (shaped(x).cuda(), G, w.cuda(), shaped(dy).cuda(), b.cuda())
    got = ccv.group_norm_bwd(*arg, activation=act)
    assert ccv.ccv_last_kernel() == "gn_bwd"
    want = ref.gn_bwd(x, G, w, dy, b, silu=silu)
    for n, t in zip(("dx", "dweight", "dbias"), got):
        e, bound = want[n]
        assert ref.worst(t.view(e.shape), e, tol(e, bound, dtype if n == "dx" else wdtype)) <= 1, n
    assert all(torch.equal(p, q) for p, q in zip(got, ccv.group_norm_bwd(*arg, activation=act)))  # fixed order
    only = ccv.group_norm_bwd(arg[0], G, None, arg[3], activation=act)
    assert only[1] is None and only[2] is None
    e, bound = ref.gn_bwd(x, G, None, dy, None, silu=silu)["dx"]
    assert ref.worst(only[0].view(N, S, C), e, tol(e, bound, dtype)) <= 1


def test_gradient_against_differences():
    x, w, b, dy = (t.cuda() for t in ref.gn_inputs(3, 2, 6, 12, "f32", "f32", mean=0.5))
    got = ccv.group_norm_bwd(x, 3, w, dy, b, activation="silu")
    f = lambda *a: float((ccv.group_norm_fwd(a[0], 3, a[1], a[2], activation="silu").double() * dy).sum())  # noqa: E731
    gen = torch.Generator(device="cuda").manual_seed(4)
    h = 2.0 ** -8
    for k, g in enumerate(got):
        way = torch.randn(g.shape, generator=gen, device="cuda")
        up, down = [x, w, b], [x, w, b]
        up[k], down[k] = up[k] + h * way, down[k] - h * way
        want = float((way.double() * g.double()).sum())
        # central: h^2 of third derivatives of a few units an element, rounding 1e-5 / h
        assert abs((f(*up) - f(*down)) / (2 * h) - want) < 2e-2


def test_views_and_inner_dimensions():
    x, w, b, dy = ref.gn_inputs(5, 3, 24, 64, "bf16", "f32")
    e, bound = ref.gn_fwd(x, 4, w, b, silu=True)
    grads = ref.gn_bwd(x, 4, w, dy, b, silu=True)
    arg = (4, w.cuda(), b.cuda())
    y = ccv.group_norm_fwd(x.cuda(), *arg, activation="silu")
    x4 = x.cuda().view(3, 4, 6, 64)
    assert torch.equal(ccv.group_norm_fwd(x4, *arg, activation="swish").view(y.shape), y)
    wide = torch.zeros((3, 24, 200), dtype=x.dtype, device="cuda")
    w2 = torch.stack([w, w], 1).cuda()[:, 0]  # strided weight
    for lo in (8, 3):  # a slice with aligned rows and one without
        wide.zero_()
        wide[..., lo:lo + 64] = x.cuda()
        out = torch.full_like(wide, 7.0)
        ccv.group_norm_fwd(wide[..., lo:lo + 64], 4, w2, b.cuda(), activation="silu", out=out[..., lo:lo + 64])
        assert ref.worst(out[..., lo:lo + 64], e, tol(e, bound, "bf16")) <= 1
        assert bool((out[..., :lo] == 7).all()) and bool((out[..., lo + 64:] == 7).all())
        dx = torch.full_like(wide, 7.0)
        got = ccv.group_norm_bwd(wide[..., lo:lo + 64], 4, w2, dy.cuda(), b.cuda(), activation="silu",
                                 dx=dx[..., lo:lo + 64])
        for n, t in zip(("dx", "dweight", "dbias"), got):
            v, bd = grads[n]
            assert ref.worst(t, v, tol(v, bd, "bf16" if n == "dx" else "f32")) <= 1, n
        assert bool((dx[..., :lo] == 7).all()) and bool((dx[..., lo + 64:] == 7).all())
    t = x.cuda().transpose(1, 2).contiguous().transpose(1, 2)  # positions innermost
    assert ref.worst(ccv.group_norm_fwd(t, *arg, activation="silu"), e, tol(e, bound, "bf16")) <= 1
    for n, g in zip(("dx", "dweight", "dbias"), ccv.group_norm_bwd(t, 4, w.cuda(), dy.cuda(), b.cuda(),
                                                                   activation="silu")):
        v, bd = grads[n]
        assert ref.worst(g, v, tol(v, bd, "bf16" if n == "dx" else "f32")) <= 1, n


def test_constant_groups_large_means_and_no_rows():
    for shape in ((4, 96), (2, 40, 96)):
        x = torch.full(shape, 7.0, device="cuda")
        w, b = torch.ones(96, device="cuda"), torch.full((96,), 0.5, device="cuda")
        assert torch.equal(ccv.group_norm_fwd(x, 3, w, b), torch.full_like(x, 0.5))
    for N, S in ((30, 1), (2, 500)):
        big = (torch.randn(N, S, 128, dtype=torch.float64) + 3000).float()
        e, bound = ref.gn_fwd(big, 2, None, None)
        assert ref.worst(ccv.group_norm_fwd(big.cuda(), 2), e, tol(e, bound, "f32")) <= 1
    w = torch.ones(64, device="cuda")
    for shape in ((0, 64), (0, 3, 64), (3, 0, 64)):
        e = torch.empty(shape, device="cuda")
        assert ccv.group_norm_fwd(e, 2, w, w).shape == shape
        dx, dw, db = ccv.group_norm_bwd(e, 2, w, e, w)
        assert dx.shape == shape and not dw.any() and not db.any()


@pytest.mark.parametrize("N,S,C,G", [(40, 1, 256, 4), (4, 90, 256, 4), (4, 90, 100, 4)])
def test_what_is_not_finite_stays_in_its_group(N, S, C, G):
    x, w, b, dy = (t.cuda() for t in ref.gn_inputs(6, N, S, C, "f16", "f32"))
    y, dx = ccv.group_norm_fwd(x, G, w, b, activation="silu"), ccv.group_norm_bwd(x, G, w, dy, b, activation="silu")[0]
    x2 = x.clone()
    cg = C // G
    x2[1, S // 2, cg + 1], x2[2, 0, 0] = float("nan"), float("inf")
    hit = torch.zeros(x.shape, dtype=torch.bool, device="cuda")
    hit[1, :, cg:2 * cg] = hit[2, :, :cg] = True
    y2 = ccv.group_norm_fwd(x2, G, w, b, activation="silu")
    assert torch.equal(y2[~hit], y[~hit]) and bool(torch.isnan(y2[1, :, cg:2 * cg]).all())
    assert torch.equal(ccv.group_norm_bwd(x2, G, w, dy, b, activation="silu")[0][~hit], dx[~hit])


def test_far_activations():
    """SiLU and its derivative deep in both tails."""
    x, _, _, dy = ref.gn_inputs(7, 6, 1, 256, "f32", "f32")
    w, b = torch.full((256,), 40.0), torch.linspace(-200, 200, 256)
    e, bound = ref.gn_fwd(x, 2, w, b, silu=True)
    got = ccv.group_norm_fwd(x[:, 0].cuda(), 2, w.cuda(), b.cuda(), activation="silu")
    assert ref.worst(got[:, None], e, tol(e, bound, "f32")) <= 1
    want = ref.gn_bwd(x, 2, w, dy, b, silu=True)
    for n, t in zip(("dx", "dweight", "dbias"),
                    ccv.group_norm_bwd(x[:, 0].cuda(), 2, w.cuda(), dy[:, 0].cuda(), b.cuda(), activation="silu")):
        v, bd = want[n]
        assert ref.worst(t.view(v.shape), v, tol(v, bd, "f32")) <= 1, n


def test_refusals():
    x, w = torch.randn((4, 6, 32), device="cuda"), torch.ones(32, device="cuda")
    for bad in (dict(groups=5), dict(groups=0), dict(groups=64)):
        with pytest.raises(ccv.CcvError, match="multiple of groups"):
            ccv.group_norm_fwd(x, weight=w, **bad)
    with pytest.raises(ValueError):
        ccv.group_norm_fwd(x, 4, activation="gelu")
    with pytest.raises(ValueError):
        ccv.group_norm_fwd(x, 4, w[:16])
    with pytest.raises(ValueError):
        ccv.group_norm_fwd(x[0, 0], 4)
    with pytest.raises(ValueError):
        ccv.group_norm_fwd(x, 4, w, w.half())
    with pytest.raises(ValueError):
        ccv.group_norm_bwd(x, 4, w, x[:, :3])
    with pytest.raises(ValueError, match="collapse"):
        ccv.group_norm_fwd(torch.randn((2, 4, 6, 32), device="cuda").transpose(1, 2), 4)
    with pytest.raises(ccv.CcvError, match="must not alias"):
        ccv.group_norm_fwd(x, 4, out=x)
    with pytest.raises(ccv.CcvError, match="eps"):
        ccv.group_norm_fwd(x, 4, eps=-1.0)
    with pytest.raises(ccv.CcvError, match="workspace too small"):
        ccv.group_norm_bwd(x, 4, w, x, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,S,C,G", [(30, 1, 256, 4), (30, 1, 100, 4), (2, 90, 256, 4), (2, 90, 100, 4)])
def test_activations_beyond_any_tail(N, S, C, G, dtype):
    """SiLU and its derivative where z is huge: nothing is left of either below, not a floor times z."""
    x, _, _, dy = (t.cuda() for t in ref.gn_inputs(8, N, S, C, dtype, "f32"))
    w, far = torch.ones(C, device="cuda"), torch.zeros(C, device="cuda")
    for k, z in enumerate((-150.0, -1e5, -1e20, -1e30, -3e38, 1e30)):
        far[k::9] = z
    y = ccv.group_norm_fwd(shaped(x), G, w, far, activation="silu").view(N, S, C)
    plain = ccv.group_norm_fwd(shaped(x), G, w, far).view(N, S, C)
    assert float(y[..., far < 0].abs().max()) < 1e-30
    # a sigmoid of one, by the hardware's functions (four of 2^-22), and two roundings to the type
    ratio = y[..., far > 1].double() / plain[..., far > 1].double()
    assert float((ratio - 1).abs().max()) <= 4 * 2.0 ** -22 + 1.01 * torch.finfo(y.dtype).eps
    _, dw, db = ccv.group_norm_bwd(shaped(x), G, w, shaped(dy), far, activation="silu")
    assert float(db[far < 0].abs().max()) < 1e-28 and float(dw[far < 0].abs().max()) < 1e-28
    # a derivative of one (five of 2^-22): the sum of N S values, each addition rounded
    total = dy.double().sum((0, 1))[far > 1]
    assert bool(((db[far > 1] - total).abs() <= (N * S + 24) * 2.0 ** -24 * dy.double().abs().sum((0, 1))[far > 1]).all())
    # a parameter that is not finite stays in its channel
    bad = far.clone()
    bad[C // 2] = float("nan")
    y2 = ccv.group_norm_fwd(shaped(x), G, w, bad, activation="silu").view(N, S, C)
    keep = torch.arange(C, device="cuda") != C // 2
    assert torch.equal(y2[..., keep], y[..., keep]) and bool(y2[..., ~keep].isnan().all())
    db2 = ccv.group_norm_bwd(shaped(x), G, w, shaped(dy), bad, activation="silu")[2]
    assert torch.equal(db2[keep], db[keep]) and bool(db2[~keep].isnan().all())


@pytest.mark.parametrize("N,S,C,G", [(3, 77, 1000, 8), (2, 150, 515, 1)])
def test_few_large_groups(N, S, C, G):
    """Groups of 9625 and 77250 elements in blocks of 1024 threads, fewer and more channels than a block has."""
    x, w, b, dy = ref.gn_inputs(9, N, S, C, "f32", "f32")
    e, bound = ref.gn_fwd(x, G, w, b, silu=True)
    assert ref.worst(ccv.group_norm_fwd(x.cuda(), G, w.cuda(), b.cuda(), activation="silu"), e, tol(e, bound, "f32")) <= 1
    want = ref.gn_bwd(x, G, w, dy, b, silu=True)
    got = ccv.group_norm_bwd(x.cuda(), G, w.cuda(), dy.cuda(), b.cuda(), activation="silu")
    for n, t in zip(("dx", "dweight", "dbias"), got):
        v, bd = want[n]
        assert ref.worst(t, v, tol(v, bd, "f32")) <= 1, n
