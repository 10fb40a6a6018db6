"""SiLU and its derivative in group normalisation over their whole range, on every kernel.

With a weight of zero the activation's argument is the bias, whatever x is: out = silu(bias), dbias = sum of dout
silu'(bias).  Bounds: the exponent z log2(e) is rounded at a magnitude of up to 1.4427 |z| + 63 (the kernels shift it), so
e^-z is off by U (|z| + 44) and by |z| 1.4e-8 from the constant; exponential, reciprocal and products 4 H.  Where the
sigmoid is below 2^-86 the kernels let go of an absolute 2^-125 of it, in the derivative 2^-115."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU-only machines
    pytest.skip("needs a CUDA device", allow_module_level=True)

import causal_depthwise_conv1d_gb300 as ccv  # noqa: E402
from tests import rec_ref as ref  # noqa: E402

U, H = ref.U, ref.H

# rows of whole vectors; narrow groups; a cluster of one and of several blocks; slabs (unaligned, and many of them)
SHAPES = [(1, 1, 4096, 32), (3, 1, 4096, 8), (1, 1, 4095, 65), (1, 4, 4096, 16), (1, 1500, 4096, 32), (1, 3, 4095, 3),
          (1, 5000, 455, 5)]


def values(C):
    """From -130 to 130, denser around zero, and far beyond."""
    z = torch.linspace(-130, 130, C - 64, dtype=torch.float64)
    near = torch.linspace(-3, 3, 58, dtype=torch.float64)
    return torch.cat([z, near, torch.tensor([-1e4, -1e38, 1e4, 1e37, 0.0, -0.0], dtype=torch.float64)]).float()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,S,C,G", SHAPES)
def test_over_the_range(N, S, C, G, dtype):
    gen = torch.Generator().manual_seed(60)
    x = torch.randn((N, S, C), generator=gen).to(ref.DT[dtype])
    bias = values(C)
    dout = (torch.randint(0, 2, (N, S, C), generator=gen) * 2 - 1).to(ref.DT[dtype])
    w = torch.zeros(C)
    shaped = (lambda t: t[:, 0]) if S == 1 else (lambda t: t)
    z = bias.double()
    s, om = torch.sigmoid(z), torch.sigmoid(-z)
    rel = U * (z.abs() + 44) + 1.4e-8 * z.abs() + 4 * H
    y = torch.where(z < -700, 0.0, z * s)
    out = ccv.group_norm_fwd(shaped(x).cuda(), G, w.cuda(), bias.cuda(), activation="silu").view(N, S, C)
    want = y.expand(N, S, C)
    assert ref.worst(out, want, want.abs() * torch.where(z > 50, U, rel) + 2.0 ** -118 + ref.rounding(want, dtype)) <= 1
    size = s * (1 + z.abs() * om)
    act = torch.where(z < -700, 0.0, s * (1 + z * om))
    err = torch.where(z < -700, 0.0, size * (3 * rel + 4 * H)) + 2.0 ** -107
    _, _, db = ccv.group_norm_bwd(shaped(x).cuda(), G, w.cuda(), shaped(dout).cuda(), bias.cuda(), activation="silu")
    total = dout.double().sum((0, 1))
    assert ref.worst(db, total * act, N * S * err + (N * S + 64) * U * N * S * act.abs() + U * (total * act).abs()) <= 1
