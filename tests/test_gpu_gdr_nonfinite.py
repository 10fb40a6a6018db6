"""Gradients beside values that are not finite: where one is finite it is right, where the definition's is not it is
not, and what such a value cannot reach by the definition stays exact in other sequences of the same chunk."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU-only machines
    pytest.skip("needs a CUDA device", allow_module_level=True)

import causal_depthwise_conv1d_gb300 as ccv  # noqa: E402
from tests import gdr_bounds, mixer_ref as ref  # noqa: E402

NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dinitial_state")


def backward(c):
    d = {n: None if x is None else x.cuda() for n, x in c.items()}
    return dict(zip(NAMES, ccv.gated_delta_rule_bwd(
        d["q"], d["k"], d["v"], d["g"], d["beta"], d["dout"], seq_idx=d["seq_idx"], initial_state=d["initial_state"],
        dfinal_state=d["dfinal_state"], return_dinitial_state=True)))


def case(dtype, L, Dv=32):
    c = ref.gdr_inputs(61, 1, L, 1, 2, 64, Dv, dtype, state=True, grads=True)
    ids = torch.zeros((1, L), dtype=torch.int32)
    ids[:, 20:] = 1
    ids[:, 44:] = 2
    c["seq_idx"] = ids
    return c


@pytest.mark.parametrize("value", ["nan", "inf"])
@pytest.mark.parametrize("what", ["dout", "v", "beta", "q", "k", "g", "initial_state", "dfinal_state"])
@pytest.mark.parametrize("dtype,L,Dv", [("f32", 150, 32), ("f16", 64, 64), ("bf16", 150, 160)])
def test_non_finite_values(dtype, L, Dv, what, value):
    c = case(dtype, L, Dv)
    bad = float(value)
    if what in ("initial_state", "dfinal_state"):
        c[what][0, 0, 3, 5] = bad
    elif what in ("beta", "g"):
        c[what][0, 30, 0] = bad
    else:
        c[what][0, 30, 0, 7] = bad
    got = backward(c)
    want = gdr_bounds.gdr_bwd(c)
    for n, (e, bound) in want.items():
        if n not in ("dg", "dinitial_state"):
            bound = bound + ref.rounding(e, dtype)
        g, bound = got[n].double().cpu(), bound.expand_as(e)
        known = torch.isfinite(e) & torch.isfinite(bound)
        at = known & torch.isfinite(g)
        assert bool(((g - e).abs() <= bound)[at].all()), n
        assert not bool(torch.isfinite(g)[~torch.isfinite(e)].any()), n
        if n == "dinitial_state":
            continue
        if what in ("dout", "v", "beta", "q", "k"):  # the other sequences of the chunk
            assert bool(torch.isfinite(g[:, :20]).all()) and bool(torch.isfinite(g[:, 44:]).all()), n
        if what == "dout" or (what == "v" and n != "dg"):  # and the tokens that the definition leaves alone
            assert bool((torch.isfinite(g) == torch.isfinite(e)).all()), n


@pytest.mark.parametrize("what", ["dout", "v", "k"])
@pytest.mark.parametrize("heads,L", [((40, 160), 66), ((16, 64), 70)])  # four and eight groups of channels a block
def test_many_heads(heads, L, what):
    c = ref.gdr_inputs(62, 1, L, *heads, 64, 64, "bf16", state=True, grads=True)
    ids = torch.zeros((1, L), dtype=torch.int32)
    ids[:, 20:] = 1
    ids[:, 44:] = 2
    c["seq_idx"] = ids
    c[what][0, 30, 3, 7] = float("nan")
    got = backward(c)
    for n, (e, bound) in gdr_bounds.gdr_bwd(c).items():
        if n not in ("dg", "dinitial_state"):
            bound = bound + ref.rounding(e, "bf16")
        g, bound = got[n].double().cpu(), bound.expand_as(e)
        at = torch.isfinite(e) & torch.isfinite(bound) & torch.isfinite(g)
        assert bool(((g - e).abs() <= bound)[at].all()), n
        assert not bool(torch.isfinite(g)[~torch.isfinite(e)].any()), n
        if n != "dinitial_state":
            assert bool(torch.isfinite(g[:, :20]).all()) and bool(torch.isfinite(g[:, 44:]).all()), n
            assert bool(torch.isfinite(g[:, :, -1]).all()), n  # a head without one
