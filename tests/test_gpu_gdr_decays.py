"""Decays that forget everything: minus infinity, and very negative numbers in the place of it."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU-only machines
    pytest.skip("needs a CUDA device", allow_module_level=True)

import causal_depthwise_conv1d_gb300 as ccv  # noqa: E402
from tests import gdr_bounds, mixer_ref as ref  # noqa: E402
from tests.test_gpu_gdr_nonfinite import backward  # noqa: E402


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("low", [-1e9, -1e12, -1e30, torch.finfo(torch.float32).min, float("-inf")])
@pytest.mark.parametrize("at", [(30,), (7, 12, 13, 70), tuple(range(40, 64))], ids=str)
def test_forward_and_backward(at, low, dtype):
    c = ref.gdr_inputs(71, 1, 130, 1, 2, 64, 64, dtype, state=True, grads=True)
    for i, t in enumerate(at):
        c["g"][0, t] = low * (1 - 0.3 * (i % 2))
    d = {n: None if x is None else x.cuda() for n, x in c.items()}
    out, fin = ccv.gated_delta_rule_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"],
                                        initial_state=d["initial_state"], return_final_state=True)
    o, s, eo, es = ref.gdr(c["q"], c["k"], c["v"], c["g"], c["beta"], None, c["initial_state"])
    assert ref.worst(out, o, eo + ref.rounding(o, dtype)) <= 1
    assert ref.worst(fin, s, es) <= 1
    got = backward(c)
    for n, (e, bound) in gdr_bounds.gdr_bwd(c).items():
        if n not in ("dg", "dinitial_state"):
            bound = bound + ref.rounding(e, dtype)
        assert ref.worst(got[n], e, bound + 1e-30) <= 1, n
