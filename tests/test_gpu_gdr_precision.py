"""How precise the gated delta rule's outputs are beyond the bounds of one FP32 evaluation."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU-only machines
    pytest.skip("needs a CUDA device", allow_module_level=True)

import causal_depthwise_conv1d_gb300 as ccv  # noqa: E402
from tests import mixer_ref as ref  # noqa: E402


def dev(c):
    return {n: None if x is None else x.cuda() for n, x in c.items()}


@pytest.mark.parametrize("size,state", [((1, 200, 1, 2, 128, 128), False), ((1, 256, 2, 2, 64, 64), True),
                                        ((2, 65, 2, 4, 64, 128), True), ((4, 64, 20, 40, 128, 128), False)], ids=str)
def test_bf16_outputs_are_the_exact_values_rounded_once(size, state):
    """An error before the rounding moves an output to another bf16 number where the exact value lies nearer than
    that to the middle of two.  Normal noise of 2^-16 of the outputs' rms moves 1.5 % of them, of 2^-18 0.5 %;
    operands in one term of 11 bits make errors of 2^-13 to 2^-12 and move 8 to 13 %."""
    c = ref.gdr_inputs(41, *size, "bf16", state=state)
    d = dev(c)
    out = ccv.gated_delta_rule_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], initial_state=d["initial_state"])
    assert ccv.ccv_last_kernel() == "gdr_chunk"
    o = ref.gdr(c["q"], c["k"], c["v"], c["g"], c["beta"], None, c["initial_state"])[0]
    moved = float((out.cpu() != o.to(torch.bfloat16)).double().mean())
    assert moved < 0.015, moved
