"""The backward pass's kernels under bounds that stay below the gradients at any length."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU-only machines
    pytest.skip("needs a CUDA device", allow_module_level=True)

import causal_depthwise_conv1d_gb300 as ccv  # noqa: E402
from tests import gdr_bounds, mixer_ref as ref  # noqa: E402

NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dinitial_state")
SIZES = [  # (B, L, Hk, Hv, Dk, Dv), packed sequences, states
    ((1, 1, 1, 1, 128, 128), 0, False), ((2, 3, 1, 2, 64, 64), 0, True), ((1, 63, 2, 2, 128, 128), 0, True),
    ((1, 64, 1, 3, 128, 64), 0, False), ((2, 65, 2, 4, 64, 128), 0, False), ((1, 200, 1, 1, 128, 128), 0, False),
    ((1, 129, 2, 2, 72, 100), 0, False), ((1, 130, 1, 1, 1, 1), 0, False), ((1, 70, 1, 1, 33, 17), 0, True),
    ((1, 513, 1, 1, 128, 16), 0, False), ((1, 300, 1, 1, 64, 512), 0, True), ((2, 150, 1, 2, 128, 64), 4, True),
    ((1, 64, 1, 1, 64, 64), 64, True), ((1, 200, 2, 6, 64, 160), 3, True), ((2, 70, 8, 32, 64, 128), 2, True),
    ((1, 66, 40, 160, 64, 64), 2, True)]


def check(c, dtype):
    d = {n: None if x is None else x.cuda() for n, x in c.items()}
    got = dict(zip(NAMES, ccv.gated_delta_rule_bwd(
        d["q"], d["k"], d["v"], d["g"], d["beta"], d["dout"], seq_idx=d["seq_idx"], initial_state=d["initial_state"],
        dfinal_state=d["dfinal_state"], return_dinitial_state=True)))
    for n, (e, bound) in gdr_bounds.gdr_bwd(c).items():
        if n not in ("dg", "dinitial_state"):
            bound = bound + ref.rounding(e, dtype)
        assert ref.worst(got[n], e, bound) <= 1, n


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size,seqs,state", SIZES, ids=str)
def test_backward(size, seqs, state, dtype):
    check(ref.gdr_inputs(51, *size, dtype, seqs=seqs, state=state, grads=True), dtype)
