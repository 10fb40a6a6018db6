"""Tokens of very different size in one chunk, also as sequences of their own."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU-only machines
    pytest.skip("needs a CUDA device", allow_module_level=True)

import causal_depthwise_conv1d_gb300 as ccv  # noqa: E402
from tests import gdr_bounds, mixer_ref as ref  # noqa: E402
from tests.test_gpu_gdr_nonfinite import backward  # noqa: E402


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("packed", [False, True])
def test_v_and_dout_over_nine_decades(packed, dtype):
    """Tokens of 1, 2^-10, 2^-20 and 2^-30 by turns of 16; packed: a sequence each, the smallest first."""
    c = ref.gdr_inputs(81, 1, 100, 1, 2, 64, 64, dtype, grads=True)
    size = torch.arange(100).div(16, rounding_mode="floor").add(1).mul(-1).remainder(4).mul(-10).double().exp2()
    for n in ("v", "dout"):
        c[n] = (c[n].double() * size[None, :, None, None]).to(c[n].dtype)
    if packed:
        c["seq_idx"] = torch.arange(100).div(16, rounding_mode="floor").to(torch.int32)[None]
    d = {n: None if x is None else x.cuda() for n, x in c.items()}
    out, fin = ccv.gated_delta_rule_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], seq_idx=d["seq_idx"],
                                        return_final_state=True)
    o, s, eo, es = ref.gdr(c["q"], c["k"], c["v"], c["g"], c["beta"], c["seq_idx"])
    fo, fs = gdr_bounds.gdr_floor(c)
    assert ref.worst(out, o, eo + ref.rounding(o, dtype) + fo) <= 1
    assert ref.worst(fin, s, es + fs) <= 1
    got = backward(c)
    for n, (e, bound) in gdr_bounds.gdr_bwd(c, floor=True).items():
        if n != "dg":
            bound = bound + ref.rounding(e, dtype)
        assert ref.worst(got[n], e, bound) <= 1, n
    if packed:  # and the floor is of use: a sequence 2^-20 of its neighbours' size keeps more than its first seven bits
        e = o[:, 16:32]
        assert float(size[16]) == 2.0 ** -20
        assert float((out.cpu().double()[:, 16:32] - e).norm() / e.norm()) < 2.0 ** -7
