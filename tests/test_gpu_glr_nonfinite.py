"""The recurrence around gates, states and gradients that are not finite."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU-only machines
    pytest.skip("needs a CUDA device", allow_module_level=True)

import causal_depthwise_conv1d_gb300 as ccv  # noqa: E402
from tests import rec_ref as ref  # noqa: E402

ARGS = ("x", "decay_gate", "input_gate", "rate")


def dev(c):
    return {n: None if t is None else t.cuda() for n, t in c.items()}


def forward(d, **kw):
    return ccv.gated_linear_recurrence_fwd(*(d[n] for n in ARGS), seq_idx=d["seq_idx"],
                                           initial_state=d["initial_state"], **kw)


def backward(d, **kw):
    return ccv.gated_linear_recurrence_bwd(*(d[n] for n in ARGS), d["dout"], seq_idx=d["seq_idx"],
                                           initial_state=d["initial_state"], dfinal_state=d["dfinal_state"],
                                           return_dinitial_state=True, **kw)


# Rows of 64 channels take tensor copies, rows of 61 plain loads; 400 tokens are seven tiles along the time (a chain), 200
# four (one block), 60 a single one.  In 61 channels every one has its own place of the start inside a run of eight tokens
# and of the NaN behind it.
@pytest.mark.parametrize("dtype,C", [("bf16", 64), ("f32", 64), ("f16", 61), ("f32", 61)])
@pytest.mark.parametrize("L,start", [(400, 328), (400, 140), (200, 96), (60, 40)])
def test_a_gate_that_is_no_number_stays_in_its_sequence(L, start, dtype, C):
    for s in range(start, start + 8):
        c = ref.glr_inputs(20, 1, L, C, dtype, state=True, grads=True)
        c["seq_idx"] = (torch.arange(L)[None] >= s).to(torch.int32)
        clean = dev(c)
        want_out, want = forward(clean), backward(clean)
        bad = dict(clean, decay_gate=clean["decay_gate"].clone())
        ch = torch.arange(C, device="cuda")
        bad["decay_gate"][0, s + ch % 8, ch] = float("nan")
        out, got = forward(bad), backward(bad)
        assert torch.equal(out[:, :s], want_out[:, :s])
        at = s + ch % 8
        assert bool(torch.isnan(out[0, at, ch]).all())
        # the gradients of the sequence before, and the one that leaves at its first token
        for a, b, n in zip(got[:3], want[:3], ("dx", "ddecay_gate", "dinput_gate")):
            assert torch.equal(a[:, :s], b[:, :s]), (n, s)
        assert torch.equal(got[4], want[4]), s
