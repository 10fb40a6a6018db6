"""The gated linear recurrence with rates on both sides of 0.85, where its decay changes from the polynomial to the
hardware's exponential, and up to those that keep a hundredth or less of a state a token."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU-only machines
    pytest.skip("needs a CUDA device", allow_module_level=True)

import causal_depthwise_conv1d_gb300 as ccv  # noqa: E402
from tests import rec_ref as ref  # noqa: E402

ARGS = ("x", "decay_gate", "input_gate", "rate")
GRADS = ("dx", "ddecay_gate", "dinput_gate", "drate", "dinitial_state")
U, H = ref.U, ref.H


@pytest.fixture
def tight(monkeypatch):
    """Bounds of the decay's own error: the hardware's exponential only where the logarithm is below -0.85.

    a there: the exponent's product and constant rounded (2 U |l|) and the exponential (2 H), together `far`.  m^2 =
    (1 - a)(1 + a) with a <= 0.43: the first factor's error is at most 0.75 far, the second's 0.3 far, so m's is at most
    0.53 far, taken as far.  Above -0.85 (less the rounding of l itself) nothing of that."""
    loose = ref._factors

    def factors(c):
        f = loose(c)
        far = (f["l"] < -0.85 * (1 - 1e-5)).double() * (2 * H + 2 * U * f["l"].abs())
        return dict(f, ea=f["l"].abs() * f["el"] + 4 * U + far, em=f["el"] + 8 * U + far + H)

    monkeypatch.setattr(ref, "_factors", factors)


def rates(kind, C, seed):
    gen = torch.Generator().manual_seed(seed)
    u = torch.rand(C, generator=gen, dtype=torch.float64)
    return {"at the switch": 0.80 + 0.15 * u,            # logarithms on both sides, warps of both codes
            "one to thirty": 10 ** (1.48 * u),           # decays mostly from the exponential
            "all": 10 ** (4.5 * u - 3)}[kind].float()    # 0.001 to 31, mixed inside a warp


def case(kind, B, L, C, dtype, spread, seqs, grads=False):
    c = ref.glr_inputs(30, B, L, C, dtype, seqs=seqs, state=True, grads=grads, spread=spread)
    c["rate"] = rates(kind, C, 31)
    return c, {n: None if t is None else t.cuda() for n, t in c.items()}


CASES = [(kind, *s) for kind in ("at the switch", "one to thirty", "all")
         for s in ((2, 300, 128, 2.0, 0), (1, 700, 61, 4.0, 3), (3, 50, 64, 3.0, 2))]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind,B,L,C,spread,seqs", CASES)
def test_forward(tight, kind, B, L, C, spread, seqs, dtype):
    c, d = case(kind, B, L, C, dtype, spread, seqs)
    got = ccv.gated_linear_recurrence_fwd(*(d[n] for n in ARGS), seq_idx=d["seq_idx"], initial_state=d["initial_state"],
                                          return_final_state=True, return_chunk_states=True)
    want = ref.glr(c)
    for n, t in zip(("out", "final_state", "chunk_states"), got):
        v, e = want[n]
        assert ref.worst(t, v, e + (ref.rounding(v, dtype) if n == "out" else 1e-30)) <= 1, n


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind,B,L,C,spread,seqs", CASES)
def test_backward(tight, kind, B, L, C, spread, seqs, dtype):
    c, d = case(kind, B, L, C, dtype, spread, seqs, grads=True)
    got = ccv.gated_linear_recurrence_bwd(*(d[n] for n in ARGS), d["dout"], seq_idx=d["seq_idx"],
                                          initial_state=d["initial_state"], dfinal_state=d["dfinal_state"],
                                          return_dinitial_state=True)
    want = ref.glr_bwd(c)
    for n, t in zip(GRADS, got):
        v, e = want[n]
        assert ref.worst(t, v, e + (ref.rounding(v, dtype) if n[1:] in ARGS[:3] else 0) + 1e-30) <= 1, n


# single channels a thread, and four
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,C", [(2, 61), (300, 512)])
@pytest.mark.parametrize("kind", ["at the switch", "one to thirty", "all"])
def test_step(tight, kind, B, C, dtype):
    c, d = case(kind, B, 3, C, dtype, 3.0, 0)
    state = d["initial_state"].clone()
    out = ccv.gated_linear_recurrence_step(*(d[n] for n in ARGS), state)
    want = ref.glr(c)
    v, e = want["out"]
    assert ref.worst(out, v, e + ref.rounding(v, dtype)) <= 1
    v, e = want["final_state"]
    assert ref.worst(state, v, e + 1e-30) <= 1
