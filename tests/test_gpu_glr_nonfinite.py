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


# Rate 1: decays of a run of tokens far above the smallest FP32 number.  8 and 30: a run's or a tile's product is below it.
# 1000: a single decay is.
@pytest.mark.parametrize("dtype,C", [("bf16", 64), ("f32", 64), ("f16", 61), ("f32", 61)])
@pytest.mark.parametrize("L,start", [(400, 333), (200, 131), (60, 43)])
def test_an_infinite_state_stays_infinite(L, start, dtype, C):
    """Decays are positive, so an infinite state keeps its sign until its sequence ends; the same for gradients."""
    c = ref.glr_inputs(21, 1, L, C, dtype, state=True, grads=True)
    c["rate"] = torch.tensor([1.0, 8.0, 30.0, 1000.0])[torch.arange(C) % 4]
    c["decay_gate"] = (c["decay_gate"].double() + 3).to(c["x"].dtype)
    c["seq_idx"] = (torch.arange(L)[None] >= start).to(torch.int32)
    clean = dev(c)
    want, want_last = forward(clean, return_final_state=True)
    inf = float("inf") * torch.where(torch.arange(C, device="cuda") % 3 == 0, -1.0, 1.0)
    # from the initial state, to the end of the first sequence
    out, last, chunks = forward(dict(clean, initial_state=inf[None]), return_final_state=True, return_chunk_states=True)
    assert torch.equal(out[0, :start].float(), inf.expand(start, C))
    assert torch.equal(out[:, start:], want[:, start:]) and torch.equal(last, want_last)
    n = start // 64 + 1
    assert torch.equal(chunks[0, :n], inf.expand(n, C)) and bool(torch.isfinite(chunks[0, n:]).all())
    # from one token of x to the end of the whole, where there is one sequence
    x = clean["x"].clone()
    x[0, 5] = inf.to(x.dtype)
    out, last = forward(dict(clean, x=x, seq_idx=None), return_final_state=True)
    assert torch.equal(out[0, 5:].float(), inf.expand(L - 5, C)) and torch.equal(last[0], inf)
    assert torch.equal(out[:, :5], want[:, :5])
    # and backwards, from the gradient of the final state to the start of the last sequence
    good = backward(clean)
    got = backward(dict(clean, dfinal_state=inf[None]))
    assert torch.equal(got[0][0, start:].float(), inf.expand(L - start, C))
    for a, b in zip(got[:3], good[:3]):
        assert torch.equal(a[:, :start], b[:, :start])
    assert torch.equal(got[4], good[4])
    got = backward(dict(clean, dfinal_state=inf[None], seq_idx=None))
    assert torch.equal(got[0][0].float(), inf.expand(L, C)) and torch.equal(got[4][0], inf)


@pytest.mark.parametrize("B,C", [(1, 64), (300, 512)])
def test_an_infinite_state_of_a_step(B, C):
    """Single channels and vectors of four."""
    c = ref.glr_inputs(22, B, 3, C, "bf16")
    c["rate"] = torch.tensor([1.0, 8.0, 30.0, 1000.0])[torch.arange(C) % 4]
    c["decay_gate"] = (c["decay_gate"].double() + 3).to(c["x"].dtype)
    d = dev(c)
    inf = float("inf") * torch.where(torch.arange(C, device="cuda") % 3 == 0, -1.0, 1.0)
    state = inf.expand(B, C).contiguous()
    out = ccv.gated_linear_recurrence_step(*(d[n] for n in ARGS), state)
    assert torch.equal(out.float(), inf.expand(B, 3, C)) and torch.equal(state, inf.expand(B, C))
