"""Calls on a stream that is not the current one: where their memory comes from."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU-only machines
    pytest.skip("needs a CUDA device", allow_module_level=True)

import causal_depthwise_conv1d_gb300 as ccv  # noqa: E402
from tests import mixer_ref as ref  # noqa: E402


def tensors(x):
    return [t for t in (x if isinstance(x, (tuple, list)) else (x,)) if t is not None]


def calls():
    c = {n: None if x is None else x.cuda() for n, x in
         ref.gdr_inputs(31, 4, 256, 4, 8, 64, 128, "bf16", state=True, grads=True).items()}
    arg = [c[n] for n in ("q", "k", "v", "g", "beta")]
    x, w = torch.randn((2048, 1024), device="cuda"), torch.ones(1024, device="cuda")
    states = [c["initial_state"].clone() for _ in range(2)]  # a step advances its own
    return {
        "fwd": lambda **kw: ccv.gated_delta_rule_fwd(*arg, initial_state=c["initial_state"], return_final_state=True,
                                                     **kw),
        "bwd": lambda **kw: ccv.gated_delta_rule_bwd(*arg, c["dout"], initial_state=c["initial_state"],
                                                     dfinal_state=c["dfinal_state"], return_dinitial_state=True, **kw),
        "step": lambda **kw: ccv.gated_delta_rule_step(*(t[:, 0] for t in arg), states.pop(), **kw),
        "ln_fwd": lambda **kw: ccv.layer_norm_fwd(x, w, w, **kw),
        "ln_bwd": lambda **kw: ccv.layer_norm_bwd(x, w, x, w, **kw)}


@pytest.mark.parametrize("name", ["fwd", "bwd", "step", "ln_fwd", "ln_bwd"])
def test_outputs_and_workspace_take_no_memory_of_the_current_stream(name):
    """A block that the current stream has freed may be in use by kernels still queued there."""
    call = calls()[name]
    want = [t.clone() for t in tensors(call())]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    block = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")  # one segment, free on the current stream
    at = block.data_ptr()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # what the call allocates stays in use while this looks
    del block
    got = tensors(call(stream=side))
    segments = torch.cuda.memory_snapshot()
    freed = [s for s in segments if s["address"] == at]
    assert len(freed) == 1 and freed[0]["active_size"] == 0
    for t in got:
        home = [s for s in segments if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]]
        assert len(home) == 1 and home[0]["stream"] == side.cuda_stream
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
