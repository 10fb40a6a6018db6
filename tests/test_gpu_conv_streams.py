"""The convolution's calls on a stream that is not the current one: where their memory comes from."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU-only machines
    pytest.skip("needs a CUDA device", allow_module_level=True)

import causal_depthwise_conv1d_gb300 as ccv  # noqa: E402
from tests.test_gpu_mixer_streams import tensors  # noqa: E402


def calls():
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, dout = (torch.randn((2, 512, 2048), generator=gen, device="cuda").bfloat16() for _ in range(2))
    w, b = torch.randn((512, 4), generator=gen, device="cuda").bfloat16(), torch.zeros(512, device="cuda").bfloat16()
    init = torch.randn((2, 512, 3), generator=gen, device="cuda").bfloat16()
    states = [init.clone() for _ in range(2)]  # a step advances its own
    return {
        "fwd": lambda **kw: ccv.causal_conv1d_fwd(x, w, b, activation="silu", initial_states=init,
                                                  return_final_states=True, **kw),
        "update": lambda **kw: ccv.causal_conv1d_update(x[..., :1], states.pop(), w, b, activation="silu", **kw),
        "bwd": lambda **kw: ccv.causal_conv1d_bwd(x, w, dout, b, activation="silu", initial_states=init,
                                                  return_dinitial_states=True, **kw)}


@pytest.mark.parametrize("name", ["fwd", "update", "bwd"])
def test_outputs_and_workspace_take_no_memory_of_the_current_stream(name):
    call = calls()[name]
    want = [t.clone() for t in tensors(call())]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    block = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    at = block.data_ptr()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
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
