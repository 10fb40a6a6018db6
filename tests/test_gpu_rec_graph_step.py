"""The recurrence's decode step in a replayed graph: its cache is advanced in place, replay after replay."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU-only machines
    pytest.skip("needs a CUDA device", allow_module_level=True)

import causal_depthwise_conv1d_gb300 as ccv  # noqa: E402
from tests import rec_ref as ref  # noqa: E402

ARGS = ("x", "decay_gate", "input_gate", "rate")


def tokens(seed, B, S, C, dtype):
    return {n: t.cuda() for n, t in ref.glr_inputs(seed, B, S, C, dtype).items() if t is not None}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,S,C,slots", [(1, 1, 5120, 1), (6, 1, 61, 9), (300, 1, 512, 320), (5, 3, 64, 8)])
def test_replays_advance_the_state_as_calls_do(B, S, C, slots, dtype):
    gen = torch.Generator(device="cuda").manual_seed(40)
    d = tokens(41, B, S, C, dtype)
    idx = torch.randperm(slots, generator=gen, device="cuda")[:B].to(torch.int32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # once before the captures
        ccv.gated_linear_recurrence_step(*(d[n] for n in ARGS), torch.zeros((slots, C), device="cuda"), state_indices=idx)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):  # two captures, each with a cache of its own
        state, g = torch.zeros((slots, C), device="cuda"), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = ccv.gated_linear_recurrence_step(*(d[n] for n in ARGS), state, state_indices=idx)
        graphs.append((g, state, out))
    caches = [torch.randn((slots, C), generator=gen, device="cuda") for _ in graphs]
    for (_, state, _), cache in zip(graphs, caches):
        state.copy_(cache)
    for k in range(3):  # new tokens, and other requests' slots, each time
        new = tokens(50 + k, B, S, C, dtype)
        for n in ARGS:
            d[n].copy_(new[n])
        idx.copy_(torch.randperm(slots, generator=gen, device="cuda")[:B])
        for (g, state, out), cache in zip(graphs, caches):
            before = cache.clone()
            want = ccv.gated_linear_recurrence_step(*(new[n] for n in ARGS), cache, state_indices=idx)
            g.replay()
            assert torch.equal(out, want) and torch.equal(state, cache)
            rest = torch.ones(slots, dtype=torch.bool, device="cuda")
            rest[idx.long()] = False
            assert torch.equal(cache[rest], before[rest]) and not torch.equal(cache[~rest], before[~rest])
