"""The recurrence and group norm on other streams, at the same time, captured into graphs, and far into memory."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU-only machines
    pytest.skip("needs a CUDA device", allow_module_level=True)

import causal_depthwise_conv1d_gb300 as ccv  # noqa: E402
from tests import rec_ref as ref  # noqa: E402

ARGS = ("x", "decay_gate", "input_gate", "rate")
NAMES = ["rec_fwd", "rec_bwd", "rec_step", "gn_fwd", "gn_bwd", "gn_rows"]


def tensors(x):
    return [t for t in (x if isinstance(x, (tuple, list)) else (x,)) if t is not None]


def inputs(seed=1, B=2, L=1500, C=512, dtype="bf16"):
    return {n: None if t is None else t.cuda()
            for n, t in ref.glr_inputs(seed, B, L, C, dtype, seqs=3, state=True, grads=True).items()}


def calls(d):
    arg = [d[n] for n in ARGS]
    x, w = d["x"], torch.linspace(0.5, 1.5, d["x"].shape[-1], device="cuda")
    states = [d["initial_state"].clone() for _ in range(8)]  # a step advances its own
    return {
        "rec_fwd": lambda **kw: ccv.gated_linear_recurrence_fwd(*arg, seq_idx=d["seq_idx"],
                                                                initial_state=d["initial_state"],
                                                                return_final_state=True, return_chunk_states=True, **kw),
        "rec_bwd": lambda **kw: ccv.gated_linear_recurrence_bwd(*arg, d["dout"], seq_idx=d["seq_idx"],
                                                                initial_state=d["initial_state"],
                                                                dfinal_state=d["dfinal_state"],
                                                                return_dinitial_state=True, **kw),
        "rec_step": lambda **kw: ccv.gated_linear_recurrence_step(*(t[:, 0] for t in arg[:3]), arg[3], states.pop(), **kw),
        "gn_fwd": lambda **kw: ccv.group_norm_fwd(x, 4, w, w, activation="silu", **kw),
        "gn_bwd": lambda **kw: ccv.group_norm_bwd(x, 4, w, d["dout"], w, activation="silu", **kw),
        "gn_rows": lambda **kw: ccv.group_norm_bwd(x.flatten(0, 1), 4, w, d["dout"].flatten(0, 1), w, activation="silu",
                                                   **kw)}


@pytest.mark.parametrize("name", NAMES)
def test_outputs_and_workspace_take_no_memory_of_the_current_stream(name):
    """A block that the current stream has freed may be in use by kernels still queued there."""
    call = calls(inputs())[name]
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


@pytest.mark.parametrize("name", ["rec_fwd", "rec_bwd", "gn_bwd"])
def test_calls_at_the_same_time(name):
    """Several calls on streams of their own: blocks of one never wait for blocks that have not started."""
    sets = [inputs(seed, B=1 + seed % 3, L=900 + 400 * seed) for seed in range(4)]
    call = [calls(d)[name] for d in sets]
    want = [[t.clone() for t in tensors(c())] for c in call]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in call]
    for _ in range(5):
        got = [tensors(c(stream=s)) for c, s in zip(call, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert ccv.ccv_device_fault() == 0


@pytest.mark.parametrize("name", ["rec_fwd", "rec_bwd", "rec_step", "gn_fwd", "gn_bwd", "gn_rows"])
def test_captured_and_replayed_on_new_inputs(name):
    d = inputs(5)
    other = inputs(6)
    want = [t.clone() for t in tensors(calls(other)[name]())]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(d)[name]()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):  # two captures, each with memory of its own
        g = torch.cuda.CUDAGraph()
        call = calls(d)[name]
        with torch.cuda.graph(g):
            out = tensors(call())
        graphs.append((g, out))
    state = d["initial_state"].clone()
    for n in d:
        if d[n] is not None:
            d[n].copy_(other[n])
    for k in range(2):
        for g, out in graphs:
            if name == "rec_step" and k == 1:
                continue  # its state has advanced
            g.replay()
    torch.cuda.synchronize()
    del state
    for g, out in graphs:
        if name == "rec_step":
            # the captured state was cloned before the inputs changed: only the shape of the run is looked at
            assert all(bool(torch.isfinite(t.float()).all()) for t in out)
        else:
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_a_given_workspace_with_any_contents():
    d = inputs(7)
    want = calls(d)["rec_bwd"]()
    for fill in (0, 0xff, 0x7f):
        ws = torch.full((64 << 20,), fill, dtype=torch.uint8, device="cuda")
        got = calls(d)["rec_bwd"](workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(calls(d)["rec_fwd"](workspace=ws), calls(d)["rec_fwd"]()))
        assert all(torch.equal(a, b) for a, b in zip(calls(d)["gn_bwd"](workspace=ws), calls(d)["gn_bwd"]()))


def test_offsets_beyond_32_bits():
    """Rows more than 2^31 elements apart, and a state cache of more than 2^31 elements."""
    far = 2 ** 31 + 64
    base = torch.zeros(far + 400 * 64, dtype=torch.bfloat16, device="cuda")
    for L, C in ((300, 64), (300, 63)):
        c = ref.glr_inputs(8, 2, L, C, "bf16")
        d = {n: None if t is None else t.cuda() for n, t in c.items()}
        x = base.as_strided((2, L, C), (far, 64, 1))
        x.copy_(d["x"])
        out = ccv.gated_linear_recurrence_fwd(x, d["decay_gate"], d["input_gate"], d["rate"])
        assert torch.equal(out, ccv.gated_linear_recurrence_fwd(*(d[n] for n in ARGS)))
        y = ccv.group_norm_fwd(x, 1, activation="silu")
        assert torch.equal(y, ccv.group_norm_fwd(d["x"], 1, activation="silu"))
    del base, x
    slots = 2 ** 31 // 4096 + 8
    state = torch.zeros((slots, 4096), device="cuda")
    c = ref.glr_inputs(9, 2, 1, 4096, "bf16")
    d = {n: None if t is None else t.cuda() for n, t in c.items()}
    idx = torch.tensor([slots - 1, 3], dtype=torch.int32, device="cuda")
    out = ccv.gated_linear_recurrence_step(*(d[n] for n in ARGS), state, state_indices=idx)
    v, e = ref.glr(c)["out"]
    assert ref.worst(out, v, e + ref.rounding(v, "bf16")) <= 1
    v, e = ref.glr(c)["final_state"]
    assert ref.worst(state[idx.long()], v, e + 1e-30) <= 1 and not state[4:slots - 1].any()


def test_no_wait_ran_out():
    assert ccv.ccv_device_fault() == 0
