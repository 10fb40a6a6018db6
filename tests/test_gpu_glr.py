"""The gated linear recurrence's kernels against the FP64 definition."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU-only machines
    pytest.skip("needs a CUDA device", allow_module_level=True)

import causal_depthwise_conv1d_gb300 as ccv  # noqa: E402
from tests import rec_ref as ref  # noqa: E402

ARGS = ("x", "decay_gate", "input_gate", "rate")
SIZES = [(1, 1, 1), (1, 2, 3), (2, 63, 64), (1, 64, 72), (2, 65, 130), (3, 77, 101), (1, 300, 200), (2, 1001, 40),
         (1, 1500, 8), (5, 129, 64), (1, 256, 72), (2, 257, 72), (90, 150, 520)]
GRADS = ("dx", "ddecay_gate", "dinput_gate", "drate", "dinitial_state")


def dev(c):
    return {n: None if t is None else t.cuda() for n, t in c.items()}


def forward(d, **kw):
    return ccv.gated_linear_recurrence_fwd(*(d[n] for n in ARGS), seq_idx=d["seq_idx"],
                                           initial_state=d["initial_state"], **kw)


def backward(d, **kw):
    return ccv.gated_linear_recurrence_bwd(*(d[n] for n in ARGS), d["dout"], seq_idx=d["seq_idx"],
                                           initial_state=d["initial_state"], dfinal_state=d["dfinal_state"],
                                           return_dinitial_state=True, **kw)


def check_forward(c, got, dtype):
    want = ref.glr(c)
    for n, t in zip(("out", "final_state", "chunk_states"), got):
        v, e = want[n]
        assert ref.worst(t, v, e + (ref.rounding(v, dtype) if n == "out" else 1e-30)) <= 1, n


def check_backward(c, got, dtype):
    want = ref.glr_bwd(c)
    for n, t in zip(GRADS, got):
        if t is not None:
            v, e = want[n]
            assert ref.worst(t, v, e + (ref.rounding(v, dtype) if n[1:] in ARGS[:3] else 0) + 1e-30) <= 1, n


@pytest.mark.parametrize("seqs,state", [(0, False), (4, True)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,L,C", SIZES)
def test_forward(B, L, C, dtype, seqs, state):
    c = ref.glr_inputs(1, B, L, C, dtype, seqs=seqs, state=state)
    got = forward(dev(c), return_final_state=True, return_chunk_states=True)
    assert ccv.ccv_last_kernel() == "glr_fwd"
    check_forward(c, got, dtype)
    alone = forward(dev(c))
    assert torch.equal(alone, got[0])


@pytest.mark.parametrize("seqs,state", [(0, False), (4, True)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,L,C", SIZES)
def test_backward(B, L, C, dtype, seqs, state):
    c = ref.glr_inputs(2, B, L, C, dtype, seqs=seqs, state=state, grads=True)
    d = dev(c)
    got = backward(d)
    assert ccv.ccv_last_kernel() == "glr_bwd"
    assert (got[4] is None) == (not state)
    check_backward(c, got, dtype)
    states = forward(d, return_chunk_states=True)[1]
    kept = backward(d, chunk_states=states)
    again = backward(d, chunk_states=states)
    check_backward(c, kept, dtype)
    # fixed order: the states are the same ones, whoever has computed them
    for a, b, e in zip(got, kept, again):
        assert (a is None and b is None) or (torch.equal(a, b) and torch.equal(b, e))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,S,C", [(1, 1, 1), (1, 1, 5120), (3, 1, 77), (7, 5, 64), (130, 1, 264), (2, 70, 40)])
def test_step(B, S, C, dtype):
    c = ref.glr_inputs(3, B, S, C, dtype)
    d = dev(c)
    gen = torch.Generator().manual_seed(4)
    cache = torch.randn((B + 3, C), generator=gen)
    slots = torch.randperm(B + 3, generator=gen)[:B].to(torch.int32)
    state = cache.cuda()
    out = ccv.gated_linear_recurrence_step(*(d[n] for n in ARGS), state, state_indices=slots.cuda())
    assert ccv.ccv_last_kernel() == "glr_step"
    c["initial_state"] = cache[slots.long()]
    check_forward(c, (out, state[slots.long().cuda()]), dtype)
    rest = [i for i in range(B + 3) if i not in slots.tolist()]
    assert torch.equal(state[rest].cpu(), cache[rest])
    if S == 1:
        state2 = cache.cuda()
        one = ccv.gated_linear_recurrence_step(*(d[n][:, 0] for n in ARGS[:3]), d["rate"], state2,
                                               state_indices=slots.cuda())
        assert torch.equal(one, out[:, 0]) and torch.equal(state2, state)


def test_step_padding_rows_and_views():
    c = ref.glr_inputs(5, 6, 1, 40, "bf16")
    d = dev(c)
    base = torch.randn((9, 64), device="cuda")
    before = base.clone()
    state = base[1:8, 3:43]
    idx = torch.tensor([6, -1, 2, 7, 0, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    out = torch.full((6, 1, 50), 7.0, dtype=torch.bfloat16, device="cuda")
    ccv.gated_linear_recurrence_step(*(d[n] for n in ARGS), state, state_indices=idx, out=out[..., 5:45])
    used = [0, 2, 4]
    slots = idx[used].long()
    sub = {n: t[used] if n in ARGS[:3] else t for n, t in c.items()}
    sub["initial_state"] = before[1:8, 3:43][slots].cpu()
    check_forward(sub, (out[used][..., 5:45], state[slots]), "bf16")
    assert not out[[1, 3, 5]][..., 5:45].any()
    assert bool((out[..., :5] == 7).all()) and bool((out[..., 45:] == 7).all())
    base[slots + 1, 3:43] = before[slots + 1, 3:43]
    assert torch.equal(base, before)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_layouts(dtype):
    """Gates as slices of one projection, x and dout with time or batch innermost, unaligned slices, outputs in views."""
    B, L, C = 2, 200, 48
    c = ref.glr_inputs(6, B, L, C, dtype, seqs=3, state=True, grads=True)
    d = dev(c)
    both = torch.cat([d["decay_gate"], d["input_gate"]], -1)
    wide = torch.zeros((B, L, C + 5), dtype=both.dtype, device="cuda")
    wide[..., 3:3 + C] = d["decay_gate"]
    views = [dict(decay_gate=both[..., :C], input_gate=both[..., C:]),
             dict(x=d["x"].transpose(1, 2).contiguous().transpose(1, 2)),
             dict(x=d["x"].permute(1, 2, 0).contiguous().permute(2, 0, 1), dout=d["dout"].transpose(0, 1).contiguous().transpose(0, 1)),
             dict(decay_gate=wide[..., 3:3 + C]),
             dict(seq_idx=torch.stack([d["seq_idx"]] * 2, -1)[..., 1], rate=torch.stack([d["rate"]] * 3, 1)[:, 1],
                  initial_state=d["initial_state"].t().contiguous().t())]
    for v in views:
        e = dict(d, **v)
        out = torch.full((B, L, 2 * C + 3), 5.0, dtype=d["x"].dtype, device="cuda")
        res = forward(e, out=out[..., 1:1 + C], return_final_state=True, return_chunk_states=True)
        check_forward(c, res, dtype)
        assert bool((out[..., 0] == 5).all()) and bool((out[..., 1 + C:] == 5).all())
        grads = torch.full((B, L, 2 * C + 8), 5.0, dtype=d["x"].dtype, device="cuda")
        check_backward(c, backward(e, ddecay_gate=grads[..., :C], dinput_gate=grads[..., C:2 * C]), dtype)
        assert bool((grads[..., 2 * C:] == 5).all())


def test_chunks_of_a_sequence_equal_the_whole():
    c = dev(ref.glr_inputs(7, 2, 500, 96, "f32", state=True))
    whole, last = forward(c, return_final_state=True)
    state = c["initial_state"]
    for lo, hi in ((0, 1), (1, 130), (130, 131), (131, 500)):
        part = dict(c, x=c["x"][:, lo:hi], decay_gate=c["decay_gate"][:, lo:hi], input_gate=c["input_gate"][:, lo:hi],
                    initial_state=state)
        out, state = forward(part, return_final_state=True)
        assert float((out - whole[:, lo:hi]).abs().max()) < 1e-5 * 20  # two evaluations, each within its bound
    assert float((state - last).abs().max()) < 1e-5 * 20


def test_gradients_against_differences():
    c = ref.glr_inputs(8, 1, 90, 5, "f32", seqs=2, state=True, grads=True, rate=0.5)
    d = dev(c)
    got = dict(zip(GRADS, backward(d)))

    def loss(e):
        out, last = forward(e, return_final_state=True)
        return float((out.double() * d["dout"]).sum() + (last.double() * d["dfinal_state"]).sum())
    gen = torch.Generator(device="cuda").manual_seed(9)
    for n in ("x", "decay_gate", "input_gate", "rate", "initial_state"):
        way = torch.randn(d[n].shape, generator=gen, device="cuda")
        if n == "rate":
            way = way * d["rate"]  # relative: it stays positive
        h = 2.0 ** -9
        up, down = (loss(dict(d, **{n: d[n] + s * h * way})) for s in (1, -1))
        want = float((way.double() * got["d" + n].double()).sum())
        size = float((way.double() * got["d" + n].double()).square().sum().sqrt())
        # central: h^2 of third derivatives of order `size`; rounding of a loss of a few hundred terms 1e-5 / h
        assert abs((up - down) / (2 * h) - want) < 1e-2 * (1 + size), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_extreme_gates_and_rates(dtype):
    """Gates closed and open completely, rates of zero and of a thousand: the root and its derivative."""
    c = ref.glr_inputs(10, 1, 150, 64, dtype, grads=True, state=True)
    c["decay_gate"][:, :, :8] = -60.0    # 1 - a^2 of the order of e^-60
    c["decay_gate"][:, :, 8:16] = 60.0
    c["input_gate"][:, :, 16:24] = 60.0
    c["input_gate"][:, :, 24:32] = -60.0
    c["rate"][32:36] = 0.0
    c["rate"][36:40] = 1000.0
    c["rate"][40:44] = 1e-6
    c["decay_gate"][:, :, 44:48] = float("-inf")
    c["decay_gate"][:, :, 48:52] = float("inf")
    c["input_gate"][:, :, 52:56] = float("-inf")
    c["decay_gate"][:, ::2, 56:60] = -200.0
    d = dev(c)
    check_forward(c, forward(d, return_final_state=True), dtype)
    got = backward(d)
    want = ref.glr_bwd(c)
    for n, t in zip(GRADS, got):
        v, e = want[n]
        assert bool(torch.isfinite(t).all()), n
        assert ref.worst(t, v, e + (ref.rounding(v, dtype) if n[1:] in ARGS[:3] else 0) + 1e-15) <= 1, n


def test_what_is_not_finite_stays_in_its_sequence():
    c = ref.glr_inputs(11, 2, 260, 72, "bf16", state=True, grads=True)
    c["seq_idx"] = torch.zeros((2, 260), dtype=torch.int32)
    c["seq_idx"][:, 100:] = 1
    c["seq_idx"][:, 180:] = 2
    d = dev(c)
    clean, clean_grads = forward(d, return_final_state=True), backward(d)
    bad = {n: None if t is None else t.clone() for n, t in d.items()}
    bad["x"][0, 130, 5] = float("inf")
    bad["x"][1, 120, 7] = float("nan")
    bad["decay_gate"][0, 140, 9] = float("nan")
    bad["initial_state"][1, 11] = float("inf")
    out, last = forward(bad, return_final_state=True)
    touched = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
    touched[0, 130:180, 5] = touched[1, 120:180, 7] = touched[0, 140:180, 9] = True
    touched[1, :100, 11] = True
    assert torch.equal(out[~touched], clean[0][~touched]) and torch.equal(last, clean[1])
    assert bool(torch.isnan(out[1, 120:180, 7]).all()) and bool(torch.isnan(out[0, 140:180, 9]).all())
    assert bool(torch.isinf(out[0, 130, 5]))
    whole = torch.zeros_like(touched)
    whole[0, 100:180, [5, 9]] = whole[1, 100:180, 7] = True
    whole[1, :100, 11] = True
    for a, b in zip(backward(bad)[:3], clean_grads[:3]):
        assert torch.equal(a[~whole], b[~whole])
    # and a gradient that is not finite
    worse = dict(d, dout=d["dout"].clone())
    worse["dout"][0, 150, 3] = float("nan")
    whole.zero_()
    whole[0, 100:151, 3] = True
    for a, b in zip(backward(worse)[:3], clean_grads[:3]):
        assert torch.equal(a[~whole], b[~whole]) and bool(torch.isnan(a[0, 150, 3]))


def test_no_tokens():
    c = dev(ref.glr_inputs(12, 2, 3, 16, "f16", state=True, grads=True))
    for n in ("x", "decay_gate", "input_gate", "dout"):
        c[n] = c[n][:, :0]
    out, last, chunks = forward(c, return_final_state=True, return_chunk_states=True)
    assert out.shape == (2, 0, 16) and chunks.shape == (2, 0, 16) and torch.equal(last, c["initial_state"])
    got = backward(c)
    assert torch.equal(got[4], c["dfinal_state"]) and not got[3].any()
    e = dev(ref.glr_inputs(12, 0, 5, 16, "f16", grads=True))
    assert forward(e).shape == (0, 5, 16)
    assert not backward(e)[3].any()


def test_refusals():
    c = dev(ref.glr_inputs(13, 2, 10, 16, "f16", state=True, grads=True))
    for n, t in (("x", c["x"][0]), ("decay_gate", c["decay_gate"][:, 1:]), ("input_gate", c["input_gate"].float()),
                 ("rate", c["rate"].half()), ("rate", c["rate"][:8]), ("initial_state", c["initial_state"].half()),
                 ("rate", c["rate"].cpu())):
        with pytest.raises(ValueError):
            forward(dict(c, **{n: t}))
    with pytest.raises(ValueError):
        forward(dict(c, x=c["x"].double()))
    with pytest.raises(ccv.CcvError, match="must not alias"):
        forward(c, out=c["x"])
    with pytest.raises(ValueError):
        backward(c, chunk_states=torch.zeros((2, 2, 16), device="cuda"))
    with pytest.raises(ccv.CcvError, match="workspace too small"):
        backward(c, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ccv.CcvError, match="requires initial_state"):
        backward(dict(c, initial_state=None), dinitial_state=torch.empty((2, 16), device="cuda"))
    with pytest.raises(ccv.CcvError, match="n_slots"):
        ccv.gated_linear_recurrence_step(*(c[n][:, 0] for n in ARGS[:3]), c["rate"], torch.zeros((1, 16), device="cuda"))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_channels_that_end_inside_a_vector(dtype):
    """77 channels in rows of 80 on 16-byte boundaries: what lies beside them is neither used nor written."""
    B, L, C, W = 2, 333, 77, 80
    c = ref.glr_inputs(11, B, L, C, dtype, seqs=3, state=True, grads=True)
    d = dev(c)

    def padded(t, fill):
        w = torch.full((B, L + 9, W), fill, dtype=d["x"].dtype, device="cuda")
        if t is not None:
            w[:, :L, :C] = t
        return w

    e = dict(d, **{n: padded(d[n], float("nan"))[:, :L, :C] for n in (*ARGS[:3], "dout")})
    bufs = [padded(None, 5.0) for _ in range(4)]
    out, dx, dp, dq = (t[:, :L, :C] for t in bufs)
    check_forward(c, forward(e, out=out, return_final_state=True, return_chunk_states=True), dtype)
    check_backward(c, backward(e, dx=dx, ddecay_gate=dp, dinput_gate=dq), dtype)
    for t in bufs:
        assert bool((t[:, L:] == 5).all()) and bool((t[..., C:] == 5).all())
    # the same channels for every batch row: a stride of zero
    same = dict(d, decay_gate=e["decay_gate"][:1].expand(B, L, C), dout=e["dout"][:, :1].expand(B, L, C))
    c2 = dict(c, decay_gate=c["decay_gate"][:1].expand(B, L, C), dout=c["dout"][:, :1].expand(B, L, C))
    check_forward(c2, forward(same, return_final_state=True, return_chunk_states=True), dtype)
    check_backward(c2, backward(same), dtype)
