"""The gated delta rule's kernels against the FP64 definition."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU-only machines
    pytest.skip("needs a CUDA device", allow_module_level=True)

import causal_depthwise_conv1d_gb300 as ccv  # noqa: E402
from tests import mixer_ref as ref  # noqa: E402


def dev(c):
    return {n: None if x is None else x.cuda() for n, x in c.items()}


def check_fwd(c, dtype, d=None, **kw):
    d = dev(c) if d is None else d
    out, fin = ccv.gated_delta_rule_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], seq_idx=d["seq_idx"],
                                        initial_state=d["initial_state"], return_final_state=True, **kw)
    o, s, eo, es = ref.gdr(c["q"], c["k"], c["v"], c["g"], c["beta"], c["seq_idx"], c["initial_state"])
    assert ref.worst(fin, s, es) <= 1
    assert ref.worst(out, o, eo + out_bound(c, o, eo, dtype)) <= 1
    return out, fin


def out_bound(c, o, eo, dtype):
    # one rounding to the dtype; bf16 outputs may take their operands in 11
    # bits, at most half that rounding again on the terms' norms (eo / gamma)
    extra = 0.0
    if dtype == "bf16":
        extra = eo / ((c["q"].shape[3] + 64) * 2.0 ** -24) * 2.0 ** -11
    return ref.rounding(o, dtype) + extra


SIZES = [  # B, L, Hk, Hv, Dk, Dv
    (1, 1, 1, 1, 128, 128), (2, 3, 1, 2, 64, 64), (1, 63, 2, 2, 128, 128), (1, 64, 1, 3, 128, 64),
    (2, 65, 2, 4, 64, 128), (1, 200, 1, 1, 128, 128), (1, 129, 2, 2, 72, 100), (1, 97, 1, 2, 16, 8),
    (1, 130, 1, 1, 1, 1), (1, 70, 1, 1, 33, 17), (1, 90, 1, 2, 200, 48), (1, 513, 1, 1, 128, 16),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward(size, dtype):
    c = ref.gdr_inputs(hash(size) % 1000, *size, dtype)
    check_fwd(c, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size,seqs", [((2, 150, 1, 2, 128, 64), 4), ((1, 64, 1, 1, 64, 64), 64),
                                       ((1, 300, 2, 2, 128, 128), 3), ((3, 40, 1, 1, 64, 32), 2)], ids=str)
def test_packed_sequences_and_states(size, seqs, dtype):
    c = ref.gdr_inputs(5, *size, dtype, seqs=seqs, state=True)
    check_fwd(c, dtype)


MANY = [  # enough heads for every block shape of the scans, a last round of few heads among them
    (2, 70, 8, 32, 64, 128), (1, 66, 40, 160, 64, 64), (4, 66, 20, 40, 128, 128), (1, 66, 160, 160, 32, 128)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", MANY, ids=str)
def test_many_heads(size, dtype):
    check_fwd(ref.gdr_inputs(17, *size, dtype, seqs=2, state=True), dtype)


def test_a_sequence_that_begins_at_a_chunk_boundary():
    c = ref.gdr_inputs(6, 1, 200, 1, 1, 128, 64, "f32", state=True)
    ids = torch.zeros(1, 200, dtype=torch.int32)
    ids[:, 64:] = 7
    ids[:, 128:] = 3  # ids need not grow
    c["seq_idx"] = ids
    check_fwd(c, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_views(dtype):
    """Channel slices of one buffer, an odd offset, and a transposed layout."""
    B, L, Hk, Hv, Dk, Dv = 2, 100, 2, 2, 64, 64
    c = ref.gdr_inputs(7, B, L, Hk, Hv, Dk, Dv, dtype)
    buf = torch.cat([c[n].flatten(2) for n in ("q", "k", "v")], 2).cuda()
    n = Hk * Dk
    d = dev(c)
    d["q"], d["k"], d["v"] = (buf[..., i * n:(i + 1) * n].unflatten(-1, (Hk, Dk)) for i in range(3))
    a, fa = check_fwd(c, dtype, d)
    odd = torch.empty(buf.numel() + 1, dtype=buf.dtype, device="cuda")[1:].view(buf.shape)  # off by one element
    odd.copy_(buf)
    d["q"], d["k"], d["v"] = (odd[..., i * n:(i + 1) * n].unflatten(-1, (Hk, Dk)) for i in range(3))
    out = torch.empty((B, Hv, Dv, L), dtype=buf.dtype, device="cuda").permute(0, 3, 1, 2)
    b, fb = check_fwd(c, dtype, d, out=out)
    assert b is out
    assert torch.equal(a, b) and torch.equal(fa, fb)
    d["g"] = d["g"].transpose(1, 2).contiguous().transpose(1, 2)
    d["beta"] = d["beta"].transpose(0, 1).contiguous().transpose(0, 1)
    check_fwd(c, dtype, d)


def test_empty():
    c = dev(ref.gdr_inputs(8, 2, 0, 1, 2, 64, 32, "bf16", state=True))
    out, fin = ccv.gated_delta_rule_fwd(c["q"], c["k"], c["v"], c["g"], c["beta"], initial_state=c["initial_state"],
                                        return_final_state=True)
    assert out.shape == (2, 0, 2, 32) and torch.equal(fin, c["initial_state"])
    fin = ccv.gated_delta_rule_fwd(c["q"], c["k"], c["v"], c["g"], c["beta"], return_final_state=True)[1]
    assert not fin.any()
    e = dev(ref.gdr_inputs(8, 0, 5, 1, 2, 64, 32, "bf16"))
    assert ccv.gated_delta_rule_fwd(e["q"], e["k"], e["v"], e["g"], e["beta"]).shape == (0, 5, 2, 32)


@pytest.mark.parametrize("L", [20, 150])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("what", ["q", "k", "v", "g", "beta", "inf", "-inf g", "state"])
def test_non_finite_values_stay_where_the_definition_puts_them(what, dtype, L):
    """Nothing before their token and nothing in the next sequence."""
    c = ref.gdr_inputs(9, 1, L, 1, 2, 64, 32, dtype, state=True)
    at, nxt = L // 2 + 1, L - 6
    ids = torch.zeros(1, L, dtype=torch.int32)
    ids[:, nxt:] = 1
    c["seq_idx"] = ids
    if what == "state":
        c["initial_state"][0, 0, 3, 5] = float("inf")
        at = 0
    elif what == "inf":
        c["v"][0, at, 0, 3] = float("inf")
    elif what == "-inf g":
        c["g"][0, at] = float("-inf")  # forgets everything: finite
    else:
        c[what][0, at, 0] = float("nan")
    clean = ref.gdr_inputs(9, 1, L, 1, 2, 64, 32, dtype, state=True)
    o, s, eo, es = ref.gdr(c["q"], c["k"], c["v"], c["g"], c["beta"], ids, c["initial_state"])
    d = dev(c)
    out, fin = ccv.gated_delta_rule_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], seq_idx=d["seq_idx"],
                                        initial_state=d["initial_state"], return_final_state=True)
    fine = torch.isfinite(o) & torch.isfinite(eo)
    got = out.cpu().double()
    assert bool(torch.isfinite(got)[fine].all())
    err = (got - o).abs()
    assert bool((err[fine] <= (eo + out_bound(clean, o, eo, dtype))[fine]).all())
    assert bool((~torch.isfinite(got[~torch.isfinite(o)])).all())
    assert bool(fine[:, :at].all()) or what == "state"
    assert bool(fine[:, nxt:].all()) and bool(torch.isfinite(fin).all())
    assert ref.worst(fin, s, es) <= 1


def test_large_and_small_magnitudes():
    """Rows of very different scale; values outside FP16's range."""
    c = ref.gdr_inputs(10, 1, 150, 1, 1, 64, 32, "bf16")
    c["v"] = (c["v"].float() * torch.logspace(-20, 20, 32)).to(torch.bfloat16)
    c["k"][:, 40:80] = (c["k"][:, 40:80].float() * 1e-12).to(torch.bfloat16)
    c["q"] = (c["q"].float() * 1e9).to(torch.bfloat16)
    check_fwd(c, "bf16")
    z = ref.gdr_inputs(11, 1, 150, 1, 1, 64, 32, "f16")
    z["k"][:, 10:90] = 0
    z["beta"][:, 100:120] = 0
    z["g"][:, 30] = -200.0  # exp underflows
    z["g"][:, 90:] = 0.0    # no decay
    check_fwd(z, "f16")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("S", [1, 2, 9])
@pytest.mark.parametrize("B,slots,size", [(1, 1, (2, 4, 128, 128)), (5, 8, (2, 2, 64, 128)), (3, 3, (1, 2, 72, 100)),
                                          (2, 4, (1, 1, 24, 7)), (2, 2, (1, 1, 256, 16)),
                                          (170, 200, (2, 4, 128, 128))], ids=str)
def test_step(B, slots, size, S, dtype):
    if B > 100 and S == 9:
        S = 3
    Hk, Hv, Dk, Dv = size
    c = ref.gdr_inputs(12, B, S, Hk, Hv, Dk, Dv, dtype)
    gen = torch.Generator().manual_seed(3)
    state = torch.randn((slots, Hv, Dk, Dv), generator=gen)
    idx = torch.randperm(slots, generator=gen)[:B].to(torch.int32)
    o, s, eo, es = ref.gdr(c["q"], c["k"], c["v"], c["g"], c["beta"], None, state[idx.long()])
    d, st = dev(c), state.cuda()
    out = ccv.gated_delta_rule_step(d["q"], d["k"], d["v"], d["g"], d["beta"], st, state_indices=idx.cuda())
    assert ccv.ccv_last_kernel() == "gdr_step"
    assert ref.worst(out, o, eo + ref.rounding(o, dtype)) <= 1
    assert ref.worst(st[idx.long().cuda()], s, es) <= 1
    rest = torch.ones(slots, dtype=torch.bool)
    rest[idx.long()] = False
    assert torch.equal(st.cpu()[rest], state[rest])  # other slots untouched


def test_step_one_token_padding_rows_and_views():
    c = dev(ref.gdr_inputs(13, 4, 1, 1, 2, 64, 32, "bf16"))
    base = torch.randn((3, 2, 64, 40), device="cuda")
    state = base[..., 4:36]  # a view
    want = state.clone()
    idx = torch.tensor([2, -1, 0, 3], dtype=torch.int32, device="cuda")
    one = {n: c[n][:, 0] for n in ("q", "k", "v", "g", "beta")}
    out = ccv.gated_delta_rule_step(*(one[n] for n in ("q", "k", "v", "g", "beta")), state, state_indices=idx)
    assert out.shape == (4, 2, 32)
    assert not out[1].any() and not out[3].any()
    assert torch.equal(state[1], want[1])
    ok = [0, 2]
    w = want[[2, 0]].contiguous()
    o2 = ccv.gated_delta_rule_step(*(one[n][ok] for n in ("q", "k", "v", "g", "beta")), w)
    assert torch.equal(o2, out[ok]) and torch.equal(w, state[[2, 0]])
    edge = base.clone()
    edge[..., 4:36] = 0
    assert torch.equal(edge[..., :4], base[..., :4]) and torch.equal(edge[..., 36:], base[..., 36:])


def test_steps_continue_a_forward_pass():
    c = ref.gdr_inputs(14, 2, 90, 1, 2, 64, 64, "f32")
    d = dev(c)
    arg = ("q", "k", "v", "g", "beta")
    _, st = ccv.gated_delta_rule_fwd(*(d[n][:, :80] for n in arg), return_final_state=True)
    out = torch.cat([ccv.gated_delta_rule_step(*(d[n][:, t:t + 1] for n in arg), st) for t in range(80, 90)], 1)
    o, s, eo, es = ref.gdr(*(c[n] for n in arg))
    assert ref.worst(out, o[:, 80:], (eo + ref.rounding(o, "f32"))[:, 80:]) <= 1
    assert ref.worst(st, s, es) <= 1


def test_other_stream_and_graph_capture():
    c = dev(ref.gdr_inputs(15, 2, 150, 1, 2, 64, 64, "bf16"))
    arg = [c[n] for n in ("q", "k", "v", "g", "beta")]
    want = ccv.gated_delta_rule_fwd(*arg)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ccv.gated_delta_rule_fwd(*arg, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    n = ccv.ccv_gdr_fwd_workspace_size(2, 150, 1, 2, 64, 64, 2)
    ws, out = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda"), torch.zeros_like(want)
    ccv.gated_delta_rule_fwd(*arg, out=out, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        ccv.gated_delta_rule_fwd(*arg, out=out, workspace=ws)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_back_to_back_calls_keep_stream_order():
    """Each call reads what the one before it wrote."""
    c = dev(ref.gdr_inputs(16, 1, 150, 1, 1, 64, 64, "bf16"))
    k, g, beta = c["k"], c["g"], c["beta"]

    def chain(sync):
        v, outs = c["v"], []
        st = torch.zeros((1, 1, 64, 64), device="cuda")
        for _ in range(6):
            v, st = ccv.gated_delta_rule_fwd(c["q"], k, v, g, beta, initial_state=st, return_final_state=True)
            if sync:
                torch.cuda.synchronize()
            outs.append(v)
        return torch.cat(outs), st

    (a, sa), (b, sb) = chain(False), chain(True)
    assert torch.equal(a, b) and torch.equal(sa, sb)


NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dinitial_state")


def run_bwd(d, **kw):
    return dict(zip(NAMES, ccv.gated_delta_rule_bwd(
        d["q"], d["k"], d["v"], d["g"], d["beta"], d["dout"], seq_idx=d["seq_idx"], initial_state=d["initial_state"],
        dfinal_state=d["dfinal_state"], return_dinitial_state=True, **kw)))


def check_bwd(c, dtype, d=None, **kw):
    got = run_bwd(dev(c) if d is None else d, **kw)
    assert ccv.ccv_last_kernel() == "gdr_bwd"
    want = ref.gdr_bwd(c)
    assert (got["dinitial_state"] is None) == (c["initial_state"] is None)
    for n, (e, bound) in want.items():
        if n not in ("dg", "dinitial_state"):
            bound = bound + ref.rounding(e, dtype)
        assert ref.worst(got[n], e, bound) <= 1, n
    return got


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", [s for s in SIZES if s[4] <= 128], ids=str)
def test_backward(size, dtype):
    check_bwd(ref.gdr_inputs(21, *size, dtype, grads=True), dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size,seqs", [((2, 150, 1, 2, 128, 64), 4), ((1, 64, 1, 1, 64, 64), 64),
                                       ((1, 200, 2, 6, 64, 160), 3), ((3, 40, 1, 1, 64, 32), 2)], ids=str)
def test_backward_of_packed_sequences_and_states(size, seqs, dtype):
    c = ref.gdr_inputs(22, *size, dtype, seqs=seqs, state=True, grads=True)
    got = check_bwd(c, dtype)
    again = run_bwd(dev(c))
    assert all(torch.equal(got[n], again[n]) for n in NAMES)  # fixed order
    first = torch.zeros_like(c["seq_idx"], dtype=torch.bool)
    first[:, 1:] = c["seq_idx"][:, 1:] != c["seq_idx"][:, :-1]
    assert not got["dg"].cpu()[first].any()  # nothing decays into a new sequence


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", MANY, ids=str)
def test_backward_many_heads(size, dtype):
    check_bwd(ref.gdr_inputs(29, *size, dtype, seqs=2, state=True, grads=True), dtype)


def test_backward_against_differences_of_the_forward():
    """f32: directional derivatives of the forward kernel itself."""
    c = ref.gdr_inputs(23, 1, 130, 1, 2, 64, 64, "f32", seqs=2, state=True, grads=True)
    d = dev(c)
    got = run_bwd(d)

    def loss(n, delta):
        x = dict(d)
        x[n] = d[n] + delta
        o, s = ccv.gated_delta_rule_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], seq_idx=x["seq_idx"],
                                        initial_state=x["initial_state"], return_final_state=True)
        return float((o.double() * d["dout"].double()).sum() + (s.double() * d["dfinal_state"].double()).sum())

    gen = torch.Generator(device="cuda").manual_seed(6)
    for n in ("q", "k", "v", "g", "beta", "initial_state"):
        way = torch.randn(d[n].shape, generator=gen, device="cuda") * d[n].abs().mean()
        want = float((way.double() * got["d" + n].double()).sum())
        size = float((way.double() * got["d" + n].double()).abs().sum())
        h = 2.0 ** -8
        # the third derivative's share is of order h^2, the outputs' roundings of order 2^-22 / h
        assert abs((loss(n, h * way) - loss(n, -h * way)) / (2 * h) - want) < 2e-3 * size, n


def test_backward_views_and_outputs():
    """Gradients written into channel slices of one buffer; strided inputs."""
    B, L, Hk, Hv, Dk, Dv = 2, 100, 2, 2, 64, 64
    c = ref.gdr_inputs(24, B, L, Hk, Hv, Dk, Dv, "bf16", grads=True)
    d = dev(c)
    plain = check_bwd(c, "bf16", d)
    n = Hk * Dk
    for off in (0, 1):  # aligned slices, and slices off by one element
        buf = torch.zeros(B * L * 3 * n + off, dtype=torch.bfloat16, device="cuda")[off:].view(B, L, 3 * n)
        x = torch.cat([d[m].flatten(2) for m in ("q", "k", "v")], 2)
        src = torch.empty(x.numel() + off, dtype=x.dtype, device="cuda")[off:].view(x.shape)
        src.copy_(x)
        e = dict(d)
        e["q"], e["k"], e["v"] = (src[..., i * n:(i + 1) * n].unflatten(-1, (Hk, Dk)) for i in range(3))
        e["dout"] = d["dout"].transpose(1, 2).contiguous().transpose(1, 2)
        dq, dk, dv = (buf[..., i * n:(i + 1) * n].unflatten(-1, (Hk, Dk)) for i in range(3))
        got = run_bwd(e, dq=dq, dk=dk, dv=dv)
        assert all(torch.equal(got[m], plain[m]) for m in ("dq", "dk", "dv", "dg", "dbeta"))


def test_backward_empty():
    d = dev(ref.gdr_inputs(25, 2, 0, 1, 2, 64, 32, "bf16", state=True, grads=True))
    got = run_bwd(d)
    assert got["dq"].shape == (2, 0, 1, 64) and torch.equal(got["dinitial_state"], d["dfinal_state"])
    e = dev(ref.gdr_inputs(25, 0, 5, 1, 2, 64, 32, "bf16", grads=True))
    assert run_bwd(e)["dv"].shape == (0, 5, 2, 32)


def test_backward_magnitudes():
    """Rows of q and k of very different length keep gradients of full precision; zero rows too."""
    c = ref.gdr_inputs(26, 1, 100, 1, 2, 64, 64, "bf16", grads=True)
    c["k"][:, 5:9] = (c["k"][:, 5:9].float() * 1e-12).to(torch.bfloat16)
    c["q"][:, 20:30] = (c["q"][:, 20:30].float() * 1e-12).to(torch.bfloat16)
    c["k"][:, 40] = 0
    c["q"][:, 41] = 0
    c["beta"][:, 50:60] = 0
    c["g"][:, 70] = -300.0
    check_bwd(c, "bf16")


def test_backward_non_finite_sequences_leave_others_alone():
    c = ref.gdr_inputs(27, 1, 256, 1, 2, 64, 32, "bf16", state=True, grads=True)
    ids = torch.zeros(1, 256, dtype=torch.int32)
    ids[:, 64:] = 1
    ids[:, 192:] = 2
    c["seq_idx"] = ids
    clean = ref.gdr_bwd(c)
    for n in ("q", "k", "v", "g", "beta", "dout"):
        d = dev(c)
        d[n][0, 100, 0] = float("nan")  # in the second sequence, chunks 1 and 2
        got = run_bwd(d)
        for m in ("dq", "dk", "dv", "dg", "dbeta"):
            e, bound = clean[m]
            if m != "dg":
                bound = bound + ref.rounding(e, "bf16")
            for part in (slice(0, 64), slice(192, 256)):
                assert ref.worst(got[m][:, part], e[:, part], bound[:, part]) <= 1, (n, m)


def test_backward_other_stream_and_workspace():
    d = dev(ref.gdr_inputs(28, 1, 150, 1, 2, 64, 64, "f16", state=True, grads=True))
    want = run_bwd(d)
    ws = torch.full((ccv.ccv_gdr_bwd_workspace_size(1, 150, 1, 2, 64, 64, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run_bwd(d, workspace=ws, stream=side)
    side.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in NAMES)
    with pytest.raises(ccv.CcvError, match="workspace too small"):
        run_bwd(d, workspace=ws[:-256])
