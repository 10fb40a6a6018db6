"""Refusals of the recurrence's and group norm's entry points, on the host:
nothing is launched and no GPU is needed."""
import ctypes

import pytest

from tests.test_mixer_abi import mx, status  # noqa: F401

F = 1 << 24  # fake addresses far apart, never dereferenced
B, L, C = 2, 130, 48
ROW, ST = (L * C, C, 1), (C, 1)


def tensors(mx, a, names):
    out = []
    for n in names:
        out += [a[n], a["s_" + n] if n in ("rate", "drate", "idx") else mx._arr(a["s_" + n])]
    return out


def glr_args(mx, kind, **kw):
    a = dict(x=F, p=2 * F, q=3 * F, rate=4 * F, seq=None, s0=None, out=5 * F, s1=None, cs=None, dout=6 * F, ds1=None,
             dx=7 * F, dp=8 * F, dq=9 * F, drate=10 * F, ds0=None, state=11 * F, idx=None, n_slots=B, ws=12 * F,
             wsb=1 << 23, B=B, L=L, C=C, dtype=2, s_x=ROW, s_p=ROW, s_q=ROW, s_rate=1, s_seq=(L, 1), s_s0=ST,
             s_out=ROW, s_s1=ST, s_cs=(3 * C, C, 1), s_dout=ROW, s_ds1=ST, s_dx=ROW, s_dp=ROW, s_dq=ROW, s_drate=1,
             s_ds0=ST, s_state=ST, s_idx=1)
    a.update(kw)
    sizes = [a[n] for n in ("B", "L", "C", "dtype")] + [None]
    head = ("x", "p", "q", "rate")
    if kind == "step":
        return tensors(mx, a, head + ("state",)) + [a["n_slots"]] + tensors(mx, a, ("idx", "out")) + sizes
    if kind == "fwd":
        return tensors(mx, a, head + ("seq", "s0", "out", "s1", "cs")) + [a["ws"], a["wsb"]] + sizes
    return tensors(mx, a, head + ("seq", "s0", "dout", "ds1", "cs", "dx", "dp", "dq", "drate", "ds0")) + \
        [a["ws"], a["wsb"]] + sizes


COMMON = [
    (dict(dtype=7), "unknown dtype"), (dict(B=-1), ">= 0"), (dict(C=-1), ">= 0"), (dict(x=None), "x is required"),
    (dict(p=None), "decay_gate is required"), (dict(q=None), "input_gate is required"),
    (dict(rate=None), "rate is required"), (dict(s_x=None), "x needs its strides"),
    (dict(x=F + 1), "x must be aligned"), (dict(rate=4 * F + 2), "rate must be aligned"),
    (dict(s_p=(1 << 61, C, 1)), "overflows"), (dict(B=1 << 40), "too large"), (dict(L=1 << 32), "too large"),
]


@pytest.mark.parametrize("kw,needle", COMMON + [
    (dict(out=None), "out is required"), (dict(out=F), "must not alias"), (dict(out=2 * F + 8), "must not alias"),
    (dict(s_out=(L * C, 0, 1)), "zero stride"), (dict(seq=13 * F + 2), "seq_idx must be aligned"),
    (dict(s1=14 * F, s_s1=(0, 1)), "zero stride"), (dict(s0=14 * F, s1=14 * F), "must not alias"),
    (dict(cs=5 * F), "must not alias"), (dict(cs=14 * F, s_cs=None), "chunk_states_out needs its strides"),
])
def test_forward_refusals(mx, kw, needle):  # noqa: F811
    rc, msg = status(mx, "ccv_glr_fwd", glr_args(mx, "fwd", **kw))
    assert rc == 1 and needle in msg, msg


@pytest.mark.parametrize("kw,needle", COMMON + [
    (dict(state=None), "state is required"), (dict(n_slots=1), "n_slots"), (dict(n_slots=-1), "n_slots"),
    (dict(idx=13 * F + 1), "state_indices must be aligned"), (dict(out=11 * F), "must not alias"),
    (dict(s_state=(0, 1)), "zero stride"), (dict(state=3 * F), "must not alias"),
])
def test_step_refusals(mx, kw, needle):  # noqa: F811
    rc, msg = status(mx, "ccv_glr_step", glr_args(mx, "step", **kw))
    assert rc == 1 and needle in msg, msg


@pytest.mark.parametrize("kw,needle", COMMON + [
    (dict(dout=None), "dout is required"), (dict(dx=None), "dx is required"), (dict(dp=None), "ddecay_gate is req"),
    (dict(dq=None), "dinput_gate is req"), (dict(drate=None), "drate is required"),
    (dict(ds0=14 * F), "requires initial_state"), (dict(ws=None), "workspace too small"),
    (dict(wsb=64), "workspace too small"), (dict(ws=12 * F + 16), "workspace must be aligned"),
    (dict(dx=6 * F), "must not alias"), (dict(dp=9 * F), "must not alias"), (dict(dq=F), "must not alias"),
    (dict(cs=7 * F), "must not alias"), (dict(ws=8 * F), "must not alias"), (dict(s_drate=0), "zero stride"),
])
def test_backward_refusals(mx, kw, needle):  # noqa: F811
    rc, msg = status(mx, "ccv_glr_bwd", glr_args(mx, "bwd", **kw))
    assert rc == 1 and needle in msg, msg


def test_gate_gradients_as_slices_of_one_buffer_pass(mx):  # noqa: F811
    st = (L * 2 * C, 2 * C, 1)
    ok = dict(dp=8 * F, dq=8 * F + 2 * C, s_dp=st, s_dq=st)
    # (the aliasing check comes last: drate at the workspace shows that it got that far)
    rc, msg = status(mx, "ccv_glr_bwd", glr_args(mx, "bwd", drate=12 * F, **ok))
    assert rc == 1 and "drate" in msg and "workspace" in msg
    rc, msg = status(mx, "ccv_glr_bwd", glr_args(mx, "bwd", **dict(ok, dq=8 * F + 2 * C - 2)))
    assert rc == 1 and "must not alias" in msg


def test_empty_recurrences_are_no_ops(mx):  # noqa: F811
    for kw in (dict(B=0), dict(C=0)):
        assert status(mx, "ccv_glr_fwd", glr_args(mx, "fwd", **kw))[0] == 0
        assert status(mx, "ccv_glr_step", glr_args(mx, "step", **kw))[0] == 0
    assert status(mx, "ccv_glr_fwd", glr_args(mx, "fwd", L=0))[0] == 0
    assert status(mx, "ccv_glr_step", glr_args(mx, "step", L=0))[0] == 0
    assert status(mx, "ccv_glr_bwd", glr_args(mx, "bwd", C=0))[0] == 0


def gn_args(mx, kind, **kw):
    a = dict(x=F, w=2 * F, b=3 * F, out=4 * F, dout=5 * F, dx=6 * F, dw=7 * F, db=8 * F, ws=9 * F, wsb=1 << 23, N=2,
             S=130, C=C, G=4, eps=1e-5, act=1, dtype=2, wdtype=0, s_x=ROW, s_w=1, s_b=1, s_out=ROW, s_dout=ROW,
             s_dx=ROW, s_dw=1, s_db=1)
    a.update(kw)
    arr = mx._arr
    tail = [a[n] for n in ("ws", "wsb", "N", "S", "C", "G", "eps", "act", "dtype", "wdtype")] + [None]
    head = [a["x"], arr(a["s_x"]), a["w"], a["s_w"], a["b"], a["s_b"]]
    if kind == "fwd":
        return head + [a["out"], arr(a["s_out"])] + tail
    return head + [a["dout"], arr(a["s_dout"]), a["dx"], arr(a["s_dx"]), a["dw"], a["s_dw"], a["db"], a["s_db"]] + tail


GN_COMMON = [
    (dict(dtype=5), "unknown dtype"), (dict(wdtype=5), "unknown weight dtype"), (dict(act=3), "unknown activation"),
    (dict(N=-1), ">= 0"), (dict(G=0), "multiple of groups"), (dict(G=5), "multiple of groups"),
    (dict(G=-2), "multiple of groups"), (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"),
    (dict(x=None), "x is required"), (dict(s_x=None), "x needs its strides"), (dict(x=F + 1), "x must be aligned"),
    (dict(w=2 * F + 2), "weight must be aligned"), (dict(N=1 << 40), "too large"), (dict(S=1 << 40), "too large"),
    (dict(s_x=(1 << 61, C, 1)), "overflows"),
]


@pytest.mark.parametrize("kw,needle", GN_COMMON + [
    (dict(out=None), "out is required"), (dict(out=F), "must not alias"), (dict(s_out=(L * C, C, 0)), "zero stride"),
])
def test_group_norm_forward_refusals(mx, kw, needle):  # noqa: F811
    rc, msg = status(mx, "ccv_gn_fwd", gn_args(mx, "fwd", **kw))
    assert rc == 1 and needle in msg, msg


@pytest.mark.parametrize("kw,needle", GN_COMMON + [
    (dict(dout=None), "dout is required"), (dict(dx=None), "dx is required"), (dict(dx=5 * F), "must not alias"),
    (dict(dw=8 * F), "must not alias"), (dict(db=2 * F), "must not alias"), (dict(ws=None), "workspace too small"),
    (dict(ws=9 * F + 8), "workspace must be aligned"), (dict(wsb=8), "workspace too small"),
    (dict(s_dw=0), "zero stride"), (dict(ws=6 * F), "must not alias"),
])
def test_group_norm_backward_refusals(mx, kw, needle):  # noqa: F811
    rc, msg = status(mx, "ccv_gn_bwd", gn_args(mx, "bwd", **kw))
    assert rc == 1 and needle in msg, msg


def test_empty_norms_are_no_ops(mx):  # noqa: F811
    for kw in (dict(N=0), dict(S=0), dict(C=0)):
        assert status(mx, "ccv_gn_fwd", gn_args(mx, "fwd", **kw))[0] == 0
        assert status(mx, "ccv_gn_bwd", gn_args(mx, "bwd", dw=None, db=None, **kw))[0] == 0


def test_workspaces_are_told_on_the_host(mx):  # noqa: F811
    n = ctypes.c_uint64(0)
    for name, key in (("ccv_glr_fwd", (B, L, C, 2)), ("ccv_glr_bwd", (B, L, C, 2)), ("ccv_gn_fwd", (2, 130, C, 4)),
                      ("ccv_gn_bwd", (2, 130, C, 4))):
        assert mx._fn(name + "_workspace_size")(*key, ctypes.byref(n)) == 0
        assert mx._fn(name + "_workspace_size")(*key, None) == 1
        assert mx._fn(name + "_workspace_size")(-1, *key[1:], ctypes.byref(n)) == 1


@pytest.mark.parametrize("kind", ["fwd", "bwd"])
def test_groups_of_too_many_channels(mx, kind):  # noqa: F811
    wide = 1 << 19
    n = ctypes.c_uint64()
    assert mx._fn(f"ccv_gn_{kind}_workspace_size")(1, 1, wide, 2, ctypes.byref(n)) == 0
    assert mx._fn(f"ccv_gn_{kind}_workspace_size")(1, 1, wide, 1, ctypes.byref(n)) == 1
    rc, msg = status(mx, "ccv_gn_" + kind, gn_args(mx, kind, N=1, S=1, C=wide, G=1))
    assert rc == 1 and "262144 channels" in msg, msg
