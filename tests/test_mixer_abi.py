"""Refusals of the gated delta rule's and layer normalisation's entry points,
on the host: nothing is launched and no GPU is needed."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def mx():
    from causal_depthwise_conv1d_gb300 import build
    build.build()
    from causal_depthwise_conv1d_gb300 import mixer
    mixer.load_library()
    return mixer


F = 1 << 24  # fake addresses far apart, never dereferenced


def status(mx, name, args):
    rc = mx._fn(name)(*args)
    return rc, mx.load_library().ccv_last_error().decode()


def gdr_args(mx, step=False, **kw):
    B, L, Hk, Hv, Dk, Dv = 2, 8, 2, 4, 16, 32
    a = dict(q=F, qs=(L * Hk * Dk, Hk * Dk, Dk, 1), k=2 * F, ks=(L * Hk * Dk, Hk * Dk, Dk, 1), v=3 * F,
             vs=(L * Hv * Dv, Hv * Dv, Dv, 1), g=4 * F, gs=(L * Hv, Hv, 1), beta=5 * F, bs=(L * Hv, Hv, 1), seq=None,
             ss=None, s0=None, s0s=None, out=6 * F, os=(L * Hv * Dv, Hv * Dv, Dv, 1), s1=None, s1s=None, ws=None,
             wsb=0, B=B, L=L, Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, scale=1.0, dtype=2, state=7 * F,
             sts=(Hv * Dk * Dv, Dk * Dv, Dv, 1), n_slots=2, idx=None, idxs=1)
    a.update(kw)
    arr = mx._arr
    head = [a["q"], arr(a["qs"]), a["k"], arr(a["ks"]), a["v"], arr(a["vs"]), a["g"], arr(a["gs"]), a["beta"],
            arr(a["bs"])]
    sizes = [a[n] for n in ("B", "L", "Hk", "Hv", "Dk", "Dv", "scale", "dtype")] + [None]
    if step:
        return head + [a["state"], arr(a["sts"]), a["n_slots"], a["idx"], a["idxs"], a["out"], arr(a["os"])] + sizes
    return head + [a["seq"], arr(a["ss"]), a["s0"], arr(a["s0s"]), a["out"], arr(a["os"]), a["s1"], arr(a["s1s"]),
                   a["ws"], a["wsb"]] + sizes


COMMON = [
    (dict(dtype=9), 1, "unknown dtype"), (dict(B=-1), 1, ">= 0"), (dict(Hv=3), 1, "multiple of Hk"),
    (dict(Hk=0), 1, "multiple of Hk"), (dict(Dk=257), 2, "at most 256"), (dict(Dk=0), 1, "Dk must be >= 1"),
    (dict(q=None), 1, "q is required"), (dict(g=None), 1, "g is required"), (dict(beta=None), 1, "beta is required"),
    (dict(out=None), 1, "out is required"), (dict(vs=None), 1, "v needs its strides"),
    (dict(v=3 * F + 1), 1, "v must be aligned"), (dict(g=4 * F + 2), 1, "g must be aligned"),
    (dict(os=(1024, 0, 32, 1)), 1, "zero stride"), (dict(out=3 * F), 1, "must not alias"),
    (dict(out=3 * F + 64), 1, "must not alias"), (dict(ks=(1 << 61, 32, 16, 1)), 1, "overflows"),
    (dict(B=1 << 50), 1, "too large"),
]


@pytest.mark.parametrize("kw,st,needle", COMMON + [
    (dict(seq=8 * F), 1, "seq_idx needs its strides"), (dict(seq=8 * F + 2, ss=(8, 1)), 1, "seq_idx must be aligned"),
    (dict(s0=7 * F), 1, "initial_state needs its strides"),
    (dict(s1=7 * F, s1s=(2048, 512, 0, 1)), 1, "zero stride"),
    (dict(s0=7 * F, s0s=(2048, 512, 32, 1), s1=7 * F, s1s=(2048, 512, 32, 1)), 1, "must not alias"),
    (dict(L=1 << 32), 1, "too large"),
])
def test_forward_refusals(mx, kw, st, needle):
    rc, msg = status(mx, "ccv_gdr_fwd", gdr_args(mx, **kw))
    assert rc == st and needle in msg, msg


@pytest.mark.parametrize("kw,st,needle", COMMON + [
    (dict(state=None), 1, "state is required"), (dict(state=7 * F + 2), 1, "state must be aligned"),
    (dict(n_slots=1), 1, "n_slots"), (dict(n_slots=-1), 1, "n_slots"),
    (dict(idx=8 * F + 1), 1, "state_indices must be aligned"), (dict(out=7 * F), 1, "must not alias"),
    (dict(sts=(0, 512, 32, 1)), 1, "zero stride"),
])
def test_step_refusals(mx, kw, st, needle):
    rc, msg = status(mx, "ccv_gdr_step", gdr_args(mx, step=True, **kw))
    assert rc == st and needle in msg, msg


@pytest.mark.parametrize("kw", [dict(B=0), dict(Hv=0, Hk=0), dict(Dv=0)])
def test_empty_problems_are_no_ops(mx, kw):
    assert status(mx, "ccv_gdr_fwd", gdr_args(mx, **kw))[0] == 0
    assert status(mx, "ccv_gdr_step", gdr_args(mx, step=True, **kw))[0] == 0
    assert status(mx, "ccv_gdr_step", gdr_args(mx, step=True, L=0))[0] == 0
    assert status(mx, "ccv_gdr_fwd", gdr_args(mx, L=0))[0] == 0


def bwd_args(mx, **kw):
    L, Hk, Hv, Dk, Dv = 8, 2, 4, 16, 32
    qs, vs, gs, ss = (L * Hk * Dk, Hk * Dk, Dk, 1), (L * Hv * Dv, Hv * Dv, Dv, 1), (L * Hv, Hv, 1), \
        (Hv * Dk * Dv, Dk * Dv, Dv, 1)
    a = dict(q=F, k=2 * F, v=3 * F, g=4 * F, beta=5 * F, seq=None, s0=None, dout=6 * F, ds1=None, dq=7 * F, dk=8 * F,
             dv=9 * F, dg=10 * F, dbeta=11 * F, ds0=None, ws=12 * F, wsb=1 << 24, B=2, L=L, Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv,
             scale=1.0, dtype=2)
    st = dict(q=qs, k=qs, v=vs, g=gs, beta=gs, seq=(L, 1), s0=ss, dout=vs, ds1=ss, dq=qs, dk=qs, dv=vs, dg=gs,
              dbeta=gs, ds0=ss)
    st.update({n[2:]: x for n, x in kw.items() if n.startswith("s_")})
    a.update({n: x for n, x in kw.items() if not n.startswith("s_")})
    arr = mx._arr
    out = []
    for n in ("q", "k", "v", "g", "beta", "seq", "s0", "dout", "ds1", "dq", "dk", "dv", "dg", "dbeta", "ds0"):
        out += [a[n], arr(st[n])]
    return out + [a["ws"], a["wsb"]] + [a[n] for n in ("B", "L", "Hk", "Hv", "Dk", "Dv", "scale", "dtype")] + [None]


@pytest.mark.parametrize("kw,st,needle", [
    (dict(dtype=4), 1, "unknown dtype"), (dict(Dk=129), 2, "at most 128"), (dict(Dv=513), 2, "at most 512"), (dict(dout=None), 1, "dout is required"),
    (dict(dq=None), 1, "dq is required"), (dict(dg=None), 1, "dg is required"), (dict(dbeta=None), 1, "dbeta is req"),
    (dict(ds0=13 * F), 1, "requires initial_state"), (dict(ws=None), 1, "workspace too small"),
    (dict(wsb=4096), 1, "workspace too small"), (dict(ws=12 * F + 16), 1, "workspace must be aligned"),
    (dict(dq=8 * F), 1, "must not alias"), (dict(dv=6 * F), 1, "must not alias"), (dict(dv=9 * F + 1), 1, "aligned"),
    (dict(s_dk=(0, 32, 16, 1)), 1, "zero stride"), (dict(ws=7 * F), 1, "must not alias"), (dict(Dv=0), 1, "Dv"),
    (dict(s_dout=None), 1, "dout needs its strides"), (dict(B=1 << 45), 1, "too large")])
def test_backward_refusals(mx, kw, st, needle):
    rc, msg = status(mx, "ccv_gdr_bwd", bwd_args(mx, **kw))
    assert rc == st and needle in msg, msg


def test_channel_slices_of_one_buffer_are_told_apart(mx):
    """dq, dk, dv as slices of one [B, L, 2 Hk Dk + Hv Dv] buffer pass; slices that share channels do not."""
    n = 2 * 2 * 16 + 4 * 32
    st = (8 * n, n, 16, 1)
    ok = dict(dq=7 * F, dk=7 * F + 2 * 32, dv=7 * F + 2 * 64, s_dq=st, s_dk=st, s_dv=(8 * n, n, 32, 1))
    # (the aliasing check comes last: an output that repeats the workspace's address shows that it got that far)
    rc, msg = status(mx, "ccv_gdr_bwd", bwd_args(mx, dg=12 * F, **ok))
    assert rc == 1 and "dg" in msg and "workspace" in msg
    rc, msg = status(mx, "ccv_gdr_bwd", bwd_args(mx, **dict(ok, dk=7 * F + 2 * 31, wsb=1 << 24)))
    assert rc == 1 and "must not alias" in msg
    rc, msg = status(mx, "ccv_gdr_bwd", bwd_args(mx, **dict(ok, dv=7 * F + 2 * 63)))
    assert rc == 1 and "must not alias" in msg


def test_workspace_sizes(mx):
    assert mx.ccv_gdr_fwd_workspace_size(1, 16, 1, 1, 128, 128, 2) == 0
    assert mx.ccv_gdr_fwd_workspace_size(1, 4096, 1, 1, 256, 128, 2) == 0  # token by token
    a = mx.ccv_gdr_fwd_workspace_size(1, 4096, 2, 4, 128, 128, 2)
    assert a > 0 and mx.ccv_gdr_fwd_workspace_size(2, 4096, 2, 4, 128, 128, 2) == 2 * a
    assert mx.ccv_gdr_bwd_workspace_size(0, 16, 1, 1, 128, 128, 2) == 0
    assert mx.ccv_gdr_bwd_workspace_size(1, 65, 1, 1, 128, 128, 2) == \
        mx.ccv_gdr_bwd_workspace_size(1, 128, 1, 1, 128, 128, 2)


def ln_args(mx, bwd=False, **kw):
    a = dict(x=F, xs=(64, 1), w=2 * F, ws=1, b=3 * F, bs=1, out=4 * F, os=(64, 1), dout=5 * F, gs=(64, 1), dw=6 * F,
             dws=1, db=7 * F, dbs=1, ws_p=8 * F, ws_n=1 << 20, N=4, D=64, eps=1e-5, dtype=2, wdtype=0)
    a.update(kw)
    arr = mx._arr
    tail = [a["N"], a["D"], a["eps"], a["dtype"], a["wdtype"], None]
    if bwd:
        return [a["x"], arr(a["xs"]), a["w"], a["ws"], a["dout"], arr(a["gs"]), a["out"], arr(a["os"]), a["dw"],
                a["dws"], a["db"], a["dbs"], a["ws_p"], a["ws_n"]] + tail
    return [a["x"], arr(a["xs"]), a["w"], a["ws"], a["b"], a["bs"], a["out"], arr(a["os"])] + tail


LN = [(dict(dtype=5), 1, "unknown dtype"), (dict(wdtype=5), 1, "unknown weight dtype"), (dict(N=-1), 1, ">= 0"),
      (dict(eps=-1.0), 1, "eps"), (dict(eps=float("nan")), 1, "eps"), (dict(x=None), 1, "x is required"),
      (dict(xs=None), 1, "needs its strides"), (dict(x=F + 1), 1, "x must be aligned"),
      (dict(w=2 * F + 2), 1, "weight must be aligned"), (dict(os=(0, 1)), 1, "zero stride"),
      (dict(out=F), 1, "must not alias"), (dict(N=1 << 33), 1, "too large"), (dict(out=F + 32), 1, "must not alias")]


@pytest.mark.parametrize("kw,st,needle", LN)
def test_ln_forward_refusals(mx, kw, st, needle):
    rc, msg = status(mx, "ccv_ln_fwd", ln_args(mx, **kw))
    assert rc == st and needle in msg, msg


@pytest.mark.parametrize("kw,st,needle", LN + [
    (dict(dout=None), 1, "dout is required"), (dict(ws_n=100), 1, "workspace too small"),
    (dict(ws_p=None), 1, "workspace too small"), (dict(ws_p=8 * F + 8), 1, "workspace must be aligned"),
    (dict(dw=7 * F), 1, "must not alias"), (dict(dws=0), 1, "zero stride"), (dict(ws_p=6 * F), 1, "must not alias")])
def test_ln_backward_refusals(mx, kw, st, needle):
    rc, msg = status(mx, "ccv_ln_bwd", ln_args(mx, bwd=True, **kw))
    assert rc == st and needle in msg, msg


def test_ln_workspace(mx):
    assert mx.ccv_ln_bwd_workspace_size(0, 64) == 0
    assert mx.ccv_ln_bwd_workspace_size(1, 4096) == 2 * 4096 * 4
    # one partial sum per block, and no more blocks than rows or than fill the device
    assert 0 < mx.ccv_ln_bwd_workspace_size(10 ** 6, 4096) <= 1024 * 2 * 4096 * 4
    with pytest.raises(Exception, match="bytes is required"):
        rc = mx._fn("ccv_ln_bwd_workspace_size")(4, 4, ctypes.POINTER(ctypes.c_uint64)())
        assert rc == 1
        raise RuntimeError(mx.load_library().ccv_last_error().decode())


def test_binding_refuses_cpu_tensors_and_wrong_shapes(mx):
    import torch
    q = torch.zeros(1, 4, 1, 8)
    g = torch.zeros(1, 4, 1)
    with pytest.raises(ValueError, match="CUDA device"):
        mx.ccv_gdr_fwd(q, q, q, g, g)
    with pytest.raises(ValueError, match=r"\[B, L, Hk, Dk\]"):
        mx.ccv_gdr_fwd(q[0], q, q, g, g)
    with pytest.raises(ValueError, match="unsupported dtype"):
        mx.ccv_gdr_fwd(q, q, q.double(), g, g)
    with pytest.raises(ValueError, match="CUDA device"):
        mx.ccv_ln_fwd(q)
    with pytest.raises(ValueError, match="supported dtype"):
        mx.ccv_ln_fwd(q.double())
