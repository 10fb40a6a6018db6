"""FP64 references of the gated linear recurrence and of group normalisation,
from their definitions, on the CPU; seeded inputs; and the error bounds that the
tests hold the kernels to.

U is the rounding of one FP32 operation, H the error of one of the hardware's
exponentials, reciprocals and square roots (both relative)."""
import torch

from tests.mixer_ref import DT, UNIT, rounding, worst  # noqa: F401

U, H = 2.0 ** -24, 2.0 ** -22


def glr_inputs(seed, B, L, C, dtype, seqs=0, state=False, grads=False, rate=0.8, spread=1.5):
    """x, gate logits, rates over three decades; None where not wanted."""
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    dt = DT[dtype]
    c = dict(x=rnd(B, L, C).to(dt), decay_gate=(spread * rnd(B, L, C)).to(dt), input_gate=(spread * rnd(B, L, C)).to(dt),
             rate=(rate * 10 ** (-3 * torch.rand(C, generator=gen, dtype=torch.float64))).float(), seq_idx=None,
             initial_state=None)
    if seqs:
        cuts = torch.rand((B, L), generator=gen).argsort(1)[:, :max(0, min(seqs, L) - 1)]
        c["seq_idx"] = torch.zeros((B, L)).scatter_(1, cuts, 1.0).cumsum(1).to(torch.int32)
    if state:
        c["initial_state"] = rnd(B, C).float()
    if grads:
        c["dout"] = rnd(B, L, C).to(dt)
        c["dfinal_state"] = rnd(B, C).float() if state else None
    return c


def _starts(seq_idx, B, L):
    new = torch.zeros((B, L), dtype=torch.bool)
    if seq_idx is not None and L > 1:
        new[:, 1:] = seq_idx[:, 1:] != seq_idx[:, :-1]
    return new


def _factors(c):
    """Gates, decays and input factors in FP64, and the relative errors of an FP32 evaluation."""
    p, q, rate = c["decay_gate"].double(), c["input_gate"].double(), c["rate"].double()
    r, i = torch.sigmoid(p), torch.sigmoid(q)
    l = -rate * r  # noqa: E741
    a, m = torch.exp(l), torch.sqrt(-torch.expm1(2 * l))

    def gate_errors(z, s):
        # e^-z: two roundings of the exponent and the exponential; 1 / (1 + e^-z): that times 1 - s, a sum, a
        # reciprocal.  Infinite z: e^-z and both results are exact
        e = 2 * U * torch.where(z.isinf(), 0.0, z.abs()) + H
        return e * (1 - s) + U + H, e + 2 * (U + H)

    er, eomr = gate_errors(p, r)
    ei, eomi = gate_errors(q, i)
    el = er + U
    far = (l < -0.34).double() * (2 * H + 2 * U * l.abs())
    ea = l.abs() * el + 4 * U + far                # of a: its exponent's error, the polynomial and the sum
    em = el + 8 * U + 3 * far + H                  # of m: 1 - a >= 0.29 where the exponential is the hardware's
    return dict(r=r, i=i, omr=torch.sigmoid(-p), omi=torch.sigmoid(-q), l=l, a=a, m=m, er=er, ei=ei, eomr=eomr,
                eomi=eomi, el=el, ea=ea, em=em)


def glr(c):
    """{name: (value, error bound)} of out, final_state, chunk_states; and what the backward pass needs.

    An evaluation in any order of association makes, at each token, an error of a
    few roundings of the terms that enter it, which then decays as the state
    does; habs is the recurrence of the magnitudes."""
    f, x = _factors(c), c["x"].double()
    B, L, C = x.shape
    new = _starts(c["seq_idx"], B, L)
    b = f["m"] * f["i"] * x
    eb = b.abs() * (f["em"] + f["ei"] + 4 * U)
    s0 = torch.zeros((B, C), dtype=torch.float64) if c["initial_state"] is None else c["initial_state"].double()
    h, habs, e = s0, s0.abs(), torch.zeros_like(s0)
    out, err, prev, eprev = (torch.empty_like(x) for _ in range(4))
    chunks = []
    for t in range(L):
        if t % 64 == 0:
            chunks.append((h, e))
        on = ~new[:, t, None]
        zero = torch.zeros((), dtype=torch.float64)
        # selected, not multiplied: nothing crosses a new sequence's start
        h, habs, e = (torch.where(on, v, zero) for v in (h, habs, e))
        prev[:, t], eprev[:, t] = h, e
        a = f["a"][:, t]
        e = a * e + (f["ea"][:, t] + 3 * U) * a * habs + eb[:, t]
        h, habs = a * h + b[:, t], a * habs + b[:, t].abs()
        e = e + 3 * U * habs
        out[:, t], err[:, t] = h, e
    res = dict(out=(out, err), final_state=(h, e), prev=(prev, eprev), factors=f, new=new)
    if chunks:
        res["chunk_states"] = tuple(torch.stack(v, 1) for v in zip(*chunks))
    return res


def glr_bwd(c):
    """{name: (gradient, error bound)}, bounds by the same argument."""
    fw = glr(c)
    f, new, (prev, eprev) = fw["factors"], fw["new"], fw["prev"]
    x, dout = c["x"].double(), c["dout"].double()
    B, L, C = x.shape
    z = torch.zeros((B, C), dtype=torch.float64)
    d = z if c["dfinal_state"] is None else c["dfinal_state"].double()
    G, eG = torch.empty_like(x), torch.empty_like(x)
    dabs, e = d.abs(), torch.zeros_like(z)
    for t in reversed(range(L)):
        d, dabs = d + dout[:, t], dabs + dout[:, t].abs()
        e = e + 3 * U * dabs
        G[:, t], eG[:, t] = d, e
        a, on = f["a"][:, t], ~new[:, t, None]
        e = torch.where(on, a * e + (f["ea"][:, t] + 3 * U) * a * dabs, z)
        d, dabs = torch.where(on, a * d, z), torch.where(on, a * dabs, z)
    m, i, a = f["m"], f["i"], f["a"]
    ix = i * x
    # the root's derivative; zero where the decay is one in FP32
    slope = torch.where(m > 2.0 ** -62, ix * a * a / m, torch.zeros((), dtype=torch.float64))
    W = a * prev - slope
    eW = a * eprev + (a * prev).abs() * (f["ea"] + 2 * U) + slope.abs() * (f["ei"] + 2 * f["ea"] + f["em"] + 8 * U)
    dx = G * m * i
    edx = (m * i) * (eG + G.abs() * (f["em"] + f["ei"] + 4 * U))
    dq = G * m * ix * f["omi"]
    edq = (m * ix * f["omi"]).abs() * (eG + G.abs() * (f["em"] + f["ei"] + f["eomi"] + 6 * U))
    k = f["l"] * f["omr"]
    eGW = eG * W.abs() + G.abs() * eW + (eG * eW)
    dp = G * W * k
    edp = k.abs() * (eGW + (G * W).abs() * (f["el"] + f["eomr"] + 6 * U))
    terms = -G * W * f["r"]
    drate = terms.sum((0, 1))
    edrate = (f["r"] * eGW + terms.abs() * (f["er"] + 6 * U)).sum((0, 1)) + (B * L + 64) * U * terms.abs().sum((0, 1))
    return dict(dx=(dx, edx), ddecay_gate=(dp, edp), dinput_gate=(dq, edq), drate=(drate, edrate),
                dinitial_state=(d, e + 3 * U * dabs))


def glr_autograd(c):
    """The gradients of sum(out dout) + sum(final_state dfinal_state) by FP64 autograd of the definition."""
    names = ["x", "decay_gate", "input_gate", "rate"] + (["initial_state"] if c["initial_state"] is not None else [])
    leaf = {n: c[n].double().requires_grad_() for n in names}
    B, L, C = leaf["x"].shape
    new = _starts(c["seq_idx"], B, L)
    h = leaf.get("initial_state", torch.zeros((B, C), dtype=torch.float64))
    loss = 0.0
    for t in range(L):
        a = torch.exp(-leaf["rate"] * torch.sigmoid(leaf["decay_gate"][:, t]))
        h = torch.where(new[:, t, None], 0.0, a * h) + \
            torch.sqrt(1 - a * a) * torch.sigmoid(leaf["input_gate"][:, t]) * leaf["x"][:, t]
        loss = loss + (h * c["dout"][:, t].double()).sum()
    if c["dfinal_state"] is not None:
        loss = loss + (h * c["dfinal_state"].double()).sum()
    return dict(zip(["dx", "ddecay_gate", "dinput_gate", "drate", "dinitial_state"],
                    torch.autograd.grad(loss, [leaf[n] for n in names])))


def gn_inputs(seed, N, S, C, dtype, wdtype, mean=3.0):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    return ((rnd(N, S, C) + mean * rnd(C)).to(DT[dtype]), (1 + 0.3 * rnd(C)).to(DT[wdtype]),
            (0.3 * rnd(C)).to(DT[wdtype]), rnd(N, S, C).to(DT[dtype]))


def _gn_parts(x, G, w, b, eps, silu):
    N, S, C = x.shape
    x = x.double()
    w = torch.ones(C, dtype=torch.float64) if w is None else w.double()
    b0 = torch.zeros(C, dtype=torch.float64) if b is None else b.double()
    mean = lambda v: v.unflatten(-1, (G, -1)).mean((1, 3)).repeat_interleave(C // G, -1)[:, None]  # noqa: E731
    mu = mean(x)
    r = 1 / torch.sqrt(mean((x - mu) ** 2) + eps)
    xh = (x - mu) * r
    z = xh * w + b0
    s = torch.sigmoid(z) if silu else None
    # a sum's chain: a thread's terms (at most one in 128 of a group, 1024 in a slab), then exchanges and merges
    g = (96 + min(S * (C // G) / 128, 2048)) * U
    dm = g * mean(x.abs()) * r                          # error of xh from the mean
    exh = dm * (1 + xh.abs()) + 3 * g * xh.abs()
    ez = w.abs() * exh + 4 * U * (z.abs() + (xh * w).abs() + b0.abs())
    return dict(w=w, r=r, xh=xh, z=z, s=s, g=g, exh=exh, ez=ez, mean=mean)


def gn_fwd(x, G, w, b, eps=1e-5, silu=False):
    """(value, error bound before the rounding to the output's type)."""
    p = _gn_parts(x, G, w, b, eps, silu)
    if not silu:
        return p["z"], p["ez"]
    y = p["z"] * p["s"]
    return y, 1.1 * p["ez"] + y.abs() * (4 * H + 3 * U * p["z"].abs())  # |silu'| <= 1.1


def gn_bwd(x, G, w, dy, b, eps=1e-5, silu=False):
    """{name: (gradient, error bound before its rounding)}."""
    p = _gn_parts(x, G, w, b, eps, silu)
    dy = dy.double()
    N, S, C = x.shape
    w, xh, z, r, mean, g = p["w"], p["xh"], p["z"], p["r"], p["mean"], p["g"]
    dz, edz = dy, torch.zeros_like(dy)
    if silu:
        s = p["s"]
        act = s * (1 + z * (1 - s))
        dz = dy * act
        # |silu''| <= 0.5; the hardware's functions in s, 1 - s and their products; below z = -80 less than 1e-30
        edz = dy.abs() * (0.5 * p["ez"] + s * (1 + z.abs() * (1 - s)) * (5 * H + 4 * U * z.abs()) + 1e-30)
    d, ed = dz * w, w.abs() * edz + 2 * U * (dz * w).abs()
    m1, m2 = mean(d), mean(d * xh)
    e1 = mean(ed) + g * mean(d.abs())
    e2 = mean(ed * xh.abs() + d.abs() * p["exh"]) + g * mean((d * xh).abs())
    dx = r * (d - m1 - xh * m2)
    rel = 3 * g + 4 * U                                  # of r
    edx = r * (ed + e1 + p["exh"] * m2.abs() + xh.abs() * e2 + p["exh"] * e2 +
               (rel + 4 * U) * (d.abs() + m1.abs() + (xh * m2).abs()))
    gn = (N * S / 8 + 2200) * U if N * S > 2400 else (N * S + 64) * U
    return dict(dx=(dx, edx),
                dweight=((dz * xh).sum((0, 1)), (edz * xh.abs() + dz.abs() * p["exh"] + edz * p["exh"] +
                                                 gn * (dz * xh).abs()).sum((0, 1))),
                dbias=(dz.sum((0, 1)), (edz + gn * dz.abs()).sum((0, 1))))
