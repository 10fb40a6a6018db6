"""FP64 references of the gated delta rule and of layer normalisation, from
their definitions, on the CPU; seeded inputs; and the error bounds that the
tests hold the kernels to."""
import numpy as np
import torch

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}   # unit roundoff
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}  # smallest subnormal


def gdr_inputs(seed, B, L, Hk, Hv, Dk, Dv, dtype, seqs=0, state=False, decay=0.2, grads=False):
    """q and k of length <= 1, beta in (0, 1), g <= 0; None where not wanted."""
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    unit = lambda x: x / (x.norm(dim=-1, keepdim=True) * 1.01 + 1e-9)  # noqa: E731
    dt = DT[dtype]
    c = dict(q=unit(rnd(B, L, Hk, Dk)).to(dt), k=unit(rnd(B, L, Hk, Dk)).to(dt), v=rnd(B, L, Hv, Dv).to(dt),
             g=(-decay * torch.nn.functional.softplus(rnd(B, L, Hv))).float(),
             beta=torch.sigmoid(rnd(B, L, Hv)).to(dt), seq_idx=None, initial_state=None)
    if seqs:
        cuts = torch.rand((B, L), generator=gen).argsort(1)[:, :max(0, min(seqs, L) - 1)]
        c["seq_idx"] = torch.zeros((B, L)).scatter_(1, cuts, 1.0).cumsum(1).to(torch.int32)
    if state:
        c["initial_state"] = (0.5 * rnd(B, Hv, Dk, Dv)).float()
    if grads:
        c["dout"] = rnd(B, L, Hv, Dv).to(dt)
        c["dfinal_state"] = (0.5 * rnd(B, Hv, Dk, Dv)).float() if state else None
    return c


def _keep(seq_idx, B, L):
    keep = torch.ones((B, L), dtype=torch.float64)
    if seq_idx is not None and L > 1:
        keep[:, 1:] = (seq_idx[:, 1:] == seq_idx[:, :-1]).double()
    return keep


def gdr(q, k, v, g, beta, seq_idx=None, initial_state=None, scale=None, unit=2.0 ** -24):
    """(out, final_state, err_out, err_state): the definition in FP64, and a
    bound of an FP32 evaluation's error.

    The bound: for |k| <= 1, 0 <= beta <= 1 and decays <= 1 a token maps the
    state by a contraction, so an error made at one token does not grow later.
    At one token, each column's prediction, write and read are sums of Dk
    products and a few terms more: an error of at most (Dk + 64) unit times the
    column's norms.  A chunk's solution of its triangular system makes the same
    error per token.  e is that sum per column, decayed with the state."""
    B, L, Hk, Dk = q.shape
    Hv, Dv = v.shape[2:]
    rep = Hv // Hk
    q, k = (x.double().repeat_interleave(rep, 2) for x in (q, k))
    v, beta, a = v.double(), beta.double(), torch.exp(g.double())
    scale = Dk ** -0.5 if scale is None else scale
    keep = _keep(seq_idx, B, L)
    S = torch.zeros((B, Hv, Dk, Dv), dtype=torch.float64) if initial_state is None else initial_state.double()
    e = torch.zeros((B, Hv, Dv), dtype=torch.float64)
    out, err = torch.empty_like(v), torch.empty_like(v)
    gamma = (Dk + 64) * unit
    for t in range(L):
        # selected, not multiplied: nothing crosses a new sequence's start
        S = torch.where(keep[:, t, None, None, None] > 0, S * a[:, t, :, None, None], torch.zeros(()).double())
        e = torch.where(keep[:, t, None, None] > 0, e * a[:, t, :, None], torch.zeros(()).double())
        u = beta[:, t, :, None] * (v[:, t] - torch.einsum("bhk,bhkv->bhv", k[:, t], S))
        e = e + gamma * (S.norm(dim=2) + v[:, t].abs() + u.abs())
        S = S + k[:, t, :, :, None] * u[:, :, None, :]
        out[:, t] = scale * torch.einsum("bhk,bhkv->bhv", q[:, t], S)
        err[:, t] = abs(scale) * q[:, t].norm(dim=-1)[..., None] * (e + gamma * S.norm(dim=2))
    return out, S, err, (e + gamma * S.norm(dim=2))[:, :, None, :]


def gdr_autograd(c, scale=None):
    """Gradients of sum(out dout) + sum(final_state dfinal_state) in FP64."""
    names = ["q", "k", "v", "g", "beta"] + (["initial_state"] if c["initial_state"] is not None else [])
    leaf = {n: c[n].double().requires_grad_() for n in names}
    out, S, _, _ = gdr(leaf["q"], leaf["k"], leaf["v"], leaf["g"], leaf["beta"], c["seq_idx"],
                       leaf.get("initial_state"), scale)
    loss = (out * c["dout"].double()).sum()
    if c["dfinal_state"] is not None:
        loss = loss + (S * c["dfinal_state"].double()).sum()
    grads = torch.autograd.grad(loss, [leaf[n] for n in names], allow_unused=True)
    return {n: torch.zeros_like(leaf[n]) if d is None else d for n, d in zip(names, grads)}


def rounding(exact, dtype):
    """Half a unit in the last place of the dtype."""
    return exact.abs() * UNIT[dtype] + TINY[dtype]


def worst(got, exact, bound):
    """Largest error over its bound; inf where finiteness differs."""
    got, exact = got.double().cpu(), exact.double().cpu()
    fin = torch.isfinite(exact)
    if not bool((torch.isfinite(got) == fin).all()):
        return float("inf")
    if not bool(fin.any()):
        return 0.0
    bound = bound.double().expand_as(exact)
    return float(((got - exact).abs()[fin] / bound[fin]).max())


def ln_fwd(x, w, b, eps=1e-5):
    x = x.double()
    m = x.mean(-1, keepdim=True)
    r = 1 / torch.sqrt(((x - m) ** 2).mean(-1, keepdim=True) + eps)
    xh = (x - m) * r
    y = xh if w is None else xh * w.double()
    return (y if b is None else y + b.double()), xh, r


def ln_bwd(x, w, dy, eps=1e-5):
    _, xh, r = ln_fwd(x, None, None, eps)
    dy = dy.double()
    d = dy if w is None else dy * w.double()
    dx = r * (d - d.mean(-1, keepdim=True) - xh * (d * xh).mean(-1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def np_rng(seed):
    return np.random.default_rng(seed)


def gdr_bwd(c, scale=None, chunk=64):
    """{name: (gradient, error bound)} from the token-by-token definition in FP64.

    The bounds follow the same argument as ``gdr``'s: for |k| <= 1,
    0 <= beta <= 1 and decays <= 1 both the state and, backwards, its gradient
    are mapped by contractions, so the errors of the tokens add up, decayed.  A
    token's own error is gamma times the norms that enter it, gamma =
    4 (D + 64) 2^-24 for the up to four sums of D products between its inputs
    and a result.  e* below are errors of norms: eS of the state, eD of its
    gradient.  dg is summed from terms of the tokens up to the end of its chunk,
    so the errors of those add to its own."""
    q, k, v, g, beta = (c[n] for n in ("q", "k", "v", "g", "beta"))
    B, L, Hk, Dk = q.shape
    Hv, Dv = v.shape[2:]
    rep = Hv // Hk
    q, k = (x.double().repeat_interleave(rep, 2) for x in (q, k))
    v, beta, a, do = v.double(), beta.double(), torch.exp(g.double()), c["dout"].double()
    scale = Dk ** -0.5 if scale is None else scale
    keep = _keep(c["seq_idx"], B, L)
    zero = torch.zeros(()).double()
    gam = 4 * (max(Dk, Dv) + 64) * 2.0 ** -24
    fro = lambda x: x.flatten(2).norm(dim=2)  # noqa: E731
    nrm = lambda x: x.norm(dim=-1)  # noqa: E731
    S = torch.zeros((B, Hv, Dk, Dv), dtype=torch.float64) if c["initial_state"] is None \
        else c["initial_state"].double()
    eS = torch.zeros((B, Hv), dtype=torch.float64)
    hist = []
    for t in range(L):
        on = keep[:, t, None]
        A = torch.where(on[..., None, None] > 0, S * a[:, t, :, None, None], zero)
        eA = torch.where(on > 0, eS * a[:, t], zero)
        w = v[:, t] - torch.einsum("bhk,bhkv->bhv", k[:, t], A)
        u = beta[:, t, :, None] * w
        ew = eA + gam * (fro(A) + nrm(v[:, t]))
        S = A + k[:, t, :, :, None] * u[:, :, None, :]
        eS = eA + gam * (fro(A) + nrm(v[:, t]) + nrm(u))
        hist.append((A, eA, w, ew, u, S, eS))
    D = torch.zeros_like(S) if c["dfinal_state"] is None else c["dfinal_state"].double()
    eD = torch.zeros((B, Hv), dtype=torch.float64)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    eq, ek, ev, eb, own = (torch.empty((B, L, Hv), dtype=torch.float64) for _ in range(5))
    dg, db = torch.empty_like(a), torch.empty_like(a)
    for t in reversed(range(L)):
        A, eA, w, ew, u, S1, eS1 = hist[t]
        d = scale * do[:, t]
        eD = eD + gam * nrm(q[:, t]) * nrm(d)
        D = D + q[:, t, :, :, None] * d[:, :, None, :]
        du = torch.einsum("bhk,bhkv->bhv", k[:, t], D)
        edu = eD + gam * fro(D)
        be = beta[:, t]
        dq[:, t] = torch.einsum("bhkv,bhv->bhk", S1, d)
        eq[:, t] = (eS1 + gam * fro(S1)) * nrm(d)
        db[:, t] = (du * w).sum(-1)
        eb[:, t] = edu * nrm(w) + nrm(du) * ew + gam * nrm(du) * (nrm(w) + nrm(v[:, t]))
        dv[:, t] = be[..., None] * du
        ev[:, t] = be * edu
        dk[:, t] = torch.einsum("bhkv,bhv->bhk", D, u) - torch.einsum("bhkv,bhv->bhk", A, dv[:, t])
        ek[:, t] = eD * nrm(u) + fro(D) * be * ew + eA * nrm(dv[:, t]) + fro(A) * ev[:, t] + \
            gam * (fro(D) * nrm(u) + fro(A) * nrm(dv[:, t]))
        dA = D - k[:, t, :, :, None] * dv[:, t, :, None, :]
        edA = eD + ev[:, t] + gam * fro(D)
        dg[:, t] = (dA * A).sum((2, 3))
        own[:, t] = edA * fro(A) + fro(dA) * eA + gam * fro(dA) * fro(A)
        on = keep[:, t, None]
        D = torch.where(on[..., None, None] > 0, dA * a[:, t, :, None, None], zero)
        eD = torch.where(on > 0, edA * a[:, t], zero)
    term = eq + 3 * ek + 2 * eb  # of one token's share of dg (|q|, |k|, beta <= 1)
    tail = torch.empty_like(term)
    for t in range(L):
        tail[:, t] = term[:, t:(t // chunk + 1) * chunk].sum(1)
        last = min(L, (t // chunk + 1) * chunk) - 1
        tail[:, t] += own[:, last] + own[:, t]
    share = lambda x: x.unflatten(2, (Hk, rep)).sum(3)  # noqa: E731
    res = {"dq": (share(dq), share(eq)[..., None]), "dk": (share(dk), share(ek)[..., None]),
           "dv": (dv, ev[..., None]), "dg": (dg, tail), "dbeta": (db, eb)}
    if c["initial_state"] is not None:
        res["dinitial_state"] = (D, eD[..., None, None] + gam * fro(D)[..., None, None])
    return res
