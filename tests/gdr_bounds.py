"""Error bounds of the gated delta rule's gradients that stay below the
gradients' own size at any length.

For |k| <= 1, 0 <= beta <= 1 and decays <= 1 the state and, backwards, its
gradient D are mapped from token to token by contractions, each column (value
channel) for itself:

    S <- (I - beta k k^T) a S + beta k v^T,      D <- a (I - beta k k^T) (D + q d^T),   d = scale dout

so an error that is there already does not grow, and only a token's own
rounding is added.  A sum of n products and the few terms that go into and out
of it is known to gam = 4 (sqrt(n) + 16) 2^-24 times the norms that enter it: up
to four such sums lie between a token's inputs and a result, and their roundings
do not all point one way (a chunk's solution of its triangular system makes the
same error per token).  Errors are kept as norms of columns; what is made of
several columns sums over them, and the errors of all earlier tokens add up.

dg is summed from terms of its sequence's tokens up to the end of the chunk, q.dq - k.dk +
2 beta k.z with z = -A du, and <S, D> there, some ten thousand roundings: those of
different columns and tokens are taken as independent, and their sum as at most
four times the root of the sum of squares.

Operands enter as two FP16 terms scaled by the largest of their row, and for a
value channel a row is its chunk of 64 tokens: beside a much larger token a value
is known to 2^-39 of the larger one.  64 of these errors, which do not all point
one way, enter a sum: four times their root sum is 2^-34.  ``floor`` adds 2^-35, in
every chunk, of each of the largest v, u, S, dout, du and D to what is made of them.
"""
import torch

from tests.mixer_ref import _keep


FLOOR = 2.0 ** -35


def gdr_floor(c, chunk=64):
    """(out, final_state) errors beside much larger tokens, to be added to ``mixer_ref.gdr``'s bounds."""
    q, k, v, g, beta = (c[n] for n in ("q", "k", "v", "g", "beta"))
    rep = v.shape[2] // q.shape[2]
    k2, a = k.double().repeat_interleave(rep, 2), torch.exp(g.double())
    keep = _keep(c["seq_idx"], *v.shape[:2])
    S = torch.zeros(v.shape[0], v.shape[2], k.shape[3], v.shape[3], dtype=torch.float64) \
        if c["initial_state"] is None else c["initial_state"].double()
    most = S.norm(dim=2)
    for t in range(v.shape[1]):
        S = S * (a[:, t] * keep[:, t, None])[..., None, None]
        u = beta.double()[:, t, :, None] * (v.double()[:, t] - torch.einsum("bhk,bhkv->bhv", k2[:, t], S))
        S = S + k2[:, t, :, :, None] * u[:, :, None, :]
        most = torch.maximum(most, v.double()[:, t].abs() + u.abs() + S.norm(dim=2))
    e = 4 * FLOOR * -(-v.shape[1] // chunk) * most
    qn = q.double().norm(dim=-1).repeat_interleave(rep, 2)
    return k.shape[3] ** -0.5 * qn[..., None] * e[:, None], e[:, :, None, :]


def gdr_bwd(c, scale=None, chunk=64, floor=False):
    """{name: (gradient, error bound)} of the token-by-token definition in FP64."""
    q, k, v, g, beta = (c[n] for n in ("q", "k", "v", "g", "beta"))
    B, L, Hk, Dk = q.shape
    Hv, Dv = v.shape[2:]
    rep = Hv // Hk
    q, k = (x.double().repeat_interleave(rep, 2) for x in (q, k))
    v, beta, a, do = v.double(), beta.double(), torch.exp(g.double()), c["dout"].double()
    scale = Dk ** -0.5 if scale is None else scale
    keep = _keep(c["seq_idx"], B, L)
    zero = torch.zeros(()).double()
    gam = 4 * (max(Dk, Dv) ** 0.5 + 16) * 2.0 ** -24
    col = lambda x: x.norm(dim=2)  # noqa: E731  columns of [B, H, Dk, Dv]
    nrm = lambda x: x.norm(dim=-1, keepdim=True)  # noqa: E731
    sq = lambda x: (x * x).sum(-1)  # noqa: E731
    rows = lambda m, x: torch.einsum("bhkv,bhv->bhk", m, x)  # noqa: E731
    S = torch.zeros((B, Hv, Dk, Dv), dtype=torch.float64) if c["initial_state"] is None \
        else c["initial_state"].double()
    eS = torch.zeros((B, Hv, Dv), dtype=torch.float64)
    hist = []
    for t in range(L):
        on = keep[:, t, None, None]
        A = torch.where(on[..., None] > 0, S * a[:, t, :, None, None], zero)
        eA = torch.where(on > 0, eS * a[:, t, :, None], zero)
        w = v[:, t] - torch.einsum("bhk,bhkv->bhv", k[:, t], A)
        u = beta[:, t, :, None] * w
        ew = eA + gam * (col(A) + v[:, t].abs())
        S = A + k[:, t, :, :, None] * u[:, :, None, :]
        eS = eA + gam * (col(A) + v[:, t].abs() + u.abs())
        hist.append((A, eA, w, ew, u, S, eS))
    D = torch.zeros_like(S) if c["dfinal_state"] is None else c["dfinal_state"].double()
    eD = torch.zeros((B, Hv, Dv), dtype=torch.float64)
    grads = [col(D)]
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    eq, ek, ev = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg, db, eb, own, end, term = (torch.empty_like(a) for _ in range(6))
    for t in reversed(range(L)):
        A, eA, w, ew, u, S1, eS1 = hist[t]
        d, be = scale * do[:, t], beta[:, t, :, None]
        end[:, t] = sq(eS1 * col(D) + col(S1) * eD + gam * col(S1) * col(D))
        eD = eD + gam * nrm(q[:, t]) * d.abs()
        D = D + q[:, t, :, :, None] * d[:, :, None, :]
        du = torch.einsum("bhk,bhkv->bhv", k[:, t], D)
        edu = nrm(k[:, t]) * (eD + gam * col(D))
        grads.append(col(D) + du.abs())
        dq[:, t] = rows(S1, d)
        eq[:, t] = ((eS1 + gam * col(S1)) * d.abs()).sum(-1, keepdim=True)
        db[:, t] = (du * w).sum(-1)
        eb[:, t] = (edu * w.abs() + du.abs() * ew + gam * du.abs() * (w.abs() + v[:, t].abs())).sum(-1)
        dv[:, t] = be * du
        ev[:, t] = be * edu
        dk[:, t] = rows(D, u) - rows(A, dv[:, t])
        ez = rows(A.abs(), edu) + ((eA + gam * col(A)) * du.abs()).sum(-1, keepdim=True)
        ek[:, t] = ((eD + gam * col(D)) * u.abs()).sum(-1, keepdim=True) + rows(D.abs(), be * ew) + be * ez
        dA = D - k[:, t, :, :, None] * dv[:, t, :, None, :]
        edA = eD + 2 * gam * col(D)
        # a sequence's first token decays nothing, whatever its gradient is
        dg[:, t] = torch.where(keep[:, t, None] > 0, (dA * A).sum((2, 3)), zero)
        own[:, t] = sq(edA * col(A) + col(dA) * eA + gam * col(dA) * col(A))
        # columns' shares of the three dot products, by their norms over the key channels
        ezc = col(A) * edu + (eA + gam * col(A)) * du.abs()
        ekc = (eD + gam * col(D)) * u.abs() + be * (col(D) * ew + ezc)
        term[:, t] = sq(nrm(q[:, t]) * (eS1 + gam * col(S1)) * d.abs() + nrm(k[:, t]) * (ekc + 2 * be * ezc))
        on = keep[:, t, None, None]
        D = torch.where(on[..., None] > 0, dA * a[:, t, :, None, None], zero)
        eD = torch.where(on > 0, edA * a[:, t, :, None], zero)
    tail = torch.empty_like(term)
    for t in range(L):  # up to the end of the chunk or of the sequence
        last = min(L, (t // chunk + 1) * chunk) - 1
        with_t = keep[:, t + 1:last + 1].cumprod(1)
        later = torch.where(with_t[..., None] > 0, term[:, t + 1:last + 1], zero).sum(1)
        at_end = torch.where(with_t[:, -1:] > 0, end[:, last], zero) if last > t else end[:, last]
        tail[:, t] = 4 * torch.sqrt(own[:, t] + at_end + term[:, t] + later)
    if floor:
        most = lambda xs: torch.stack([x.abs() for x in xs]).amax(0)  # noqa: E731  over the tokens
        f = FLOOR * -(-L // chunk)
        Md = most([scale * do[:, t] for t in range(L)])
        Mu = most([h[4] for h in hist]) + most([col(h[5]) for h in hist]) + most([col(h[0]) for h in hist])
        MD = Md + most(grads)
        fv = f * MD
        f2 = 4 * f * Dv ** 0.5 * (MD * (Mu + v.abs().amax(1))).amax(-1)[:, None]  # a product over the channels
        ev, eD = ev + fv[:, None], eD + fv
        eq, ek = eq + f2[..., None], ek + f2[..., None]
        eb, tail = eb + f2, tail + 16 * f2
    share = lambda x: x.unflatten(2, (Hk, rep)).sum(3)  # noqa: E731
    res = {"dq": (share(dq), share(eq)), "dk": (share(dk), share(ek)), "dv": (dv, ev), "dg": (dg, tail),
           "dbeta": (db, eb)}
    if c["initial_state"] is not None:
        res["dinitial_state"] = (D, (eD + gam * col(D))[:, :, None, :])
    return res
