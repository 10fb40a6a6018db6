"""Performance cases of the sequence-mixing operators: the gated delta rule
(whole sequences, its backward pass, its step for single tokens) and layer
normalisation (forward and backward).

Gated delta rule, per value head with state S [Dk, Dv] (zero, or the given
initial state; back to zero where seq_idx changes):

    S <- exp(g_t) S;   u_t = beta_t (v_t - k_t^T S);   S <- S + k_t u_t^T;   o_t = scale * q_t^T S

q and k have Hk heads, v and o Hv heads (a multiple of Hk; value head h reads
q and k of head h // (Hv // Hk)).

``run`` computes either the plain form (torch operations in FP32, rounded once
at the end) or, with ``own`` set, calls the package's operators.  ``exact``
follows the token-by-token definition in FP64.
"""
import math

import torch

own = False

CHUNK = 64
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one long prompt: few heads, a long axis; the final state goes to the cache
        dict(name="fwd prompt", op="fwd", dtype="bf16", B=1, L=8192, Hk=16, Hv=32, Dk=128, Dv=128, seqs=0, state=False),
        # a training batch: 8 x 2048 tokens, 5120 channels in heads of 128, each row packed with documents
        dict(name="fwd training batch", op="fwd", dtype="bf16", B=8, L=2048, Hk=40, Hv=40, Dk=128, Dv=128, seqs=5,
             state=False),
        # a short ragged continuation in FP32 from a cached state, head sizes that are no tile's
        dict(name="fwd short f32", op="fwd", dtype="f32", B=3, L=77, Hk=4, Hv=8, Dk=72, Dv=100, seqs=0, state=True),
        # a training step's backward pass, keys and queries shared by two value heads
        dict(name="bwd training", op="bwd", dtype="bf16", B=2, L=2048, Hk=16, Hv=32, Dk=128, Dv=128, seqs=0,
             state=False),
        # backward over an odd length with packed sequences and a state gradient
        dict(name="bwd ragged", op="bwd", dtype="f16", B=1, L=1001, Hk=8, Hv=8, Dk=64, Dv=64, seqs=3, state=True),
        # one sequence's next token: latency
        dict(name="step one", op="step", dtype="bf16", B=1, S=1, Hk=16, Hv=32, Dk=128, Dv=128, slots=1),
        # a serving batch's next tokens, states in a cache with more slots than requests
        dict(name="step batch", op="step", dtype="bf16", B=128, S=1, Hk=16, Hv=32, Dk=128, Dv=128, slots=192),
        # a few drafted tokens per request
        dict(name="step drafted", op="step", dtype="f16", B=16, S=5, Hk=16, Hv=16, Dk=64, Dv=128, slots=16),
        # the block's norm over a long batch of tokens
        dict(name="ln fwd", op="ln_fwd", dtype="bf16", N=16384, D=5120, wdtype="bf16"),
        # the norm of single heads, parameters kept in FP32
        dict(name="ln fwd heads", op="ln_fwd", dtype="f16", N=8191, D=128, wdtype="f32"),
        # the block's norm, backward
        dict(name="ln bwd", op="ln_bwd", dtype="bf16", N=8192, D=4096, wdtype="bf16"),
        # few rows of an odd size
        dict(name="ln bwd odd", op="ln_bwd", dtype="f32", N=333, D=1001, wdtype="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "step", "step", "ln_fwd", "ln_bwd"])
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    if op in ("ln_fwd", "ln_bwd"):
        D = rng.choice([rng.randint(32, 8192), 128, 2048, 4096, 5120])
        top = (16384 * 5120 if op == "ln_fwd" else 8192 * 4096) * 2 // SIZE[dtype]
        return dict(op=op, dtype=dtype, N=_log(rng, 1, max(1, min(65536, top // D))), D=D,
                    wdtype=rng.choice([dtype, "f32"]))
    Hk = rng.choice([1, 2, 4, 8, 16])
    Hv = Hk * rng.choice([1, 2, 4] if Hk < 16 else [1, 2])
    Dk = rng.choice([128, 128, 64, rng.randint(2, 16) * 8])
    Dv = rng.choice([128, 128, 64, rng.randint(2, 16) * 8])
    if op == "step":
        B = _log(rng, 1, 128)
        S = rng.choice([1, 1, 1, rng.randint(2, 6)])
        if S > 1:
            B = min(B, 32)
        return dict(op=op, dtype=dtype, B=B, S=S, Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, slots=B + rng.choice([0, B // 2]))
    tokens = _log(rng, 20, (65536 if op == "fwd" else 8192) * 16 // Hv)
    tokens = min(tokens, 16384 if op == "fwd" else 4096)
    B = min(tokens, rng.choice([1, 1, 2, 4]))
    L = max(1, tokens // B)
    return dict(op=op, dtype=dtype, B=B, L=L, Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv,
                seqs=rng.choice([0, 0, min(L, rng.randint(1, 9))]), state=rng.random() < 0.4)


def work(case):
    c, e = case, SIZE[case["dtype"]]
    if c["op"] in ("ln_fwd", "ln_bwd"):
        w = SIZE[c["wdtype"]]
        if c["op"] == "ln_fwd":
            return {"bytes": 2 * c["N"] * c["D"] * e + 2 * c["D"] * w, "flops": 8 * c["N"] * c["D"]}
        return {"bytes": 3 * c["N"] * c["D"] * e + 3 * c["D"] * w, "flops": 16 * c["N"] * c["D"]}
    T = c["B"] * (c["S"] if c["op"] == "step" else c["L"])
    qk, vo, gates = T * c["Hk"] * c["Dk"] * e, T * c["Hv"] * c["Dv"] * e, T * c["Hv"] * (4 + e)
    state = c["B"] * c["Hv"] * c["Dk"] * c["Dv"] * 4
    flops = 6 * T * c["Hv"] * c["Dk"] * c["Dv"]
    if c["op"] == "step":
        return {"bytes": 2 * qk + 2 * vo + gates + 2 * state, "flops": flops}
    ids = 4 * T if c["seqs"] else 0
    if c["op"] == "fwd":
        return {"bytes": 2 * qk + 2 * vo + gates + ids + state * (2 if c["state"] else 1), "flops": flops}
    # backward: the inputs and dout read, five gradients written; the state recomputed and its gradient carried back
    return {"bytes": 4 * qk + 3 * vo + 2 * gates + ids + state * (3 if c["state"] else 0), "flops": 3 * flops}


# ---------------------------------------------------------------- inputs

def _gates(gen, shape, dtype):
    """Log decays -A softplus(a) with a rate A per head, and write strengths sigmoid(b)."""
    H = shape[-1]
    A = torch.rand(H, generator=gen, device="cuda") * 15.9 + 0.1
    dt = torch.exp(torch.rand(H, generator=gen, device="cuda") * math.log(100.0) + math.log(1e-3))
    bias = dt + torch.log(-torch.expm1(-dt))  # softplus(bias) = dt
    a = torch.randn(shape, generator=gen, device="cuda")
    g = -A * torch.nn.functional.softplus(0.5 * a + bias)
    beta = torch.sigmoid(torch.randn(shape, generator=gen, device="cuda"))
    return g, beta.to(dtype)


def _qkv(gen, B, T, Hk, Hv, Dk, Dv, dtype):
    """q, k, v as views of one [B, T, channels] buffer, as they leave a channel-last convolution; q and k of unit length."""
    n = Hk * Dk
    x = torch.randn((B, T, 2 * n + Hv * Dv), generator=gen, device="cuda")
    x = x * torch.sigmoid(x)
    qk = x[..., :2 * n].unflatten(-1, (2 * Hk, Dk))
    qk = qk * torch.rsqrt((qk * qk).sum(-1, keepdim=True) + 1e-6)
    x = torch.cat([qk.flatten(-2), x[..., 2 * n:]], -1).to(dtype)
    return (x[..., :n].unflatten(-1, (Hk, Dk)), x[..., n:2 * n].unflatten(-1, (Hk, Dk)),
            x[..., 2 * n:].unflatten(-1, (Hv, Dv)))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c, dt, st = case, DT[case["dtype"]], {"case": dict(case)}
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    if c["op"] in ("ln_fwd", "ln_bwd"):
        shift = randn(1, c["D"])  # channels have means of their own, as a residual stream has
        st["x"] = (randn(c["N"], c["D"]) * 1.5 + shift).to(dt)
        st["weight"] = (1 + 0.2 * randn(c["D"])).to(DT[c["wdtype"]])
        st["bias"] = (0.2 * randn(c["D"])).to(DT[c["wdtype"]])
        if c["op"] == "ln_bwd":
            st["dout"] = randn(c["N"], c["D"]).to(dt)
        return st
    B, Hv, Dk, Dv = c["B"], c["Hv"], c["Dk"], c["Dv"]
    T = c["S"] if c["op"] == "step" else c["L"]
    st["q"], st["k"], st["v"] = _qkv(gen, B, T, c["Hk"], Hv, Dk, Dv, dt)
    st["g"], st["beta"] = _gates(gen, (B, T, Hv), dt)
    if c["op"] == "step":
        st["state"] = 0.3 * randn(c["slots"], Hv, Dk, Dv)
        st["slots"] = torch.randperm(c["slots"], generator=gen, device="cuda")[:B].to(torch.int32)
        return st
    st["seq_idx"] = st["init"] = st["dout"] = st["dfinal"] = None
    if c["seqs"]:
        # each row holds `seqs` documents of random lengths
        cuts = torch.rand((B, c["L"]), generator=gen, device="cuda").argsort(1)[:, :max(0, min(c["seqs"], c["L"]) - 1)]
        st["seq_idx"] = torch.zeros((B, c["L"]), device="cuda").scatter_(1, cuts, 1.0).cumsum(1).to(torch.int32)
    if c["state"]:
        st["init"] = 0.3 * randn(B, Hv, Dk, Dv)
    if c["op"] == "bwd":
        st["dout"] = randn(B, c["L"], Hv, Dv).to(dt)
        if c["state"]:
            st["dfinal"] = 0.3 * randn(B, Hv, Dk, Dv)
    return st


# ---------------------------------------------------------------- plain forms (FP32)

def _chunked(st):
    """The sequence in chunks: [B, Hv, n, CHUNK, .] tensors, the padding with k = v = beta = g = 0."""
    Hv, Hk = st["v"].shape[2], st["q"].shape[2]
    L = st["v"].shape[1]
    pad = -L % CHUNK
    n = (L + pad) // CHUNK

    def cut(x):
        x = x.float().movedim(2, 1)
        if pad:
            x = torch.cat([x, x.new_zeros(x.shape[:2] + (pad,) + x.shape[3:])], 2)
        return x.unflatten(2, (n, CHUNK))

    q, k = (cut(x).repeat_interleave(Hv // Hk, 1) for x in (st["q"], st["k"]))
    v, g, beta = cut(st["v"]), cut(st["g"]), cut(st["beta"])
    G = g.cumsum(-1)
    gam = torch.exp((G[..., :, None] - G[..., None, :]).tril()).tril()
    gi, gc, ga = torch.exp(G), torch.exp(G[..., -1:] - G), torch.exp(G[..., -1])
    if st["seq_idx"] is not None:
        # ids that count the changes; a term crosses no change
        s = st["seq_idx"]
        new = torch.cat([torch.zeros_like(s[:, :1]), (s[:, 1:] != s[:, :-1]).to(s.dtype)], 1)
        if pad:
            new = torch.cat([new, new.new_zeros(new.shape[0], pad)], 1)
        ids = new.unflatten(1, (n, CHUNK)).cumsum(-1)[:, None]
        gam = gam * (ids[..., :, None] == ids[..., None, :])
        gi = gi * (ids == 0)
        gc = gc * (ids == ids[..., -1:])
        ga = ga * (ids[..., -1] == 0)
    kk, qk = k @ k.mT, q @ k.mT
    low = (beta[..., :, None] * gam * kk).tril(-1)
    return q, k, v, beta, gam, gi, gc, ga, kk, qk, low


def _unit_lower_inverse(low):
    """(I + low)^-1 by doubling the inverted diagonal blocks: [A 0; C D]^-1 = [A' 0; -D'CA' D']."""
    T = torch.eye(CHUNK, device=low.device).expand(low.shape).contiguous()
    s = 1
    while s < CHUNK:
        m = CHUNK // (2 * s)
        idx = torch.arange(m, device=low.device)
        Tb = T.unflatten(-1, (m, 2 * s)).unflatten(-3, (m, 2 * s))  # [..., m, 2s, m, 2s]
        Lb = low.unflatten(-1, (m, 2 * s)).unflatten(-3, (m, 2 * s))
        blk, lb = Tb[..., idx, :, idx, :], Lb[..., idx, :, idx, :]  # [m, ..., 2s, 2s]
        new = blk.clone()
        new[..., s:, :s] = -blk[..., s:, s:] @ lb[..., s:, :s] @ blk[..., :s, :s]
        Tb[..., idx, :, idx, :] = new
        s *= 2
    return T


def _join(x, L):
    return x.flatten(2, 3)[:, :, :L].movedim(1, 2)


def _state0(st):
    B, L, Hv, Dv = st["v"].shape
    if st["init"] is not None:
        return st["init"]
    return torch.zeros((B, Hv, st["q"].shape[3], Dv), device="cuda")


def _plain_fwd(st):
    q, k, v, beta, gam, gi, gc, ga, kk, qk, low = _chunked(st)
    scale = q.shape[-1] ** -0.5
    T = _unit_lower_inverse(low) * beta[..., None, :]
    w, u0 = T @ (gi[..., None] * k), T @ v
    P = scale * gam * qk
    qg, kg = scale * gi[..., None] * q, gc[..., None] * k
    S = _state0(st)
    out = torch.empty_like(v)
    for c in range(v.shape[2]):
        u = u0[:, :, c] - w[:, :, c] @ S
        out[:, :, c] = qg[:, :, c] @ S + P[:, :, c] @ u
        S = ga[:, :, c, None, None] * S + kg[:, :, c].mT @ u
    return _join(out, st["v"].shape[1]).to(st["v"].dtype), S


def _plain_bwd(st):
    q, k, v, beta, gam, gi, gc, ga, kk, qk, low = _chunked(st)
    n, scale = q.shape[2], q.shape[-1] ** -0.5
    T = _unit_lower_inverse(low)
    P = gam * qk
    dO = scale * st["dout"].float().movedim(2, 1)
    if n * CHUNK > dO.shape[2]:
        dO = torch.cat([dO, dO.new_zeros(dO.shape[:2] + (n * CHUNK - dO.shape[2], dO.shape[3]))], 2)
    dO = dO.unflatten(2, (n, CHUNK))
    S0 = torch.empty(v.shape[:3] + (k.shape[-1], v.shape[-1]), device=v.device)
    D1 = torch.empty_like(S0)
    U, dR, E = torch.empty_like(v), torch.empty_like(v), torch.empty_like(v)
    S = _state0(st)
    for c in range(n):
        S0[:, :, c] = S
        E[:, :, c] = v[:, :, c] - gi[:, :, c, :, None] * (k[:, :, c] @ S)
        U[:, :, c] = T[:, :, c] @ (beta[:, :, c, :, None] * E[:, :, c])
        S = ga[:, :, c, None, None] * S + (gc[:, :, c, :, None] * k[:, :, c]).mT @ U[:, :, c]
    D = torch.zeros_like(S) if st["dfinal"] is None else st["dfinal"]
    for c in reversed(range(n)):
        D1[:, :, c] = D
        dU = P[:, :, c].mT @ dO[:, :, c] + gc[:, :, c, :, None] * (k[:, :, c] @ D)
        dR[:, :, c] = T[:, :, c].mT @ dU
        X = (beta[:, :, c] * gi[:, :, c])[..., None] * dR[:, :, c]
        D = ga[:, :, c, None, None] * D + (gi[:, :, c, :, None] * q[:, :, c]).mT @ dO[:, :, c] - k[:, :, c].mT @ X
    dv = beta[..., None] * dR
    X = gi[..., None] * dv
    dP = (dO @ U.mT).tril()
    dL = -(dR @ U.mT).tril(-1)
    DP, DL = dP * gam, dL * beta[..., None] * gam
    dq0 = gi[..., None] * (dO @ S0.mT)
    KD = gc[..., None] * (k @ D1)
    KS = k @ S0
    dq = dq0 + DP @ k
    dk = gc[..., None] * (U @ D1.mT) - X @ S0.mT + DP.mT @ q + (DL + DL.mT) @ k
    dbeta = (dR * E).sum(-1) + (dL * gam * kk).sum(-1)
    MP, ML = dP * P, dL * low
    dG = (q * dq0).sum(-1) - (X * KS).sum(-1) - (U * KD).sum(-1) + (MP + ML).sum(-1) - (MP + ML).sum(-2)
    # what the last token's cumulative decay multiplies: the carried state and every later write
    dG[..., -1] += (U * KD).sum((-1, -2)) + ga * (S0 * D1).sum((-1, -2))
    dg = dG.flip(-1).cumsum(-1).flip(-1)
    L, Hk = st["v"].shape[1], st["q"].shape[2]
    group = lambda x: x.unflatten(1, (Hk, -1)).sum(2)  # noqa: E731
    dt = st["v"].dtype
    return [_join(group(dq), L).to(dt), _join(group(dk), L).to(dt), _join(dv, L).to(dt), _join(dg, L),
            _join(dbeta, L).to(dt)] + ([D] if st["init"] is not None else [])


def _plain_step(st):
    Hv, Hk = st["v"].shape[2], st["q"].shape[2]
    q, k = (st[n].float().repeat_interleave(Hv // Hk, 2) for n in ("q", "k"))
    v, beta, a = st["v"].float(), st["beta"].float(), torch.exp(st["g"])
    scale = q.shape[-1] ** -0.5
    slots = st["slots"].long()
    S = st["state"][slots]
    out = torch.empty_like(v)
    for t in range(v.shape[1]):
        S = S * a[:, t, :, None, None]
        u = beta[:, t, :, None] * (v[:, t] - (k[:, t, :, :, None] * S).sum(-2))
        S = S + k[:, t, :, :, None] * u[:, :, None, :]
        out[:, t] = scale * (q[:, t, :, :, None] * S).sum(-2)
    st["state"][slots] = S
    return out.to(st["v"].dtype)


def _plain_ln_fwd(st):
    x = st["x"].float()
    xc = x - x.mean(-1, keepdim=True)
    y = xc * torch.rsqrt((xc * xc).mean(-1, keepdim=True) + 1e-5)
    return (y * st["weight"].float() + st["bias"].float()).to(st["x"].dtype)


def _plain_ln_bwd(st):
    x, dy, w = st["x"].float(), st["dout"].float(), st["weight"]
    xc = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((xc * xc).mean(-1, keepdim=True) + 1e-5)
    xh = xc * r
    d = dy * w.float()
    dx = r * (d - d.mean(-1, keepdim=True) - xh * (d * xh).mean(-1, keepdim=True))
    return [dx.to(st["x"].dtype), (dy * xh).sum(0).to(w.dtype), dy.sum(0).to(w.dtype)]


# ---------------------------------------------------------------- one pass

def run(st):
    op = st["case"]["op"]
    if not own:
        if op == "step":
            out = _plain_step(st)
            return [out, st["state"]]
        plain = {"fwd": _plain_fwd, "bwd": _plain_bwd, "ln_fwd": _plain_ln_fwd, "ln_bwd": _plain_ln_bwd}[op]
        return plain(st)
    import causal_depthwise_conv1d_gb300 as ccv
    if op == "fwd":
        return ccv.gated_delta_rule_fwd(st["q"], st["k"], st["v"], st["g"], st["beta"], seq_idx=st["seq_idx"],
                                        initial_state=st["init"], return_final_state=True)
    if op == "bwd":
        grads = ccv.gated_delta_rule_bwd(st["q"], st["k"], st["v"], st["g"], st["beta"], st["dout"],
                                         seq_idx=st["seq_idx"], initial_state=st["init"],
                                         dfinal_state=st["dfinal"],
                                         return_dinitial_state=st["init"] is not None)
        return list(grads[:5]) + ([grads[5]] if st["init"] is not None else [])
    if op == "step":
        out = ccv.gated_delta_rule_step(st["q"], st["k"], st["v"], st["g"], st["beta"], st["state"],
                                        state_indices=st["slots"])
        return [out, st["state"]]
    if op == "ln_fwd":
        return ccv.layer_norm_fwd(st["x"], st["weight"], st["bias"])
    return list(ccv.layer_norm_bwd(st["x"], st["weight"], st["dout"], st["bias"]))


# ---------------------------------------------------------------- FP64, token by token

def _resets(st):
    """[B, L] 1.0 where the state is carried into token t, 0.0 where a new sequence begins."""
    B, L = st["v"].shape[:2]
    keep = torch.ones((B, L), dtype=torch.float64, device="cuda")
    if st.get("seq_idx") is not None:
        keep[:, 1:] = (st["seq_idx"][:, 1:] == st["seq_idx"][:, :-1]).double()
    return keep


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op in ("ln_fwd", "ln_bwd"):
        x, w, b = (st[n].double() for n in ("x", "weight", "bias"))
        D = x.shape[1]
        mean = x.sum(1, keepdim=True) / D
        var = ((x - mean) ** 2).sum(1, keepdim=True) / D
        n = (x - mean) / torch.sqrt(var + 1e-5)
        if op == "ln_fwd":
            return n * w + b
        dy = st["dout"].double()
        dn = dy * w
        dx = (dn - dn.sum(1, keepdim=True) / D - n * ((dn * n).sum(1, keepdim=True) / D)) / torch.sqrt(var + 1e-5)
        return [dx, (dy * n).sum(0), dy.sum(0)]
    rep = case["Hv"] // case["Hk"]
    q, k = (st[n].double().repeat_interleave(rep, 2) for n in ("q", "k"))
    v, beta, a = st["v"].double(), st["beta"].double(), torch.exp(st["g"].double())
    T, scale = v.shape[1], 1.0 / math.sqrt(case["Dk"])
    out = torch.empty_like(v)

    def token(S, t, keep=None):
        """Decayed state, prediction, write, new state."""
        A = S * (a[:, t] if keep is None else a[:, t] * keep[:, t, None])[..., None, None]
        p = torch.matmul(k[:, t, :, None, :], A)[:, :, 0]
        u = beta[:, t, :, None] * (v[:, t] - p)
        return A, p, u, A + k[:, t, :, :, None] * u[:, :, None, :]

    if op == "step":
        state = st["state"].double()
        S = state[st["slots"].long()]
        for t in range(T):
            S = token(S, t)[3]
            out[:, t] = scale * torch.matmul(q[:, t, :, None, :], S)[:, :, 0]
        state[st["slots"].long()] = S
        return [out, state]
    keep = _resets(st)
    S = st["init"].double() if st["init"] is not None else \
        torch.zeros((v.shape[0], v.shape[2], case["Dk"], case["Dv"]), dtype=torch.float64, device="cuda")
    if op == "fwd":
        for t in range(T):
            S = token(S, t, keep)[3]
            out[:, t] = scale * torch.matmul(q[:, t, :, None, :], S)[:, :, 0]
        return out, S
    if S.numel() * T * 8 > 80e9:
        return None
    hist = torch.empty((T,) + tuple(S.shape), dtype=torch.float64, device="cuda")
    for t in range(T):
        hist[t] = S
        S = token(S, t, keep)[3]
    dS = torch.zeros_like(S) if st["dfinal"] is None else st["dfinal"].double()
    dq, dk, dv, dg, dbeta = (torch.zeros_like(x) for x in (q, k, v, a, a))
    dout = st["dout"].double() * scale
    for t in reversed(range(T)):
        A, p, u, S1 = token(hist[t], t, keep)
        dq[:, t] = torch.matmul(S1, dout[:, t, :, :, None])[..., 0]
        dS = dS + q[:, t, :, :, None] * dout[:, t, :, None, :]
        du = torch.matmul(k[:, t, :, None, :], dS)[:, :, 0]
        dk[:, t] = torch.matmul(dS, u[..., None])[..., 0]
        dbeta[:, t] = (du * (v[:, t] - p)).sum(-1)
        dv[:, t] = beta[:, t, :, None] * du
        dk[:, t] -= torch.matmul(A, dv[:, t, :, :, None])[..., 0]
        dA = dS - k[:, t, :, :, None] * dv[:, t, :, None, :]
        dg[:, t] = (dA * A).sum((-1, -2))
        dS = dA * (a[:, t] * keep[:, t, None])[..., None, None]
    shared = lambda x: x.unflatten(2, (case["Hk"], rep)).sum(3)  # noqa: E731
    return [shared(dq), shared(dk), dv, dg, dbeta] + ([dS] if st["init"] is not None else [])
