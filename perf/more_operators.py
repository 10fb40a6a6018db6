"""Performance cases of the gated linear recurrence (whole sequences, its
backward pass, its step for single tokens) and of group normalisation with an
activation, channels last (forward and backward).

Gated linear recurrence, per channel with a state h (zero, or the given initial
state; back to zero where seq_idx changes), gate logits p (decay) and q (input),
rate >= 0:

    a_t = exp(-rate sigmoid(p_t));   h <- a_t h + sqrt(1 - a_t^2) sigmoid(q_t) x_t;   out_t = h

Group norm of x [N, S, C]: mean and variance over the S positions and C / G
channels of a group, weight and bias per channel, then the activation.  S = 1
is the norm of each token's heads.

``run`` computes either the plain form (torch operations in FP32, rounded once
at the end) or, with ``own`` set, calls the package's operators.  ``exact``
follows the definitions in FP64, the recurrence token by token.
"""
import math

import torch

own = False

CHUNK = 64  # tokens between two states that a forward pass keeps for its backward pass
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one long prompt: few channels to split, a long axis; the final state goes to the cache
        dict(name="rec fwd prompt", op="fwd", dtype="bf16", B=1, L=8192, C=5120, seqs=0, state=False),
        # a training batch, each row packed with documents
        dict(name="rec fwd training batch", op="fwd", dtype="bf16", B=8, L=2048, C=5120, seqs=5, state=False),
        # a short ragged continuation in FP32 from a cached state, an odd number of channels
        dict(name="rec fwd short f32", op="fwd", dtype="f32", B=3, L=77, C=1001, seqs=0, state=True),
        # a training step's backward pass, the forward's states of every 64th token kept for it
        dict(name="rec bwd training", op="bwd", dtype="bf16", B=4, L=2048, C=4096, seqs=0, state=False, saved=True),
        # backward over an odd length with packed sequences and a state gradient, nothing kept from the forward
        dict(name="rec bwd ragged", op="bwd", dtype="f16", B=1, L=1001, C=512, seqs=3, state=True, saved=False),
        # one sequence's next token: latency
        dict(name="rec step one", op="step", dtype="bf16", B=1, S=1, C=5120, slots=1),
        # a serving batch's next tokens, states in a cache with more slots than requests
        dict(name="rec step batch", op="step", dtype="bf16", B=128, S=1, C=5120, slots=192),
        # the norm of every token's heads with SiLU over a long batch of tokens
        dict(name="gn fwd heads", op="gn_fwd", dtype="bf16", N=16384, S=1, C=5120, G=40, act="silu", wdtype="bf16"),
        # the norm over whole sequences, as behind a convolution, parameters kept in FP32
        dict(name="gn fwd sequences", op="gn_fwd", dtype="bf16", N=8, S=2048, C=5120, G=32, act="silu",
             wdtype="f32"),
        # few short sequences of groups that are no vector's multiple
        dict(name="gn fwd odd", op="gn_fwd", dtype="f32", N=3, S=77, C=1000, G=8, act=None, wdtype="f32"),
        # the heads' norm, backward
        dict(name="gn bwd heads", op="gn_bwd", dtype="f16", N=8192, S=1, C=4096, G=32, act="silu", wdtype="f32"),
        # the sequences' norm, backward
        dict(name="gn bwd sequences", op="gn_bwd", dtype="bf16", N=8, S=2048, C=4096, G=32, act="silu",
             wdtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "gn_fwd", "gn_fwd", "gn_bwd"])
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    if op in ("gn_fwd", "gn_bwd"):
        width = rng.choice([_log(rng, 4, 256), 8 * _log(rng, 1, 32), 64, 128])
        G = max(1, min(rng.choice([_log(rng, 1, 64), 8, 32]), 8192 // width))
        C = G * width
        rows = (16384 * 5120 if op == "gn_fwd" else 8192 * 4096) * 2 // SIZE[dtype] // C
        S = rng.choice([1, 1, _log(rng, 2, 4096)])
        return dict(op=op, dtype=dtype, N=_log(rng, 1, max(1, min(rows // S, 65536 if S == 1 else 64))), S=S, C=C,
                    G=G, act=rng.choice([None, "silu", "silu"]), wdtype=rng.choice([dtype, "f32"]))
    C = rng.choice([_log(rng, 64, 8192), 8 * _log(rng, 8, 1024), 1024, 4096, 5120])
    if op == "step":
        B, S = _log(rng, 1, 256), rng.choice([1, 1, 1, rng.randint(2, 6)])
        return dict(op=op, dtype=dtype, B=B, S=S, C=C, slots=B + rng.choice([0, B // 2]))
    most = (8 * 2048 * 5120 if op == "fwd" else 4 * 2048 * 4096) * 2 // SIZE[dtype] // C
    tokens = _log(rng, 20, min(most, 32768))
    B = min(tokens, rng.choice([1, 1, 2, 4, 8]))
    L = max(1, tokens // B)
    c = dict(op=op, dtype=dtype, B=B, L=L, C=C, seqs=rng.choice([0, 0, min(L, rng.randint(1, 9))]),
             state=rng.random() < 0.4)
    if op == "bwd":
        c["saved"] = rng.random() < 0.5
    return c


def work(case):
    c, e = case, SIZE[case["dtype"]]
    if c["op"] in ("gn_fwd", "gn_bwd"):
        n, w = c["N"] * c["S"] * c["C"], SIZE[c["wdtype"]]
        if c["op"] == "gn_fwd":
            return {"bytes": 2 * n * e + 2 * c["C"] * w, "flops": 12 * n}
        return {"bytes": 3 * n * e + 4 * c["C"] * w, "flops": 30 * n}
    T = c["B"] * (c["S"] if c["op"] == "step" else c["L"])
    stream, state, rate = T * c["C"] * e, c["B"] * c["C"] * 4, 4 * c["C"]
    if c["op"] == "step":
        return {"bytes": 4 * stream + 2 * state + rate, "flops": 25 * T * c["C"]}
    ids = 4 * T if c["seqs"] else 0
    if c["op"] == "fwd":
        return {"bytes": 4 * stream + rate + ids + state * (2 if c["state"] else 1), "flops": 25 * T * c["C"]}
    # the inputs and dout read, three gradients written, and what was kept of the forward pass
    kept = c["B"] * -(-c["L"] // CHUNK) * c["C"] * 4 if c["saved"] else 0
    return {"bytes": 7 * stream + 2 * rate + ids + kept + state * (3 if c["state"] else 0),
            "flops": 60 * T * c["C"]}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c, dt, st = case, DT[case["dtype"]], {"case": dict(case)}
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    if c["op"] in ("gn_fwd", "gn_bwd"):
        shape = (c["N"], c["C"]) if c["S"] == 1 else (c["N"], c["S"], c["C"])
        shift = randn(c["C"])  # channels have means of their own
        st["x"] = (randn(*shape) * 1.5 + shift).to(dt)
        st["weight"] = (1 + 0.2 * randn(c["C"])).to(DT[c["wdtype"]])
        st["bias"] = (0.2 * randn(c["C"])).to(DT[c["wdtype"]])
        if c["op"] == "gn_bwd":
            st["dout"] = randn(*shape).to(dt)
        return st
    B, C = c["B"], c["C"]
    T = c["S"] if c["op"] == "step" else c["L"]
    x = randn(B, T, C)
    st["x"] = (x * torch.sigmoid(x)).to(dt)  # as it leaves a convolution with SiLU
    # both gates' logits come from one projection: views of one buffer
    st["decay_gate"], st["input_gate"] = randn(B, T, 2 * C).to(dt).chunk(2, -1)
    # a fully open decay gate keeps 0.9 to 0.999 of an eighth of the state's logarithm
    st["rate"] = -8 * torch.log(0.9 + 0.099 * torch.rand(C, generator=gen, device="cuda"))
    if c["op"] == "step":
        st["state"] = 0.5 * randn(c["slots"], C)
        st["slots"] = torch.randperm(c["slots"], generator=gen, device="cuda")[:B].to(torch.int32)
        return st
    st["seq_idx"] = st["init"] = st["dout"] = st["dfinal"] = st["chunk_states"] = None
    if c["seqs"]:
        # each row holds `seqs` documents of random lengths
        cuts = torch.rand((B, T), generator=gen, device="cuda").argsort(1)[:, :max(0, min(c["seqs"], T) - 1)]
        st["seq_idx"] = torch.zeros((B, T), device="cuda").scatter_(1, cuts, 1.0).cumsum(1).to(torch.int32)
    if c["state"]:
        st["init"] = 0.5 * randn(B, C)
    if c["op"] == "bwd":
        st["dout"] = randn(B, T, C).to(dt)
        if c["state"]:
            st["dfinal"] = 0.5 * randn(B, C)
        if c["saved"]:
            # the state before every 64th token, which the training step's forward pass has left
            st["chunk_states"] = _scan(*_gates(st)[:2], st["init"])[1]
    return st


# ---------------------------------------------------------------- plain forms (FP32)

def _keep(st):
    """[B, L, 1] 1.0 where the state is carried into token t, 0.0 where a new sequence begins; or None."""
    if st.get("seq_idx") is None:
        return None
    s = st["seq_idx"]
    return torch.cat([torch.ones_like(s[:, :1]), (s[:, 1:] == s[:, :-1]).to(s.dtype)], 1)[..., None].float()


def _gates(st):
    """Carried decay, input, and the factors: a (0 across a new sequence), m i x, a, m, i, r, log a."""
    x, r, i = st["x"].float(), torch.sigmoid(st["decay_gate"].float()), torch.sigmoid(st["input_gate"].float())
    log_a = -st["rate"] * r
    a, m = torch.exp(log_a), torch.sqrt(-torch.expm1(2 * log_a))
    keep = _keep(st)
    return (a if keep is None else a * keep), m * i * x, a, m, i, r, log_a


def _scan(a, b, h):
    """h_t = a_t h_{t-1} + b_t: (all states, the states before every 64th token, the last state)."""
    B, L, C = a.shape
    n = -(-L // CHUNK)
    if n * CHUNK > L:
        a = torch.cat([a, a.new_ones(B, n * CHUNK - L, C)], 1)
        b = torch.cat([b, b.new_zeros(B, n * CHUNK - L, C)], 1)
    a, b = a.unflatten(1, (n, CHUNK)), b.unflatten(1, (n, CHUNK)).clone()
    P = a.clone()
    for t in range(1, CHUNK):  # inside all chunks at once
        b[:, :, t] += a[:, :, t] * b[:, :, t - 1]
        P[:, :, t] *= P[:, :, t - 1]
    h = a.new_zeros(B, C) if h is None else h
    first = a.new_empty(B, n, C)
    for c in range(n):
        first[:, c] = h
        h = P[:, c, -1] * h + b[:, c, -1]
    return (b + P * first[:, :, None]).flatten(1, 2)[:, :L], first, h


def _plain_fwd(st):
    a, b = _gates(st)[:2]
    h, _, last = _scan(a, b, st["init"])
    return h.to(st["x"].dtype), last


def _plain_bwd(st):
    carried, b, a, m, i, r, log_a = _gates(st)
    x, dt, init = st["x"].float(), st["x"].dtype, st["init"]
    h = _scan(carried, b, init)[0]
    before = torch.cat([torch.zeros_like(h[:, :1]) if init is None else init[:, None], h[:, :-1]], 1)
    keep = _keep(st)
    if keep is not None:
        before = before * keep
    # G_t = dout_t + a_{t+1} G_{t+1}, from the last token to the first
    shifted = torch.cat([carried[:, 1:], torch.ones_like(a[:, :1])], 1).flip(1)
    G = _scan(shifted, st["dout"].float().flip(1), st["dfinal"])[0].flip(1)
    W = a * before - torch.where(m > 0, i * x * a * a / m, torch.zeros_like(m))
    grads = [(G * m * i).to(dt), (G * W * log_a * (1 - r)).to(dt), (G * b * (1 - i)).to(dt), -(G * W * r).sum((0, 1))]
    return grads + ([carried[:, 0] * G[:, 0]] if init is not None else [])


def _plain_step(st):
    a, b = _gates(st)[:2]
    slots = st["slots"].long()
    h = st["state"][slots]
    out = torch.empty_like(b)
    for t in range(b.shape[1]):
        h = a[:, t] * h + b[:, t]
        out[:, t] = h
    st["state"][slots] = h
    return [out.to(st["x"].dtype), st["state"]]


def _grouped(st):
    """Normalised x as [N, S, G, width], its rstd, weight and bias as [G, width], all FP32."""
    c = st["case"]
    x = st["x"].float().view(c["N"], c["S"], c["G"], -1)
    w, b = (st[n].float().view(c["G"], -1) for n in ("weight", "bias"))
    xc = x - x.mean((1, 3), keepdim=True)
    rstd = torch.rsqrt((xc * xc).mean((1, 3), keepdim=True) + 1e-5)
    return xc * rstd, rstd, w, b


def _plain_gn_fwd(st):
    xh, _, w, b = _grouped(st)
    z = xh * w + b
    if st["case"]["act"]:
        z = z * torch.sigmoid(z)
    return z.view(st["x"].shape).to(st["x"].dtype)


def _plain_gn_bwd(st):
    xh, rstd, w, b = _grouped(st)
    dz = st["dout"].float().view(xh.shape)
    if st["case"]["act"]:
        z = xh * w + b
        s = torch.sigmoid(z)
        dz = dz * (s * (1 + z * (1 - s)))
    d = dz * w
    dx = rstd * (d - d.mean((1, 3), keepdim=True) - xh * (d * xh).mean((1, 3), keepdim=True))
    wt = st["weight"].dtype
    return [dx.view(st["x"].shape).to(st["x"].dtype), (dz * xh).sum((0, 1)).flatten().to(wt),
            dz.sum((0, 1)).flatten().to(wt)]


# ---------------------------------------------------------------- one pass

def run(st):
    c = st["case"]
    op = c["op"]
    if not own:
        return {"fwd": _plain_fwd, "bwd": _plain_bwd, "step": _plain_step, "gn_fwd": _plain_gn_fwd,
                "gn_bwd": _plain_gn_bwd}[op](st)
    import causal_depthwise_conv1d_gb300 as ccv
    if op == "fwd":
        return ccv.gated_linear_recurrence_fwd(st["x"], st["decay_gate"], st["input_gate"], st["rate"],
                                               seq_idx=st["seq_idx"], initial_state=st["init"],
                                               return_final_state=True)
    if op == "bwd":
        grads = ccv.gated_linear_recurrence_bwd(st["x"], st["decay_gate"], st["input_gate"], st["rate"], st["dout"],
                                                seq_idx=st["seq_idx"], initial_state=st["init"],
                                                dfinal_state=st["dfinal"], chunk_states=st["chunk_states"],
                                                return_dinitial_state=st["init"] is not None)
        return list(grads[:4]) + ([grads[4]] if st["init"] is not None else [])
    if op == "step":
        out = ccv.gated_linear_recurrence_step(st["x"], st["decay_gate"], st["input_gate"], st["rate"], st["state"],
                                               state_indices=st["slots"])
        return [out, st["state"]]
    if op == "gn_fwd":
        return ccv.group_norm_fwd(st["x"], c["G"], st["weight"], st["bias"], activation=c["act"])
    return list(ccv.group_norm_bwd(st["x"], c["G"], st["weight"], st["dout"], st["bias"], activation=c["act"]))


# ---------------------------------------------------------------- FP64

def _exact_gn(st):
    c = st["case"]
    rows = c["N"] * c["S"]
    x, w, b = st["x"].double().reshape(c["N"], c["S"], c["C"]), st["weight"].double(), st["bias"].double()
    n = c["S"] * (c["C"] // c["G"])

    def mean(v):  # of each sample's groups, spread over their channels
        per = v.sum(1).unflatten(-1, (c["G"], -1)).sum(-1) / n
        return per.repeat_interleave(c["C"] // c["G"], -1)[:, None]

    xc = x - mean(x)
    std = torch.sqrt(mean(xc * xc) + 1e-5)
    xh = xc / std
    z = xh * w + b
    silu = c["act"] is not None
    s = 1 / (1 + torch.exp(-z))
    if c["op"] == "gn_fwd":
        return (z * s if silu else z).view(st["x"].shape)
    dz = st["dout"].double().view(x.shape)
    if silu:
        dz = dz * (s + z * s * (1 - s))
    d = dz * w
    dx = (d - mean(d) - xh * mean(d * xh)) / std
    return [dx.view(st["x"].shape), (dz * xh).view(rows, -1).sum(0), dz.view(rows, -1).sum(0)]


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op in ("gn_fwd", "gn_bwd"):
        return _exact_gn(st)
    x, p, q, rate = (st[n].double() for n in ("x", "decay_gate", "input_gate", "rate"))
    B, T, C = x.shape
    new = torch.zeros((B, T), dtype=torch.bool, device=x.device)
    if st.get("seq_idx") is not None:
        new[:, 1:] = st["seq_idx"][:, 1:] != st["seq_idx"][:, :-1]

    def token(t):
        """r, i, decay, input factor of token t."""
        r, i = 1 / (1 + torch.exp(-p[:, t])), 1 / (1 + torch.exp(-q[:, t]))
        return r, i, torch.exp(-rate * r), torch.sqrt(-torch.expm1(-2 * rate * r))

    if op == "step":
        state = st["state"].double()
        h = state[st["slots"].long()]
        out = torch.empty_like(x)
        for t in range(T):
            _, i, a, m = token(t)
            h = a * h + m * i * x[:, t]
            out[:, t] = h
        state[st["slots"].long()] = h
        return [out, state]
    h = st["init"].double() if st["init"] is not None else x.new_zeros(B, C)
    out = torch.empty_like(x)
    for t in range(T):
        _, i, a, m = token(t)
        h = torch.where(new[:, t, None], 0.0, h * a) + m * i * x[:, t]
        out[:, t] = h
    if op == "fwd":
        return out, h
    dx, dp, dq, drate = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), torch.zeros_like(rate)
    dh = st["dfinal"].double() if st["dfinal"] is not None else x.new_zeros(B, C)
    for t in reversed(range(T)):
        r, i, a, m = token(t)
        dh = dh + st["dout"][:, t].double()
        h = out[:, t - 1] if t > 0 else st["init"].double() if st["init"] is not None else torch.zeros_like(dh)
        h = torch.where(new[:, t, None], 0.0, h)
        dx[:, t] = dh * m * i
        dq[:, t] = dh * m * x[:, t] * i * (1 - i)
        # through the decay and through sqrt(1 - a^2), whose derivative to log a is -a^2 / m
        dlog = dh * (h * a - i * x[:, t] * a * a / m)
        dp[:, t] = -dlog * rate * r * (1 - r)
        drate -= (dlog * r).sum(0)
        dh = torch.where(new[:, t, None], 0.0, dh * a)
    return [dx, dp, dq, drate] + ([dh] if st["init"] is not None else [])
