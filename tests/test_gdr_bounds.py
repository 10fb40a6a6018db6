"""The gradients' error bounds: below the gradients themselves at any length, above an FP32 run's errors, and
small enough that a wrong gradient does not pass."""
import pytest
import torch

from tests import gdr_bounds, mixer_ref as ref

CASES = [((1, 200, 1, 1, 128, 128), 0, False), ((1, 513, 1, 1, 128, 16), 0, False), ((2, 150, 1, 2, 128, 64), 4, True),
         ((1, 129, 2, 2, 72, 100), 0, False), ((1, 63, 2, 2, 128, 128), 0, True)]


def rms(x):
    return float(x.pow(2).mean().sqrt())


@pytest.mark.parametrize("size,seqs,state", CASES, ids=str)
def test_bounds_are_of_use(size, seqs, state):
    c = ref.gdr_inputs(21, *size, "f32", seqs=seqs, state=state, grads=True)
    old = ref.gdr_bwd(c)
    gen = torch.Generator().manual_seed(8)
    for n, (e, bound) in gdr_bounds.gdr_bwd(c).items():
        assert torch.allclose(e, old[n][0], rtol=1e-11, atol=1e-12), n
        assert rms(bound.expand_as(e)) < (0.1 if n == "dg" else 0.02) * rms(e), n
        assert ref.worst(torch.zeros_like(e), e, bound) > 1, n
        # an eighth of the tokens missing; noise of a tenth of the gradients' size
        bad = e.clone()
        bad[:, :e.shape[1] // 8 or 1] = 0
        assert ref.worst(bad, e, bound) > 1, n
        noise = torch.randn(e.shape, generator=gen, dtype=torch.float64)
        assert ref.worst(e + 0.1 * rms(e) * noise, e, bound) > 1, n


def fp32_run(c):
    """The definition in FP32, its gradients by automatic differentiation."""
    names = ["q", "k", "v", "g", "beta"] + (["initial_state"] if c["initial_state"] is not None else [])
    leaf = {n: c[n].float().clone().requires_grad_() for n in names}
    rep = c["v"].shape[2] // c["q"].shape[2]
    q, k = (leaf[n].repeat_interleave(rep, 2) for n in ("q", "k"))
    keep = ref._keep(c["seq_idx"], *c["v"].shape[:2]).float()
    S = leaf["initial_state"] if "initial_state" in leaf else \
        torch.zeros(c["v"].shape[0], c["v"].shape[2], q.shape[3], c["v"].shape[3])
    loss = 0.0
    for t in range(q.shape[1]):
        S = S * (torch.exp(leaf["g"][:, t]) * keep[:, t, None])[..., None, None]
        u = leaf["beta"][:, t, :, None] * (leaf["v"][:, t] - torch.einsum("bhk,bhkv->bhv", k[:, t], S))
        S = S + k[:, t, :, :, None] * u[:, :, None, :]
        loss = loss + (q.shape[3] ** -0.5 * torch.einsum("bhk,bhkv->bhv", q[:, t], S) * c["dout"][:, t].float()).sum()
    if c["dfinal_state"] is not None:
        loss = loss + (S * c["dfinal_state"]).sum()
    return dict(zip(("d" + n for n in names), torch.autograd.grad(loss, [leaf[n] for n in names])))


@pytest.mark.parametrize("size,seqs,state", CASES, ids=str)
def test_an_fp32_run_stays_inside(size, seqs, state):
    c = ref.gdr_inputs(22, *size, "f32", seqs=seqs, state=state, grads=True)
    got = fp32_run(c)
    for n, (e, bound) in gdr_bounds.gdr_bwd(c).items():
        assert ref.worst(got[n], e, bound) <= 1, n
