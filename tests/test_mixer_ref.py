"""The FP64 references themselves: the gradients against automatic
differentiation of the definition and against differences; an FP32 run of the
definition stays inside the bounds."""
import pytest
import torch

from tests import mixer_ref as ref


@pytest.mark.parametrize("size,seqs,state", [((2, 7, 1, 2, 5, 3), 0, True), ((1, 70, 2, 2, 4, 6), 3, True),
                                             ((1, 66, 1, 3, 8, 4), 0, False), ((1, 1, 1, 1, 3, 2), 0, True)])
def test_gradients_of_the_definition(size, seqs, state):
    c = ref.gdr_inputs(1, *size, "f32", seqs=seqs, state=state, grads=True)
    auto, mine = ref.gdr_autograd(c), ref.gdr_bwd(c)
    assert set(mine) == {"d" + n for n in auto}
    for n, d in auto.items():
        assert torch.allclose(mine["d" + n][0], d, rtol=1e-11, atol=1e-12), n


def test_gradients_against_differences():
    c = ref.gdr_inputs(2, 1, 9, 1, 2, 4, 3, "f32", state=True, grads=True)
    names = ("q", "k", "v", "g", "beta", "initial_state")
    d = ref.gdr_bwd(c)

    def loss(n, delta):
        x = {m: c[m].double() + (delta if m == n else 0) for m in names}
        o, s, _, _ = ref.gdr(x["q"], x["k"], x["v"], x["g"], x["beta"], None, x["initial_state"])
        return float((o * c["dout"].double()).sum() + (s * c["dfinal_state"].double()).sum())

    for n in names:
        gen = torch.Generator().manual_seed(4)
        way = torch.randn(c[n].shape, generator=gen, dtype=torch.float64)
        h = 1e-6
        assert abs((loss(n, h * way) - loss(n, -h * way)) / (2 * h) - float((way * d["d" + n][0]).sum())) < 1e-6, n


def test_an_fp32_run_stays_inside_the_bounds():
    c = ref.gdr_inputs(3, 1, 80, 1, 1, 32, 16, "f32", state=True)
    o, s, eo, es = ref.gdr(c["q"], c["k"], c["v"], c["g"], c["beta"], None, c["initial_state"])
    S, out = c["initial_state"].clone(), []
    for t in range(80):
        S = S * torch.exp(c["g"][:, t])[..., None, None]
        u = c["beta"][:, t, :, None] * (c["v"][:, t] - torch.einsum("bhk,bhkv->bhv", c["k"][:, t], S))
        S = S + c["k"][:, t, :, :, None] * u[:, :, None, :]
        out.append(32 ** -0.5 * torch.einsum("bhk,bhkv->bhv", c["q"][:, t], S))
    assert ref.worst(torch.stack(out, 1), o, eo) <= 1 and ref.worst(S, s, es) <= 1
    # and the bounds are of use: far below the values
    assert float(es.max()) < 1e-3 * float(s.abs().max())


def test_layer_norm_gradients():
    gen = torch.Generator().manual_seed(5)
    x, w, b, dy = (torch.randn(s, generator=gen, dtype=torch.float64, requires_grad=r)
                   for s, r in (((6, 9), True), ((9,), True), ((9,), True), ((6, 9), False)))
    y, _, _ = ref.ln_fwd(x, w, b)
    auto = torch.autograd.grad((y * dy).sum(), (x, w, b))
    for p, d in zip(ref.ln_bwd(x.detach(), w.detach(), dy), auto):
        assert torch.allclose(p, d, rtol=1e-10, atol=1e-12)
    n = torch.nn.functional.layer_norm(x.detach(), (9,), w.detach(), b.detach())
    assert torch.allclose(y.detach(), n, rtol=1e-12, atol=1e-12)
