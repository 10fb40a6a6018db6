"""The FP64 references of the recurrence and of group norm against independent forms (CPU)."""
import pytest
import torch

from tests import rec_ref as ref


@pytest.mark.parametrize("seqs,state", [(0, False), (3, True), (0, True)])
def test_gradients_against_autograd(seqs, state):
    c = ref.glr_inputs(1, 2, 40, 7, "f32", seqs=seqs, state=state, grads=True)
    want = ref.glr_autograd(c)
    for n, d in ref.glr_bwd(c).items():
        if n in want:
            assert float((d[0] - want[n]).abs().max()) < 1e-9 * (1 + float(want[n].abs().max())), n


def test_bounds_stay_useful():
    c = ref.glr_inputs(2, 2, 600, 16, "f32", state=True, grads=True)
    fw = ref.glr(c)
    for n in ("out", "final_state", "chunk_states"):
        assert float(fw[n][1].max() / fw[n][0].square().mean().sqrt()) < 1e-2, n
    for n, (v, e) in ref.glr_bwd(c).items():
        # drate adds 1200 tokens' worst cases, with states that last up to a thousand tokens
        assert float(e.max() / v.square().mean().sqrt()) < (0.25 if n == "drate" else 2e-2), n


def test_recurrence_by_hand():
    c = ref.glr_inputs(3, 1, 3, 1, "f32", state=True)
    p, q, x = (c[n].double().flatten() for n in ("decay_gate", "input_gate", "x"))
    h = float(c["initial_state"])
    for t in range(3):
        a = float(torch.exp(-c["rate"].double() * torch.sigmoid(p[t])))
        h = a * h + (1 - a * a) ** 0.5 * float(torch.sigmoid(q[t])) * float(x[t])
        assert abs(float(ref.glr(c)["out"][0][0, t, 0]) - h) < 1e-12


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("N,S,C,G", [(2, 5, 12, 3), (4, 1, 8, 2), (1, 9, 6, 6)])
def test_group_norm_against_the_framework(N, S, C, G, silu):
    x, w, b, dy = ref.gn_inputs(4, N, S, C, "f32", "f32")
    leaf = [t.double().requires_grad_() for t in (x, w, b)]
    y = torch.nn.functional.group_norm(leaf[0].transpose(1, 2), G, leaf[1], leaf[2], 1e-5).transpose(1, 2)
    y = torch.nn.functional.silu(y) if silu else y
    assert float((y - ref.gn_fwd(x, G, w, b, silu=silu)[0]).abs().max()) < 1e-10
    grads = torch.autograd.grad((y * dy.double()).sum(), leaf)
    for n, d in zip(("dx", "dweight", "dbias"), grads):
        assert float((ref.gn_bwd(x, G, w, dy, b, silu=silu)[n][0] - d).abs().max()) < 1e-9, n
