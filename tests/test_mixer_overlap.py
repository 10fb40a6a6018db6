"""Outputs that share memory with another tensor are refused, and only those.

On the host: every call here is refused, by the pair under test or else by a second pair that is checked later, so
nothing is launched."""
import itertools
import random

import pytest

from tests.test_mixer_abi import F, bwd_args, gdr_args, ln_args, mx, status  # noqa: F401


def elements(base, strides, shape, size):
    """The bytes that a tensor touches."""
    return {base + size * sum(i * s for i, s in zip(idx, strides)) + b
            for idx in itertools.product(*map(range, shape)) for b in range(size)}


def test_gradients_interleaved_by_head(mx):  # noqa: F811
    """dq, dk, dv as the thirds of each head's row in one [B, L, H, 3 D] buffer."""
    L, H, D = 8, 4, 16
    st = (L * H * 3 * D, H * 3 * D, 3 * D, 1)
    part = dict(dq=7 * F, dk=7 * F + 2 * D, dv=7 * F + 4 * D, s_dq=st, s_dk=st, s_dv=st, Hk=H, Hv=H, Dk=D, Dv=D,
                s_q=(L * H * D, H * D, D, 1), s_k=(L * H * D, H * D, D, 1), s_v=(L * H * D, H * D, D, 1),
                s_dout=(L * H * D, H * D, D, 1))
    rc, msg = status(mx, "ccv_gdr_bwd", bwd_args(mx, dg=12 * F, **part))
    assert rc == 1 and "dg" in msg and "workspace" in msg  # past the three
    rc, msg = status(mx, "ccv_gdr_bwd", bwd_args(mx, dg=12 * F, **dict(part, dk=7 * F + 2 * D - 2)))
    assert rc == 1 and "dq must not alias or overlap dk" in msg


def test_norm_rows_shifted_by_one_column(mx):  # noqa: F811
    """x and out as columns 0.. and 1.. of one buffer share all but one column; 64.. shares none."""
    st = (160, 1)
    rc, msg = status(mx, "ccv_ln_fwd", ln_args(mx, x=F, xs=st, out=F + 2, os=st, w=F + 2, wdtype=2))
    assert rc == 1 and "out must not alias or overlap x" in msg
    rc, msg = status(mx, "ccv_ln_fwd", ln_args(mx, x=F, xs=st, out=F + 128, os=st, w=F + 128, wdtype=2))
    assert rc == 1 and "out must not alias or overlap weight" in msg


def layout(rng, shape):
    """Strides of a slice of a buffer of `shape` with its dimensions in any order, some padded or run backwards."""
    order, strides, step = list(range(len(shape))), [0] * len(shape), rng.choice([1, 1, 1, 2])
    rng.shuffle(order)
    for d in order:
        strides[d] = step
        step *= shape[d] + rng.choice([0, 0, 0, 1, 2, 3])
    return [s * (-1 if rng.random() < 0.1 else 1) for s in strides]


@pytest.mark.parametrize("seed", range(8))
def test_against_the_elements_themselves(mx, seed):  # noqa: F811
    rng = random.Random(seed)
    met = 0
    for _ in range(150):
        B, L, Hk, Dk, Dv = rng.randint(1, 3), rng.randint(1, 4), rng.randint(1, 2), rng.randint(1, 5), rng.randint(1, 5)
        Hv = Hk * rng.randint(1, 2)
        qs, os = layout(rng, (B, L, Hk, Dk)), layout(rng, (B, L, Hv, Dv))
        if rng.random() < 0.5:  # slices of one buffer
            qs[:2] = os[:2] = [s * 64 for s in layout(rng, (B, L))]
            qs[2:], os[2:] = layout(rng, (Hk, Dk)), layout(rng, (Hv, Dv))
        q, out = 2 * F, 2 * F + 4 * rng.randint(-60, 60)
        want = bool(elements(q, qs, (B, L, Hk, Dk), 2) & elements(out, os, (B, L, Hv, Dv), 2))
        big = (1000, 100, 20, 1)
        rc, msg = status(mx, "ccv_gdr_fwd", gdr_args(
            mx, q=q, qs=qs, out=out, os=os, g=out, gs=(100, 20, 1), k=30 * F, ks=big, v=40 * F,
            vs=big, beta=50 * F, bs=(100, 20, 1), B=B, L=L, Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv))
        assert rc == 1 and "out must not alias or overlap" in msg, msg
        got = msg.endswith("overlap q")
        assert got or msg.endswith("overlap g")
        assert got == want, (q - out, qs, os, (B, L, Hk, Hv, Dk, Dv))
        met += want
    assert 20 < met < 130
