"""The operators together: the example block's prefill, decode and training step."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU-only machines
    pytest.skip("needs a CUDA device", allow_module_level=True)

from examples import mixer_block as mb  # noqa: E402


def setup(dtype=torch.float32, L=160):
    block = mb.Block(dim=256, key_heads=2, value_heads=4, head=64, dtype=dtype)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((2, L, 256), generator=gen, device="cuda").to(dtype)
    return block, x, torch.randn((2, L, 256), generator=gen, device="cuda")


@pytest.mark.parametrize("dtype,bound", [(torch.float32, 1e-3), (torch.bfloat16, 0.15)])
def test_decoding_continues_a_prefill(dtype, bound):
    # outputs are of order 1; a bf16 token passes five roundings of 2^-9 on either path
    block, x, _ = setup(dtype)
    whole, (conv, state) = block.prefill(x)
    first, states = block.prefill(x[:, :150].contiguous())
    tail = torch.stack([block.decode(x[:, t], states) for t in range(150, 160)], 1)
    got = torch.cat([first, tail], 1)
    assert float((got.float() - whole.float()).abs().max()) < bound
    assert float((states[1] - state).abs().max()) < bound
    assert float((states[0].float() - conv.float()).abs().max()) < bound


def test_packed_sequences_equal_separate_ones():
    block, x, _ = setup()
    ids = torch.zeros((2, 160), dtype=torch.int32, device="cuda")
    ids[:, 70:] = 1
    whole, _ = block.prefill(x, seq_idx=ids)
    a, _ = block.prefill(x[:, :70].contiguous())
    b, _ = block.prefill(x[:, 70:].contiguous())
    assert float((whole - torch.cat([a, b], 1)).abs().max()) < 1e-3


def test_training_step_against_differences_and_descends():
    block, x, target = setup()
    loss, grads = mb.train_step(block, x, target)
    gen = torch.Generator(device="cuda").manual_seed(2)
    leaves = block.params + list(block.norm) + list(block.head_norm)
    for p, d in zip(leaves, grads):
        assert bool(torch.isfinite(d).all())
        way = torch.randn(p.shape, generator=gen, device="cuda") * p.abs().mean().clamp_min(0.1) * 0.3
        h = 2.0 ** -6
        keep = p.clone()
        p.copy_(keep + h * way)
        up = float(mb.training_loss(block, x, target).double())
        p.copy_(keep - h * way)
        down = float(mb.training_loss(block, x, target).double())
        p.copy_(keep)
        want = float((way.double() * d.double()).sum())
        size = float((way.double() * d.double()).abs().sum())
        # the loss is of order 2 and known to 1e-6: 1e-4 in the quotient; the h^2 term a few percent of the whole
        assert abs((up - down) / (2 * h) - want) < 2e-4 + 0.05 * size
    losses = [float(mb.train_step(block, x, target, lr=0.5)[0]) for _ in range(6)]
    assert losses[-1] < losses[0]
