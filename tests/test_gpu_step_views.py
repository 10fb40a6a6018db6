"""A decode step whose cache is a view: nothing beside the view and no slot without a request changes."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU-only machines
    pytest.skip("needs a CUDA device", allow_module_level=True)

import causal_depthwise_conv1d_gb300 as ccv  # noqa: E402
from tests import mixer_ref as ref  # noqa: E402


@pytest.mark.parametrize("B,S,off", [(4, 1, 4), (4, 1, 3), (4, 3, 4), (400, 1, 4)])  # several kernels and loads
def test_what_lies_around_the_view_stays(B, S, off):
    c = ref.gdr_inputs(13, B, S, 1, 2, 64, 32, "bf16")
    d = {n: c[n].cuda() for n in ("q", "k", "v", "g", "beta")}
    base = torch.randn((B + 2, 2, 66, 40), device="cuda")
    before = base.clone()
    state = base[:, :, 1:65, off:off + 32]
    idx = torch.arange(B, 0, -1, dtype=torch.int32, device="cuda")  # slots B .. 1
    idx[1] = -1
    out = ccv.gated_delta_rule_step(*d.values(), state, state_indices=idx)
    used = [i for i in range(B) if i != 1]
    slots = [B - i for i in used]
    o, s, eo, es = ref.gdr(*(c[n][used] for n in ("q", "k", "v", "g", "beta")), None,
                           before[slots, :, 1:65, off:off + 32].cpu())
    assert ref.worst(out[used], o, eo + ref.rounding(o, "bf16")) <= 1
    assert ref.worst(state[slots], s, es) <= 1
    assert not out[1].any()
    base[slots, :, 1:65, off:off + 32] = before[slots, :, 1:65, off:off + 32]
    assert torch.equal(base, before)
