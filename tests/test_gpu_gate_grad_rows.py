"""GPU tests of moe_gate_backward on rows that routing leaves in an odd state: padding, NaN logits,
masked scores, slots that are dropped between routing and the experts."""
import pytest
import torch

from test_gpu_dispatch_grad import GATING, gen, moe, run_gate  # noqa: F401

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("gating", GATING)
def test_padding_has_no_gradient(moe, gating, whole, bad):  # noqa: F811
    """A token without an expert in any slot is in no loss: zeros, whatever its logits hold, one of them
    or all; its neighbours' gradients are those of a batch without it."""
    T, E, k = 9, 70, 4
    g = gen(5)
    z = torch.randn((T, E), generator=g, device="cuda")
    ids = torch.tensor([[3, 30, 31, 69]] * T, dtype=torch.int32, device="cuda")
    dw = torch.randn((T, k), generator=g, device="cuda")
    pad = torch.tensor([1, 4, 8], device="cuda")
    ids[pad] = -1
    want = run_gate(moe, z, ids, dw, gating, 2.0)
    z[pad] = bad if whole else torch.where(torch.arange(E, device="cuda") == 30, bad, z[pad])
    dw[pad] = bad
    got = run_gate(moe, z, ids, dw, gating, 2.0)
    assert torch.all(got[pad] == 0) and torch.all(torch.isfinite(got))
    assert torch.equal(got, want)
