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


@pytest.mark.parametrize("k", [1, 4, 7, 8])
@pytest.mark.parametrize("gating", GATING)
def test_nan_logits_reach_the_gradient(moe, gating, k):  # noqa: F811
    """Weights made of NaN logits are NaN, and so are their gradients: of every chosen expert, and in
    the softmax over all experts of the whole row.  Rows beside them are as ever."""
    T, E = 6, 33
    g = gen(k)
    z = torch.randn((T, E), generator=g, device="cuda")
    ids = torch.arange(2, 2 + k, dtype=torch.int32, device="cuda").repeat(T, 1).contiguous()
    dw = torch.randn((T, k), generator=g, device="cuda")
    want = run_gate(moe, z, ids, dw, gating, 1.5)
    z[0] = NAN                               # a token whose row is NaN
    z[2, 2] = NAN                            # one chosen logit ...
    z[3, 2], z[3, 3:] = NAN, -INF            # ... the others masked
    z[4, 2:2 + k] = NAN                      # the chosen ones
    z[5, 20] = NAN                           # one that is not chosen
    got = run_gate(moe, z, ids, dw, gating, 1.5)
    assert torch.equal(got[1], want[1])
    for t in (0, 2, 3, 4):
        assert torch.all(torch.isnan(got[t, 2:2 + k])), t
        if gating == "softmax":
            assert torch.all(torch.isnan(got[t])), t
        else:
            assert torch.all(got[t, :2] == 0) and torch.all(got[t, 2 + k:] == 0), t
    if gating == "softmax":
        assert torch.all(torch.isnan(got[5]))
    else:
        assert torch.equal(got[5], want[5])
