"""GPU tests of moe_combine for every k, with and without slots that have no row, plain and with the
normalised second output: equal to the bit to the sum in fp32, j in order, one rounding at the end."""
import pytest
import torch

from test_gpu_dispatch_grad import dispatch, gen, moe  # noqa: F401

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("k", range(1, 9))
@pytest.mark.parametrize("T,H", [(1, 7168), (37, 520), (19, 32768), (300, 1032)])
@pytest.mark.parametrize("drop", [0.0, 0.15, 0.6])
@pytest.mark.parametrize("extra", [False, True])
def test_combine_every_k(moe, k, T, H, drop, extra):  # noqa: F811
    """Products of whole numbers: the sums are exact, so that any order and any fused addition gives the
    same value, and what rows and weights of slots without a row hold shows at once."""
    g = gen(T + k)
    _, _, pos, _ = dispatch(moe, T, 16, k, drop, T + k)
    live = pos >= 0

    def whole(*shape):
        return torch.randint(-8, 9, shape, generator=g, device="cuda").to(BF)
    y, sh, res = whole(T * k, H), whole(T, H), whole(T, H)
    y[int(live.sum()):] = float("nan")
    w = torch.randint(1, 9, (T, k), generator=g, device="cuda") * 0.25
    w[~live] = float("inf")
    gate = torch.randint(1, 5, (T,), generator=g, device="cuda") * 0.25
    want = (torch.where(live[:, :, None], y[pos.clamp_min(0).long()].double(), 0.0)
            * torch.where(live, w, 0.0).double()[:, :, None]).sum(1)
    if extra:
        want += gate.double()[:, None] * sh.double()
    want = want.float().to(BF)
    if extra:
        want = (want.float() + res.float()).to(BF)
    args = (y, pos, w, T, k, H, sh if extra else None, gate if extra else None, res if extra else None)
    out, again, normed = (torch.full((T + 1, H), 7.0, dtype=BF, device="cuda") for _ in range(3))
    moe.moe_combine(*args, out)
    moe.moe_combine(*args, again, out_normed=normed, norm_eps=1e-6)
    assert torch.equal(out[:T], want) and torch.equal(again[:T], want)
    assert torch.all(out[T] == 7.0) and torch.all(again[T] == 7.0) and torch.all(normed[T] == 7.0)
    # the sum of squares is off by (H + 2) 2^-24 of itself, half of it in the root, which rounds, as do the
    # quotient and the product (2^-22 in all); the result by half a step of bf16 more
    x = want.double()
    ref = x / torch.sqrt((x * x).mean(1, keepdim=True) + 1e-6)
    tol = ref.abs() * ((H + 2) * 2.0 ** -25 + 2.0 ** -22)
    assert torch.all((normed[:T].double() - ref).abs() <= tol + (ref.abs() + tol) * 2.0 ** -8)
