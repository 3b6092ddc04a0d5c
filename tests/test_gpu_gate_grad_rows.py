"""GPU tests of moe_gate_backward on rows that routing leaves in an odd state: padding, NaN logits,
masked scores, slots that are dropped between routing and the experts."""
import os

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


def readme_example():
    """The training example of README.md: its block of calls."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "README.md")) as f:
        lines = f.read().split("\n")
    first = next(i for i, line in enumerate(lines) if line.startswith("    moe.moe_sort_tokens("))
    block = []
    for line in lines[first:]:
        if not line.startswith("    "):
            break
        block.append(line[4:])
    return "\n".join(block)


@pytest.mark.parametrize("gating,scale", [("softmax_renorm", 1.0), ("softmax", 1.0),
                                          ("sigmoid_bias_renorm", 2.5)])
def test_dropped_slots_through_the_documented_calls(moe, gating, scale):  # noqa: F811
    """README's training example, run as it stands, on a batch whose single slots are dropped between
    routing and the experts: the gradient of the library's own weights, which are normalised over all k
    slots, against 64-bit differentiation of them.  A dropped expert's logit has a gradient through the
    weights of the others."""
    T, H, N, E, k = 61, 256, 192, 20, 4
    g = gen(33)
    i32 = dict(dtype=torch.int32, device="cuda")
    bf = torch.bfloat16
    x = torch.randn((T, H), generator=g, device="cuda").to(bf)
    w_r = torch.randn((H, E), generator=g, device="cuda") * 0.1
    ids, w, logits = torch.empty((T, k), **i32), torch.empty((T, k), device="cuda"), torch.empty(
        (T, E), device="cuda")
    disp = [torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty((T, k), **i32),
            torch.empty(T * k, **i32)]
    nb = moe.moe_route_workspace_size(T, H, E, k)
    moe.moe_route_topk(x, w_r, None, None, None, None, T, H, E, k, gating, scale, ids, w, *disp, logits,
                       None, None, torch.empty(nb, dtype=torch.uint8, device="cuda"), nb)
    drop = torch.rand((T, k), generator=g, device="cuda") < 0.25
    drop[7], drop[8] = True, False
    kept = torch.where(drop, -1, ids)
    ws_bytes = moe.moe_sort_tokens_workspace_size(T, E, k)
    n4 = moe.moe_grouped_gemv_int4_workspace_size(T * k, E, N, H)
    u8 = dict(dtype=torch.uint8, device="cuda")
    names = dict(
        moe=moe, T=T, E=E, k=k, H=H, N=N, ids=ids, kept=kept, x=x, w=w, logits=logits,
        counts=torch.empty(E, **i32), offsets=torch.empty(E + 1, **i32), pos=torch.empty((T, k), **i32),
        src=torch.empty(T * k, **i32), ws=torch.empty(max(ws_bytes, 4), **u8), ws_bytes=ws_bytes,
        x_perm=torch.empty((T * k, H), dtype=bf, device="cuda"),
        w4=torch.randint(0, 256, (E, N, H // 2), generator=g, **u8),
        scales=(torch.rand((E, N, H // 128), generator=g, device="cuda") * 0.02).to(bf),
        zeros=torch.randint(0, 17, (E, N, H // 128), generator=g, **u8),
        y=torch.empty((T * k, N), dtype=bf, device="cuda"), ws4=torch.empty(n4, **u8), n4=n4,
        out=torch.empty((T, N), dtype=bf, device="cuda"),
        dout=torch.randn((T, N), generator=g, device="cuda").to(bf),
        dy=torch.zeros((T * k, N), dtype=bf, device="cuda"), dw=torch.empty((T, k), device="cuda"),
        dlogits=torch.empty((T, E), device="cuda"),
        dx_perm=torch.randn((T * k, H), generator=g, device="cuda").to(bf),
        dx=torch.empty((T, H), device="cuda"))
    code = readme_example().replace('"softmax_renorm", 1.0', "gating, scale")
    exec(code, names | dict(gating=gating, scale=scale))
    assert int(names["offsets"][-1]) == int((~drop).sum())
    assert torch.all(names["dw"][drop] == 0)
    # the framework's own weights in 64 bits: over all k slots, whatever the dispatch drops
    z = logits.double().requires_grad_(True)
    zj = z.gather(1, ids.long())
    if gating == "softmax":
        w64 = torch.softmax(z, 1).gather(1, ids.long()) * scale
    else:
        v = torch.sigmoid(zj) if gating == "sigmoid_bias_renorm" else torch.exp(zj)
        w64 = v / v.sum(1, keepdim=True) * scale
    assert torch.all((w64.detach() - w.double()).abs() <= w64.detach() * (E + 40) * 2.0 ** -23)
    y, pos = names["y"], names["pos"]
    yt = torch.where(drop[:, :, None], 0.0, y[pos.clamp_min(0).long()].double())
    dots = torch.einsum("th,tkh->tk", names["dout"].double(), yt)
    (want,) = torch.autograd.grad((w64 * dots).sum(), z)
    # dw is off by (N + 2) 2^-24 of its terms' magnitudes, the gating by (E + 64) 2^-23 of its own; both
    # reach an element with a factor of at most 2 scale
    size = torch.einsum("th,tkh->tk", names["dout"].abs().double(), yt.abs()).sum(1, keepdim=True)
    got = names["dlogits"].double()
    assert torch.all((got - want).abs() <= 2 * scale * size * (N + E + 66) * 2.0 ** -23)
    part = drop & ~drop.all(1, keepdim=True)
    assert torch.all(got.gather(1, ids.long())[part] != 0) and torch.all(got[7] == 0)


@pytest.mark.parametrize("gating", GATING)
@pytest.mark.parametrize("low", [-60.0, -100.0, -300.0, -INF])
def test_weights_and_gradient_of_low_scores(moe, gating, low):  # noqa: F811
    """Group-limited routing and the gradient follow one rule where scores are so low that nothing, or
    next to nothing, is left: logits (the bias alone) around `low`, every weight finite and its gradient
    that of the weights as routing made them."""
    T, H, E, k, scale = 5, 64, 32, 4, 1.5
    g = gen(17)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    w_r = torch.zeros((H, E), device="cuda")
    bias = torch.randn(E, generator=g, device="cuda") + low
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, w, z = torch.empty((T, k), **i32), torch.empty((T, k), device="cuda"), torch.empty(
        (T, E), device="cuda")
    disp = [torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty((T, k), **i32),
            torch.empty(T * k, **i32)]
    nb = moe.moe_route_workspace_size(T, H, E, k)
    moe.moe_route_topk_grouped(x, w_r, bias, None, None, T, H, E, k, 4, 2, gating, scale, ids, w, *disp, z,
                               None, None, torch.empty(nb, dtype=torch.uint8, device="cuda"), nb)
    assert torch.all(torch.isfinite(w))
    dw = torch.randn((T, k), generator=g, device="cuda")
    got = run_gate(moe, z, ids, dw, gating, scale)
    if low == -INF:
        assert torch.all(w == 0) and torch.all(got == 0)
        return
    assert torch.all(z[0] == bias)
    r = w.double() / scale
    D = (r * dw.double()).sum(1, keepdim=True)
    if gating == "softmax":
        want = -scale * torch.softmax(z.double(), 1) * D
        want.scatter_add_(1, ids.long(), scale * r * dw.double())
    else:
        want = torch.zeros_like(z, dtype=torch.float64)
        slope = torch.sigmoid(-z.double()).gather(1, ids.long()) if "sigmoid" in gating else 1.0
        want.scatter_(1, ids.long(), scale * r * (dw.double() - D) * slope)
    # both the weights and the gradient are off by the rounding of exponents of at most 2 |low| and a
    # few products: (2 |low| + E + 16) 2^-23 of the terms each
    mag = scale * dw.double().abs().sum(1, keepdim=True)
    assert torch.all((got.double() - want).abs() <= 4 * mag * (2 * abs(low) + E + 16) * 2.0 ** -23)
    assert torch.any(got != 0)
