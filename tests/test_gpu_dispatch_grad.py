"""GPU tests of the slot sort and of the gradients of permute, combine and gating, against plain
64-bit forms of their definitions.

Tolerances.  Whole numbers are equal.  A sum of n products in fp32 may be off by n + 2 roundings of
2^-24 of the sum of its terms' magnitudes; a bf16 result by half a step, 2^-8 of its value, more.
The gating's exponentials: the rounding of an exponent's argument, whose largest magnitude is D,
shows as a relative error D 2^-24, and the exponential itself, the sum over E and the few products
after it add at most (E + 16) 2^-23.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import expert_dispatch_streaming_gb300 as m
    return m


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def sort_ref(ids, E):
    T, k = ids.shape
    flat = ids.reshape(-1)
    has = (flat >= 0) & (flat < E)
    counts = np.bincount(flat[has], minlength=E)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    slots = np.nonzero(has)[0]
    order = slots[np.argsort(flat[slots], kind="stable")]
    src = np.full(T * k, -1)
    src[:order.size] = order
    pos = np.full(T * k, -1)
    pos[order] = np.arange(order.size)
    return counts, offsets, pos.reshape(T, k), src


def run_sort(moe, ids, E, stream=None):
    T, k = ids.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    out = [torch.full((E,), 77, **i32), torch.full((E + 1,), 77, **i32),
           torch.full((T, k), 77, **i32), torch.full((T * k,), 77, **i32)]
    nb = moe.moe_sort_tokens_workspace_size(T, E, k)
    ws = torch.full((max(nb, 4),), 0x5A, dtype=torch.uint8, device="cuda")
    moe.moe_sort_tokens(ids, T, E, k, *out, ws, nb, stream)
    return out


def make_ids(T, E, k, drop, seed, kind="distinct"):
    rng = np.random.default_rng(seed)
    if kind == "repeat":
        ids = rng.integers(0, E, (T, k))
    elif kind == "one":
        ids = np.full((T, k), E - 1)
    else:
        ids = np.argsort(rng.random((T, E)), axis=1)[:, :k]
    if drop:
        ids = np.where(rng.random((T, k)) < drop, rng.choice([-1, E, -2 ** 31, 2 ** 31 - 1], (T, k)),
                       ids)
    return ids.astype(np.int32)


SORT = [(1, 1, 1, 0.0, "distinct"), (1, 256, 8, 0.0, "distinct"), (33, 60, 4, 0.3, "distinct"),
        (2, 8, 2, 1.0, "distinct"), (255, 256, 8, 0.0, "repeat"), (256, 7, 8, 0.1, "repeat"),
        (257, 256, 8, 0.0, "one"), (341, 3, 6, 0.5, "repeat"), (1024, 16, 8, 0.02, "repeat"),
        (1025, 256, 8, 0.02, "distinct"), (2049, 255, 7, 0.0, "distinct"),
        (8192, 256, 8, 0.03, "distinct"), (32768, 256, 8, 0.0, "repeat"), (50001, 8, 2, 0.2, "repeat"),
        (40009, 256, 8, 0.1, "repeat"), (9000, 1, 1, 0.4, "repeat"), (4097, 33, 1, 0.0, "one")]


@pytest.mark.parametrize("T,E,k,drop,kind", SORT)
def test_sort_tokens(moe, T, E, k, drop, kind):
    ids = make_ids(T, E, k, drop, T + E + k, kind)
    got = run_sort(moe, torch.from_numpy(ids).cuda(), E)
    for g, r in zip(got, sort_ref(ids, E)):
        assert np.array_equal(g.cpu().numpy(), r)


def test_sort_no_tokens(moe):
    counts = torch.full((9,), 7, dtype=torch.int32, device="cuda")
    offsets = torch.full((10,), 7, dtype=torch.int32, device="cuda")
    moe.moe_sort_tokens(None, 0, 9, 2, counts, offsets, None, None, None, 0)
    assert counts.abs().sum() == 0 and offsets.abs().sum() == 0


def test_sort_matches_routing(moe):
    """The dispatch of the router's own choice, from its ids."""
    T, H, E, k = 300, 256, 64, 6
    g = gen(3)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    w_r = torch.randn((H, E), generator=g, device="cuda") * 0.05
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, w = torch.empty((T, k), **i32), torch.empty((T, k), device="cuda")
    disp = [torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty((T, k), **i32),
            torch.empty(T * k, **i32)]
    nb = moe.moe_route_workspace_size(T, H, E, k)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    moe.moe_route_topk(x, w_r, None, None, None, None, T, H, E, k, "softmax", 1.0, ids, w, *disp,
                       None, None, None, ws, nb)
    for a, b in zip(run_sort(moe, ids, E), disp):
        assert torch.equal(a, b)


def dispatch(moe, T, E, k, drop, seed):
    ids = torch.from_numpy(make_ids(T, E, k, drop, seed, "repeat")).cuda()
    _, offsets, pos, src = run_sort(moe, ids, E)
    return ids, offsets, pos, src


SHAPES = [(1, 8, 1, 8), (1, 256, 8, 7168), (3, 8, 2, 264), (37, 60, 4, 2048), (130, 16, 8, 1032),
          (65, 4, 3, 4104), (257, 256, 5, 520), (40, 9, 6, 16), (19, 30, 7, 1000)]


@pytest.mark.parametrize("T,E,k,H", SHAPES)
@pytest.mark.parametrize("drop", [0.0, 0.4])
def test_permute_and_combine_with_padding(moe, T, E, k, H, drop):
    """The forward pair on a dispatch with slots that have no row: rows that no slot takes read
    zero, their NaNs and infinite weights reach no output."""
    g = gen(T + H)
    ids, _, pos, src = dispatch(moe, T, E, k, drop, T)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    xp = torch.full((T * k, H), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_permute(x, src, T, k, H, xp)
    ref = torch.where((src >= 0)[:, None], x[(src.clamp_min(0) // k).long()], 0.0)
    assert torch.equal(xp, ref.to(torch.bfloat16))
    live = (pos >= 0)
    y = torch.randn((T * k, H), generator=g, device="cuda").to(torch.bfloat16)
    y[int(live.sum()):] = float("nan")
    w = torch.rand((T, k), generator=g, device="cuda")
    w[~live] = float("inf")
    terms = (torch.where(live[:, :, None], y[pos.clamp_min(0).long()].double(), 0.0)
             * torch.where(live, w, 0.0).double()[:, :, None])
    want, mag = terms.sum(1), terms.abs().sum(1)
    res = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    for residual in (None, res):
        for normed in (False, True):
            out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
            on = torch.empty_like(out) if normed else None
            moe.moe_combine(y, pos, w, T, k, H, None, None, residual, out, out_normed=on)
            tol = mag * (k + 2) * 2.0 ** -24 + want.abs() * 2.0 ** -8
            total = want
            if residual is not None:
                total = want + residual.double()
                tol = tol + (total.abs() + tol) * 2.0 ** -8
            assert torch.all((out.double() - total).abs() <= tol)


@pytest.mark.parametrize("T,E,k,H", SHAPES)
@pytest.mark.parametrize("drop", [0.0, 0.4, 1.0])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("add", [False, True])
def test_permute_backward(moe, T, E, k, H, drop, out, add):
    g = gen(T * 3 + H)
    _, _, pos, src = dispatch(moe, T, E, k, drop, T + 1)
    live = pos >= 0
    d = torch.randn((T * k, H), generator=g, device="cuda").to(torch.bfloat16)
    d[int(live.sum()):] = float("nan")       # rows that no slot takes
    a = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16) if add else None
    dx = torch.full((T + 1, H), 5.0, device="cuda",
                    dtype=torch.bfloat16 if out == "bf16" else torch.float32)
    moe.moe_permute_backward(d, pos, a, T, k, H, out, dx)
    terms = torch.where(live[:, :, None], d[pos.clamp_min(0).long()].double(), 0.0)
    if add:
        terms = torch.cat([terms, a.double()[:, None]], 1)
    want, mag = terms.sum(1), terms.abs().sum(1)
    tol = mag * (k + 2) * 2.0 ** -24
    if out == "bf16":
        tol = tol + want.abs() * 2.0 ** -8
    assert torch.all((dx[:T].double() - want).abs() <= tol)
    assert torch.all(dx[T] == 5.0)


def test_permute_backward_in_place(moe):
    """dx in the buffer of the gradient that is added: the result of separate buffers."""
    T, E, k, H = 70, 16, 4, 520
    g = gen(31)
    _, _, pos, _ = dispatch(moe, T, E, k, 0.2, 6)
    d = torch.randn((T * k, H), generator=g, device="cuda").to(torch.bfloat16)
    a = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    dx = torch.empty_like(a)
    moe.moe_permute_backward(d, pos, a, T, k, H, "bf16", dx)
    moe.moe_permute_backward(d, pos, a, T, k, H, "bf16", a)
    assert torch.equal(a, dx)


@pytest.mark.parametrize("T,E,k,H", SHAPES)
@pytest.mark.parametrize("drop", [0.0, 0.4, 1.0])
@pytest.mark.parametrize("shared", ["none", "plain", "gated"])
def test_combine_backward(moe, T, E, k, H, drop, shared):
    g = gen(T * 5 + H)
    _, _, pos, _ = dispatch(moe, T, E, k, drop, T + 2)
    live = pos >= 0
    rows = int(live.sum())
    dout = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    y = torch.randn((T * k, H), generator=g, device="cuda").to(torch.bfloat16)
    y[rows:] = float("nan")
    w = torch.randn((T, k), generator=g, device="cuda")
    w[~live] = float("nan")
    sh = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    gate = torch.rand(T, generator=g, device="cuda")
    dy = torch.full((T * k + 1, H), 5.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((T + 1, k), 5.0, device="cuda")
    dsh = torch.full((T + 1, H), 5.0, dtype=torch.bfloat16, device="cuda")
    dg = torch.full((T + 1,), 5.0, device="cuda")
    moe.moe_combine_backward(dout, y, pos, w, T, k, H, sh if shared == "gated" else None,
                             gate if shared == "gated" else None, dy, dw,
                             dsh if shared != "none" else None, dg if shared == "gated" else None)
    at = pos.clamp_min(0).long()
    prod = dout.double()[:, None] * torch.where(live[:, :, None], y[at].double(), 0.0)
    tol = prod.abs().sum(2) * (H + 2) * 2.0 ** -24
    assert torch.all((dw[:T].double() - prod.sum(2)).abs() <= tol)
    assert torch.all(dw[:T][~live] == 0) and torch.all(dw[T] == 5.0)
    want = torch.full((T * k, H), 5.0, dtype=torch.float64, device="cuda")
    want[pos[live].long()] = (dout.double()[:, None] * w.double()[:, :, None])[live]
    # (the product rounded to fp32, then to bf16)
    tol = want.abs() * (2.0 ** -8 + 2.0 ** -23)
    tol[rows:] = 0
    assert torch.all((dy[:T * k].double() - want).abs() <= tol) and torch.all(dy[T * k] == 5.0)
    if shared == "none":
        assert torch.all(dsh == 5.0) and torch.all(dg == 5.0)
        return
    gs = gate.double() if shared == "gated" else torch.ones(T, dtype=torch.float64, device="cuda")
    want = dout.double() * gs[:, None]
    assert torch.all((dsh[:T].double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -23))
    assert torch.all(dsh[T] == 5.0)
    if shared == "gated":
        prod = dout.double() * sh.double()
        tol = prod.abs().sum(1) * (H + 2) * 2.0 ** -24
        assert torch.all((dg[:T].double() - prod.sum(1)).abs() <= tol) and dg[T] == 5.0


@pytest.mark.parametrize("which", ["dy", "dw", "dshared", "dgate"])
def test_combine_backward_one_output(moe, which):
    """Each output alone is the one of a call with all of them, to the bit."""
    T, E, k, H = 37, 12, 4, 520
    g = gen(9)
    _, _, pos, _ = dispatch(moe, T, E, k, 0.2, 5)
    dout, sh = (torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    y = torch.randn((T * k, H), generator=g, device="cuda").to(torch.bfloat16)
    w, gate = torch.randn((T, k), generator=g, device="cuda"), torch.rand(T, generator=g, device="cuda")

    def outs():
        return dict(dy=torch.zeros((T * k, H), dtype=torch.bfloat16, device="cuda"),
                    dw=torch.zeros((T, k), device="cuda"),
                    dshared=torch.zeros((T, H), dtype=torch.bfloat16, device="cuda"),
                    dgate=torch.zeros(T, device="cuda"))
    full, one = outs(), outs()
    moe.moe_combine_backward(dout, y, pos, w, T, k, H, sh, gate, full["dy"], full["dw"],
                             full["dshared"], full["dgate"])
    pick = {n: one[n] if n == which else None for n in one}
    moe.moe_combine_backward(dout, y if which == "dw" else None, pos, w, T, k, H,
                             sh if which == "dgate" else None, gate, pick["dy"], pick["dw"],
                             pick["dshared"], pick["dgate"])
    assert torch.equal(full[which], one[which])
    assert all(torch.all(one[n] == 0) for n in one if n != which)


def test_permute_is_the_adjoint(moe):
    """<dx_perm, permute(x)> = <permute_backward(dx_perm), x>, on small whole numbers, where both are exact."""
    T, E, k, H = 45, 12, 5, 136
    g = gen(51)
    _, _, pos, src = dispatch(moe, T, E, k, 0.3, 8)
    x, d = (torch.randint(-8, 9, s, generator=g, device="cuda").to(torch.bfloat16)
            for s in ((T, H), (T * k, H)))
    xp, dx = torch.empty_like(d), torch.empty((T, H), device="cuda")
    moe.moe_permute(x, src, T, k, H, xp)
    moe.moe_permute_backward(d, pos, None, T, k, H, "fp32", dx)
    assert (d.double() * xp.double()).sum() == (dx.double() * x.double()).sum()


def test_combine_backward_differences(moe):
    """The gradients of <dout, combine(...)> are its differences: the sum is linear in each of y_perm, w,
    shared and shared_gate, and the values are chosen so that nothing rounds (whole numbers and halves
    whose sums stay below 2^7)."""
    T, E, k, H = 9, 6, 3, 16
    g = gen(52)
    _, _, pos, _ = dispatch(moe, T, E, k, 0.2, 9)
    live = pos >= 0

    def whole(*shape):
        return torch.randint(-3, 4, shape, generator=g, device="cuda").float()
    y, sh, dout = whole(T * k, H), whole(T, H), whole(T, H)
    w, gate = whole(T, k) * 0.5, whole(T) * 0.5

    def loss(y, w, sh, gate):
        out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
        moe.moe_combine(y.to(torch.bfloat16), pos, w, T, k, H, sh.to(torch.bfloat16), gate, None, out)
        return (out.double() * dout.double()).sum()

    bf = torch.bfloat16
    dy, dsh = torch.zeros((T * k, H), dtype=bf, device="cuda"), torch.empty((T, H), dtype=bf, device="cuda")
    dw, dg = torch.empty((T, k), device="cuda"), torch.empty(T, device="cuda")
    moe.moe_combine_backward(dout.to(bf), y.to(bf), pos, w, T, k, H, sh.to(bf), gate, dy, dw, dsh, dg)
    base = loss(y, w, sh, gate)

    def moved(v, at, by=1.0):
        v = v.clone()
        v[at] += by
        return v
    for t in range(T):
        assert loss(y, w, sh, moved(gate, t)) - base == dg[t]
        assert loss(y, w, moved(sh, (t, 5)), gate) - base == dsh[t, 5]
        for j in range(k):
            assert loss(y, moved(w, (t, j)), sh, gate) - base == dw[t, j]
            if live[t, j]:
                at = (int(pos[t, j]), 11)
                assert loss(moved(y, at), w, sh, gate) - base == dy[at]


def gate_weights(z, ids, gating, scale):
    """w [T][k] in 64 bits, zero at slots without an expert."""
    has = (ids >= 0) & (ids < z.shape[1])
    at = torch.where(has, ids, 0).long()
    if gating == "softmax":
        return torch.where(has, torch.softmax(z, 1).gather(1, at), 0.0) * scale
    if gating == "softmax_renorm":
        v = z.gather(1, at)
    else:
        v = torch.nn.functional.logsigmoid(z.gather(1, at))
    v = torch.where(has, v, -torch.inf)
    some = has.any(1, keepdim=True)
    w = torch.softmax(torch.where(some, v, 0.0), 1)
    return torch.where(has, w, 0.0) * scale


def run_gate(moe, z, ids, dw, gating, scale):
    T, E = z.shape
    dl = torch.full((T + 1, E), 5.0, device="cuda")
    moe.moe_gate_backward(z, ids, dw, T, E, ids.shape[1], gating, scale, dl)
    assert torch.all(dl[T] == 5.0)
    return dl[:T]


GATING = ["softmax_renorm", "softmax", "sigmoid_bias_renorm"]


@pytest.mark.parametrize("gating", GATING)
@pytest.mark.parametrize("T,E,k,drop", [(1, 1, 1, 0.0), (1, 256, 8, 0.0), (33, 60, 4, 0.3),
                                        (17, 8, 8, 0.0), (50, 33, 5, 0.2), (700, 255, 7, 0.05),
                                        (9, 100, 3, 1.0), (300, 64, 8, 0.5)])
@pytest.mark.parametrize("kind", ["distinct", "repeat"])
@pytest.mark.parametrize("spread", [1.0, 12.0])
def test_gate_backward(moe, gating, T, E, k, drop, kind, spread):
    g = gen(T + E)
    z = torch.randn((T, E), generator=g, device="cuda") * spread
    ids = torch.from_numpy(make_ids(T, E, k, drop, E, kind)).cuda()
    dw = torch.randn((T, k), generator=g, device="cuda")
    has = (ids >= 0) & (ids < E)
    dw[~has] = float("nan")                  # not read
    got = run_gate(moe, z, ids, dw, gating, 2.5).double()
    z64 = z.double().requires_grad_(True)
    w = gate_weights(z64, ids, gating, 2.5)
    up = torch.where(has, dw, 0.0).double()
    (want,) = torch.autograd.grad((w * up).sum(), z64)
    # magnitude of the terms of each element: its own weights' and, through D, everyone's
    w = w.detach()
    at = torch.where(has, ids, 0).long()
    own = torch.zeros_like(want).scatter_add_(1, at, w * up.abs())
    p = torch.softmax(z64.detach(), 1) if gating == "softmax" else torch.zeros_like(want).scatter_add_(
        1, at, w) / 2.5
    mag = own + p * (w * up.abs()).sum(1, keepdim=True)
    depth = 2 * z.double().abs().amax()
    tol = mag * (2 * depth + E + 16) * 2.0 ** -23 + 1e-37
    assert torch.all((got - want).abs() <= tol)


@pytest.mark.parametrize("gating", GATING)
def test_gate_backward_masked_scores(moe, gating):
    """Experts masked with -infinity, rows whose every score is, sigmoids below fp32's range."""
    E, k = 40, 4
    g = gen(4)
    z = torch.randn((5, E), generator=g, device="cuda")
    ids = torch.tensor([[0, 3, 7, 9]] * 5, dtype=torch.int32, device="cuda")
    dw = torch.randn((5, k), generator=g, device="cuda")
    inf = float("inf")
    z[0, 3] = -inf                               # one of the chosen
    z[1] = -inf                                  # everything
    z[2, ids[2].long()] = torch.tensor([-inf] * 4, device="cuda")
    z[3, 20:] = -inf                             # others only
    z[4, ids[4].long()] = torch.tensor([-200.0, -201.0, -203.0, -200.5], device="cuda")
    got = run_gate(moe, z, ids, dw, gating, 1.0).double()
    assert torch.all(torch.isfinite(got))
    assert torch.all(got[1] == 0)
    if gating == "softmax":
        p = torch.softmax(z.double(), 1)
        p[1] = 0
    else:
        v = z.gather(1, ids.long()).double()
        if gating == "sigmoid_bias_renorm":
            v = torch.nn.functional.logsigmoid(v)
        r = torch.nan_to_num(torch.softmax(v, 1))
        p = torch.zeros_like(got).scatter_(1, ids.long(), r)
    r = p.gather(1, ids.long())
    D = (r * dw.double()).sum(1, keepdim=True)
    if gating == "softmax":
        want = -p * D
        want.scatter_add_(1, ids.long(), r * dw.double())
    else:
        slope = 1.0
        if gating == "sigmoid_bias_renorm":
            slope = 1 - torch.sigmoid(z.gather(1, ids.long()).double())
        want = torch.zeros_like(got).scatter_(1, ids.long(), r * (dw.double() - D) * slope)
    mag = dw.abs().double().sum(1, keepdim=True)
    assert torch.all((got - want).abs() <= mag * (3 * 2 + E + 210) * 2.0 ** -23)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("gating", GATING)
def test_gate_backward_weights_of_zero(moe, gating, bad):
    """What stands in dw for a chosen expert whose logit is -infinity, or for a token all of whose
    logits are, reaches nothing."""
    E, k, T = 37, 3, 6
    g = gen(11)
    z = torch.randn((T, E), generator=g, device="cuda")
    ids = torch.tensor([[1, 30, 36]] * T, dtype=torch.int32, device="cuda")
    dw = torch.randn((T, k), generator=g, device="cuda")
    z[0, 30], z[2, 1], z[2, 36] = [-float("inf")] * 3
    z[4] = -float("inf")
    off = torch.isinf(z.gather(1, ids.long()))
    got = run_gate(moe, z, ids, torch.where(off, bad, dw), gating, 1.5)
    want = run_gate(moe, z, ids, torch.where(off, 0.0, dw), gating, 1.5)
    assert torch.equal(got, want) and torch.all(torch.isfinite(got))
    assert torch.all(got[4] == 0) and got[0, 30] == 0


def test_gate_backward_differences(moe):
    """The gradient against central differences of the library's own gating weights: w of
    moe_route_topk with an identity router, whose logits are the tokens' values."""
    E = H = 32
    k, T = 4, 6
    g = gen(8)
    step = 2.0 ** -3
    x = (torch.randint(-12, 13, (T, H), generator=g, device="cuda") * 0.25)
    eye = torch.eye(E, device="cuda")
    dw = torch.randn((T, k), generator=g, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    ids = torch.from_numpy(make_ids(T, E, k, 0.0, 1)).cuda()
    nb = moe.moe_route_workspace_size(T, H, E, k)

    def weights(xv, gating):
        w, logits = torch.empty((T, k), device="cuda"), torch.empty((T, E), device="cuda")
        o = [torch.empty((T, k), **i32), w, torch.empty(E, **i32), torch.empty(E + 1, **i32),
             torch.empty((T, k), **i32), torch.empty(T * k, **i32)]
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        moe.moe_route_topk(xv.to(torch.bfloat16), eye, None, None, None, ids, T, H, E, k, gating, 1.5,
                           *o, logits, None, None, ws, nb)
        return w.double(), logits

    for gating in GATING:
        _, z = weights(x, gating)
        assert torch.equal(z, x)
        got = run_gate(moe, z, ids, dw, gating, 1.5).double()
        for e in range(E):
            d = torch.zeros_like(x)
            d[:, e] = step
            up, _ = weights(x + d, gating)
            dn, _ = weights(x - d, gating)
            num = ((up - dn) * dw.double()).sum(1) / (2 * step)
            # the difference is off by step^2 / 6 of a third derivative, at most 1 for a softmax
            # weight (its derivatives are products of weights), and by the weights' fp32 roundings
            tol = 1.5 * dw.abs().double().sum(1) * (step ** 2 / 6 + 64 * 2.0 ** -24 / step)
            assert torch.all((got[:, e] - num).abs() <= tol)


def test_programmatic_launches(moe):
    """The chain with every kernel allowed to start beside its predecessor's end: the results of plain
    launches, to the bit, call after call on the same buffers."""
    T, E, k, H = 3001, 64, 8, 256
    i32 = dict(dtype=torch.int32, device="cuda")
    g = gen(40)
    sets = []
    for seed in range(3):
        ids = torch.from_numpy(make_ids(T, E, k, 0.1, seed)).cuda()
        x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
        sets.append((ids, x, torch.rand((T, k), generator=g, device="cuda")))
    nb = moe.moe_sort_tokens_workspace_size(T, E, k)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    b = dict(ids=torch.empty((T, k), **i32), counts=torch.empty(E, **i32),
             offsets=torch.empty(E + 1, **i32), pos=torch.empty((T, k), **i32),
             src=torch.empty(T * k, **i32),
             xp=torch.empty((T * k, H), dtype=torch.bfloat16, device="cuda"),
             out=torch.empty((T, H), dtype=torch.bfloat16, device="cuda"),
             dy=torch.zeros((T * k, H), dtype=torch.bfloat16, device="cuda"),
             dw=torch.empty((T, k), device="cuda"), dx=torch.empty((T, H), device="cuda"),
             z=torch.randn((T, E), generator=g, device="cuda"), dz=torch.empty((T, E), device="cuda"))

    def chain(ids, x, w):
        b["ids"].copy_(ids)
        moe.moe_sort_tokens(b["ids"], T, E, k, b["counts"], b["offsets"], b["pos"], b["src"], ws, nb)
        moe.moe_permute(x, b["src"], T, k, H, b["xp"])
        moe.moe_combine(b["xp"], b["pos"], w, T, k, H, None, None, None, b["out"])
        moe.moe_combine_backward(b["out"], b["xp"], b["pos"], w, T, k, H, None, None, b["dy"], b["dw"])
        moe.moe_gate_backward(b["z"], b["ids"], b["dw"], T, E, k, "softmax_renorm", 1.0, b["dz"])
        moe.moe_permute_backward(b["dy"], b["pos"], None, T, k, H, "fp32", b["dx"])
        return {n: v.clone() for n, v in b.items()}

    plain = [chain(*s) for s in sets]
    moe.set_pdl(True)
    try:
        for _ in range(3):
            for s, want in zip(sets, plain):
                got = chain(*s)
                for n in want:
                    if n != "dy":        # (its last rows are the calls' before)
                        assert torch.equal(got[n], want[n]), n
    finally:
        moe.set_pdl(False)


def test_captured_training_step(moe):
    """The sort and the gradients captured into one graph on a side stream and replayed on new
    inputs in the same buffers: the results of eager calls, to the bit."""
    T, E, k, H = 300, 16, 4, 512
    s = torch.cuda.Stream()
    g = gen(12)
    st = {}
    i32 = dict(dtype=torch.int32, device="cuda")

    def fill(seed):
        g = gen(seed)
        return dict(ids=torch.from_numpy(make_ids(T, E, k, 0.1, seed)).cuda(),
                    dout=torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16),
                    y=torch.randn((T * k, H), generator=g, device="cuda").to(torch.bfloat16),
                    w=torch.rand((T, k), generator=g, device="cuda"),
                    z=torch.randn((T, E), generator=g, device="cuda"))

    def step(b, stream):
        moe.moe_sort_tokens(b["ids"], T, E, k, b["counts"], b["offsets"], b["pos"], b["src"],
                            b["ws"], b["ws"].numel(), stream)
        moe.moe_combine_backward(b["dout"], b["y"], b["pos"], b["w"], T, k, H, None, None, b["dy"],
                                 b["dw"], stream=stream)
        moe.moe_gate_backward(b["z"], b["ids"], b["dw"], T, E, k, "softmax_renorm", 1.0, b["dz"],
                              stream)
        moe.moe_permute_backward(b["dy"], b["pos"], b["dout"], T, k, H, "fp32", b["dx"], stream)

    def buffers():
        nb = moe.moe_sort_tokens_workspace_size(T, E, k)
        return dict(counts=torch.empty(E, **i32), offsets=torch.empty(E + 1, **i32),
                    pos=torch.empty((T, k), **i32), src=torch.empty(T * k, **i32),
                    ws=torch.empty(nb, dtype=torch.uint8, device="cuda"),
                    dy=torch.zeros((T * k, H), dtype=torch.bfloat16, device="cuda"),
                    dw=torch.empty((T, k), device="cuda"), dz=torch.empty((T, E), device="cuda"),
                    dx=torch.empty((T, H), device="cuda"))

    st = {**fill(1), **buffers()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(st, s)
    for seed in (2, 3):
        new = fill(seed)
        for n, v in new.items():
            st[n].copy_(v)
        st["dy"].zero_()
        graph.replay()
        ref = {**new, **buffers()}
        step(ref, None)
        torch.cuda.synchronize()
        for n in ("counts", "offsets", "pos", "src", "dy", "dw", "dz", "dx"):
            assert torch.equal(st[n], ref[n]), n
