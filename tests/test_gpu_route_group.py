"""GPU tests of group-limited routing (moe_route_topk_grouped) against a plain 64-bit form.

Ids and the dispatch tables are compared exactly (tokens whose 64-bit gap at the group or the
expert boundary is below 1e-6 are checked for a valid choice instead).  An fp32 logit may be off
by (2 H + 64) * 2^-24 times the sum of its terms' magnitudes (each product and addition rounded
once, products split in up to three pieces); a weight, a ratio of exponentials or sigmoids of
logits, by 2.5 times that relatively, plus 2^-20 for the functions themselves.
"""
import numpy as np
import pytest
import torch

from oracle import moe_ref

pytestmark = pytest.mark.gpu

MODES = ["sigmoid_bias_renorm", "softmax", "softmax_renorm"]


@pytest.fixture(scope="module")
def moe():
    import expert_dispatch_streaming_gb300 as m
    return m


def inputs(seed, T, H, E, mode, logit_bias=None, sel_bias=None):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16)
    w_r = (rng.standard_normal((H, E)) * 0.05).astype(np.float32)
    if mode == "sigmoid_bias_renorm":
        sb = (0.1 * rng.standard_normal(E)).astype(np.float32) if sel_bias is None else sel_bias
        return x, w_r, logit_bias, sb
    lb = rng.standard_normal(E).astype(np.float32) if logit_bias is None else logit_bias
    return x, w_r, lb, None


def run(moe, x, w_r, lb, sb, E, k, groups, take, mode, scale=1.0, w_gate=None, stream=None):
    T, H = x.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    o = dict(ids=torch.full((T, k), -1, **i32), w=torch.full((T, k), -1.0, device="cuda"),
             counts=torch.full((E,), -1, **i32), offsets=torch.full((E + 1,), -1, **i32),
             pos=torch.full((T, k), -1, **i32), src=torch.full((T * k,), -1, **i32),
             logits=torch.full((T, E), -1.0, device="cuda"),
             sg=torch.full((T,), -1.0, device="cuda"), tie=torch.full((T,), -1, **i32))
    dev = lambda a: None if a is None else torch.from_numpy(np.asarray(a)).cuda()  # noqa: E731
    n = moe.moe_route_workspace_size(T, H, E, k)
    ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    moe.moe_route_topk_grouped(x.cuda(), dev(w_r), dev(lb), dev(sb),
                               None if w_gate is None else w_gate.cuda(), T, H, E, k, groups,
                               take, mode, scale, o["ids"], o["w"], o["counts"], o["offsets"],
                               o["pos"], o["src"], o["logits"],
                               None if w_gate is None else o["sg"], o["tie"], ws, n, stream)
    torch.cuda.synchronize()
    assert moe.moe_workspace_error(ws) == 0
    return {n: t.cpu().numpy() for n, t in o.items()}


def reference(x, w_r, lb, sb, k, groups, take, mode, scale):
    """(ids, w, gap of the groups, gap of the experts, selection scores, logit error bound)."""
    xd, wd = x.double().numpy(), w_r.astype(np.float64)
    with np.errstate(invalid="ignore"):
        l = xd @ wd + (0 if lb is None else lb.astype(np.float64))
        s = 1 / (1 + np.exp(-l)) if mode == "sigmoid_bias_renorm" else l
        c = s + (0 if sb is None else sb.astype(np.float64))
    c = np.where(np.isnan(c), -np.inf, c)
    T, E = c.shape
    gs = E // groups
    ids, w, ggap, egap = np.zeros((T, k), np.int32), np.zeros((T, k)), np.zeros(T), np.zeros(T)
    with np.errstate(all="ignore"):
        for t in range(T):
            per = -np.sort(-c[t].reshape(groups, gs), axis=1)
            G = per[:, :2].sum(1) if mode == "sigmoid_bias_renorm" else per[:, 0]
            G = np.where(np.isnan(G), -np.inf, G)
            order = np.lexsort((np.arange(groups), -G))
            ggap[t] = G[order[take - 1]] - G[order[take]] if take < groups else np.inf
            open_ = np.concatenate([np.arange(g * gs, (g + 1) * gs) for g in sorted(order[:take])])
            eo = open_[np.lexsort((open_, -c[t, open_]))]
            egap[t] = c[t, eo[k - 1]] - c[t, eo[k]] if k < len(eo) else np.inf
            ids[t] = np.sort(eo[:k])
            z = l[t, ids[t]]
            if mode == "softmax":
                w[t] = np.exp(z - l[t].max()) / np.exp(l[t] - l[t].max()).sum()
            else:
                v = s[t, ids[t]] if mode == "sigmoid_bias_renorm" else np.exp(z - z.max())
                w[t] = v / v.sum()
            if not np.any(s[t, ids[t]] > (0 if mode == "sigmoid_bias_renorm" else -np.inf)):
                w[t] = 0
    H = x.shape[1]
    bound = (2 * H + 64) * 2.0 ** -24 * (np.abs(xd) @ np.abs(wd)).max(1)
    return ids, w * scale, ggap, egap, c, bound


def check(got, ref, k, E):
    ids, w, ggap, egap, c, bound = ref
    near = (ggap < 1e-6) | (egap < 1e-6)          # -inf - -inf (masked): nan, compared exactly
    bad = np.where(~near & np.any(got["ids"] != ids, 1))[0]
    assert bad.size == 0, (bad[:5], got["ids"][bad[:5]], ids[bad[:5]], ggap[bad[:5]], egap[bad[:5]])
    for t in np.where(near)[0]:
        assert len(set(got["ids"][t].tolist())) == k
    ok = ~near
    tol = np.abs(w) * (2.5 * bound[:, None] + 2.0 ** -20)
    assert np.array_equal(np.isnan(got["w"][ok]), np.isnan(w[ok]))
    assert np.all(~(np.abs(got["w"] - w) > tol)[ok])
    counts, offsets, pos, src = moe_ref.dispatch(got["ids"], E)
    for n, r in (("counts", counts), ("offsets", offsets), ("pos", pos), ("src", src)):
        assert np.array_equal(got[n], r), n
    return int(near.sum())


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("E,groups,take,k", [(256, 8, 4, 8), (60, 6, 3, 4), (64, 32, 5, 7),
                                             (8, 1, 1, 2), (8, 8, 3, 3), (250, 5, 2, 8),
                                             (96, 16, 16, 6), (4, 2, 1, 2)])
@pytest.mark.parametrize("T", [1, 7, 16, 17, 300])
def test_grouped_routing(moe, T, E, groups, take, k, mode):
    H = 320
    x, w_r, lb, sb = inputs(T + E + groups, T, H, E, mode)
    got = run(moe, x, w_r, lb, sb, E, k, groups, take, mode, 2.5)
    check(got, reference(x, w_r, lb, sb, k, groups, take, mode, 2.5), k, E)


@pytest.mark.parametrize("H,T", [(8, 5), (200, 40), (7168, 3), (2048, 1030)])
def test_grouped_routing_hidden_sizes(moe, H, T):
    x, w_r, lb, sb = inputs(H, T, H, 128, MODES[0])
    got = run(moe, x, w_r, lb, sb, 128, 6, 8, 3, MODES[0])
    check(got, reference(x, w_r, lb, sb, 6, 8, 3, MODES[0], 1.0), 6, 128)


def test_large_batch(moe):
    T, H, E = 8192, 512, 256
    x, w_r, lb, sb = inputs(1, T, H, E, MODES[0])
    got = run(moe, x, w_r, lb, sb, E, 8, 8, 4, MODES[0], 2.5)
    near = check(got, reference(x, w_r, lb, sb, 8, 8, 4, MODES[0], 2.5), 8, E)
    assert near < 100
    again = run(moe, x, w_r, lb, sb, E, 8, 8, 4, MODES[0], 2.5)
    assert all(np.array_equal(got[n], again[n]) for n in got)


@pytest.mark.parametrize("T", [3, 20, 260])
@pytest.mark.parametrize("mode", MODES)
def test_one_group_or_all_groups_equals_ungrouped(moe, mode, T):
    """take == n_group leaves nothing out: the ids and weights of moe_route_topk."""
    H, E, k = 256, 64, 6
    x, w_r, lb, sb = inputs(T, T, H, E, mode)
    a = run(moe, x, w_r, lb, sb, E, k, 8, 8, mode)
    b = run(moe, x, w_r, lb, sb, E, k, 1, 1, mode)
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, w = torch.empty((T, k), **i32), torch.empty((T, k), device="cuda")
    n = moe.moe_route_workspace_size(T, H, E, k)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    dev = lambda v: None if v is None else torch.from_numpy(v).cuda()  # noqa: E731
    moe.moe_route_topk(x.cuda(), dev(w_r), dev(lb), dev(sb), None, None, T, H, E, k, mode, 1.0, ids,
                       w, torch.empty(E, **i32), torch.empty(E + 1, **i32),
                       torch.empty((T, k), **i32), torch.empty(T * k, **i32), None, None, None,
                       ws, n)
    ids, w = ids.cpu().numpy(), w.cpu().numpy()
    for o in (a, b):
        assert np.array_equal(o["ids"], ids)
        assert np.allclose(o["w"], w, rtol=2.0 ** -20, atol=0)


@pytest.mark.parametrize("T", [2, 40, 300])
def test_ties_go_to_the_lowest(moe, T):
    """Identical groups and identical experts: lower groups and lower ids win, and the ties are
    flagged."""
    H, E, groups, k = 256, 64, 8, 4
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16)
    col = (rng.standard_normal((H, E // groups)) * 0.05).astype(np.float32)
    got = run(moe, x, np.tile(col, groups), None, None, E, k, groups, 2, MODES[0])
    assert (got["ids"] < 2 * (E // groups)).all() and (got["tie"] == 2).all()
    one = (rng.standard_normal((H, 1)) * 0.05).astype(np.float32)
    got = run(moe, x, np.tile(one, E), None, None, E, k, groups, 2, MODES[1])
    assert np.array_equal(got["ids"], np.tile(np.arange(k), (T, 1))) and (got["tie"] == 2).all()


@pytest.mark.parametrize("T", [1, 9, 300])
def test_close_groups_and_experts_are_resolved_exactly(moe, T):
    """Router columns that differ by parts in 1e5 put many scores inside the fp32 margin: the
    64-bit order decides, at both boundaries."""
    H, E, groups = 256, 64, 8
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16)
    base = np.tile((rng.standard_normal((H, 8)) * 0.05).astype(np.float32), (1, groups))
    w_r = (base + rng.standard_normal((H, E)).astype(np.float32) * 1e-6).astype(np.float32)
    for mode in MODES:
        got = run(moe, x, w_r, None, None, E, 5, groups, 3, mode)
        check(got, reference(x, w_r, None, None, 5, groups, 3, mode, 1.0), 5, E)
        assert (got["tie"] >= 1).all()


def test_large_batch_with_every_token_rescored(moe):
    H, E, groups, T = 128, 256, 8, 4100
    rng = np.random.default_rng(4)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16)
    base = np.tile((rng.standard_normal((H, 32)) * 0.05).astype(np.float32), (1, groups))
    w_r = (base + rng.standard_normal((H, E)).astype(np.float32) * 1e-6).astype(np.float32)
    got = run(moe, x, w_r, None, None, E, 5, groups, 3, MODES[0])
    check(got, reference(x, w_r, None, None, 5, groups, 3, MODES[0], 1.0), 5, E)
    assert (got["tie"] >= 1).all()
    again = run(moe, x, w_r, None, None, E, 5, groups, 3, MODES[0])
    assert all(np.array_equal(got[n], again[n]) for n in got)


@pytest.mark.parametrize("T", [2, 30, 300])
@pytest.mark.parametrize("mode", MODES)
def test_masked_experts_and_groups(moe, mode, T):
    """Biases of -infinity mask experts, whole groups, and everything; +infinity and the lowest
    finite value."""
    H, E, groups, take, k = 128, 32, 8, 3, 4
    low = np.finfo(np.float32).min
    rng = np.random.default_rng(5)
    for pattern in range(5):
        b = (0.1 * rng.standard_normal(E)).astype(np.float32)
        if pattern == 0:
            b[::3] = -np.inf
        elif pattern == 1:
            b[4:28] = -np.inf                      # two groups left for three places
        elif pattern == 2:
            b[:] = -np.inf
        elif pattern == 3:
            b[:20] = low
        else:
            b[3] = -np.inf
            b[17] = -np.inf
        lb, sb = (None, b) if mode == MODES[0] else (b, None)
        x, w_r, _, _ = inputs(pattern, T, H, E, mode)
        got = run(moe, x, w_r, lb, sb, E, k, groups, take, mode)
        check(got, reference(x, w_r, lb, sb, k, groups, take, mode, 1.0), k, E)
    x, w_r, _, _ = inputs(9, T, H, E, MODES[0])
    none = np.full(E, -np.inf, np.float32)          # every logit -infinity: no weight left
    got = run(moe, x, w_r, none, None, E, k, groups, take, mode)
    assert (got["w"] == 0).all() and np.array_equal(got["ids"], np.tile(np.arange(k), (T, 1)))


def test_nan_rows_stay_valid(moe):
    """A NaN activation makes every score NaN: the first experts are taken, ids stay distinct
    and in range, other tokens are untouched."""
    for T in (4, 40, 300):
        x, w_r, lb, sb = inputs(T, T, 128, 32, MODES[0])
        x[1, 5] = float("nan")
        got = run(moe, x, w_r, lb, sb, 32, 4, 8, 3, MODES[0])
        assert np.array_equal(got["ids"][1], np.arange(4))
        keep = [t for t in range(T) if t != 1]
        ref = reference(x[keep], w_r, lb, sb, 4, 8, 3, MODES[0], 1.0)
        assert np.array_equal(got["ids"][keep], ref[0])
        _, _, pos, src = moe_ref.dispatch(got["ids"], 32)
        assert np.array_equal(got["src"], src) and np.array_equal(got["pos"], pos)


@pytest.mark.parametrize("T", [1, 16, 60, 400])
def test_shared_gate_and_logits(moe, T):
    H, E = 192, 48
    x, w_r, lb, sb = inputs(T, T, H, E, MODES[0])
    wg = (torch.from_numpy(np.random.default_rng(1).standard_normal(H)) * 0.05).to(torch.bfloat16)
    got = run(moe, x, w_r, lb, sb, E, 4, 6, 2, MODES[0], w_gate=wg)
    ref = reference(x, w_r, lb, sb, 4, 6, 2, MODES[0], 1.0)
    check(got, ref, 4, E)
    l = x.double().numpy() @ w_r.astype(np.float64)
    assert np.all(np.abs(got["logits"] - l) <= ref[5][:, None])
    z = x.double().numpy() @ wg.double().numpy()
    zb = (2 * H + 64) * 2.0 ** -24 * (np.abs(x.double().numpy()) @ np.abs(wg.double().numpy()))
    assert np.all(np.abs(got["sg"] - 1 / (1 + np.exp(-z))) <= zb + 2.0 ** -20)


@pytest.mark.parametrize("T,H,E,groups,gate", [
    (511, 320, 64, 8, True), (512, 64, 16, 4, False), (515, 7168, 256, 8, True),
    (1025, 2048, 60, 6, False), (700, 320, 250, 5, True), (20001, 128, 64, 8, False),
    (640, 4096, 8, 2, True), (8200, 192, 256, 32, False)])
def test_batches_on_the_tensor_cores(moe, T, H, E, groups, gate):
    """One and two column tiles and the gate column's third, ragged token tiles, more tiles than
    SMs, one to many parts of H; every logit."""
    x, w_r, lb, sb = inputs(T, T, H, E, MODES[0])
    wg = (torch.from_numpy(np.random.default_rng(1).standard_normal(H)) * 0.05).to(torch.bfloat16)
    a = dict(w_gate=wg if gate else None)
    got = run(moe, x, w_r, lb, sb, E, 4, groups, max(1, groups // 2), MODES[0], **a)
    ref = reference(x, w_r, lb, sb, 4, groups, max(1, groups // 2), MODES[0], 1.0)
    check(got, ref, 4, E)
    l = x.double().numpy() @ w_r.astype(np.float64)
    assert np.all(np.abs(got["logits"] - l) <= ref[5][:, None])
    if gate:
        z = x.double().numpy() @ wg.double().numpy()
        zb = (2 * H + 64) * 2.0 ** -24 * (np.abs(x.double().numpy()) @ np.abs(wg.double().numpy()))
        assert np.all(np.abs(got["sg"] - 1 / (1 + np.exp(-z))) <= zb + 2.0 ** -20)
    again = run(moe, x, w_r, lb, sb, E, 4, groups, max(1, groups // 2), MODES[0], **a)
    assert all(np.array_equal(got[n], again[n]) for n in got)


def test_empty_batch(moe):
    i32 = dict(dtype=torch.int32, device="cuda")
    counts, offsets = torch.full((16,), -1, **i32), torch.full((17,), -1, **i32)
    n = moe.moe_route_workspace_size(0, 64, 16, 2)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    moe.moe_route_topk_grouped(None, None, None, None, None, 0, 64, 16, 2, 4, 2, MODES[0], 1.0,
                               None, None, counts, offsets, None, None, None, None, None, ws, n)
    assert (counts == 0).all() and (offsets == 0).all()
