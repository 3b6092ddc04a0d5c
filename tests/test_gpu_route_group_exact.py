"""GPU tests of group-limited routing where both selections are near their boundaries: the exact
(re-scored) choice against a 64-bit form, token by token.

A re-scored score is a compensated fp32 dot product: its second-order error is (n 2^-24)^2 times
the sum of its terms' magnitudes for chains of n additions (8 terms a thread, H <= 2048, five
shuffles and at most 32 warps: n = 45); the 64-bit form's own product is off by H 2^-53 times that
sum, a sigmoid (whose slope is at most a quarter) by 2^-52 more.  A group's score adds two of them
and a gap compares two groups, so ids are compared exactly where the 64-bit gap is above four times
a score's error, about 4e-10.  What lies below (hardly any token) is held to that: groups and experts
within that much of the best that could stand in their place.  The flag is 2 where a gap is below
1e-6 and less than 2 where it is above, by more than that error.
"""
import numpy as np
import pytest
import torch

from oracle import moe_ref
from test_gpu_route_group import MODES, reference, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import expert_dispatch_streaming_gb300 as m
    return m


def score_error(x, w_r):
    H = x.shape[1]
    mag = (x.double().abs().numpy() @ np.abs(w_r.astype(np.float64))).max()
    return (45 ** 2 * 2.0 ** -48 + H * 2.0 ** -53) * mag + 2.0 ** -50


def check_exact(got, x, w_r, lb, sb, k, groups, take, mode):
    """Returns the fraction of tokens that re-scoring cannot tell apart."""
    E = w_r.shape[1]
    gs = E // groups
    ids, _, ggap, egap, c, _ = reference(x, w_r, lb, sb, k, groups, take, mode, 1.0)
    err = score_error(x, w_r)
    near = np.minimum(ggap, egap) <= 4 * err
    assert np.array_equal(got["ids"][~near], ids[~near])
    for t in np.where(near)[0]:
        mine = got["ids"][t]
        assert len(set(mine.tolist())) == k
        per = -np.sort(-c[t].reshape(groups, gs), axis=1)
        G = per[:, :2].sum(1) if mode == MODES[0] and gs > 1 else per[:, 0]
        used = np.unique(mine // gs)
        assert len(used) <= take and G[used].min() >= np.sort(G)[::-1][take - 1] - 4 * err
        # every expert left out of a used group is at most that much better than the worst taken
        left = np.setdiff1d(np.concatenate([np.arange(g * gs, (g + 1) * gs) for g in used]), mine)
        assert left.size == 0 or c[t, left].max() <= c[t, mine].min() + 4 * err
    # weights of the ids that were returned (an fp32 logit, as the fp32 tests)
    l = x.double().numpy() @ w_r.astype(np.float64) + (0 if lb is None else lb.astype(np.float64))
    z = np.take_along_axis(l, got["ids"].astype(np.int64), 1)
    if mode == "softmax":
        w = np.exp(z - l.max(1, keepdims=True)) / np.exp(l - l.max(1, keepdims=True)).sum(1, keepdims=True)
    else:
        v = 1 / (1 + np.exp(-z)) if mode == MODES[0] else np.exp(z - z.max(1, keepdims=True))
        w = v / v.sum(1, keepdims=True)
    H = x.shape[1]
    lerr = (2 * H + 64) * 2.0 ** -24 * (np.abs(x.double().numpy()) @ np.abs(w_r.astype(np.float64)))
    assert np.all(np.abs(got["w"] - w) <= w * (2.5 * lerr.max(1, keepdims=True) + 2.0 ** -20))
    # the flags
    gap = np.fmin(ggap, egap)
    assert (got["tie"][gap < 1e-6 - 4 * err] == 2).all()
    assert (got["tie"][gap > 1e-6 + 4 * err] < 2).all()
    counts, offsets, pos, src = moe_ref.dispatch(got["ids"], E)
    for n, r in (("counts", counts), ("offsets", offsets), ("pos", pos), ("src", src)):
        assert np.array_equal(got[n], r), n
    return near.mean()


def near_columns(rng, H, E, distinct):
    """Router columns that repeat with a period of `distinct`, apart by parts in 1e5."""
    base = np.tile((rng.standard_normal((H, distinct)) * 0.05).astype(np.float32),
                   (1, E // distinct))
    return (base + rng.standard_normal((H, E)).astype(np.float32) * 1e-6).astype(np.float32)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("T", [1, 9, 16, 17, 300, 600, 4100])
@pytest.mark.parametrize("H,E,groups,take,k,distinct", [(256, 64, 8, 3, 5, 8),
                                                        (128, 256, 8, 3, 5, 32),
                                                        (192, 60, 6, 2, 4, 10)])
def test_near_boundaries_token_by_token(moe, mode, T, H, E, groups, take, k, distinct):
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16)
    w_r = near_columns(rng, H, E, distinct)
    got = run(moe, x, w_r, None, None, E, k, groups, take, mode)
    near = check_exact(got, x, w_r, None, None, k, groups, take, mode)
    assert near <= (0.01 if T >= 300 else 0.12)
    assert (got["tie"] >= 1).all()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("T", [1, 5, 16, 300, 600, 4100])
@pytest.mark.parametrize("E,groups,k", [(256, 4, 8), (128, 4, 8)])
def test_group_boundary_then_a_long_list_of_experts(moe, mode, T, E, groups, k):
    """Two requests for one token: two groups close to the last place (their best experts are
    re-scored), then, inside the group that is clear, every expert but two close to the last
    place (62 of 64 or 30 of 32, none of them scored yet: several batches)."""
    H, gs = 256, E // groups
    rng = np.random.default_rng(11)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16)
    w_r = near_columns(rng, H, E, 1)
    level = np.full(E, -1.0, np.float32)
    level[:gs] = 0.0
    level[[0, 1]] = 2.0
    level[[gs, gs + 1, 2 * gs, 2 * gs + 1]] = 1.0
    lb, sb = (None, level) if mode == MODES[0] else (level, None)
    got = run(moe, x, w_r, lb, sb, E, k, groups, 2, mode)
    near = check_exact(got, x, w_r, lb, sb, k, groups, 2, mode)
    assert near <= (0.01 if T >= 300 else 0.12)
    assert (got["tie"] >= 1).all()
    again = run(moe, x, w_r, lb, sb, E, k, groups, 2, mode)
    assert all(np.array_equal(got[n], again[n]) for n in got)
