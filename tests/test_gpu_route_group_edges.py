"""GPU tests of group-limited routing at the edges of fp32: biases near the largest finite values
and sigmoids below the smallest, against the 64-bit form of test_gpu_route_group."""
import numpy as np
import pytest
import torch  # noqa: F401

from test_gpu_route_group import MODES, check, inputs, reference, run

pytestmark = pytest.mark.gpu

LOW = np.finfo(np.float32).min
INF = np.float32(np.inf)


@pytest.fixture(scope="module")
def moe():
    import expert_dispatch_streaming_gb300 as m
    return m


@pytest.mark.parametrize("T", [2, 30, 300, 600])
@pytest.mark.parametrize("first,second,third", [
    (-INF, LOW, 0.75 * LOW), (-INF, LOW, LOW), (LOW, -INF, 0.6 * LOW), (-LOW, -INF, INF),
    (-0.75 * LOW, -LOW, -LOW)])
@pytest.mark.parametrize("mode", MODES)
def test_masks_of_the_largest_finite_values(moe, mode, T, first, second, third):
    """One group of ordinary experts, two places and eight experts: the second group is one whose
    experts are all masked, by -infinity, by the lowest value or by a part of it (two of which add
    up past fp32's range); or, with the signs turned, favoured."""
    H, E, groups, take, k = 128, 32, 8, 2, 8
    rng = np.random.default_rng(8)
    b = (0.1 * rng.standard_normal(E)).astype(np.float32)
    for g, v in ((0, first), (1, second), (2, third), (3, -INF), (4, -INF), (6, -INF), (7, -INF)):
        b[4 * g:4 * g + 4] = v
    lb, sb = (None, b) if mode == MODES[0] else (b, None)
    x, w_r, _, _ = inputs(T, T, H, E, mode)
    got = run(moe, x, w_r, lb, sb, E, k, groups, take, mode)
    check(got, reference(x, w_r, lb, sb, k, groups, take, mode, 1.0), k, E)


@pytest.mark.parametrize("T", [1, 30, 300, 600])
@pytest.mark.parametrize("k", [1, 4])
@pytest.mark.parametrize("level", [-70, -87, -88, -88.3, -89, -104, -300, -680])
def test_weights_of_far_negative_logits(moe, level, k, T):
    """Sigmoids below fp32's range: their ratios are not."""
    H, E = 64, 32
    x, w_r, _, sb = inputs(T, T, H, E, MODES[0])
    lb = (level + 0.3 * np.random.default_rng(1).standard_normal(E)).astype(np.float32)
    got = run(moe, x, w_r, lb, sb, E, k, 8, 3, MODES[0], 2.5)
    ids, w, ggap, egap, c, bound = reference(x, w_r, lb, sb, k, 8, 3, MODES[0], 2.5)
    clear = np.fmin(ggap, egap) > 1e-6
    assert clear.mean() > 0.9 and np.array_equal(got["ids"][clear], ids[clear])
    # a logit is off by its product's error and half a step of its own size (adding the bias), a
    # weight by twice that relatively, and the functions' own 2^-20
    tol = w * (2.5 * bound[:, None] + 2 * 2.0 ** -24 * (abs(level) + 8) + 2.0 ** -20)
    assert np.all(np.abs(got["w"] - w)[clear] <= tol[clear])


@pytest.mark.parametrize("T,E,groups", [(600, 60, 6), (4100, 256, 8)])
def test_nan_rows_of_large_batches(moe, T, E, groups):
    """A NaN activation on the tensor-core product: its own token takes the first experts, the
    others are untouched."""
    x, w_r, lb, sb = inputs(T, T, 128, E, MODES[0])
    bad = [0, 1, 127, 128, T - 1]
    x[bad, [0, 5, 63, 64, 127]] = float("nan")
    got = run(moe, x, w_r, lb, sb, E, 4, groups, 3, MODES[0])
    assert np.array_equal(got["ids"][bad], np.tile(np.arange(4), (5, 1)))
    keep = np.setdiff1d(np.arange(T), bad)
    x2, _, _, _ = inputs(T, T, 128, E, MODES[0])
    want = run(moe, x2, w_r, lb, sb, E, 4, groups, 3, MODES[0])
    assert np.array_equal(got["ids"][keep], want["ids"][keep])
    assert np.array_equal(got["w"][keep], want["w"][keep])


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("pattern", ["thirds", "groups", "all", "low"])
def test_masks_of_large_batches(moe, pattern, mode):
    T, H, E, groups, take, k = 4100, 128, 256, 8, 3, 6
    b = (0.1 * np.random.default_rng(5).standard_normal(E)).astype(np.float32)
    if pattern == "thirds":
        b[::3] = -np.inf
    elif pattern == "groups":
        b[40:] = -np.inf                            # one group and a quarter for three places
    elif pattern == "all":
        b[:] = -np.inf
    else:
        b[:224] = LOW
    lb, sb = (None, b) if mode == MODES[0] else (b, None)
    x, w_r, _, _ = inputs(1, T, H, E, mode)
    got = run(moe, x, w_r, lb, sb, E, k, groups, take, mode)
    check(got, reference(x, w_r, lb, sb, k, groups, take, mode, 1.0), k, E)
    if pattern == "all" and mode != MODES[0]:
        assert (got["w"] == 0).all()
