"""GPU tests of group-limited routing's logits and weights, held to what fp32 rounding allows
(route_bounds), and of every gating mode, with logit and selection biases, on the tensor-core
product and the two-step gating of large batches.  Ids are compared exactly where the 64-bit gap
is above 1e-6."""
import numpy as np
import pytest
import torch

import route_bounds as rb
from oracle import moe_ref
from test_gpu_route_group import MODES, reference, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import expert_dispatch_streaming_gb300 as m
    return m


def held(moe, x, w_r, lb, sb, k, groups, take, mode, scale, spread):
    T, E = x.shape[0], w_r.shape[1]
    got = run(moe, x, w_r, lb, sb, E, k, groups, take, mode, scale)
    exact, s = spread(x, w_r, lb, "cuda")
    assert rb.logits_ok(got["logits"], exact, s)
    assert rb.weights_ok(got["w"], rb.weights(exact, got["ids"], mode, scale), s)
    ids, _, ggap, egap, _, _ = reference(x, w_r, lb, sb, k, groups, take, mode, scale)
    clear = np.fmin(ggap, egap) > 1e-6
    assert clear.mean() > 0.99 or T < 200
    assert np.array_equal(got["ids"][clear], ids[clear])
    counts, offsets, pos, src = moe_ref.dispatch(got["ids"], E)
    for n, r in (("counts", counts), ("offsets", offsets), ("pos", pos), ("src", src)):
        assert np.array_equal(got[n], r), n


def made(seed, T, H, E, std):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16)
    w_r = (rng.standard_normal((H, E)) * std).astype(np.float32)
    return x, w_r, rng.standard_normal(E).astype(np.float32), (
        0.1 * rng.standard_normal(E)).astype(np.float32)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("T", [3, 40, 516])
def test_full_width(moe, mode, T):
    x, w_r, lb, sb = made(T, T, 7168, 256, 0.02)
    sb, lb = (sb, None) if mode == MODES[0] else (None, lb)
    held(moe, x, w_r, lb, sb, 8, 8, 4, mode, 2.5, rb.spread if T >= 512 else rb.spread_chain)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,groups,take,k", [(60, 6, 3, 4), (256, 8, 4, 8), (160, 8, 3, 6)])
@pytest.mark.parametrize("T", [512, 1100, 4100])
def test_modes_of_large_batches(moe, T, E, groups, take, k, biased, mode):
    x, w_r, lb, sb = made(T + E, T, 1024, E, 0.03)
    held(moe, x, w_r, lb if biased else None, sb if mode == MODES[0] and biased else None, k,
         groups, take, mode, 1.0, rb.spread)


@pytest.mark.parametrize("T", [3, 40, 300, 520, 1100])
def test_one_value_a_row(moe, T):
    """Every logit is one product, good to 2^-22, on every way of computing it."""
    H, E = 7168, 256
    rng = np.random.default_rng(T)
    x = rb.one_hot_rows(rng, T, H)
    w_r = (rng.standard_normal((H, E)) * 0.02).astype(np.float32)
    got = run(moe, x, w_r, None, None, E, 8, 8, 4, "softmax")
    assert rb.one_hot_ok(got["logits"], x, w_r)
