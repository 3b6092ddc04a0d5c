"""The routing tests' limits have to fail wrong sums: a restatement of the router product in numpy
(three bf16 pieces, an instruction of 16 products cut off at a time, blocks of 64 added in fp32)
passes, and fails with any one of the pieces left out or with the blocks summed in 16 bits."""
import numpy as np
import pytest
import torch

from route_bounds import logits_ok, one_hot_ok, one_hot_rows, spread, weights, weights_ok

H, E, T = 7168, 64, 96


def pieces(w):
    out, rest = [], torch.from_numpy(w)
    for _ in range(3):
        p = rest.to(torch.bfloat16).float()
        out.append(p.numpy())
        rest = rest - p
    assert not rest.any()
    return out


def cut(v):
    """fp64 to fp32 towards zero."""
    f = v.astype(np.float32)
    return np.where(np.abs(f.astype(np.float64)) > np.abs(v), np.nextafter(f, np.float32(0)), f)


def product(x, w, left_out=None, half=False):
    xf, acc = x.float().numpy(), np.zeros((x.shape[0], w.shape[1]), np.float32)
    for h in range(0, x.shape[1], 64):
        run = np.zeros_like(acc)
        for i, p in enumerate(pieces(w)):
            for c in range(h, h + 64, 16):
                if i != left_out:
                    run = cut(run + xf[:, c:c + 16].astype(np.float64) @ p[c:c + 16].astype(np.float64))
        acc = acc + (run.astype(np.float16).astype(np.float32) if half else run)
    return acc


@pytest.fixture(scope="module")
def dense():
    rng = np.random.default_rng(2)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16)
    w = (rng.standard_normal((H, E)) * 0.02).astype(np.float32)
    return (x, w) + spread(x, w)


def test_limits_pass_the_product_and_fail_each_piece_left_out(dense):
    x, w, exact, s = dense
    assert np.sqrt((s ** 2).mean()) < 2e-6
    assert logits_ok(product(x, w), exact, s)
    for i in range(3):
        assert not logits_ok(product(x, w, i), exact, s), i
    assert not logits_ok(product(x, w, half=True), exact, s)


@pytest.mark.parametrize("mode", ["sigmoid_bias_renorm", "softmax", "softmax_renorm"])
def test_weights_likewise(dense, mode):
    x, w, exact, s = dense
    ids = np.argsort(-exact, 1)[:, :6]
    ref = weights(exact, ids, mode, 2.5)
    assert weights_ok(weights(product(x, w).astype(np.float64), ids, mode, 2.5).astype(np.float32),
                      ref, s)
    for i in range(2):      # (without the low piece, 2^-18, weights are off by less than the limit)
        assert not weights_ok(weights(product(x, w, i).astype(np.float64), ids, mode, 2.5), ref, s)


def test_one_hot_rows_fail_each_piece_left_out():
    rng = np.random.default_rng(3)
    x = one_hot_rows(rng, T, H)
    w = (rng.standard_normal((H, E)) * 0.02).astype(np.float32)
    assert one_hot_ok(product(x, w), x, w)
    for i in range(3):
        assert not one_hot_ok(product(x, w, i), x, w), i
