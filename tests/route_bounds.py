"""What fp32 rounding allows of the logits and weights of group-limited routing (512 tokens and
more: blocks of 64 products of three bf16 pieces summed by the tensor cores, the blocks added in
fp32), as limits that the routing tests hold results to.

A logit's error is the sum of these roundings, each at most

  * 2^-23 of the largest of an instruction's 16 products, its running sum before and after it, for
    each of a block's 12 instructions (the block's sum is cut off, not rounded, there);
  * 2^-24 of the running sum, for each block added and for up to 16 parts of H added at the end;
  * 2^-24 of the logit, for its bias.

`spread` is the root of the sum of their squares.  Independent roundings add up to less than it in
the mean square (a rounding's own mean square is a third of its largest), which is asked of every
token over its experts; and to less than 7 times it in any one logit (Hoeffding: 5e-11).
"""
import numpy as np
import torch


def spread(x, w_r, lb=None, device="cpu"):
    """(fp64 logits, spread of their errors), [T][E]."""
    x, w = x.to(device).double(), torch.as_tensor(w_r).to(device).double()
    T, H = x.shape
    E = w.shape[1]
    total = torch.zeros((T, E), dtype=torch.float64, device=device)
    var, most = torch.zeros_like(total), torch.zeros_like(total)
    for h0 in range(0, H, 64):
        run = torch.zeros_like(total)
        for c in range(h0, min(h0 + 64, H), 16):
            xc, wc = x[:, c:c + 16], w[c:c + 16]
            big = xc.abs().amax(1, keepdim=True) * wc.abs().amax(0, keepdim=True)
            after = run + xc @ wc
            big = torch.maximum(big, torch.maximum(run.abs(), after.abs()))
            var += (2.0 ** -23 * big) ** 2
            run = after
        var += 8 * (2.0 ** -23 * run) ** 2            # the middle and the low piece
        total = total + run
        most = torch.maximum(most, total.abs())
        var += (2.0 ** -24 * total) ** 2
    var += 16 * (2.0 ** -24 * most) ** 2
    if lb is not None:
        total = total + torch.as_tensor(lb).to(device).double()
        var += (2.0 ** -24 * total) ** 2
    return total.cpu().numpy(), var.sqrt().cpu().numpy()


def spread_chain(x, w_r, lb=None, device="cpu"):
    """The same for fewer than 256 tokens: fp32 products and additions, each rounded to 2^-24, in
    one chain over H (cut into parts, the running sums and their number are smaller)."""
    x, w = x.to(device).double(), torch.as_tensor(w_r).to(device).double()
    total = torch.zeros((x.shape[0], w.shape[1]), dtype=torch.float64, device=device)
    var = torch.zeros_like(total)
    for h0 in range(0, x.shape[1], 64):
        terms = x[:, h0:h0 + 64, None] * w[None, h0:h0 + 64]
        run = total[:, None] + terms.cumsum(1)
        var += (2.0 ** -48) * (terms ** 2 + run ** 2).sum(1)
        total = run[:, -1]
    if lb is not None:
        total = total + torch.as_tensor(lb).to(device).double()
        var += (2.0 ** -24 * total) ** 2
    return total.cpu().numpy(), var.sqrt().cpu().numpy()


def logits_ok(got, exact, s):
    err = got.astype(np.float64) - exact
    mean = np.sqrt((err ** 2).mean(1)) <= np.sqrt((s ** 2).mean(1))
    return bool(mean.all() and (np.abs(err) <= 7 * s).all())


def one_hot_rows(rng, T, H):
    """Rows with one value each: a logit is one product, no rounding hides the others."""
    x = torch.zeros((T, H))
    at = rng.integers(0, H, T)
    at[:2] = 0, H - 1
    x[torch.arange(T), torch.from_numpy(at)] = torch.from_numpy(
        rng.uniform(0.5, 2.0, T).astype(np.float32) * rng.choice([-1, 1], T).astype(np.float32))
    return x.to(torch.bfloat16)


def one_hot_ok(got, x, w_r):
    """The three pieces' products are exact and their two additions cut off by at most 2^-23."""
    exact = x.double().numpy() @ w_r.astype(np.float64)
    return bool((np.abs(got - exact) <= 1.001 * 2.0 ** -22 * np.abs(exact)).all())


def weights(l, ids, mode, scale):
    z = np.take_along_axis(l, ids.astype(np.int64), 1)
    if mode == "softmax":
        top = l.max(1, keepdims=True)
        return scale * np.exp(z - top) / np.exp(l - top).sum(1, keepdims=True)
    v = 1 / (1 + np.exp(-z)) if mode == "sigmoid_bias_renorm" else np.exp(z - z.max(1, keepdims=True))
    return scale * v / v.sum(1, keepdims=True)


def weights_ok(got, ref, s):
    """A weight is a ratio of exponentials or sigmoids: off by at most twice its logits' errors,
    and 2^-20 for the functions themselves (each good to a few steps of 2^-23)."""
    rel = np.abs(got / ref - 1)
    mean = np.sqrt((rel ** 2).mean()) <= 2 * np.sqrt((s ** 2).mean()) + 2.0 ** -20
    return bool(mean and (rel <= 14 * s.max(1, keepdims=True) + 2.0 ** -20).all())
