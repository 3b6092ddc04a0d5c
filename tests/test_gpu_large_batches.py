"""GPU tests of the dispatch and its gradients at batches whose sizes come near 2^31, with the smallest
rows: index arithmetic has to hold up to the documented limit T * k < 2^31.  Values are compared in pieces;
a test that does not find the memory it needs is skipped."""
import pytest
import torch

from test_gpu_dispatch_grad import gen, moe  # noqa: F401

pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
PIECE = 1 << 26


def need(gigabytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < (gigabytes + 8) << 30:
        pytest.skip(f"needs {gigabytes} GB")


@pytest.fixture(autouse=True)
def free_again():
    yield
    torch.cuda.empty_cache()


def rows_of(n, H, seed):
    """[n][H] bf16 of small whole numbers, a different row for any two neighbours."""
    x = torch.empty((n, H), dtype=BF, device="cuda")
    g = gen(seed)
    for lo in range(0, n, PIECE):
        m = min(PIECE, n - lo)
        x[lo:lo + m] = torch.randint(-8, 9, (m, H), generator=g, device="cuda", dtype=torch.int8)
    return x


def pieces(n):
    return [(lo, min(lo + PIECE, n)) for lo in range(0, n, PIECE)]


def test_combine_backward_of_more_than_two_to_the_thirtieth_tokens(moe):  # noqa: F811
    """A token a CTA: the index of the last ones passes 2^30.  Sums of whole numbers are exact."""
    need(50)
    T, H = (1 << 30) + 5, 8
    dout, y = rows_of(T, H, 1), rows_of(T, H, 2)
    pos = torch.arange(T - 1, -1, -1, dtype=I32, device="cuda")
    w, dw = torch.ones(T, device="cuda"), torch.full((T,), 5.5, device="cuda")
    moe.moe_combine_backward(dout, y, pos, w, T, 1, H, None, None, None, dw)
    for lo, hi in pieces(T):
        want = (dout[lo:hi].float() * y[T - hi:T - lo].flip(0).float()).sum(1)
        assert torch.equal(dw[lo:hi], want)


def test_permute_backward_and_combine_of_the_largest_batch(moe):  # noqa: F811
    """T * k = 2^31 - 1, rows in reverse order: a block's steps over the tokens end past 2^31."""
    need(125)
    T, H = (1 << 31) - 1, 8
    y, pos = rows_of(T, H, 3), torch.arange(T - 1, -1, -1, dtype=I32, device="cuda")
    out = torch.full((T, H), 5.5, dtype=BF, device="cuda")
    moe.moe_permute_backward(y, pos, None, T, 1, H, "bf16", out)
    for lo, hi in pieces(T):
        assert torch.equal(out[lo:hi], y[T - hi:T - lo].flip(0))
    w = torch.full((T,), 0.5, device="cuda")
    moe.moe_combine(y, pos, w, T, 1, H, None, None, None, out)
    for lo, hi in pieces(T):
        assert torch.equal(out[lo:hi], y[T - hi:T - lo].flip(0) * 0.5)
    # whole rows of equal values: their root mean square is the value
    w[:] = 2.0
    for lo, hi in pieces(T):
        y[lo:hi] = y[lo:hi, :1] + 9
    normed = torch.full((T, H), 5.5, dtype=BF, device="cuda")
    moe.moe_combine(y, pos, w, T, 1, H, None, None, None, out, out_normed=normed, norm_eps=0.0)
    for lo, hi in pieces(T):
        assert torch.equal(out[lo:hi], y[T - hi:T - lo].flip(0) * 2.0)
        assert torch.all(normed[lo:hi] == 1.0)


@pytest.mark.parametrize("T,k", [((1 << 26) + 3, 1), ((1 << 26) + 1, 2), ((1 << 31) - 1, 1)])
def test_permute_of_large_batches(moe, T, k):  # noqa: F811
    """One warp a row: the threads in all pass 2^31 and 2^32."""
    rows, H = T * k, 8
    need(90 if rows > 1 << 30 else 8)
    x = rows_of(T, H, 4)
    src = torch.arange(rows - 1, -1, -1, dtype=I32, device="cuda")
    src[::5] = -1
    xp = torch.full((rows, H), 5.5, dtype=BF, device="cuda")
    moe.moe_permute(x, src, T, k, H, xp)
    for lo, hi in pieces(rows):
        s = src[lo:hi].long()
        want = x[s.clamp_min(0) // k] * (s >= 0)[:, None]
        assert torch.equal(xp[lo:hi], want)


def test_sort_of_the_most_slots(moe):  # noqa: F811
    """2^31 - 1 slots, experts in turn and every fifth slot without one."""
    need(40)
    n, E = (1 << 31) - 1, 4
    ids = torch.empty(n, dtype=I32, device="cuda")
    for lo, hi in pieces(n):
        ids[lo:hi] = torch.arange(lo, hi, device="cuda") % 5          # 4: no expert
    i32 = dict(dtype=I32, device="cuda")
    counts, offsets = torch.full((E,), 7, **i32), torch.full((E + 1,), 7, **i32)
    pos, src = torch.full((n,), 7, **i32), torch.full((n,), 7, **i32)
    nb = moe.moe_sort_tokens_workspace_size(n, E, 1)
    moe.moe_sort_tokens(ids, n, E, 1, counts, offsets, pos, src,
                        torch.empty(nb, dtype=torch.uint8, device="cuda"), nb)
    per = [(n - e + 4) // 5 for e in range(E)]
    at = [sum(per[:e]) for e in range(E + 1)]
    assert counts.tolist() == per and offsets.tolist() == at
    start = torch.tensor(at[:E] + [0], device="cuda")
    for lo, hi in pieces(n):
        s = torch.arange(lo, hi, device="cuda")
        assert torch.equal(pos[lo:hi].long(), torch.where(s % 5 < 4, start[s % 5] + s // 5, -1))
        e = (s[:, None] >= torch.tensor(at[1:], device="cuda")).sum(1)
        assert torch.equal(src[lo:hi].long(), torch.where(e < 4, 5 * (s - start[e]) + e, -1))
