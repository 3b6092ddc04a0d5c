"""GPU tests on whole numbers: inputs whose every product and partial sum is a whole number (of halves)
below 2^24, so that fp32 rounds nothing in whatever order it adds, and results are compared with
equality.  One term left out, taken twice or multiplied by another's scale shows at any length.

The 4-bit products here give each CTA several items: the weights' ring, the steps' order and the first
values ahead of an item run on from one item to the next, with items of 16, 32 and 48 weight rows,
wide and single loads of scales, and K steps that are and are not a multiple of the warps."""
import numpy as np
import pytest
import torch

from test_gpu_dispatch_grad import dispatch, gen, moe  # noqa: F401
from test_gpu_gemv_int4 import run, values

pytestmark = pytest.mark.gpu


def slots():
    """CTAs that run side by side."""
    return 2 * torch.cuda.get_device_properties(0).multi_processor_count


def height(E, N, rows):
    """Units of 16 weight rows of an item, by the library's rule: the rounds of items times what one
    costs, ties to the higher."""
    most = (rows + 7 * min(E, rows)) // 8
    passes = max(1, min(most, (E + 1) // 2 + rows // 8))
    cost = {n: -(-passes * -(-N // (16 * n)) // slots()) * (n + 1) for n in (1, 2, 3)}
    return max(n for n in cost if cost[n] == min(cost.values()))


def uneven(E, passes, seed):
    """Rows of E experts, some without any, of about `passes` eights in all (no fewer)."""
    rng = np.random.default_rng(seed)
    c = rng.integers(1, 2 * (8 * passes // E), E)
    c[rng.permutation(E)[:E // 6]] = 0
    c[0] = 1
    c[-1] += max(0, 8 * (passes - sum(-(-int(v) // 8) for v in c)))
    return [int(v) for v in c]


def shapes():
    """(units of an item, rows per expert, N) with at least three items a CTA (six for the third), by name."""
    s = slots()
    few = [1, 2, 0, 1, 1, 9, 1, 1]                     # eight passes, six by the rule of the height
    return {
        "16 rows, one tile": (1, uneven(24, 3 * s, 1), 13),
        "16 rows, full tile": (1, uneven(200, 3 * s, 2), 16),
        "32 rows, tiles": (2, few, 32 * (19 * s // 4 // 6) - 3),
        "32 rows, one tile": (2, uneven(24, 3 * s, 3), 29),
        "48 rows, one tile": (3, uneven(24, 3 * s, 4), 48),
        "48 rows, tiles": (3, few, 48 * -(-3 * s // 8) + 5),
        "48 rows, passes and tiles": (3, uneven(9, s // 2, 5), 48 * 7 - 1),
        "48 rows, dense": (3, [5], 48 * 3 * s - 5),
    }


NAMES = ["16 rows, one tile", "16 rows, full tile", "32 rows, tiles", "32 rows, one tile", "48 rows, one tile",
         "48 rows, tiles", "48 rows, passes and tiles", "48 rows, dense"]


@pytest.mark.parametrize("K", [2304, 2400, 4096, 7136])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("name", NAMES)
def test_gemv_several_items_a_cta(moe, name, group, zero, K):  # noqa: F811
    units, counts, N = shapes()[name]
    E, rows = len(counts), sum(counts)
    assert height(E, N, rows) == units
    items = sum(-(-c // 8) for c in counts) * -(-N // (16 * units))
    assert items >= 3 * slots()
    if N > 10000:
        K = min(K, 2400 if K % 256 else 2304)          # (memory of the 64-bit form)
    g = gen(N + K + group)
    ng = -(-K // group)
    w = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.exp2(torch.randint(-1, 2, (E, N, ng), generator=g, device="cuda").float())
    s = (s * (1 - 2 * torch.randint(0, 2, (E, N, ng), generator=g, device="cuda"))).to(torch.bfloat16)
    z = (torch.randint(0, 17, (E, N, ng), generator=g, device="cuda", dtype=torch.uint8) if zero
         else None)
    x = torch.randint(-2, 3, (rows, K), generator=g, device="cuda").to(torch.bfloat16)
    # |code - zero| <= 16, |x| <= 2, |s| <= 2, in halves
    assert 16 * 2 * 2 * 2 * K < 2 ** 24
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    want = torch.empty((rows, N), device="cuda")
    r0 = 0
    for e, n in enumerate(counts):
        if n:
            v = values(w[e], s[e], None if z is None else z[e], group)
            want[r0:r0 + n] = (x[r0:r0 + n].double() @ v.T).float()
        r0 += n
    for out, ref in (("fp32", want), ("bf16", want.to(torch.bfloat16))):
        y, ws = run(moe, x, w, s, z, off if E > 1 else None, group, rows, out, N, K, E)
        assert moe.moe_workspace_error(ws) == 0
        assert torch.equal(y[:rows], ref) and torch.all(y[rows:] == 5.0)


@pytest.mark.parametrize("T,E,k,H", [(1, 8, 2, 7168), (37, 60, 8, 7168), (300, 256, 8, 7168), (9, 4, 3, 16376)])
def test_combine_backward_long_rows(moe, T, E, k, H):  # noqa: F811
    """Dot products over long rows."""
    g = gen(T)
    _, _, pos, _ = dispatch(moe, T, E, k, 0.2, 3)
    live = pos >= 0
    dout, sh = (torch.randint(-8, 9, (T, H), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    y = torch.randint(-8, 9, (T * k, H), generator=g, device="cuda").to(torch.bfloat16)
    w, gate = torch.ones((T, k), device="cuda"), torch.ones(T, device="cuda")
    dw, dg = torch.empty((T, k), device="cuda"), torch.empty(T, device="cuda")
    moe.moe_combine_backward(dout, y, pos, w, T, k, H, sh, gate, None, dw, None, dg)
    at = torch.where(live[:, :, None], y[pos.clamp_min(0).long()].double(), 0.0)
    assert torch.equal(dw.double(), (dout.double()[:, None] * at).sum(2))
    assert torch.equal(dg.double(), (dout.double() * sh.double()).sum(1))


@pytest.mark.parametrize("T,E,k,H", [(1, 8, 8, 7168), (37, 60, 8, 7168), (130, 9, 5, 1032)])
def test_permute_backward_whole_numbers(moe, T, E, k, H):  # noqa: F811
    g = gen(T)
    _, _, pos, _ = dispatch(moe, T, E, k, 0.2, 4)
    d = torch.randint(-8, 9, (T * k, H), generator=g, device="cuda").to(torch.bfloat16)
    add = torch.randint(-8, 9, (T, H), generator=g, device="cuda").to(torch.bfloat16)
    want = torch.where((pos >= 0)[:, :, None], d[pos.clamp_min(0).long()].double(), 0.0).sum(1) + add.double()
    for out, t in (("fp32", torch.float32), ("bf16", torch.bfloat16)):
        dx = torch.empty((T, H), device="cuda", dtype=t)
        moe.moe_permute_backward(d, pos, add, T, k, H, out, dx)
        assert torch.equal(dx.double(), want)        # (|sums| <= 72: whole numbers that bf16 holds)


@pytest.mark.parametrize("rows", [1, 40])
def test_gemv_of_no_rows(moe, rows):  # noqa: F811
    """Offsets that give no expert a row: nothing is written, and no error recorded."""
    N, K, E = 50, 320, 5
    g = gen(1)
    w = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.ones((E, N, K // 32), dtype=torch.bfloat16, device="cuda")
    x = torch.ones((rows, K), dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    y, ws = run(moe, x, w, s, None, off, 32, rows, "fp32", N, K, E)
    assert torch.all(y == 5.0) and moe.moe_workspace_error(ws) == 0
