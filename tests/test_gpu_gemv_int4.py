"""GPU tests of moe_grouped_gemv_int4 against its definition in 64 bits, and of a run of the operators
together: sort, permute, 4-bit products, combine and the router's gradient.

Tolerances.  The products of a group (code minus zero point times a bf16 value) are exact; the fp32
sums of the K products of an output and of its groups may be off by one unit of the last place
(2^-23) of the sum S of the terms' magnitudes per addition, so by (K + groups) * 2^-23 * S; a bf16
result by half a step (2^-8 of its value) more.
"""
import numpy as np
import pytest
import torch

from test_gpu_dispatch_grad import dispatch, gate_weights, gen, moe, run_sort  # noqa: F401

pytestmark = pytest.mark.gpu


def weights(g, E, N, K, group, zero):
    ng = -(-K // group)
    w = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.randn((E, N, ng), generator=g, device="cuda") * 0.02).to(torch.bfloat16)
    z = (torch.randint(0, 17, (E, N, ng), generator=g, device="cuda", dtype=torch.uint8)
         if zero else None)
    return w, s, z


def values(w, s, z, group):
    """64-bit values of one expert's weights, and their codes."""
    N, K = w.shape[0], w.shape[1] * 2
    q = torch.stack([w & 15, w >> 4], 2).view(N, K).double()
    at = torch.arange(K, device=w.device) // group
    zero = 8.0 if z is None else z.double()[:, at]
    return (q - zero) * s.double()[:, at]


def run(moe, x, w, s, z, off, group, max_rows, out, N, K, E, y=None, stream=None):
    nb = moe.moe_grouped_gemv_int4_workspace_size(max_rows, E, N, K)
    ws = torch.full((nb,), 0x5A, dtype=torch.uint8, device="cuda")
    if y is None:
        y = torch.full((max_rows + 1, N), 5.0, device="cuda",
                       dtype=torch.bfloat16 if out == "bf16" else torch.float32)
    moe.moe_grouped_gemv_int4(x, w, s, z, off, E, N, K, group, max_rows, out, y, ws, nb, stream)
    return y, ws


def check(x, w, s, z, counts, group, out, y):
    E, r0 = w.shape[0], 0
    for e in range(E):
        n = counts[e]
        if n:
            v = values(w[e], s[e], None if z is None else z[e], group)
            xe = x[r0:r0 + n].double()
            want, mag = xe @ v.T, xe.abs() @ v.abs().T
            tol = mag * (v.shape[1] + s.shape[2]) * 2.0 ** -23
            if out == "bf16":
                tol = tol + want.abs() * 2.0 ** -8
            assert torch.all((y[r0:r0 + n].double() - want).abs() <= tol), e
        r0 += n
    assert torch.all(y[r0:] == 5.0)


CASES = [  # counts of rows per expert, N, K
    ([1], 1, 32), ([1], 17, 96), ([2], 63, 1440), ([1], 4096, 7168), ([8], 130, 256),
    ([9], 100, 160), ([16], 33, 2080), ([17], 128, 1024), ([33], 65, 992), ([64], 257, 544),
    ([130], 48, 320), ([0, 3, 0, 1, 12, 0], 1000, 1440), ([0] * 255 + [1], 31, 128),
    ([1] * 256, 16, 64), ([5, 0, 41, 1, 8, 7, 0, 2], 95, 416), ([1, 1, 1, 1, 1, 1, 1, 1], 2049, 736),
]


@pytest.mark.parametrize("counts,N,K", CASES, ids=lambda v: str(v)[:24])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_gemv(moe, counts, N, K, group, zero, out):  # noqa: F811
    E, rows = len(counts), sum(counts)
    g = gen(N + K + rows)
    w, s, z = weights(g, E, N, K, group, zero)
    x = torch.randn((rows, K), generator=g, device="cuda").to(torch.bfloat16)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    y, ws = run(moe, x, w, s, z, off, group, rows, out, N, K, E)
    check(x, w, s, z, counts, group, out, y)
    assert moe.moe_workspace_error(ws) == 0
    if E == 1:
        y2, _ = run(moe, x, w, s, z, None, group, rows, out, N, K, E)
        assert torch.equal(y, y2)


@pytest.mark.parametrize("group", [32, 128])
def test_gemv_rows_do_not_mix(moe, group):  # noqa: F811
    """A NaN or an infinity in a token row reaches that row only, one in a scale its weight row."""
    counts, N, K = [3, 0, 9], 40, 288
    g = gen(2)
    w, s, z = weights(g, 3, N, K, group, True)
    x = torch.randn((12, K), generator=g, device="cuda").to(torch.bfloat16)
    off = torch.tensor([0, 3, 3, 12], dtype=torch.int32, device="cuda")
    ref, _ = run(moe, x, w, s, z, off, group, 12, "fp32", N, K, 3)
    x2, s2 = x.clone(), s.clone()
    x2[5, 17], x2[1, 280] = float("nan"), float("inf")
    s2[2, 21, 1] = float("nan")
    got, _ = run(moe, x2, w, s2, z, off, group, 12, "fp32", N, K, 3)
    bad = torch.zeros((13, N), dtype=torch.bool, device="cuda")
    bad[5] = bad[1] = True
    bad[3:12, 21] = True
    assert torch.all(torch.isnan(got[5])) and torch.all(torch.isnan(got[3:12, 21]))
    assert not torch.any(torch.isfinite(got[1]))
    assert torch.equal(got[~bad], ref[~bad])


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("K", [32, 288, 1440, 2048])
def test_gemv_infinite_last_scale(moe, K, group, zero):  # noqa: F811
    """An infinite scale of a row's last group: infinity with the sign of that group's sum."""
    N, rows = 70, 5
    g = gen(K + group)
    w, s, z = weights(g, 1, N, K, group, zero)
    x = torch.randn((rows, K), generator=g, device="cuda").to(torch.bfloat16)
    s[0, 33, -1] = float("inf")
    y, _ = run(moe, x, w, s, z, None, group, rows, "fp32", N, K, 1)
    one = torch.ones_like(s)
    one[0, :, :-1] = 0
    last = x.double() @ values(w[0], one[0], None if z is None else z[0], group).T
    assert torch.all(last[:, 33] != 0)
    assert torch.equal(y[:rows, 33].double(), torch.sign(last[:, 33]) * float("inf"))
    assert torch.all(torch.isfinite(y[:rows, :33])) and torch.all(torch.isfinite(y[:rows, 34:]))


@pytest.mark.parametrize("group", [32, 64, 128])
def test_gemv_unaligned_scales(moe, group):  # noqa: F811
    """Scales and zero points that start on no 16-byte boundary: the aligned call's result, to the bit."""
    counts, N, K = [1, 5], 70, 768
    g = gen(group)
    w, s, z = weights(g, 2, N, K, group, True)
    x = torch.randn((6, K), generator=g, device="cuda").to(torch.bfloat16)
    off = torch.tensor([0, 1, 6], dtype=torch.int32, device="cuda")
    ref, _ = run(moe, x, w, s, z, off, group, 6, "fp32", N, K, 2)
    check(x, w, s, z, counts, group, "fp32", ref)
    s2 = torch.empty(s.numel() + 1, dtype=s.dtype, device="cuda")[1:].copy_(s.view(-1))
    z2 = torch.empty(z.numel() + 3, dtype=z.dtype, device="cuda")[3:].copy_(z.view(-1))
    assert s2.data_ptr() % 16 == 2 and z2.data_ptr() % 16 == 3
    for a, b in ((s2, z), (s, z2), (s2, z2)):
        got, _ = run(moe, x, w, a, b, off, group, 6, "fp32", N, K, 2)
        assert torch.equal(got, ref)


def test_gemv_all_zero_points_and_codes(moe):  # noqa: F811
    """Every code against every documented zero point: the value is exact."""
    N, K = 16, 32
    codes = torch.arange(16, dtype=torch.uint8, device="cuda")
    w = (codes | (codes << 4))[:, None].expand(N, K // 2).contiguous()[None]
    x = torch.zeros((1, K), dtype=torch.bfloat16, device="cuda")
    x[0, 5] = 1.0
    s = torch.ones((1, N, 1), dtype=torch.bfloat16, device="cuda")
    for zp in range(128):
        z = torch.full((1, N, 1), zp, dtype=torch.uint8, device="cuda")
        y, _ = run(moe, x, w, s, z, None, 32, 1, "fp32", N, K, 1)
        assert torch.equal(y[0], codes.float() - zp)


def test_gemv_clips_ranges(moe):  # noqa: F811
    N, K = 24, 64
    g = gen(6)
    w, s, z = weights(g, 3, N, K, 32, False)
    x = torch.randn((6, K), generator=g, device="cuda").to(torch.bfloat16)
    off = torch.tensor([-2, 3, 5, 11], dtype=torch.int32, device="cuda")
    y, ws = run(moe, x, w, s, z, off, 32, 6, "fp32", N, K, 3)
    check(x, w, s, z, [3, 2, 1], 32, "fp32", y)
    assert moe.moe_workspace_error(ws) == 8
    # the next call on the workspace reports its own state
    off = torch.tensor([0, 3, 5, 6], dtype=torch.int32, device="cuda")
    moe.moe_grouped_gemv_int4(x, w, s, z, off, 3, N, K, 32, 6, "fp32", y, ws, ws.numel())
    assert moe.moe_workspace_error(ws) == 0
    # ranges that run backwards are empty
    off = torch.tensor([4, 2, 2, 6], dtype=torch.int32, device="cuda")
    y.fill_(5.0)
    moe.moe_grouped_gemv_int4(x, w, s, z, off, 3, N, K, 32, 6, "fp32", y, ws, ws.numel())
    assert torch.all(y[:2] == 5.0) and torch.all(y[2:6] != 5.0)


def test_gemv_past_32_bits(moe):  # noqa: F811
    """Weights of more than 4 GB: the last expert's are reached."""
    E, N, K = 256, 4112, 8256
    assert E * N * (K // 2) > 2 ** 32
    g = gen(7)
    w = torch.empty((E, N, K // 2), dtype=torch.uint8, device="cuda")
    w[:] = 0x88
    w[-1] = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.ones((E, N, K // 32 + (K % 32 > 0)), dtype=torch.bfloat16, device="cuda")
    x = torch.randn((3, K), generator=g, device="cuda").to(torch.bfloat16)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = 1
    off[E] = 3
    y, _ = run(moe, x, w, s, None, off, 32, 3, "fp32", N, K, E)
    assert torch.all(y[0] == 0)
    v = values(w[-1], s[-1], None, 32)
    xe = x[1:].double()
    assert torch.all((y[1:3].double() - xe @ v.T).abs() <= (xe.abs() @ v.abs().T) * (K + 258) * 2.0 ** -23)


def test_gemv_streams_and_graph(moe):  # noqa: F811
    """Two streams with a workspace each, and a captured call replayed with other rows."""
    counts, N, K, E = [4, 0, 1, 7], 200, 480, 4
    g = gen(10)
    w, s, z = weights(g, E, N, K, 64, True)
    off = torch.tensor([0, 4, 4, 5, 12], dtype=torch.int32, device="cuda")
    xs = [torch.randn((12, K), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    refs = [run(moe, x, w, s, z, off, 64, 12, "bf16", N, K, E)[0] for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    ys = [torch.empty((12, N), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    wss = [torch.empty(256, dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for i in range(2):
            moe.moe_grouped_gemv_int4(xs[i], w, s, z, off, E, N, K, 64, 12, "bf16", ys[i], wss[i],
                                      256, streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(ys[i], refs[i][:12])
    graph = torch.cuda.CUDAGraph()
    xin, yout = xs[0].clone(), torch.full((13, N), 5.0, dtype=torch.bfloat16, device="cuda")
    ooff = off.clone()
    with torch.cuda.graph(graph, stream=streams[0]):
        moe.moe_grouped_gemv_int4(xin, w, s, z, ooff, E, N, K, 64, 12, "bf16", yout, wss[0], 256,
                                  streams[0])
    xin.copy_(xs[1])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(yout[:12], refs[1][:12])
    ooff.copy_(torch.tensor([0, 0, 2, 2, 3], dtype=torch.int32))
    yout.fill_(5.0)
    graph.replay()
    torch.cuda.synchronize()
    check(xin, w, s, z, [0, 2, 0, 1], 64, "bf16", yout)


@pytest.mark.parametrize("gating,scale", [("softmax_renorm", 1.0), ("softmax", 1.0),
                                          ("sigmoid_bias_renorm", 2.5)])
def test_router_training_step(moe, gating, scale):  # noqa: F811
    """A router's training step around frozen 4-bit experts: route, drop the padding, sort, permute,
    the experts' products, combine; then the way back to the logits and to the tokens.  Every stage
    against 64 bits on the stage's own inputs."""
    T, H, E, k, group = 77, 288, 20, 4, 32
    g = gen(21)
    i32 = dict(dtype=torch.int32, device="cuda")
    bf = torch.bfloat16
    x = torch.randn((T, H), generator=g, device="cuda").to(bf)
    w_r = torch.randn((H, E), generator=g, device="cuda") * 0.05
    ids, wt = torch.empty((T, k), **i32), torch.empty((T, k), device="cuda")
    logits = torch.empty((T, E), device="cuda")
    disp = [torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty((T, k), **i32),
            torch.empty(T * k, **i32)]
    nb = moe.moe_route_workspace_size(T, H, E, k)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    moe.moe_route_topk(x, w_r, None, None, None, None, T, H, E, k, gating, scale, ids, wt, *disp,
                       logits, None, None, ws, nb)
    ids[60:] = -1                                     # the batch's padding
    counts, off, pos, src = run_sort(moe, ids, E)
    rows = int(off[-1])
    assert rows == 60 * k
    xp = torch.empty((T * k, H), dtype=bf, device="cuda")
    moe.moe_permute(x, src, T, k, H, xp)
    w4, s4, z4 = weights(g, E, H, H, group, True)
    y, ws4 = run(moe, xp, w4, s4, z4, off, group, T * k, "bf16", H, H, E)
    check(xp, w4, s4, z4, counts.tolist(), group, "bf16", y)
    y = y[:T * k]
    out = torch.empty((T, H), dtype=bf, device="cuda")
    moe.moe_combine(y, pos, wt, T, k, H, None, None, None, out)
    assert torch.all(out[60:] == 0)
    dout = torch.randn((T, H), generator=g, device="cuda").to(bf)
    dy = torch.zeros_like(y)
    dw = torch.empty((T, k), device="cuda")
    dz = torch.empty((T, E), device="cuda")
    dx = torch.empty((T, H), device="cuda")
    moe.moe_combine_backward(dout, y, pos, wt, T, k, H, None, None, dy, dw)
    moe.moe_gate_backward(logits, ids, dw, T, E, k, gating, scale, dz)
    moe.moe_permute_backward(dy, pos, None, T, k, H, "fp32", dx)
    # the loss <dout, out> as a function of the logits, on the products' own values
    z64 = logits.double().requires_grad_(True)
    w64 = gate_weights(z64, ids, gating, scale)
    yt = torch.where((pos >= 0)[:, :, None], y[pos.clamp_min(0).long()].double(), 0.0)
    dots = torch.einsum("th,tkh->tk", dout.double(), yt)
    (want,) = torch.autograd.grad((w64 * dots).sum(), z64)
    size = torch.einsum("th,tkh->tk", dout.abs().double(), yt.abs()).sum(1, keepdim=True)
    # dw is off by (H + 2) 2^-24 of its terms' magnitudes, the gating by (E + 64) 2^-23 (see the
    # gating's own test); both reach an element with a factor of at most 2 scale
    assert torch.all((dz.double() - want).abs() <= 2 * scale * size * (H + E + 66) * 2.0 ** -23)
    assert torch.all(dz[60:] == 0) and torch.all(dx[60:] == 0)
    dy64 = torch.where((pos >= 0)[:, :, None], dy[pos.clamp_min(0).long()].double(), 0.0)
    assert torch.all((dx.double() - dy64.sum(1)).abs() <= dy64.abs().sum(1) * (k + 2) * 2.0 ** -24)
