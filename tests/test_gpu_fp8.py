"""GPU tests of the FP8 expert path: quantisation, the grouped FP8 product and the SwiGLU expert
FFN on FP8 bundles, against plain 64-bit forms of their definitions.

Tolerances.  Quantisation is compared bit for bit: its definition is a fixed sequence of fp32
operations.  A product's fp32 result may be off by one unit of the last place (2^-23) of the
sum of its terms' magnitudes S per addition: within a block of 128 and over the blocks, so by
(128 + blocks + 3) * 2^-23 * S; a bf16 result by half a step (2^-8 relative) more.  The SwiGLU's
result also carries the rounding of h to E4M3: an h within the fp32 error of a rounding border
may take the neighbouring code, so it is held to the layer's tolerance (max |err| <= 2e-2 max
|ref|, sum |err| <= 5e-3 sum |ref|).
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
NB = lambda n: -(-n // 128)  # noqa: E731


@pytest.fixture(scope="module")
def moe():
    import expert_dispatch_streaming_gb300 as m
    return m


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def quant_ref(x):
    """The definition in fp32, on the CPU: codes and scales of fp32 rows."""
    x = x.float().cpu()
    R, H = x.shape
    pad = torch.zeros((R, NB(H) * 128))
    pad[:, :H] = x
    b = pad.view(R, NB(H), 128)
    amax = torch.nan_to_num(b.abs(), nan=0.0, posinf=float("inf")).amax(2)
    amax = torch.maximum(amax, torch.tensor(2.0 ** -96))
    v = b * (torch.tensor(448.0) / amax)[:, :, None]
    return v.to(F8).view(R, -1)[:, :H].contiguous(), amax / 448.0


def quantize(moe, x, src=None, k=0, stream=None):
    T, H = x.shape
    rows = T * k if src is not None else T
    q = torch.full((rows, H), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((rows, NB(H)), -1.0, device="cuda")
    moe.moe_quantize_fp8(x, src, T, k, H, q, s, stream)
    return q, s


def same_codes(q, ref):
    a, b = q.cpu(), ref.view(torch.uint8)
    nan_a, nan_b = (a & 0x7F) == 0x7F, (b & 0x7F) == 0x7F
    return torch.equal(nan_a, nan_b) and torch.equal(a[~nan_a], b[~nan_b])


# ------------------------------------------------------------------------------ quantisation
@pytest.mark.parametrize("H", [16, 128, 144, 2048, 7168])
@pytest.mark.parametrize("T", [1, 3, 130])
def test_quantize_rows(moe, T, H):
    g = gen(T * 10007 + H)
    x = (randn(g, T, H) * torch.exp(2 * randn(g, T, 1))).to(torch.bfloat16)
    q, s = quantize(moe, x)
    rq, rs = quant_ref(x)
    assert same_codes(q, rq) and torch.equal(s.cpu(), rs)


@pytest.mark.parametrize("T,k,H", [(1, 8, 256), (5, 1, 48), (67, 3, 400), (300, 8, 1024)])
def test_quantize_gathers_rows(moe, T, k, H):
    g = gen(T + H)
    x = randn(g, T, H).to(torch.bfloat16)
    src = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32)
    q, s = quantize(moe, x, src, k)
    rq, rs = quant_ref(x[(src // k).long()])
    assert same_codes(q, rq) and torch.equal(s.cpu(), rs)


def test_quantize_special_values(moe):
    """Zero blocks, tiny and huge magnitudes, NaN (kept, ignored by the scale), infinities
    (their block's scale is infinite) and negative zeros."""
    x = torch.zeros((9, 256), dtype=torch.bfloat16, device="cuda")
    x[1, :128] = 1e-38
    x[2] = torch.linspace(-3e38, 3e38, 256, device="cuda").to(torch.bfloat16)
    x[3, 5] = float("nan")
    x[3, 6:20] = 2.5
    x[4, 7] = float("inf")
    x[4, 8] = 1.0
    x[4, 200] = 3.0
    x[5] = -0.0
    x[6, 3] = float("-inf")
    x[7] = float("nan")
    x[8, 130] = 2.0 ** -100
    q, s = quantize(moe, x)
    rq, rs = quant_ref(x)
    assert same_codes(q, rq) and torch.equal(s.cpu(), rs)
    assert s[4, 0].isinf() and s[4, 1] == 3.0 / 448 and s[3, 0] == 2.5 / 448


def test_quantize_out_of_range_sources_give_zero_rows(moe):
    x = torch.ones((4, 64), dtype=torch.bfloat16, device="cuda")
    src = torch.tensor([0, 8, -1, 7, 2 ** 31 - 1, -2 ** 31, 3, 5], dtype=torch.int32, device="cuda")
    q, s = quantize(moe, x, src, 2)
    zero = (q == 0).all(1).cpu().tolist()
    assert zero == [False, True, True, False, True, True, False, False]


def test_quantize_offsets_past_32_bits(moe):
    """More than 2^31 codes: the last rows are right too."""
    T, H = 300_000, 7168
    x = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    x.fill_(1.0)
    x[-3:] = randn(gen(1), 3, H).to(torch.bfloat16)
    q, s = quantize(moe, x)
    rq, rs = quant_ref(x[-3:])
    assert same_codes(q[-3:], rq) and torch.equal(s[-3:].cpu(), rs)


# ------------------------------------------------------------------------------ products
def fp8_rows(g, rows, K):
    x = randn(g, rows, K)
    q, s = quant_ref(x) if rows * K < 1 << 22 else quant_gpu(x)
    return q.cuda(), s.cuda()


def quant_gpu(x):
    R, K = x.shape
    pad = torch.nn.functional.pad(x, (0, -K % 128)).view(R, NB(K), 128)
    amax = pad.abs().amax(2).clamp_min(2.0 ** -96)
    return (pad * (448.0 / amax)[:, :, None]).to(F8).view(R, -1)[:, :K].contiguous(), amax / 448.0


def fp8_weights(g, E, N, K):
    w = torch.empty((E, N, K), dtype=F8, device="cuda")
    s = torch.empty((E, NB(N), NB(K)), device="cuda")
    for e in range(E):
        v = torch.nn.functional.pad(randn(g, N, K) * 0.02, (0, -K % 128, 0, -N % 128))
        b = v.view(NB(N), 128, NB(K), 128)
        amax = b.abs().amax(dim=(1, 3))
        s[e] = amax / 448.0
        w[e] = (b * (448.0 / amax)[:, None, :, None]).to(F8).view(v.shape)[:N, :K]
    return w, s


def spread(s, n, dim):
    return s.double().repeat_interleave(128, dim).narrow(dim, 0, n)


def product_ref(q, xs, w, ws):
    """64-bit product of FP8 rows and one weight, and the sum of its terms' magnitudes."""
    K, N = q.shape[1], w.shape[0]
    x = q.double() * spread(xs, K, 1)
    m = w.double() * spread(spread(ws, N, 0), K, 1)
    return x @ m.T, x.abs() @ m.abs().T


def offsets_of(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def run_gemm(moe, q, xs, w, ws, offsets, out, max_rows=None, stream=None, y=None):
    E, N, K = w.shape
    rows = q.shape[0] if max_rows is None else max_rows
    if y is None:
        y = torch.full((rows, N), -77.0, device="cuda",
                       dtype=torch.bfloat16 if out == "bf16" else torch.float32)
    n = moe.moe_grouped_gemm_fp8_workspace_size(rows, E, N, K)
    scratch = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    moe.moe_grouped_gemm_fp8(q, xs, w, ws, offsets, E, N, K, rows, out, y, scratch, n, stream)
    return y, scratch


def check_rows(y, ref, mag, K, out):
    err = (y.double() - ref).abs()
    tol = (128 + NB(K) + 3) * 2.0 ** -23 * mag
    if out == "bf16":
        tol = tol + 2.0 ** -8 * ref.abs()
    worst = (err - tol).max().item() if err.numel() else 0.0
    assert worst <= 0, f"off by {(err / mag.clamp_min(1e-30)).max().item():.3e} of the terms' sum"


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("N,K", [(128, 128), (256, 512), (1, 16), (130, 144), (1000, 1200),
                                 (384, 2048), (77, 4096)])
@pytest.mark.parametrize("rows", [1, 33, 200])
def test_dense_product(moe, rows, N, K, out):
    g = gen(rows + 31 * N + K)
    q, xs = fp8_rows(g, rows, K)
    w, ws = fp8_weights(g, 1, N, K)
    y, _ = run_gemm(moe, q, xs, w, ws, None, out)
    ref, mag = product_ref(q, xs, w[0], ws[0])
    check_rows(y, ref, mag, K, out)


COUNTS = [
    [0, 1, 0, 127, 128, 129, 0, 300],
    [5, 0, 0, 0],
    [0, 0, 0, 7],
    [1] * 40,
    [64, 65, 63, 1, 2, 31, 32, 33, 255, 257],
]


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "x".join(map(str, c[:8])))
@pytest.mark.parametrize("N,K", [(256, 384), (200, 272)])
def test_grouped_product(moe, counts, N, K):
    g = gen(sum(counts) + N)
    q, xs = fp8_rows(g, sum(counts), K)
    w, ws = fp8_weights(g, len(counts), N, K)
    off = offsets_of(counts)
    y, _ = run_gemm(moe, q, xs, w, ws, off, "bf16")
    y2, _ = run_gemm(moe, q, xs, w, ws, off, "bf16")
    assert torch.equal(y.view(torch.int16), y2.view(torch.int16)), "second run differs"
    o = off.tolist()
    for e, n in enumerate(counts):
        if n:
            ref, mag = product_ref(q[o[e]:o[e + 1]], xs[o[e]:o[e + 1]], w[e], ws[e])
            check_rows(y[o[e]:o[e + 1]], ref, mag, K, "bf16")


@pytest.mark.parametrize("counts,N,K", [
    ([100], 512, 8192), ([128], 100, 14336), ([3], 512, 8192), ([1, 4, 2], 1000, 7168),
    ([5, 130, 37], 256, 4112), ([1] * 11, 4096, 2048), ([130] * 8, 2560, 8192),
    ([90] * 30, 1536, 4096)])
def test_tiles_in_several_ranges(moe, counts, N, K):
    """Few tiles with many steps: every way of sharing their steps among the CTAs (pieces of one
    tile, ranges over tiles, whole tiles), few rows and many."""
    g = gen(sum(counts) + N + K)
    q, xs = fp8_rows(g, sum(counts), K)
    w, ws = fp8_weights(g, len(counts), N, K)
    off = offsets_of(counts)
    o = off.tolist()
    for out in ("fp32", "bf16"):
        y, scratch = run_gemm(moe, q, xs, w, ws, off, out)
        assert moe.moe_workspace_error(scratch) == 0
        y2, _ = run_gemm(moe, q, xs, w, ws, off, out)
        assert torch.equal(y, y2), "second run differs"
        for e, n in enumerate(counts):
            ref, mag = product_ref(q[o[e]:o[e + 1]], xs[o[e]:o[e + 1]], w[e], ws[e])
            check_rows(y[o[e]:o[e + 1]], ref, mag, K, out)


def test_rows_outside_every_expert_stay_as_they_are(moe):
    """offsets[E] below max_rows: the rows past it are not written, whatever they hold."""
    g = gen(3)
    q, xs = fp8_rows(g, 300, 256)
    q.view(torch.uint8)[170:] = 0x7F
    xs[170:] = float("inf")
    w, ws = fp8_weights(g, 3, 256, 256)
    off = torch.tensor([0, 40, 40, 170], dtype=torch.int32, device="cuda")
    y, _ = run_gemm(moe, q, xs, w, ws, off, "fp32")
    assert (y[170:] == -77.0).all()
    for e, lo, hi in ((0, 0, 40), (2, 40, 170)):
        ref, mag = product_ref(q[lo:hi], xs[lo:hi], w[e], ws[e])
        check_rows(y[lo:hi], ref, mag, 256, "fp32")


def test_ranges_past_max_rows_are_clipped_and_reported(moe):
    g = gen(4)
    q, xs = fp8_rows(g, 64, 128)
    w, ws = fp8_weights(g, 2, 128, 128)
    off = torch.tensor([0, 50, 90], dtype=torch.int32, device="cuda")
    y, scratch = run_gemm(moe, q, xs, w, ws, off, "fp32", max_rows=64)
    assert moe.moe_workspace_error(scratch) == 8
    ref, mag = product_ref(q[50:64], xs[50:64], w[1], ws[1])
    check_rows(y[50:64], ref, mag, 128, "fp32")
    off = torch.tensor([-5, 10, 4], dtype=torch.int32, device="cuda")
    y, scratch = run_gemm(moe, q, xs, w, ws, off, "fp32", max_rows=64)
    assert moe.moe_workspace_error(scratch) == 8
    assert (y[10:] == -77.0).all()


def test_nan_and_infinity_stay_in_their_rows_and_columns(moe):
    g = gen(5)
    q, xs = fp8_rows(g, 140, 384)
    w, ws = fp8_weights(g, 1, 300, 384)
    q.view(torch.uint8)[7, 200] = 0x7F
    xs[9, 1] = float("inf")
    w.view(torch.uint8)[0, 131, 5] = 0xFF
    y, _ = run_gemm(moe, q, xs, w, ws, None, "fp32")
    ref, mag = product_ref(q, xs, w[0], ws[0])
    assert torch.equal(torch.isfinite(y), torch.isfinite(ref))
    fine = torch.isfinite(ref)
    assert fine.sum() == (140 - 2) * 299
    check_rows(y[fine], ref[fine], mag[fine], 384, "fp32")


def test_scales_reach_their_own_block_only(moe):
    """Codes of one: with a scale of 2^b in block b and zero elsewhere, each result is exact."""
    K, N = 640, 384
    q = torch.full((130, K), 0x38, dtype=torch.uint8, device="cuda")          # 1.0
    w = torch.full((1, N, K), 0x38, dtype=torch.uint8, device="cuda")
    xs = torch.arange(130 * 5, device="cuda", dtype=torch.float32).view(130, 5)
    ws = torch.tensor([[1., 2, 4, 8, 16], [3, 0, 0, 0, 0], [0, 0, 0, 0, 5]], device="cuda")[None]
    y, _ = run_gemm(moe, q.view(F8), xs, w.view(F8), ws, None, "fp32")
    ref = 128.0 * (xs.double() @ ws[0].double().T).repeat_interleave(128, 1)
    assert torch.equal(y.double(), ref)


def test_gemm_weights_past_32_bits(moe):
    """Weight offsets past 2^31 and 2^32 bytes: the last expert's product is right."""
    E, N, K = 80, 7168, 8192
    g = gen(6)
    w = torch.empty((E, N, K), dtype=F8, device="cuda")
    w.view(torch.uint8).fill_(0x38)
    ws = torch.ones((E, N // 128, K // 128), device="cuda")
    w[-1:], ws[-1:] = fp8_weights(g, 1, N, K)
    q, xs = fp8_rows(g, 9, K)
    off = torch.tensor([0] * (E - 1) + [4, 9], dtype=torch.int32, device="cuda")
    y, _ = run_gemm(moe, q, xs, w, ws, off, "fp32")
    ref, mag = product_ref(q[4:], xs[4:], w[-1], ws[-1])
    check_rows(y[4:], ref, mag, K, "fp32")


def test_gemm_outputs_past_32_bits(moe):
    rows, N, K = 160_000, 14336, 256
    g = gen(7)
    q, xs = fp8_rows(g, rows, K)
    w, ws = fp8_weights(g, 2, N, K)
    off = torch.tensor([0, rows - 200, rows], dtype=torch.int32, device="cuda")
    y, _ = run_gemm(moe, q, xs, w, ws, off, "bf16")
    for e, lo, hi in ((0, 0, 3), (0, rows - 203, rows - 200), (1, rows - 200, rows)):
        ref, mag = product_ref(q[lo:hi], xs[lo:hi], w[e], ws[e])
        check_rows(y[lo:hi], ref, mag, K, "bf16")


# ------------------------------------------------------------------------------ SwiGLU experts
def swiglu_ref(q, xs, w13, s13, w2, s2):
    gu, _ = product_ref(q, xs, w13, s13)
    g, u = gu.chunk(2, 1)
    h = g / (1 + torch.exp(-g)) * u
    R, I = h.shape
    b = h.view(R, I // 128, 128)
    amax = b.abs().amax(2).clamp_min(2.0 ** -96)
    hv = (b * (448.0 / amax)[:, :, None]).float().to(F8).double() * (amax / 448.0)[:, :, None]
    N, K = w2.shape
    return hv.view(R, I) @ (w2.double() * spread(spread(s2, N, 0), K, 1)).T


def layer_close(y, ref):
    err = (y.double() - ref).abs()
    scale = ref.abs().max().item()
    mx, mean = err.max().item() / scale, (err.sum() / ref.abs().sum()).item()
    assert mx <= 2e-2 and mean <= 5e-3, (mx, mean)


def bundles_of(moe, H, I, w13, s13, w2, s2):
    nb = moe.moe_bundle_bytes(H, I, "fp8_b128")
    out = torch.full((w13.shape[0], nb), 0xEE, dtype=torch.uint8, device="cuda")
    for e in range(w13.shape[0]):
        moe.moe_pack_bundle_fp8_device(H, I, w13[e], s13[e], w2[e], s2[e], out[e])
    return out


def run_swiglu(moe, q, xs, off, bundles, E, H, I, rows, stream=None):
    y = torch.full((rows, H), -77.0, dtype=torch.bfloat16, device="cuda")
    n = moe.moe_grouped_swiglu_fp8_workspace_size(rows, E, H, I)
    ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    moe.moe_grouped_swiglu_fp8(q, xs, off, bundles, E, H, I, rows, y, ws, n, stream)
    return y, ws


def test_device_packer_equals_host_packer(moe):
    H, I = 384, 256
    g = gen(8)
    w13, s13 = fp8_weights(g, 1, 2 * I, H)
    w2, s2 = fp8_weights(g, 1, H, I)
    d = bundles_of(moe, H, I, w13, s13, w2, s2)[0].cpu().numpy()
    host = np.zeros_like(d)
    lay = moe.bundle_layout(H, I, "fp8_b128")
    moe.moe_pack_bundle_fp8(H, I, w13[0].view(torch.uint8).cpu(), s13[0].cpu(),
                            w2[0].view(torch.uint8).cpu(), s2[0].cpu(), host)
    for at, n in ((0, 3 * H * I), (lay.gate_up_scale_offset, 4 * s13.numel()),
                  (lay.down_scale_offset, 4 * s2.numel())):
        assert np.array_equal(d[at:at + n], host[at:at + n])


@pytest.mark.parametrize("H,I", [(128, 128), (256, 384), (640, 256), (1024, 640)])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "x".join(map(str, c[:8])))
def test_grouped_swiglu_fp8(moe, counts, H, I):
    E = len(counts)
    g = gen(sum(counts) + H + I)
    q, xs = fp8_rows(g, sum(counts), H)
    w13, s13 = fp8_weights(g, E, 2 * I, H)
    w2, s2 = fp8_weights(g, E, H, I)
    b = bundles_of(moe, H, I, w13, s13, w2, s2)
    ptrs = [b[e] if n else None for e, n in enumerate(counts)]     # no bundle for an empty expert
    off = offsets_of(counts)
    y, ws = run_swiglu(moe, q, xs, off, ptrs, E, H, I, sum(counts))
    y2, _ = run_swiglu(moe, q, xs, off, ptrs, E, H, I, sum(counts))
    assert torch.equal(y.view(torch.int16), y2.view(torch.int16)), "second run differs"
    assert moe.moe_workspace_error(ws) == 0
    o = off.tolist()
    ref = torch.cat([swiglu_ref(q[o[e]:o[e + 1]], xs[o[e]:o[e + 1]], w13[e], s13[e], w2[e], s2[e])
                     for e in range(E) if counts[e]])
    layer_close(y, ref)


@pytest.mark.parametrize("counts,H,I", [([70], 8192, 256), ([2, 1], 14336, 128),
                                        ([200, 3, 64], 7168, 384), ([1] * 5, 4096, 4096)])
def test_swiglu_tiles_in_several_ranges(moe, counts, H, I):
    E = len(counts)
    g = gen(sum(counts) + H + I)
    q, xs = fp8_rows(g, sum(counts), H)
    w13, s13 = fp8_weights(g, E, 2 * I, H)
    w2, s2 = fp8_weights(g, E, H, I)
    b = bundles_of(moe, H, I, w13, s13, w2, s2)
    off = offsets_of(counts)
    y, ws = run_swiglu(moe, q, xs, off, [b[e] for e in range(E)], E, H, I, sum(counts))
    assert moe.moe_workspace_error(ws) == 0
    o = off.tolist()
    ref = torch.cat([swiglu_ref(q[o[e]:o[e + 1]], xs[o[e]:o[e + 1]], w13[e], s13[e], w2[e], s2[e])
                     for e in range(E)])
    layer_close(y, ref)


@pytest.mark.parametrize("T,E,k,H,I", [(1, 256, 8, 7168, 2048), (33, 60, 4, 2048, 1408),
                                       (700, 16, 8, 7168, 2048)])
def test_grouped_swiglu_fp8_full_shapes(moe, T, E, k, H, I):
    """The DeepSeek-V3- and Qwen1.5-MoE-shaped experts on randomly routed tokens."""
    g = gen(T + E)
    ids = torch.argsort(torch.rand((T, E), generator=g, device="cuda"), 1)[:, :k]
    counts = torch.bincount(ids.flatten(), minlength=E).tolist()
    q, xs = fp8_rows(g, T * k, H)
    used = [e for e in range(E) if counts[e]]
    w13, s13 = fp8_weights(g, len(used), 2 * I, H)
    w2, s2 = fp8_weights(g, len(used), H, I)
    b = bundles_of(moe, H, I, w13, s13, w2, s2)
    ptrs = [None] * E
    for i, e in enumerate(used):
        ptrs[e] = b[i]
    off = offsets_of(counts)
    y, _ = run_swiglu(moe, q, xs, off, ptrs, E, H, I, T * k)
    o = off.tolist()
    ref = torch.cat([swiglu_ref(q[o[e]:o[e + 1]], xs[o[e]:o[e + 1]], w13[i], s13[i], w2[i], s2[i])
                     for i, e in enumerate(used)])
    layer_close(y, ref)


def test_an_expert_with_rows_but_no_bundle_is_skipped(moe):
    H, I, counts = 256, 256, [3, 40, 0, 150]
    g = gen(21)
    q, xs = fp8_rows(g, sum(counts), H)
    w13, s13 = fp8_weights(g, 4, 2 * I, H)
    w2, s2 = fp8_weights(g, 4, H, I)
    b = bundles_of(moe, H, I, w13, s13, w2, s2)
    y, ws = run_swiglu(moe, q, xs, offsets_of(counts), [b[0], None, None, b[3]], 4, H, I,
                       sum(counts))
    assert moe.moe_workspace_error(ws) == 10
    assert (y[3:43] == -77).all()
    layer_close(y[:3], swiglu_ref(q[:3], xs[:3], w13[0], s13[0], w2[0], s2[0]))
    layer_close(y[43:], swiglu_ref(q[43:], xs[43:], w13[3], s13[3], w2[3], s2[3]))


def test_zero_and_nan_rows_through_the_experts(moe):
    """A row of zeros gives zeros; a NaN row gives NaN there and nowhere else."""
    H, I = 256, 256
    g = gen(11)
    q, xs = fp8_rows(g, 140, H)
    q.view(torch.uint8)[3] = 0
    q.view(torch.uint8)[130, 17] = 0x7F
    w13, s13 = fp8_weights(g, 1, 2 * I, H)
    w2, s2 = fp8_weights(g, 1, H, I)
    b = bundles_of(moe, H, I, w13, s13, w2, s2)
    y, _ = run_swiglu(moe, q, xs, offsets_of([140]), [b[0]], 1, H, I, 140)
    assert (y[3] == 0).all() and y[130].isnan().all()
    keep = [r for r in range(140) if r != 130]
    assert torch.isfinite(y[keep]).all()
    layer_close(y[keep], swiglu_ref(q[keep], xs[keep], w13[0], s13[0], w2[0], s2[0]))


def test_side_stream_and_graph_replay(moe):
    """Quantise -> experts on a side stream, captured once and replayed on other inputs."""
    T, k, E, H, I = 5, 2, 4, 256, 384
    g = gen(12)
    w13, s13 = fp8_weights(g, E, 2 * I, H)
    w2, s2 = fp8_weights(g, E, H, I)
    b = bundles_of(moe, H, I, w13, s13, w2, s2)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    src = torch.tensor([0, 3, 4, 7, 8, 1, 2, 5, 6, 9], dtype=torch.int32, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    q = torch.empty((T * k, H), dtype=torch.uint8, device="cuda")
    xs = torch.empty((T * k, H // 128), device="cuda")
    y = torch.empty((T * k, H), dtype=torch.bfloat16, device="cuda")
    n = moe.moe_grouped_swiglu_fp8_workspace_size(T * k, E, H, I)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    tab = moe.bundle_table([b[e] for e in range(E)])

    def step(st):
        moe.moe_quantize_fp8(x, src, T, k, H, q, xs, st)
        moe.moe_grouped_swiglu_fp8(q, xs, off, tab, E, H, I, T * k, y, ws, n, st)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(side)
    for counts in ([4, 0, 5, 1], [0, 0, 0, 10], [3, 3, 3, 1]):
        x.copy_(randn(g, T, H).to(torch.bfloat16))
        off.copy_(offsets_of(counts))
        graph.replay()
        torch.cuda.synchronize()
        rq, rs = quant_ref(x[(src // k).long()])
        rq, rs = rq.cuda(), rs.cuda()
        o = off.tolist()
        ref = torch.cat([swiglu_ref(rq[o[e]:o[e + 1]], rs[o[e]:o[e + 1]], w13[e], s13[e], w2[e],
                                    s2[e]) for e in range(E) if counts[e]])
        layer_close(y, ref)
