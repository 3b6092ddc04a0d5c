"""Host-side checks of the FP8 expert path: the bundle layout and packer, and the refusals of
every new entry point (sizes, alignment, null pointers, workspaces).  No GPU is used: a refused
call returns before any CUDA work."""
import numpy as np
import pytest

from oracle import moe_ref


@pytest.fixture(scope="module")
def moe():
    import expert_dispatch_streaming_gb300 as m
    return m


def _untile_fp8(buf, rows, K):
    """Inverse of the tiled E4M3 image: tiles of 128 rows x 128 k, chunk c of row r at
    r*128 + ((c ^ (r % 8)) * 16)."""
    t = buf[:rows * K].reshape(rows // 128, K // 128, 128, 8, 16)
    r, c = np.arange(128)[:, None], np.arange(8)[None, :]
    return t[:, :, r, c ^ (r % 8), :].transpose(0, 2, 1, 3, 4).reshape(rows, K)


def _expert(H, I, seed=0):
    rng = np.random.default_rng(seed)
    w13 = rng.integers(0, 0x7F, (2 * I, H)).astype(np.uint8)
    w2 = (rng.integers(0, 0x7F, (H, I)) | 0x80).astype(np.uint8)
    s13 = rng.uniform(0.5, 2.0, (2 * I // 128, H // 128)).astype(np.float32)
    s2 = rng.uniform(0.5, 2.0, (H // 128, I // 128)).astype(np.float32)
    return w13, s13, w2, s2


def test_pack_fp8_layout(moe):
    H, I = 256, 384
    w13, s13, w2, s2 = _expert(H, I)
    lay = moe.bundle_layout(H, I, "fp8_b128")
    buf = np.zeros(lay.total_bytes, np.uint8)
    moe.moe_pack_bundle_fp8(H, I, w13, s13, w2, s2, buf)
    assert np.array_equal(_untile_fp8(buf[lay.gate_up_offset:], 2 * I, H), w13)
    assert np.array_equal(_untile_fp8(buf[lay.down_offset:], H, I), w2)
    got = buf[lay.gate_up_scale_offset:][:4 * s13.size].view(np.float32)
    assert np.array_equal(got.reshape(s13.shape), s13)
    got = buf[lay.down_scale_offset:][:4 * s2.size].view(np.float32)
    assert np.array_equal(got.reshape(s2.shape), s2)
    assert lay.down_offset == 2 * H * I and lay.gate_up_scale_offset == 3 * H * I
    # hand check of one code: row 130 (tile 1, r = 2), k = 150 (k tile 1, chunk 1, byte 6)
    at = (1 * (H // 128) + 1) * 16384 + 2 * 128 + ((1 ^ 2) << 4) + 6
    assert buf[lay.gate_up_offset + at] == w13[130, 150]


def test_fp8_bundle_sizes(moe):
    assert moe.moe_bundle_bytes(7168, 2048, "fp8_b128") == 3 * 7168 * 2048 + 4 * 3 * 56 * 16
    assert moe.moe_bundle_bytes(200, 128, "fp8_b128") == 0


@pytest.mark.parametrize("field", ["code", "code_neg", "scale_inf", "scale_nan", "null"])
def test_pack_fp8_refusals(moe, field):
    H, I = 128, 128
    w13, s13, w2, s2 = _expert(H, I)
    if field == "code":
        w13[3, 5] = 0x7F
    elif field == "code_neg":
        w2[3, 5] = 0xFF
    elif field == "scale_inf":
        s2[0, 0] = np.inf
    elif field == "scale_nan":
        s13[1, 0] = np.nan
    buf = np.zeros(moe.moe_bundle_bytes(H, I, "fp8_b128"), np.uint8)
    with pytest.raises(moe.MoEError) as ei:
        moe.moe_pack_bundle_fp8(H, I, w13, None if field == "null" else s13, w2, s2, buf)
    assert ei.value.status == moe.MOE_ERR_INVALID_ARG


def test_generic_packer_refuses_fp8(moe):
    q = np.zeros((128, 128), np.uint8)
    buf = np.zeros(moe.moe_bundle_bytes(128, 128, "fp8_b128"), np.uint8)
    with pytest.raises(moe.MoEError):
        moe.moe_pack_bundle(128, 128, "fp8_b128", q, q, q, q, q, q, buf)


def test_e4m3_max_and_block_formula():
    """448 is E4M3's largest value and amax * (448 / amax) never rounds past it: the nearest
    code of any value up to 448 * (1 + 2^-23) is 448 (the next step would be 480)."""
    vals = moe_ref.decode_e4m3(np.arange(256))
    assert np.nanmax(vals) == 448.0
    amax = np.random.default_rng(0).uniform(1e-20, 1e20, 100000).astype(np.float32)
    assert np.all(amax * (np.float32(448) / amax) < 464)


A = 1 << 20          # stands for a device pointer: the calls below never touch it
BIG = 1 << 34


@pytest.mark.parametrize("bad", [
    dict(n_group=0), dict(n_group=33, E=66), dict(n_group=7), dict(topk_group=0),
    dict(topk_group=9), dict(k=0), dict(k=9), dict(topk_group=1, k=5, E=32), dict(E=264),
    dict(H=60), dict(T=-1), dict(gating=3), dict(gating=-1), dict(x=None), dict(w_r=None),
    dict(ids=None), dict(src=None), dict(ws=None), dict(ws_bytes=256), dict(w_gate=A)])
def test_route_grouped_refusals(moe, bad):
    a = dict(x=A, w_r=A, w_gate=None, T=4, H=64, E=64, k=4, n_group=8, topk_group=4, gating=2,
             ids=A, src=A, ws=A, ws_bytes=BIG)
    a.update(bad)
    with pytest.raises(moe.MoEError) as ei:
        moe.moe_route_topk_grouped(a["x"], a["w_r"], None, None, a["w_gate"], a["T"], a["H"],
                                   a["E"], a["k"], a["n_group"], a["topk_group"], a["gating"],
                                   1.0, a["ids"], A, A, A, A, a["src"], None, None, None,
                                   a["ws"], a["ws_bytes"], 0)
    assert ei.value.status == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(H=0), dict(H=24), dict(x=None), dict(q=None), dict(scale=None),
    dict(x=A + 8), dict(q=A + 4), dict(src=A, k=0), dict(src=A, k=1 << 20, T=1 << 20),
    dict(scale=A + 2), dict(src=A + 1, k=1)])
def test_quantize_refusals(moe, bad):
    a = dict(x=A, src=None, T=4, k=0, H=64, q=A, scale=A)
    a.update(bad)
    with pytest.raises(moe.MoEError) as ei:
        moe.moe_quantize_fp8(a["x"], a["src"], a["T"], a["k"], a["H"], a["q"], a["scale"], 0)
    assert ei.value.status == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    dict(E=0), dict(E=257), dict(N=0), dict(K=0), dict(K=24), dict(rows=-1), dict(out=2),
    dict(offsets=None, E=2), dict(xq=None), dict(xs=None), dict(w=None), dict(w_scale=None),
    dict(y=None), dict(ws=None), dict(ws_bytes=0), dict(xq=A + 8), dict(w=A + 8), dict(y=A + 8),
    dict(xs=A + 2), dict(w_scale=A + 1), dict(ws=A + 16)])
def test_gemm_refusals(moe, bad):
    a = dict(xq=A, xs=A, w=A, w_scale=A, offsets=A, E=4, N=64, K=64, rows=8, out=0, y=A, ws=A,
             ws_bytes=BIG)
    a.update(bad)
    with pytest.raises(moe.MoEError) as ei:
        moe.moe_grouped_gemm_fp8(a["xq"], a["xs"], a["w"], a["w_scale"], a["offsets"], a["E"],
                                 a["N"], a["K"], a["rows"], a["out"], a["y"], a["ws"],
                                 a["ws_bytes"], 0)
    assert ei.value.status == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    dict(E=0), dict(E=257), dict(H=64), dict(I=192), dict(rows=-1), dict(xq=None), dict(xs=None),
    dict(offsets=None), dict(y=None), dict(ws=None), dict(ws_bytes=512), dict(xq=A + 8),
    dict(y=A + 2), dict(ws=A + 128)])
def test_swiglu_refusals(moe, bad):
    a = dict(xq=A, xs=A, offsets=A, E=4, H=128, I=128, rows=8, y=A, ws=A, ws_bytes=BIG)
    a.update(bad)
    with pytest.raises(moe.MoEError) as ei:
        moe.moe_grouped_swiglu_fp8(a["xq"], a["xs"], a["offsets"], [A] * max(a["E"], 1), a["E"],
                                   a["H"], a["I"], a["rows"], a["y"], a["ws"], a["ws_bytes"], 0)
    assert ei.value.status == moe.MOE_ERR_INVALID_ARG


def test_empty_calls_return_without_work(moe):
    moe.moe_quantize_fp8(None, None, 0, 0, 64, None, None, 0)
    moe.moe_grouped_gemm_fp8(None, None, None, None, None, 1, 64, 64, 0, 0, None, None, 0, 0)
    moe.moe_grouped_swiglu_fp8(None, None, None, [A], 1, 128, 128, 0, None, None, 0, 0)
    assert moe.moe_grouped_gemm_fp8_workspace_size(8, 300, 64, 64) == 0
    assert moe.moe_grouped_swiglu_fp8_workspace_size(8, 4, 100, 128) == 0


def _layer(moe, **kw):
    d = moe.moe_layer()
    d.H, d.E, d.k, d.I, d.Is = 256, 16, 4, 128, 0
    d.gating, d.scale, d.wdtype = moe.MOE_GATING_SOFTMAX, 1.0, moe.WDTYPE["fp8_b128"]
    for n, v in kw.items():
        setattr(d, n, v)
    return d


def test_layer_refuses_bad_groups_and_sizes(moe):
    g = moe.MOE_GATING_SOFTMAX + moe.MOE_GATING_GROUPED
    ok = dict(gating=g, n_group=4, topk_group=2)
    assert moe.moe_layer_workspace_size(_layer(moe), 8) > 0
    assert moe.moe_layer_workspace_size(_layer(moe, **ok), 8) > 0
    # the groups are read with the flag only
    assert moe.moe_layer_workspace_size(_layer(moe, n_group=-3, topk_group=99), 8) > 0
    for bad in (dict(n_group=3), dict(n_group=0), dict(n_group=64), dict(topk_group=0),
                dict(topk_group=5), dict(n_group=16, topk_group=3)):
        assert moe.moe_layer_workspace_size(_layer(moe, **{**ok, **bad}), 8) == 0, bad
    for bad in (dict(H=200), dict(I=100), dict(Is=64), dict(k=9), dict(wdtype=4)):
        assert moe.moe_layer_workspace_size(_layer(moe, **bad), 8) == 0, bad


def test_layer_refuses_forced_ids_with_groups(moe):
    """Addresses that are never followed: the call returns before any CUDA work."""
    one = 1 << 20
    d = _layer(moe, gating=moe.MOE_GATING_SOFTMAX + moe.MOE_GATING_GROUPED, n_group=4,
               topk_group=2, w_r=one)
    table = moe.bundle_table([one] * 16)
    d.bundles = table
    with pytest.raises(moe.MoEError):
        moe.moe_layer_forward(d, one, 8, one, None, one, None, one, 1 << 40)
    d.gating = 3 + moe.MOE_GATING_GROUPED
    with pytest.raises(moe.MoEError):
        moe.moe_layer_forward(d, one, 8, None, None, one, None, one, 1 << 40)


def test_fp8_recipe_and_rounding():
    """The workload's codes are finite with the stated deviation; the oracle's rounding is the
    nearest E4M3 value."""
    import workloads as wl
    cfg = wl.custom("f8", H=256, I=128, wdtype="fp8_b128")
    wg, wu, wd = moe_ref.expert_matrices(wl.expert(cfg, 0, 0))
    for m, shape in ((wg, (256, 128)), (wu, (256, 128)), (wd, (128, 256))):
        assert m.shape == shape and np.isfinite(m).all()
        assert 0.4 * cfg.w_std < m.std() < 1.6 * cfg.w_std
    vals = np.unique(moe_ref.decode_e4m3(np.arange(0x7F)))
    mids = (vals[1:] + vals[:-1]) / 2
    even = np.where(np.arange(len(mids)) % 2 == 0, vals[:-1], vals[1:])
    assert np.array_equal(moe_ref.round_e4m3(mids), even)
    assert np.array_equal(moe_ref.round_e4m3(-vals), -vals)
    assert np.array_equal(moe_ref.round_e4m3(np.array([449.0, 1e9, -500.0])), [448, 448, -448])


def test_misaligned_bundles_are_refused(moe):
    """As above, addresses that are never followed."""
    one = 1 << 20
    d = _layer(moe, w_r=one)
    d.bundles = moe.bundle_table([one] * 15 + [one + 8])
    with pytest.raises(moe.MoEError):
        moe.moe_layer_forward(d, one, 8, None, None, one, None, one, 1 << 40)
    d = _layer(moe, w_r=one, Is=128, shared_bundle=one + 4)
    d.bundles = moe.bundle_table([one] * 16)
    with pytest.raises(moe.MoEError):
        moe.moe_layer_forward(d, one, 8, None, None, one, None, one, 1 << 40)
    with pytest.raises(moe.MoEError):
        moe.moe_grouped_swiglu_fp8(one, one, one, [one, one + 8], 2, 256, 128, 8, one, one, 1 << 40)


@pytest.mark.parametrize("bad", [dict(x=A + 8), dict(ws=A + 16)])
def test_route_grouped_refuses_misaligned_rows_and_workspaces(moe, bad):
    test_route_grouped_refusals(moe, bad)
