"""GPU tests of the whole layer with FP8 experts and with group-limited selection: against the
fp64 oracle, against the same layer composed of its single calls, with experts resident and
through the expert-slot cache, and replayed as a CUDA graph.

Tolerance as for the other formats: max |err| <= 2e-2 max |ref|, sum |err| <= 5e-3 sum |ref|.
"""
import numpy as np
import pytest
import torch

import workloads as wl
from oracle import bf16, moe_ref

from gpu_util import assert_close, spread_rows
from test_gpu_cache import make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import expert_dispatch_streaming_gb300 as m
    return m


@pytest.fixture(scope="module")
def syn(moe):
    from expert_dispatch_streaming_gb300 import synthetic
    return synthetic


SMALL = [
    wl.custom("f8plain", cfg_id=170, H=256, E=16, k=4, I=384, gating="softmax_renorm",
              wdtype="fp8_b128"),
    wl.custom("f8qwenlike", cfg_id=171, H=512, E=60, k=4, I=256, gating="softmax", Is=384,
              shared_gate="sigmoid", zipf_s=1.0, bias_kind="logit", wdtype="fp8_b128",
              n_group=6, topk_group=2),
    wl.custom("f8dslike", cfg_id=172, H=512, E=64, k=8, I=256, gating="sigmoid_bias_renorm",
              scale=2.5, Is=256, shared_gate="one", zipf_s=1.1, bias_kind="select",
              wdtype="fp8_b128", n_group=8, topk_group=4),
]
GROUPED_OTHER = [
    wl.custom("gbf16", cfg_id=173, H=256, E=16, k=4, I=384, gating="softmax_renorm", n_group=4,
              topk_group=2),
    wl.custom("gint4", cfg_id=174, H=256, E=32, k=4, I=256, gating="sigmoid_bias_renorm",
              scale=2.5, Is=256, shared_gate="one", zipf_s=1.1, bias_kind="select",
              wdtype="int4_g128", n_group=8, topk_group=3),
    wl.custom("gfp4", cfg_id=175, H=512, E=60, k=4, I=256, gating="softmax", Is=384,
              shared_gate="sigmoid", zipf_s=1.0, bias_kind="logit", wdtype="nvfp4", n_group=12,
              topk_group=4),
]


def check_grouped_ids(cfg, ids, ref):
    """Equal to the oracle's except where its group or expert gap is below 1e-6."""
    clear = ref["gap"] >= 1e-6
    assert clear.mean() > 0.9 and np.array_equal(ids[clear], ref["ids_selected"][clear])


def _layer_case(moe, syn, cfg, T, rows=None, cache=None, dl=None):
    dl = dl or syn.DeviceLayer(cfg)
    xb = wl.tokens(cfg, T)
    x = syn.to_device_bits(xb)
    ws = dl.workspace(T)
    ws.fill_(0xA5)
    ids = torch.full((T, cfg.k), -1, dtype=torch.int32, device="cuda")
    out, st = dl.forward(x, ws, ids_out=ids, cache=cache)
    out2, _ = dl.forward(x, ws, cache=cache)
    torch.cuda.synchronize()
    assert moe.moe_workspace_error(ws) == 0 and st.fused_decode == 0
    got = syn.bits_of(out)
    if cache is None:
        assert np.array_equal(got, syn.bits_of(out2)), "second run differs"
    ids = ids.cpu().numpy()
    if isinstance(rows, str):
        rows = spread_rows(ids, cfg.E)
    ref = moe_ref.layer_forward(cfg, 0, xb, forced_ids=ids, rows=rows)
    check_grouped_ids(cfg, ids, ref)
    assert_close(got[ref["rows"]], ref["out"], f"{cfg.name} T={T}")
    assert_close(syn.bits_of(out2)[ref["rows"]], ref["out"], f"{cfg.name} T={T} again")
    return st


@pytest.mark.parametrize("cfg", SMALL, ids=lambda c: c.name)
@pytest.mark.parametrize("T", [1, 2, 16, 17, 133, 300])
def test_layer_forward_fp8(moe, syn, cfg, T):
    _layer_case(moe, syn, cfg, T)


@pytest.mark.parametrize("cfg", GROUPED_OTHER, ids=lambda c: c.name)
@pytest.mark.parametrize("T", [1, 16, 133])
def test_layer_forward_grouped_other_weights(moe, syn, cfg, T):
    _layer_case(moe, syn, cfg, T)


@pytest.mark.parametrize("T", [1, 32, 512])
def test_layer_forward_deepseek_fp8(moe, syn, T, deepseek):
    """The full DeepSeek-V3 shape with FP8 experts; sampled rows."""
    _layer_case(moe, syn, wl.DEEPSEEK_FP8, T, rows="spread", dl=deepseek)


@pytest.fixture(scope="module")
def deepseek(syn):
    yield syn.DeviceLayer(wl.DEEPSEEK_FP8)


@pytest.mark.parametrize("T", [1, 16, 40, 1100])
def test_layer_equals_its_single_calls(moe, syn, T):
    """route -> quantise and gather -> experts -> combine, called one by one, with a shared
    expert and a residual: the layer's output bit for bit."""
    cfg = SMALL[2]
    dl = syn.DeviceLayer(cfg)
    H, E, k, I, Is = cfg.H, cfg.E, cfg.k, cfg.I, cfg.Is
    x, res = (syn.to_device_bits(wl.tokens(cfg, T, step=s)) for s in (0, 1))
    out, _ = dl.forward(x, dl.workspace(T), residual=res)

    i32 = dict(dtype=torch.int32, device="cuda")
    u8 = dict(dtype=torch.uint8, device="cuda")
    ids, pos, src = (torch.empty(T * k, **i32) for _ in range(3))
    w = torch.empty((T, k), device="cuda")
    counts, off = torch.empty(E, **i32), torch.empty(E + 1, **i32)
    n = moe.moe_route_workspace_size(T, H, E, k)
    moe.moe_route_topk_grouped(x, dl.w_r, dl.logit_bias, dl.sel_bias, None, T, H, E, k,
                               cfg.n_group, cfg.topk_group, cfg.gating, cfg.scale, ids, w,
                               counts, off, pos, src, None, None, None, torch.empty(n, **u8), n)

    def experts(src, kk, rows, off, bundles, n_e, inner):
        q, s = torch.empty((rows, H), **u8), torch.empty((rows, H // 128), device="cuda")
        moe.moe_quantize_fp8(x, src, T, kk, H, q, s)
        y = torch.empty((rows, H), dtype=torch.int16, device="cuda")
        n = moe.moe_grouped_swiglu_fp8_workspace_size(rows, n_e, H, inner)
        moe.moe_grouped_swiglu_fp8(q, s, off, bundles, n_e, H, inner, rows, y,
                                   torch.empty(n, **u8), n)
        return y

    y = experts(src, k, T * k, off, [dl.routed[e] for e in range(E)], E, I)
    shared = experts(None, 0, T, torch.tensor([0, T], **i32), [dl.shared[0]], 1, Is)
    ref = torch.empty_like(x)
    moe.moe_combine(y, pos, w, T, k, H, shared, None, res, ref)
    assert torch.equal(out, ref)


def test_residual_and_normed_output(moe, syn):
    cfg, T = SMALL[1], 21
    dl = syn.DeviceLayer(cfg)
    xb, rb = wl.tokens(cfg, T), wl.tokens(cfg, T, step=1)
    ids = torch.empty((T, cfg.k), dtype=torch.int32, device="cuda")
    normed = torch.empty((T, cfg.H), dtype=torch.int16, device="cuda")
    events = [torch.cuda.Event(enable_timing=True) for _ in range(moe.MOE_N_PHASE_EVENTS)]
    for e in events:
        e.record()
    out, _ = dl.forward(syn.to_device_bits(xb), dl.workspace(T), ids_out=ids, out_normed=normed,
                        residual=syn.to_device_bits(rb), phase_events=events)
    torch.cuda.synchronize()
    assert all(a.elapsed_time(b) >= 0 for a, b in zip(events, events[1:]))
    ref = moe_ref.layer_forward(cfg, 0, xb, forced_ids=ids.cpu().numpy())["out"]
    total = bf16.round_rne(ref + bf16.decode(rb))
    assert_close(syn.bits_of(out), total)
    assert_close(syn.bits_of(normed),
                 moe_ref.rms_normalize(bf16.decode(syn.bits_of(out)), wl.STACK_NORM_EPS))


@pytest.mark.parametrize("mode", ["host", "device"])
@pytest.mark.parametrize("T", [1, 24])
def test_fp8_bundles_through_the_cache(moe, syn, mode, T):
    """All experts miss on the first call; on the second some or all hit."""
    cfg = SMALL[2]
    cache, store, table = make_cache(moe, syn, cfg, cfg.E, device_lru=int(mode == "device"))
    try:
        st = _layer_case(moe, syn, cfg, T, cache=cache, dl=syn.DeviceLayer(cfg, cached=True))
        if mode == "host":
            assert st.n_missed == st.n_unique > 0
    finally:
        moe.moe_expert_cache_destroy(cache)


def test_device_lru_with_too_few_slots(moe, syn):
    """The error word says so, and the experts that got no slot are skipped."""
    cfg = SMALL[2]
    cache, store, table = make_cache(moe, syn, cfg, 2, device_lru=1)
    try:
        dl = syn.DeviceLayer(cfg, cached=True)
        ws = dl.workspace(6)
        dl.forward(syn.to_device_bits(wl.tokens(cfg, 6)), ws, cache=cache)
        torch.cuda.synchronize()
        assert moe.moe_workspace_error(ws) == 20
    finally:
        moe.moe_expert_cache_destroy(cache)


def test_fp8_layer_graph_replay(moe, syn):
    """Captured once on a side stream, replayed on other tokens: equal to the eager calls."""
    cfg, T = SMALL[2], 5
    dl = syn.DeviceLayer(cfg)
    xs = [syn.to_device_bits(wl.tokens(cfg, T, step=s)) for s in range(4)]
    ws = dl.workspace(T)
    eager = [dl.forward(x, ws)[0].clone() for x in xs]
    x, out = xs[0].clone(), torch.empty_like(xs[0])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        dl.forward(x, ws, out=out, stream=side)
    for a, want in zip(xs, eager):
        x.copy_(a)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_programmatic_launches(moe, syn):
    """MOE_OPT_PDL only changes when kernels may start."""
    cfg = SMALL[2]
    dl = syn.DeviceLayer(cfg)
    for T in (3, 200):
        x, ws = syn.to_device_bits(wl.tokens(cfg, T)), dl.workspace(T)
        want = dl.forward(x, ws)[0].clone()
        moe.moe_set_option(moe.MOE_OPT_PDL, 1)
        try:
            got = [dl.forward(x, ws)[0].clone() for _ in range(3)]
            torch.cuda.synchronize()
        finally:
            moe.moe_set_option(moe.MOE_OPT_PDL, 0)
        assert all(torch.equal(g, want) for g in got)
